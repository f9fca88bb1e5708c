// Paged 8-bit cache of exact keys and values: the append that quantises, the read
// that gives rows back, and decode attention.
//
// A page holds P tokens of one sequence; per head its keys (rotated) and its values
// are P x d int8 codes with one fp32 scale each, value = code * scale.  Layout
// [n_pages][H][P][d], so one head's part of a page is one contiguous run of bytes.
//
// The scale of a page and head is amax / 127 over the tokens of the call that opened
// the page.  A later append with a larger value grows it to at least kQ8Grow times
// its old value and rounds the codes already there again: growing by a constant
// factor bounds the sum of those roundings by a geometric series, whereas following
// every small rise would let a code survive many rescalings unrounded and drift.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "lla_internal.cuh"
#include "lla_rows.cuh"
#include "lla_sm100.cuh"

namespace lla {
namespace {

constexpr float kQ8Grow = 1.25f;
constexpr float kQ8Tiny = 1e-30f;    // a largest value at or below this stores zeros

// ---------------------------------------------------------------- append

constexpr int kAppendThreads = 128;

// The page that unit u of an append works on: units floor(tok_start[b] / P) + 2 b and
// up belong to sequence b, enough for every page its tokens can touch.
struct AppendUnit {
  int b, page, off, count;    // rows [off, off + count) of the page are new
  int tok;                    // first of their tokens
};

__device__ __forceinline__ bool append_unit(const Q8AppendArgs& a, int u, bool tell,
                                            AppendUnit& r) {
  const int P = 1 << a.shift;
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((a.tok_start[mid] >> a.shift) + 2 * mid <= u) lo = mid;
    else hi = mid;
  }
  const int s = a.tok_start[lo], e = a.tok_start[lo + 1];
  const int after = a.ctx_len[lo];
  if (s < 0 || e < s || e > a.n_tok || after < e - s ||
      after > (long long)a.max_pages << a.shift) {
    if (tell && a.status) atomicOr(a.status, LLA_STATUS_CTX_RANGE);
    return false;
  }
  const int before = after - (e - s);
  const int j = u - ((s >> a.shift) + 2 * lo);
  const long long page_at = (long long)(before >> a.shift) + j;
  const long long p0 = page_at << a.shift;
  if (j < 0 || e == s || p0 >= after) return false;
  r.b = lo;
  r.page = a.block_table[(long long)lo * a.max_pages + page_at];
  if (r.page < 0 || r.page >= a.n_pages) {
    if (tell && a.status) atomicOr(a.status, LLA_STATUS_PAGE_RANGE);
    return false;
  }
  r.off = before > p0 ? (int)(before - p0) : 0;
  r.count = (int)(after - p0 < P ? after - p0 : P) - r.off;
  r.tok = s + (int)(p0 + r.off - before);
  return true;
}

// Scale of the page after the append, from the largest new value.
__device__ __forceinline__ float grown_scale(float amax, float older) {
  const float asked = amax > kQ8Tiny ? __fdiv_rn(amax, 127.f) : 0.f;
  return asked > older ? fmaxf(asked, older * kQ8Grow) : older;
}

__device__ __forceinline__ int quantise(float x, float inv) {
  const float y = x * inv;
  return y == y ? __float2int_rn(fminf(fmaxf(y, -127.f), 127.f)) : 0;
}

__device__ __forceinline__ uint32_t quantise4(const float* v, float inv) {
  return (quantise(v[0], inv) & 255) | (quantise(v[1], inv) & 255) << 8 |
         (quantise(v[2], inv) & 255) << 16 | (uint32_t)quantise(v[3], inv) << 24;
}

// grid (units, H, 2): z = 0 keys, z = 1 values.
template <typename T>
__global__ void __launch_bounds__(kAppendThreads) q8_append_kernel(Q8AppendArgs a) {
  __shared__ float red[kAppendThreads / 32];
  const int h = blockIdx.y;
  const bool is_k = blockIdx.z == 0;
  const bool tell = h == 0 && is_k && threadIdx.x == 0;
  AppendUnit un;
  if (!append_unit(a, blockIdx.x, tell, un)) return;
  const int tpr = a.d / 8, rpp = kAppendThreads / tpr;      // threads per row, rows per pass
  const int row0 = threadIdx.x / tpr, c = threadIdx.x % tpr;
  const bool works = row0 < rpp;
  const bool turn = is_k && a.rope;
  const RowChunk rc = row_chunk(c, a.d, a.rd, turn ? a.layout : LLA_ROPE_INTERLEAVED);
  const T* src = static_cast<const T*>(is_k ? a.k : a.v) + (long long)h * a.d;
  const long long stride = is_k ? a.k_stride : a.v_stride;
  const long long run = (((long long)un.page * a.H + h) << a.shift) * a.d;
  int8_t* codes = (is_k ? a.kc : a.vc) + run;
  float* scale = (is_k ? a.ks : a.vs) + (long long)un.page * a.H + h;

  auto value = [&](int r, float* v) {
    const long long tok = un.tok + r;
    load_chunk(src + tok * stride, rc, v);
    if (turn) {
      const int pos = checked_position(a.positions[tok], a.rope_max_pos, a.status, h == 0 && c == 0);
      rotate_chunk(a.rope + (size_t)pos * (a.rd / 2), rc, 1.f, v);
    }
  };
  float amax = 0.f;
  bool strange = false;
  if (works)
    for (int r = row0; r < un.count; r += rpp) {
      float v[8];
      value(r, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = fabsf(v[j]);
        if (x <= FLT_MAX) amax = fmaxf(amax, x);
        else strange = true;
      }
    }
  if (strange && a.status) atomicOr(a.status, LLA_STATUS_NONFINITE);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  float older = un.off > 0 ? *scale : 0.f;
  if (!(older > 0.f && older <= FLT_MAX)) older = 0.f;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, red[w]);
  const float now = grown_scale(amax, older);
  const float inv = now > 0.f ? __fdiv_rn(1.f, now) : 0.f;
  if (threadIdx.x == 0) *scale = now;
  if (now > older && un.off > 0) {
    const float ratio = __fdiv_rn(older, now);
    uint32_t* words = reinterpret_cast<uint32_t*>(codes);
    for (int i = threadIdx.x; i < un.off * a.d / 4; i += kAppendThreads) {
      const uint32_t w = words[i];
      const float v[4] = {(float)(int8_t)w, (float)(int8_t)(w >> 8), (float)(int8_t)(w >> 16),
                          (float)(int8_t)(w >> 24)};
      words[i] = quantise4(v, ratio);
    }
  }
  if (works)
    for (int r = row0; r < un.count; r += rpp) {
      float v[8];
      value(r, v);
      int8_t* row = codes + (long long)(un.off + r) * a.d;
      *reinterpret_cast<uint32_t*>(row + rc.lo) = quantise4(v, inv);
      *reinterpret_cast<uint32_t*>(row + rc.hi) = quantise4(v + 4, inv);
    }
}

// ---------------------------------------------------------------- read

// One thread per eight dims of one head's row; grid.y: 0 keys, 1 values.
__global__ void __launch_bounds__(256) q8_read_kernel(Q8ReadArgs a) {
  const int tpr = a.d / 8, per_row = a.H * tpr;
  const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long row = idx / per_row;
  if (row >= a.n_rows) return;
  const int rest = (int)(idx % per_row), h = rest / tpr, c = rest % tpr;
  const bool is_k = blockIdx.y == 0;
  __nv_bfloat16* out = is_k ? a.k_out : a.v_out;
  const long long slot = a.slot[row];
  if (slot < 0 || slot >= (long long)a.n_pages << a.shift) {
    if (rest == 0 && is_k && a.status) atomicOr(a.status, LLA_STATUS_SLOT_RANGE);
    return;
  }
  const long long page = slot >> a.shift;
  const int r = (int)(slot & ((1 << a.shift) - 1));
  const float s = (is_k ? a.ks : a.vs)[page * a.H + h];
  const int8_t* p = (is_k ? a.kc : a.vc) + (((page * a.H + h) << a.shift) + r) * a.d + c * 8;
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = s * (float)(int8_t)(w.x >> (8 * j));
    v[4 + j] = s * (float)(int8_t)(w.y >> (8 * j));
  }
  *reinterpret_cast<uint4*>(out + (row * a.H + h) * a.d + c * 8) =
      make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]),
                 bf16x2_bits(v[6], v[7]));
}

// ---------------------------------------------------------------- decode attention
//
// q8_decode_kernel<T, D>: HBM-bound (2 D bytes per token and head against 4 D
// operations), so the codes never become floats one by one:
//   scores   q is split once per item into three 7-bit integers, q = qs (q1 2^14 + q2 2^7
//            + q3), and the dot products of four codes are one instruction each, exact in
//            int32 (dp4a); the page's scale multiplies the finished score.
//   values   a token's weight times its page's value scale, relative to the largest so
//            far, is a 24-bit integer; its three bytes, of four tokens each, meet the codes
//            of four tokens and one dim in dp4a, exact in int32 until a new largest weight
//            rescales the sum in fp32.
// About 1.5 instructions per code instead of the five of convert-and-multiply.
//
// Work: the tokens of all (sequence, head) items, in tiles of 4 KB of keys, divided among
// the blocks from the lengths on the device, so that uneven sequences and few long ones
// load every SM alike (see "the block's range").  Warps take a block's tiles in turn, each
// with a ring of its own filled by bulk copies, so no warp waits for another inside an
// item.  Pieces of one item leave partials; the last block to bring one merges them in
// order.

constexpr int kQ8Warps = 4;
constexpr int kQ8Threads = 32 * kQ8Warps;
constexpr int kQ8BlocksPerSm = 3;
constexpr int kQ8Stages = 2;
constexpr int kQ8MinTiles = 4;              // tiles worth a block
constexpr int kQ8FlushGroups = 8192;        // 4 * 255 * 128 per group and dim stays below 2^31
constexpr float kQ8Weight = 16777215.f;     // 2^24 - 1
constexpr float kQ8SmallRef = 1e-31f;       // least reference of the weights

template <int D>
struct Q8Shape {
  static constexpr int kGroups = D == 96 ? 2 : 256 / D;     // 16-token groups per tile
  static constexpr int kTile = 16 * kGroups;                // tokens per tile
  static constexpr int kWords = D / 32;                     // 4-code words per lane and row
  static constexpr int kGroupBytes = 16 * D;
  static constexpr int kHalf = kGroups * kGroupBytes;       // keys of a stage, then its values
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kRing = kQ8Stages * kStage;
  // shared memory: rings, warp partials, rotated q, barriers
  static constexpr int kPartOff = kQ8Warps * kRing;
  static constexpr int kQOff = kPartOff + kQ8Warps * (D + 4) * 4;
  static constexpr int kBarOff = kQOff + D * 4;
  static constexpr int kBytes = kBarOff + kQ8Warps * kQ8Stages * 8;
};

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// sum of four products, unsigned bytes of a with signed bytes of b
__device__ __forceinline__ int dp4a_us(uint32_t a, uint32_t b, int c) {
  int d;
  asm("dp4a.u32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

template <int W>
__device__ __forceinline__ void load_words(const unsigned char* p, uint32_t* w) {
  if constexpr (W == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x;
    w[1] = u.y;
    w[2] = u.z;
    w[3] = u.w;
  } else if constexpr (W == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x;
    w[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
}

// Length of sequence b, clamped into its block table.
__device__ __forceinline__ int q8_length(const Q8DecodeArgs& a, int b, bool tell) {
  const long long cap = (long long)a.max_pages << a.shift;
  const int n = a.ctx_len[b];
  if (n >= 0 && n <= cap) return n;
  if (tell) atomicOr(a.status, LLA_STATUS_CTX_RANGE);
  return n < 0 ? 0 : (int)cap;
}

// What a block works on: tiles [t0, t1) of an item (sequence b, head h of n tokens).
struct Q8Item {
  int b, h, n, t0, t1;
  int c0, pieces;       // first block with a piece of the item, and how many there are
  int slot, first_slot; // partial slot (of two per block) of this block's and of c0's piece
};

__device__ __forceinline__ long long q8_div(long long x, int q) {
  return x >> 32 ? x / q : (long long)((uint32_t)x / (uint32_t)q);
}

// Sums over the block before this thread and in all, of four ints each (0 <= sums < 2^31).
struct Int4Scan {
  int before[4], total[4];
};
__device__ __forceinline__ Int4Scan block_scan4(const int* v, int (*sums)[4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = v[j];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x[j], o);
      if (lane >= o) x[j] += y;
    }
    if (lane == 31) sums[warp][j] = x[j];
  }
  __syncthreads();
  Int4Scan r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r.before[j] = x[j] - v[j];
    r.total[j] = 0;
#pragma unroll
    for (int w = 0; w < kQ8Warps; ++w) {
      if (w < warp) r.before[j] += sums[w][j];
      r.total[j] += sums[w][j];
    }
  }
  return r;
}

template <typename T, int D>
__global__ void __launch_bounds__(kQ8Threads, kQ8BlocksPerSm) q8_decode_kernel(Q8DecodeArgs a) {
  using S = Q8Shape<D>;
  constexpr int W = S::kWords;
  extern __shared__ __align__(128) unsigned char sm[];
  float* parts = reinterpret_cast<float*>(sm + S::kPartOff);      // [warps][4 + D]
  float* qs = reinterpret_cast<float*>(sm + S::kQOff);
  __shared__ long long sums64[kQ8Warps];
  __shared__ int sums4[kQ8Warps][4];
  __shared__ long long start_at;      // units (aligned: pieces) before the first item's sequence
  __shared__ int start_b;
  __shared__ int abort_word, is_last, told;
  __shared__ float self_score;
  volatile int* abort_flag = &abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = blockIdx.x;
  unsigned char* ring = sm + warp * S::kRing;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kBarOff) + warp * kQ8Stages;

  // ---------------------------------------------------------------- the block's range
  // Units: one per tile and head, one for an empty item.  When the grid can give every
  // item blocks of its own, each block gets one piece of one item (`aligned`: pieces of up
  // to q tiles, for the least q of four that fits the grid); otherwise range c is
  // units [c q, c q + q) and may hold the end of one item, whole ones and a beginning.
  const int per = (a.B + kQ8Threads - 1) / kQ8Threads;
  const int seg0 = min(tid * per, a.B), seg1 = min(seg0 + per, a.B);
  auto tiles_of = [&](int b, bool tell) {
    return max(1, (int)(((long long)q8_length(a, b, tell) + S::kTile - 1) / S::kTile));
  };
  long long mine = 0;
  for (int b = seg0; b < seg1; ++b) mine += tiles_of(b, c == 0);
  if (tid == 0) {
    abort_word = 0;
    told = 0;
    start_b = 0;
    start_at = 0;
  }
  if (lane == 0) {
    for (int s = 0; s < kQ8Stages; ++s) sm100::mbar_init(&bars[s], 1);
    sm100::fence_mbar_init();
  }
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) sums64[warp] = upto;
  __syncthreads();
  long long before = upto - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kQ8Warps; ++w) {
    if (w < warp) before += sums64[w];
    total += sums64[w];
  }
  const long long units = total * a.H;
  int q = max(kQ8MinTiles, (int)q8_div(units + gridDim.x - 1, gridDim.x));
  bool aligned = false;
  int blocks, start_pieces = 0, mine_pieces = 0;
  if ((long long)a.B * a.H <= gridDim.x) {
    int qj[4], v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) qj[j] = q + (q * j + 3) / 4;
    for (int b = seg0; b < seg1; ++b) {
      const int tiles = tiles_of(b, false);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += min((tiles + qj[j] - 1) / qj[j], (int)gridDim.x + 1);
    }
    const Int4Scan sc = block_scan4(v, sums4);
#pragma unroll
    for (int j = 3; j >= 0; --j)
      if ((long long)sc.total[j] * a.H <= gridDim.x) {
        aligned = true;
        q = qj[j];
        blocks = sc.total[j] * a.H;
        start_pieces = sc.before[j];
        mine_pieces = v[j];
      }
  }
  if (!aligned) blocks = (int)q8_div(units + q - 1, q);
  if (c >= blocks) return;
  {
    const long long x = aligned ? c : (long long)c * q;
    long long at = (aligned ? start_pieces : before) * a.H;
    if (x >= at && x < at + (aligned ? mine_pieces : mine) * a.H) {
      int b = seg0;
      for (; b < seg1; ++b) {
        const int tiles = tiles_of(b, false);
        const long long len = (long long)(aligned ? (tiles + q - 1) / q : tiles) * a.H;
        if (x < at + len) break;
        at += len;
      }
      start_b = b;
      start_at = at;
    }
  }
  __syncthreads();

  // ---------------------------------------------------------------- its items
  const int r = lane >> 3, col = lane & 7;          // token row of a group of four, dims' eighth
  uint32_t used = 0;                                // tiles this warp has put through its ring
  bool aborted = false;
  long long seq_at = start_at, u = (long long)c * q;   // range: first unit of sequence b, next unit
  const long long u1 = min(u + q, units);
  Q8Item it;
  it.b = start_b;
  // the item that unit u lies in (range), or the block's piece (aligned)
  auto find_item = [&]() {
    if (aligned) {
      it.n = q8_length(a, it.b, false);
      const int tiles = tiles_of(it.b, false), pieces = (tiles + q - 1) / q;
      const int k = c - (int)seq_at;
      it.h = k / pieces;
      const int part = k - it.h * pieces, base = tiles / pieces, rem = tiles - base * pieces;
      it.t0 = part * base + min(part, rem);
      it.t1 = it.t0 + base + (part < rem ? 1 : 0);
      it.c0 = c - part;
      it.pieces = pieces;
      it.slot = it.first_slot = 0;
      return;
    }
    int tiles;
    for (;;) {
      it.n = q8_length(a, it.b, false);
      tiles = tiles_of(it.b, false);
      if (u < seq_at + (long long)tiles * a.H) break;
      seq_at += (long long)tiles * a.H;
      ++it.b;
    }
    it.h = (int)q8_div(u - seq_at, tiles);
    const long long item0 = seq_at + (long long)it.h * tiles;
    it.t0 = (int)(u - item0);
    it.t1 = (int)min((long long)tiles, u1 - item0);
    it.c0 = (int)q8_div(item0, q);
    it.pieces = (int)q8_div(item0 + tiles - 1, q) - it.c0 + 1;
    // slot 0: the first item of a block's range, slot 1: a later one, which is its last
    it.slot = u == (long long)c * q ? 0 : 1;
    it.first_slot = (long long)it.c0 * q == item0 ? 0 : 1;
    u = item0 + it.t1;
  };

  // Lane g < kGroups looks after group g of each tile: its page id (loaded two tiles
  // ahead of the tile's use), its copies, its scales (loaded one tile ahead).
  const size_t page_step = (size_t)a.H << a.shift;             // rows per page, all heads
  bool bad = false;
  auto group_id = [&](int t) {
    if (lane >= S::kGroups || t >= it.t1) return -1;
    const int tok = t * S::kTile + lane * 16;                  // lengths stay below 2^31
    return tok < it.n ? __ldg(a.block_table + (long long)it.b * a.max_pages + (tok >> a.shift)) : -1;
  };
  auto checked = [&](int t, int id) {                          // -1 for what is not there
    const bool there = lane < S::kGroups && t < it.t1 && t * S::kTile + lane * 16 < it.n;
    const bool ok = there && id >= 0 && id < a.n_pages;
    bad |= there && !ok;
    return ok ? id : -1;
  };
  auto issue = [&](int t, int id, uint32_t seq) {              // tile t, the warp's seq-th
    if (t >= it.t1) return;
    const int s = seq % kQ8Stages;
    const unsigned live = __ballot_sync(0xffffffffu, id >= 0);
    if (lane == 0) sm100::mbar_arrive_expect_tx(&bars[s], __popc(live) * 2 * S::kGroupBytes);
    __syncwarp();
    if (id >= 0) {
      const int tok = t * S::kTile + lane * 16;
      const size_t run = (id * page_step + ((size_t)it.h << a.shift) +
                          (tok & ((1 << a.shift) - 1))) * D;
      unsigned char* st = ring + s * S::kStage + lane * S::kGroupBytes;
      sm100::bulk_load(st, a.kc + run, S::kGroupBytes, &bars[s]);
      sm100::bulk_load(st + S::kHalf, a.vc + run, S::kGroupBytes, &bars[s]);
    }
  };
  auto scale_of = [&](const float* scales, int id) {
    return id >= 0 ? __ldg(scales + (size_t)id * a.H + it.h) : 0.f;
  };
  int id0 = -1, id1 = -1, id2 = -1;                            // tiles t, t + 4, t + 8
  float ks0 = 0.f, vs0 = 0.f;
  auto start_item = [&]() {
    const int first = it.t0 + warp;
    id0 = group_id(first);
    id1 = group_id(first + kQ8Warps);
    id2 = group_id(first + 2 * kQ8Warps);
    id0 = checked(first, id0);
    id1 = checked(first + kQ8Warps, id1);
    if (!aborted) {
      issue(first, id0, used);
      issue(first + kQ8Warps, id1, used + 1);
    }
    ks0 = scale_of(a.ks, id0);
    vs0 = scale_of(a.vs, id0);
  };
  find_item();
  start_item();
  for (bool more = true; more;) {
    const int first = it.t0 + warp;
    const size_t bh = (size_t)it.b * a.H + it.h;

    // q rotated at q_pos, into shared memory; the in-flight token's score, which needs no
    // rotation, both sitting at q_pos
    float v_own = 0.f;
    if (tid < 32) {
      float acc = 0.f;
      if (tid < D / 8) {
        const bool turn = a.rope != nullptr;
        const RowChunk rc = row_chunk(tid, D, a.rd, turn ? a.layout : LLA_ROPE_INTERLEAVED);
        float v[8], k[8];
        load_chunk(static_cast<const T*>(a.q) + bh * D, rc, v);
        if (a.k_self) {
          load_chunk(static_cast<const T*>(a.k_self) + bh * D, rc, k);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc = fmaf(v[j], k[j], acc);
        }
        if (turn) {
          const int pos = checked_position(a.q_pos[it.b], a.rope_max_pos, nullptr, false);
          if (tid == 0 && pos != a.q_pos[it.b]) {
            atomicOr(a.status, LLA_STATUS_POSITION_RANGE);
            told = 1;
          }
          rotate_chunk(a.rope + (size_t)pos * (a.rd / 2), rc, 1.f, v);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          qs[rc.lo + j] = v[j];
          qs[rc.hi + j] = v[4 + j];
        }
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
      if (tid == 0) self_score = acc * a.kappa;
    }
    if (a.k_self && tid < D) v_own = as_float(static_cast<const T*>(a.v_self)[bh * D + tid]);
    __syncthreads();
    // this lane's dims as three signed digits of 7 bits, the largest |q| at 127 * 2^14
    uint32_t q1[W], q2[W], q3[W];
    float score_scale;
    bool strange = false;                                       // a NaN or an infinity in q
    {
      float v[4 * W], amax = 0.f;
#pragma unroll
      for (int j = 0; j < 4 * W; ++j) {
        v[j] = qs[col * 4 * W + j];
        amax = fmaxf(amax, fabsf(v[j]));
        strange |= !(fabsf(v[j]) <= FLT_MAX);
      }
      strange = __any_sync(0xffffffffu, strange);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      constexpr float kTop = 127.f * 16384.f;
      const float inv = amax > kQ8Tiny ? kTop / amax : 0.f;
      score_scale = strange ? 0.f : a.kappa * amax / kTop;      // strange: pl becomes NaN below
#pragma unroll
      for (int w = 0; w < W; ++w) {
        q1[w] = q2[w] = q3[w] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          int x = __float2int_rn(v[4 * w + j] * inv);
          const int lo = ((x + 64) & 127) - 64;
          x = (x - lo) >> 7;
          const int mid = ((x + 64) & 127) - 64;
          x = (x - mid) >> 7;
          q1[w] |= (uint32_t)(x & 255) << (8 * j);
          q2[w] |= (uint32_t)(mid & 255) << (8 * j);
          q3[w] |= (uint32_t)(lo & 255) << (8 * j);
        }
      }
    }

    // Sums are relative to 2^m, m the largest score so far: l of 2^(s - m), o of
    // 2^(s - m) v.  acc holds weights w = 2^(s - m) vs / R * (2^24 - 1) times codes, R
    // the reference that no weight since the last flush exceeds.  A larger weight flushes
    // acc into o; a larger score rescales l, o and R.
    float m = -INFINITY, l = 0.f, R = 0.f, wf = 0.f;             // wf = (2^24 - 1) / R
    float o[4 * W];
    int acc1[4 * W], acc2[4 * W], acc3[4 * W];
#pragma unroll
    for (int j = 0; j < 4 * W; ++j) {
      o[j] = 0.f;
      acc1[j] = acc2[j] = acc3[j] = 0;
    }
    int groups = 0;
    auto flush = [&]() {
      const float f = R * (1.f / kQ8Weight);
#pragma unroll
      for (int j = 0; j < 4 * W; ++j) {
        o[j] = fmaf(f, fmaf((float)acc1[j], 65536.f, fmaf((float)acc2[j], 256.f, (float)acc3[j])),
                    o[j]);
        acc1[j] = acc2[j] = acc3[j] = 0;
      }
      groups = 0;
    };

    const int i_own = ((col >> 1) & 1) | ((col >> 1) & 2);      // row group this lane ends up with
    uint32_t seq = used;
    for (int t = first; t < it.t1 && !aborted; t += kQ8Warps, ++seq) {
      const int s = seq % kQ8Stages;
      const unsigned live = __ballot_sync(0xffffffffu, id0 >= 0);
      // scales of the next tile, page ids of the one after it
      const float ks1 = scale_of(a.ks, id1), vs1 = scale_of(a.vs, id1);
      id2 = checked(t + 2 * kQ8Warps, id2);
      const int id3 = group_id(t + 3 * kQ8Warps);
      if (!sm100::mbar_wait(&bars[s], (seq / kQ8Stages) & 1u, abort_flag)) {
        // copies already issued land before the block can end
        for (int k = 0; k < kQ8Stages && t + k * kQ8Warps < it.t1; ++k) {
          const unsigned long long w0 = sm100::global_timer_ns();
          while (!sm100::mbar_try_wait(&bars[(seq + k) % kQ8Stages], ((seq + k) / kQ8Stages) & 1u) &&
                 sm100::global_timer_ns() - w0 < sm100::kWaitTimeoutNs) {
          }
        }
        aborted = true;
        break;
      }
      const unsigned char* st = ring + s * S::kStage + r * D + col * 4 * W;
      const int rows_left = it.n - t * S::kTile - r - 4 * i_own;   // of this lane's row of group 0
#pragma unroll
      for (int g = 0; g < S::kGroups; ++g) {
        if (!(live >> g & 1)) continue;                         // warp-uniform
        const float ksc = __shfl_sync(0xffffffffu, ks0, g) * score_scale;
        const float vsc = __shfl_sync(0xffffffffu, vs0, g);
        const unsigned char* kp = st + g * S::kGroupBytes;
        float part[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t kw[W];
          load_words<W>(kp + i * 4 * D, kw);
          int s1 = 0, s2 = 0, s3 = 0;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            s1 = __dp4a((int)kw[w], (int)q1[w], s1);
            s2 = __dp4a((int)kw[w], (int)q2[w], s2);
            s3 = __dp4a((int)kw[w], (int)q3[w], s3);
          }
          part[i] = fmaf((float)(s1 * 128 + s2), 128.f, (float)s3);
        }
        // sum over the row's eight lanes; a lane keeps row r + 4 i_own
        float x0 = (col & 4 ? part[2] : part[0]) +
                   __shfl_xor_sync(0xffffffffu, col & 4 ? part[0] : part[2], 4);
        const float x1 = (col & 4 ? part[3] : part[1]) +
                         __shfl_xor_sync(0xffffffffu, col & 4 ? part[1] : part[3], 4);
        x0 = (col & 2 ? x1 : x0) + __shfl_xor_sync(0xffffffffu, col & 2 ? x0 : x1, 2);
        x0 += __shfl_xor_sync(0xffffffffu, x0, 1);
        const float sc = rows_left > 16 * g ? x0 * ksc : -INFINITY;
        if (__any_sync(0xffffffffu, sc > m)) {
          float mt = sc;
#pragma unroll
          for (int off = 2; off < 32; off <<= 1)
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
          const float f = exp2f(m - mt);                        // 0 the first time
          m = mt;
          l *= f;
          R *= f;
#pragma unroll
          for (int j = 0; j < 4 * W; ++j) o[j] *= f;
          if (R < kQ8SmallRef) {                                // 1 / R stays finite
            flush();
            R = kQ8SmallRef;
          }
          wf = kQ8Weight / R;
        }
        const float p = exp2f(sc - m);
        l += col & 1 ? 0.f : p;
        if (vsc > R || groups >= kQ8FlushGroups) {              // p <= 1
          flush();
          R = fmaxf(R, vsc);
          wf = kQ8Weight / R;
        }
        ++groups;
        const uint32_t wt = __float2uint_rn(fminf(p * (vsc * wf), kQ8Weight));
        // the four rows' weights, then their bytes: hi, mid, lo words of four tokens
        const uint32_t w2 = __shfl_xor_sync(0xffffffffu, wt, 2);
        const uint32_t e0 = col & 2 ? w2 : wt, e1 = col & 2 ? wt : w2;
        const uint32_t f0 = __shfl_xor_sync(0xffffffffu, e0, 4);
        const uint32_t f1 = __shfl_xor_sync(0xffffffffu, e1, 4);
        const uint32_t g0 = col & 4 ? f0 : e0, g1 = col & 4 ? f1 : e1;
        const uint32_t g2 = col & 4 ? e0 : f0, g3 = col & 4 ? e1 : f1;
        const uint32_t a01 = __byte_perm(g0, g1, 0x5140), a23 = __byte_perm(g2, g3, 0x5140);
        const uint32_t h01 = __byte_perm(g0, g1, 0x0062), h23 = __byte_perm(g2, g3, 0x0062);
        const uint32_t wlo = __byte_perm(a01, a23, 0x5410), wmid = __byte_perm(a01, a23, 0x7632);
        const uint32_t whi = __byte_perm(h01, h23, 0x5410);
        uint32_t vw[4][W];
#pragma unroll
        for (int i = 0; i < 4; ++i) load_words<W>(kp + S::kHalf + i * 4 * D, vw[i]);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          // four rows of four dims, turned into four dims of four rows
          const uint32_t y0 = __byte_perm(vw[0][w], vw[1][w], 0x5140);
          const uint32_t y1 = __byte_perm(vw[2][w], vw[3][w], 0x5140);
          const uint32_t y2 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
          const uint32_t y3 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
          const uint32_t dim[4] = {__byte_perm(y0, y1, 0x5410), __byte_perm(y0, y1, 0x7632),
                                   __byte_perm(y2, y3, 0x5410), __byte_perm(y2, y3, 0x7632)};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc1[4 * w + j] = dp4a_us(whi, dim[j], acc1[4 * w + j]);
            acc2[4 * w + j] = dp4a_us(wmid, dim[j], acc2[4 * w + j]);
            acc3[4 * w + j] = dp4a_us(wlo, dim[j], acc3[4 * w + j]);
          }
        }
      }
      __syncwarp();                                             // the stage is read
      issue(t + kQ8Stages * kQ8Warps, id2, seq + kQ8Stages);
      id0 = id1;
      id1 = id2;
      id2 = id3;
      ks0 = ks1;
      vs0 = vs1;
    }
    if (it.t1 > first) used += (it.t1 - first + kQ8Warps - 1) / kQ8Warps;
    if (__any_sync(0xffffffffu, bad) && lane == 0) {
      atomicOr(a.status, LLA_STATUS_PAGE_RANGE);
      told = 1;
    }
    bad = false;
    // the next item's first tiles are on their way while this one is merged
    const Q8Item now = it;
    more = !aligned && u < u1;
    if (more) {
      find_item();
      start_item();
    }

    // ---------------------------------------------------------------- merge the warps
    flush();
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    l += __shfl_xor_sync(0xffffffffu, l, 4);
#pragma unroll
    for (int off = 8; off < 32; off <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
      for (int j = 0; j < 4 * W; ++j) o[j] += __shfl_xor_sync(0xffffffffu, o[j], off);
    }
    float* pw = parts + warp * (D + 4);
    if (r == 0) {
#pragma unroll
      for (int j = 0; j < 4 * W; ++j) pw[4 + col * 4 * W + j] = o[j];
      if (lane == 0) {
        pw[0] = m;
        pw[1] = l;
      }
    }
    __syncthreads();
    float pm = -INFINITY, pl = 0.f, po = 0.f;
#pragma unroll
    for (int w = 0; w < kQ8Warps; ++w) pm = fmaxf(pm, parts[w * (D + 4)]);
    if (pm > -INFINITY) {
#pragma unroll
      for (int w = 0; w < kQ8Warps; ++w) {
        const float f = exp2f(parts[w * (D + 4)] - pm);
        pl = fmaf(parts[w * (D + 4) + 1], f, pl);
        if (tid < D) po = fmaf(parts[w * (D + 4) + 4 + tid], f, po);
      }
    }

    // ---------------------------------------------------------------- the item's other blocks
    bool finish = true;
    if (now.pieces > 1) {
      float* mine_p = a.partials + (size_t)(2 * c + now.slot) * (D + 2);
      if (tid < D) __stcg(mine_p + 2 + tid, po);
      if (tid == 0) {
        __stcg(mine_p, pm);
        __stcg(mine_p + 1, pl);
      }
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        const unsigned got = atomicAdd(a.piece_counters + now.c0, 1u);
        is_last = got == (unsigned)now.pieces - 1;
        if (is_last) a.piece_counters[now.c0] = 0;
        __threadfence();
      }
      __syncthreads();
      finish = is_last;
      if (finish) {
        // in the order of the pieces, four at a time
        pm = -INFINITY;
        pl = po = 0.f;
        for (int k0 = 0; k0 < now.pieces; k0 += 4) {
          float mm[4], ll[4], oo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int i = k0 + k;
            const float* pp = a.partials +
                (size_t)(2 * (now.c0 + i) + (i == 0 ? now.first_slot : 0)) * (D + 2);
            mm[k] = i < now.pieces ? __ldcg(pp) : -INFINITY;
            ll[k] = i < now.pieces ? __ldcg(pp + 1) : 0.f;
            oo[k] = i < now.pieces && tid < D ? __ldcg(pp + 2 + tid) : 0.f;
          }
          const float top = fmaxf(fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3])), pm);
          if (!(top > -INFINITY)) continue;
          const float f0 = exp2f(pm - top);
          pl *= f0;
          po *= f0;
          pm = top;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float f = exp2f(mm[k] - top);
            pl = fmaf(ll[k], f, pl);
            po = fmaf(oo[k], f, po);
          }
        }
      }
    }
    if (finish) {
      if (a.k_self) {
        const float self = self_score, top = fmaxf(pm, self);
        const float f = pm > -INFINITY ? exp2f(pm - top) : 0.f, fs = exp2f(self - top);
        pl = fmaf(pl, f, fs);
        po = fmaf(po, f, fs * v_own);
      }
      if (strange && pl != 0.f) pl = NAN;
      if (tid < D) put(static_cast<T*>(a.out) + bh * D + tid, pl == 0.f ? 0.f : po / pl);
    }
    __syncthreads();                                            // parts, qs and is_last are free
  }
  if (aborted && lane == 0) {
    atomicOr(a.status, LLA_STATUS_TIMEOUT);
    told = 1;
  }
  // the last block to finish publishes the call's status word and re-arms the counter
  __syncthreads();
  if (tid == 0) {
    if (told || c == 0) __threadfence();                        // block 0 tells of lengths
    if (atomicAdd(a.counter, 1u) == (unsigned)blocks - 1) {
      __threadfence();
      a.status[1] = atomicExch(&a.status[0], 0);
      atomicExch(a.counter, 0u);
    }
  }
}

int q8_max_blocks() { return sm_count() * kQ8BlocksPerSm; }

template <typename T, int D>
cudaError_t launch_decode_td(const Q8DecodeArgs& a, cudaStream_t s) {
  using S = Q8Shape<D>;
  cudaError_t e = cudaFuncSetAttribute(q8_decode_kernel<T, D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != cudaSuccess) return e;
  const long long tiles =
      (((long long)a.max_pages << a.shift) + S::kTile - 1) / S::kTile;
  // at most one block per kQ8MinTiles tiles of every item
  const long long per_item = std::max(1LL, (tiles + kQ8MinTiles - 1) / kQ8MinTiles);
  const long long grid = std::min<long long>((long long)a.B * a.H * per_item, q8_max_blocks());
  q8_decode_kernel<T, D><<<(unsigned)grid, kQ8Threads, S::kBytes, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_decode_t(const Q8DecodeArgs& a, cudaStream_t s) {
  switch (a.d) {
    case 32: return launch_decode_td<T, 32>(a, s);
    case 64: return launch_decode_td<T, 64>(a, s);
    case 96: return launch_decode_td<T, 96>(a, s);
    case 128: return launch_decode_td<T, 128>(a, s);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace

cudaError_t launch_q8_append(const Q8AppendArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.n_tok >> a.shift) + 2 * a.B), a.H, 2);
  if (a.bf16)
    q8_append_kernel<__nv_bfloat16><<<grid, kAppendThreads, 0, s>>>(a);
  else
    q8_append_kernel<float><<<grid, kAppendThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_q8_read(const Q8ReadArgs& a, cudaStream_t s) {
  const long long n = a.n_rows * a.H * (a.d / 8);
  q8_read_kernel<<<dim3((unsigned)((n + 255) / 256), 2), 256, 0, s>>>(a);
  return cudaGetLastError();
}

// Workspace: header, one counter per block, two partials per block.
size_t q8_decode_counters_at() { return kWsHeader; }
size_t q8_decode_partials_at() { return kWsHeader + align_up((size_t)q8_max_blocks() * 4, 256); }
size_t q8_decode_ws_bytes(const lla_cfg& c, int, int) {
  return q8_decode_partials_at() + (size_t)q8_max_blocks() * 2 * (c.d_head + 2) * 4;
}

cudaError_t launch_q8_decode(const Q8DecodeArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_decode_t<__nv_bfloat16>(a, s) : launch_decode_t<float>(a, s);
}

}  // namespace lla

// Decode attention over the paged 8-bit cache (its layout and scales: lla_q8.cu).
//
// q8_decode_kernel<T, D>: HBM-bound (2 D bytes per token and head against 4 D operations):
//   scores   a lane's 16 dims of q (12 of 96) are split once per item into the three bytes of
//            24-bit integers, q = qs (q1 2^16 + q2 2^8 + q3), and the dot products of four codes
//            are one instruction each, exact in int32 (dp4a); a lane's sum meets its own qs, the
//            finished score the page's scale.  Each element of q is held to 2^-24 of the largest
//            of its 16: what fp32 sums with that element round away too, unless its keys are
//            zero.  Four 7-bit integers of the whole head's largest element cost 5 %.
//   values   fp32: a code becomes a float by a byte permutation and half of a packed add, and
//            meets its token's weight p * scale in half of a packed fma.  Weights as integers
//            (dp4a on the codes) take half the instructions, but are fixed point: beside one
//            heavy token, or a page of large values, whatever weighs 2^-24 of it is lost, while
//            the softmax's sum still counts it.
//
// Work: the tokens of all (sequence, head) items, in tiles of 4 KB of keys, divided among
// the blocks from the lengths on the device, so that uneven sequences and few long ones
// load every SM alike (see "the block's range").  Warps take a block's tiles in turn, each
// with a ring of its own filled by bulk copies, so no warp waits for another inside an
// item.  Pieces of one item leave partials; the last block to bring one merges them in
// order.

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "lla_internal.cuh"
#include "lla_rows.cuh"
#include "lla_sm100.cuh"

namespace lla {
namespace {

constexpr int kQ8Warps = 4;
constexpr int kQ8Threads = 32 * kQ8Warps;
constexpr int kQ8Stages = 2;
constexpr int kQ8MinTiles = 8;              // tiles worth a block
constexpr int kQ8ItemBlock = 12;            // start and merge of an item in tiles, for a block
constexpr int kQ8ItemWarp = 4;              // and for a warp that has it to itself

template <int D>
struct Q8Shape {
  // A row's lanes hold 16 of its codes each (12 of 96); a warp's load covers kRows rows, and
  // four of them are a group, the unit of the arithmetic.  kSubs 16-token blocks, each in
  // one page, make a group; two groups make a tile.
  static constexpr int kLanes = D == 96 ? 8 : D / 16;
  // Registers bound the blocks per SM: two take 180 a thread; three of 168 fit without spills and
  // are better for some sizes and worse for others (16 heads of 128, us with two against three:
  // 64 x 512 tokens 30 and 37, 1024 x 64 88 and 74, 128 x 1000 97 and 93, 256 x 4096 633 and 651,
  // repeated under the power limit 761 and 720).  Lanes of 96 hold 12 codes and need fewer.
  static constexpr int kBlocksPerSm = D == 96 ? 3 : 2;
  static constexpr int kWords = D / kLanes / 4;             // 4-code words per lane and row
  static constexpr int kRows = 32 / kLanes;
  static constexpr int kGroup = 4 * kRows;
  static constexpr int kSubs = kGroup / 16;
  static constexpr int kScores = kGroup > 32 ? 2 : 1;       // scores per lane
  static constexpr int kParts = 2 * kSubs;                  // 16-token blocks of a tile
  static constexpr int kTile = 16 * kParts;                 // tokens per tile
  static constexpr int kPartBytes = 16 * D;
  static constexpr int kHalf = kParts * kPartBytes;         // keys of a stage, then its values
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kRing = kQ8Stages * kStage;
  // shared memory: rings, warp partials, rotated q, barriers
  static constexpr int kPartOff = kQ8Warps * kRing;
  static constexpr int kQOff = kPartOff + kQ8Warps * (D + 4) * 4;
  static constexpr int kBarOff = kQOff + kQ8Warps * D * 4;
  static constexpr int kBytes = kBarOff + kQ8Warps * kQ8Stages * 8;
};

// 2^x of x <= 0: results below 2^-126 are zero, others within two units in the last place.
__device__ __forceinline__ float exp2_down(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// sum of four products, signed bytes of a with unsigned bytes of b
__device__ __forceinline__ int dp4a_su(uint32_t a, uint32_t b, int c) {
  int d;
  asm("dp4a.s32.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// Two floats in a register pair, and arithmetic on both, each rounded as by itself.
typedef unsigned long long float_pair;
__device__ __forceinline__ float_pair pair_of(float a, float b) {
  float_pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(float_pair p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ float_pair add2(float_pair a, float_pair b) {
  float_pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float_pair mul2(float_pair a, float_pair b) {
  float_pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float_pair fma2(float_pair a, float_pair b, float_pair c) {
  float_pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Codes j and j + 1 of a word whose sign bits are flipped, as floats: 2^23 + 128 + code has the
// byte as its lowest mantissa bits.
template <int J>
__device__ __forceinline__ float_pair codes2(uint32_t flipped) {
  const float lo = __uint_as_float(__byte_perm(flipped, 0x4b000000u, 0x7440 + J));
  const float hi = __uint_as_float(__byte_perm(flipped, 0x4b000000u, 0x7441 + J));
  return add2(pair_of(lo, hi), pair_of(-8388736.f, -8388736.f));
}

template <int W>
__device__ __forceinline__ void load_words(const unsigned char* p, uint32_t* w) {
  if constexpr (W == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x;
    w[1] = u.y;
    w[2] = u.z;
    w[3] = u.w;
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
}

// The call's counter word: blocks that finished, and the status bits above them, so that the
// last block learns of every bit from the count that it must read anyway.
constexpr int kQ8StatusShift = 16;
__device__ __forceinline__ void tell_status(const Q8DecodeArgs& a, uint32_t bits) {
  atomicOr(a.counter, bits << kQ8StatusShift);
}

// Largest of the lanes' values.
__device__ __forceinline__ float warp_largest(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// a / b for the invariant divisor of `by`, a < 2^31.
__device__ __forceinline__ uint32_t divide(uint32_t a, const Q8Divisor& by) {
  return by.factor ? __umulhi(a, by.factor) >> by.shift : a;
}

// Pieces of up to about 1 / inv_q tiles, at most `most` of them.
__device__ __forceinline__ uint32_t pieces_of(uint32_t tiles, float inv_q, uint32_t most) {
  return max(1, (int)ceilf(fminf((float)tiles * inv_q, (float)most)));
}

// Length of sequence b, clamped into its block table.
__device__ __forceinline__ int q8_length(const Q8DecodeArgs& a, int b, bool tell) {
  const long long cap = (long long)a.max_pages << a.shift;
  const int n = a.ctx_len[b];
  if (n >= 0 && n <= cap) return n;
  if (tell) tell_status(a, LLA_STATUS_CTX_RANGE);
  return n < 0 ? 0 : (int)cap;
}

// What a block (or a warp) works on: tiles [t0, t1) of an item, sequence b's head h.
struct Q8Item {
  int b, h, n, t0, t1;
  int c0, pieces;       // first block with a piece of the item, and how many there are
  int slot, first_slot; // partial slot (of two per block) of this block's and of c0's piece
};

template <typename T, int D>
__global__ void __launch_bounds__(kQ8Threads, Q8Shape<D>::kBlocksPerSm)
q8_decode_kernel(Q8DecodeArgs a) {
  using S = Q8Shape<D>;
  constexpr int W = S::kWords;
  extern __shared__ __align__(128) unsigned char sm[];
  float* parts = reinterpret_cast<float*>(sm + S::kPartOff);      // [warps][4 + D]
  __shared__ uint32_t sums[kQ8Warps];
  __shared__ int longest[kQ8Warps];
  __shared__ unsigned long long sums3[kQ8Warps];
  __shared__ uint32_t start_at[kQ8Warps];   // units (aligned: pieces) before the sequence
  __shared__ int start_b[kQ8Warps];         // of a block's, or warp's, first item
  __shared__ int abort_word, is_last;
  volatile int* abort_flag = &abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = blockIdx.x;
  unsigned char* ring = sm + warp * S::kRing;
  float* qs = reinterpret_cast<float*>(sm + S::kQOff) + warp * D;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kBarOff) + warp * kQ8Stages;

  // ---------------------------------------------------------------- the block's range
  // Units: an item's tiles (one for an empty item) after kQ8ItemBlock or kQ8ItemWarp more
  // for its start and merge; the host keeps their number below 2^31.  Three ways to divide
  // them:
  //   aligned   the grid can give every item blocks of its own: each block gets one piece of
  //             one item, of up to q tiles, for the least q of three that fits the grid
  //   ranges    block c gets units [c q, c q + q): the end of one item, whole ones and a
  //             beginning
  //   by warp   many short items: each warp gets the items that begin in its range, whole,
  //             and meets no other warp
  // The one whose busiest warp has least to do is taken.  Of up to 32 sequences every warp
  // finds its range by itself, lane b looking after sequence b (1 x 128 tokens 6.2 -> 5.9 us);
  // more are shared out over the block's threads.
  const bool few = a.B <= 32;
  const int per = (a.B + kQ8Threads - 1) / kQ8Threads;
  const int seg0 = min(tid * per, a.B), seg1 = min(seg0 + per, a.B);
  auto tiles_of = [&](int n) { return max(1, (int)(((uint32_t)n + S::kTile - 1) / S::kTile)); };
  uint32_t mine = 0, before = 0, total = 0;
  int most = 0, n_of_lane = 0, pos_of_lane = 0;
  if (few) {
    if (lane < a.B) {
      n_of_lane = q8_length(a, lane, c == 0 && warp == 0);
      if (a.rope) pos_of_lane = a.q_pos[lane];
      mine = tiles_of(n_of_lane);
    }
  } else {
    for (int b = seg0; b < seg1; ++b) {
      const int tiles = tiles_of(q8_length(a, b, c == 0));
      mine += tiles;
      most = max(most, tiles);
    }
  }
  if (tid == 0) abort_word = 0;
  if (lane == 0) {
    for (int s = 0; s < kQ8Stages; ++s) sm100::mbar_init(&bars[s], 1);
    sm100::fence_mbar_init();
  }
  if (few) {
    total = __reduce_add_sync(0xffffffffu, mine);
    most = __reduce_max_sync(0xffffffffu, mine);
  } else {
    before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 31) {
      sums[warp] = before;
      longest[warp] = most;
    }
    before -= mine;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQ8Warps; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
      most = max(most, longest[w]);
    }
  }
  const uint32_t H = a.H, items = a.B * H, grid = gridDim.x, warps = grid * kQ8Warps;
  const uint32_t block_units = (total + a.B * kQ8ItemBlock) * H;
  const uint32_t warp_units = (total + a.B * kQ8ItemWarp) * H;
  const uint32_t in_turn = divide(items + warps - 1, a.by_warps);   // items of one warp
  const uint32_t warp_cost =
      min(in_turn * (most + kQ8ItemWarp), divide(warp_units, a.by_warps) + most);
  uint32_t block_cost = divide(block_units, a.by_warps) + kQ8ItemBlock / 2;
  uint32_t q = 0, blocks = 0, start_pieces = 0, mine_pieces = 0;
  float inv_q = 0.f;                        // 1 / q, and a little less (aligned)
  bool aligned = false;
  if (items <= grid) {
    // pieces for three q, in fields of 21 bits: at most 444 sequences of 445 pieces
    const uint32_t q0 = max((uint32_t)kQ8MinTiles, divide(total * H + grid - 1, a.by_grid));
    float inv[3];
#pragma unroll
    for (int j = 0; j < 3; ++j)
      inv[j] = (1.f - 0x1p-20f) / (float)(q0 + j * kQ8ItemBlock / 2);
    if (few) {
#pragma unroll
      for (int j = 2; j >= 0; --j) {
        const uint32_t own = lane < a.B ? pieces_of(mine, inv[j], grid + 1) : 0;
        const uint32_t n = __reduce_add_sync(0xffffffffu, own);
        if (n * H > grid) continue;
        aligned = true;
        q = q0 + j * kQ8ItemBlock / 2;
        inv_q = inv[j];
        blocks = n * H;
        mine_pieces = own;
      }
    } else {
      unsigned long long v = 0;
      for (int b = seg0; b < seg1; ++b) {
        const uint32_t tiles = tiles_of(q8_length(a, b, false));
#pragma unroll
        for (int j = 0; j < 3; ++j)
          v += (unsigned long long)pieces_of(tiles, inv[j], grid + 1) << (21 * j);
      }
      unsigned long long upto = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31) sums3[warp] = upto;
      __syncthreads();
      unsigned long long all = 0;
      upto -= v;
#pragma unroll
      for (int w = 0; w < kQ8Warps; ++w) {
        if (w < warp) upto += sums3[w];
        all += sums3[w];
      }
#pragma unroll
      for (int j = 2; j >= 0; --j) {
        constexpr uint32_t kField = (1u << 21) - 1;
        const uint32_t n = (uint32_t)(all >> (21 * j)) & kField;
        if (n * H > grid) continue;
        aligned = true;
        q = q0 + j * kQ8ItemBlock / 2;
        inv_q = inv[j];
        blocks = n * H;
        start_pieces = (uint32_t)(upto >> (21 * j)) & kField;
        mine_pieces = (uint32_t)(v >> (21 * j)) & kField;
      }
    }
    if (aligned) block_cost = min(q, (uint32_t)most) / kQ8Warps + kQ8ItemBlock / 4;
  }
  const bool by_warp = warp_cost < block_cost;
  const uint32_t units = by_warp ? warp_units : block_units;
  if (by_warp) {
    aligned = false;
    q = divide(units + warps - 1, a.by_warps);
    blocks = (units + kQ8Warps * q - 1) / (kQ8Warps * q);
  } else if (!aligned) {
    q = max((uint32_t)kQ8MinTiles, divide(units + grid - 1, a.by_grid));
    blocks = (units + q - 1) / q;
  }
  if (c >= blocks) return;
  const uint32_t extra = by_warp ? kQ8ItemWarp : kQ8ItemBlock;   // an item's units before its tiles
  const int team = by_warp ? c * kQ8Warps + warp : c;
  const int step = by_warp ? 1 : kQ8Warps, lead = by_warp ? 0 : warp;   // a warp's tiles
  // the sequence that the block's (or each warp's) first unit lies in, and its first unit
  int first_b;
  uint32_t first_at;
  if (few) {
    const uint32_t len = lane < a.B ? (aligned ? mine_pieces : mine + extra) * H : 0;
    uint32_t end = len;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    const uint32_t x = aligned ? c : team * q;
    first_b = min(__popc(__ballot_sync(0xffffffffu, lane < a.B && end <= x)), a.B - 1);
    first_at = __shfl_sync(0xffffffffu, end - len, first_b);
  } else {
    const int teams = by_warp ? kQ8Warps : 1;
    const uint32_t at0 = (aligned ? start_pieces : before + seg0 * extra) * H;
    const uint32_t end0 = at0 + (aligned ? mine_pieces : mine + (seg1 - seg0) * extra) * H;
    for (int w = 0; w < teams; ++w) {
      const uint32_t x = aligned ? c : (c * teams + w) * q;
      if (x < at0 || x >= end0) continue;
      uint32_t at = at0;
      int b = seg0;
      for (; b < seg1 - 1; ++b) {
        const uint32_t tiles = tiles_of(q8_length(a, b, false));
        const uint32_t len = (aligned ? pieces_of(tiles, inv_q, grid + 1) : tiles + extra) * H;
        if (x < at + len) break;
        at += len;
      }
      start_b[w] = b;
      start_at[w] = at;
    }
    __syncthreads();
    first_b = start_b[by_warp ? warp : 0];
    first_at = start_at[by_warp ? warp : 0];
  }
  auto length = [&](int b) {
    return few ? __shfl_sync(0xffffffffu, n_of_lane, b) : q8_length(a, b, false);
  };

  // ---------------------------------------------------------------- its items
  const int r = lane / S::kLanes, col = lane % S::kLanes;      // row of a load, its dims
  uint32_t used = 0;                                // tiles this warp has put through its ring
  bool aborted = false;
  uint32_t u = team * q;                            // next unit
  const uint32_t u1 = min(u + q, units);
  uint32_t seq_at = first_at;                       // first unit (piece) of sequence it.b
  Q8Item it;
  it.b = first_b;
  // the item that unit u lies in, or the block's piece (aligned); false: there is none
  auto find_item = [&]() {
    if (aligned) {
      it.n = length(it.b);
      const uint32_t tiles = tiles_of(it.n), pieces = pieces_of(tiles, inv_q, grid + 1);
      const uint32_t k = c - seq_at;                // below 2^18 here, as c is
      const float inv = __frcp_rn((float)pieces);
      it.h = (int)(((float)k + 0.5f) * inv);
      const uint32_t part = k - it.h * pieces;
      const float each = (float)tiles * inv;
      it.t0 = (int)((float)part * each);
      it.t1 = part + 1 == pieces ? tiles : (uint32_t)((float)(part + 1) * each);
      it.c0 = c - part;
      it.pieces = pieces;
      it.slot = it.first_slot = 0;
      return true;
    }
    while (u < u1) {
      uint32_t len;
      for (;;) {
        it.n = length(it.b);
        len = tiles_of(it.n) + extra;
        if (u < seq_at + len * H) break;
        seq_at += len * H;
        ++it.b;
      }
      it.h = (u - seq_at) / len;
      const uint32_t item0 = seq_at + it.h * len, tile0 = item0 + extra;
      if (by_warp) {
        const bool begun = u > item0;               // in the range before this one
        u = item0 + len;
        if (begun) continue;
        it.t0 = 0;
        it.t1 = len - extra;
        it.pieces = 1;
        return true;
      }
      const uint32_t end = min(item0 + len, u1);
      it.t0 = u > tile0 ? u - tile0 : 0;
      it.t1 = end > tile0 ? end - tile0 : 0;
      u = end;
      if (it.t0 == it.t1) continue;                 // its tiles are all in the next range
      it.c0 = tile0 / q;
      it.pieces = (item0 + len - 1) / q - it.c0 + 1;
      // slot 0: the first item of a block's range, slot 1: a later one, which is its last
      it.slot = item0 <= c * q ? 0 : 1;
      it.first_slot = item0 <= it.c0 * q ? 0 : 1;
      return true;
    }
    return false;
  };

  // Lane g < kParts looks after block g of each tile: its page id (loaded two tiles ahead of
  // the tile's use), its copies, its scales (loaded one tile ahead).
  const size_t page_step = (size_t)a.H << a.shift;             // rows per page, all heads
  bool bad = false;
  auto part_id = [&](int t) {
    if (lane >= S::kParts || t >= it.t1) return -1;
    const int tok = t * S::kTile + lane * 16;                  // lengths stay below 2^31
    if (tok >= it.n) return -1;
    return __ldg(a.block_table + (long long)it.b * a.max_pages + (tok >> a.shift));
  };
  auto checked = [&](int t, int id) {                          // -1 for what is not there
    const bool there = lane < S::kParts && t < it.t1 && t * S::kTile + lane * 16 < it.n;
    const bool ok = there && id >= 0 && id < a.n_pages;
    bad |= there && !ok;
    return ok ? id : -1;
  };
  auto issue = [&](int t, int id, uint32_t seq) {              // tile t, the warp's seq-th
    if (t >= it.t1) return;
    const int s = seq % kQ8Stages;
    const unsigned live = __ballot_sync(0xffffffffu, id >= 0);
    if (lane == 0) sm100::mbar_arrive_expect_tx(&bars[s], __popc(live) * 2 * S::kPartBytes);
    __syncwarp();
    if (id >= 0) {
      const int tok = t * S::kTile + lane * 16;
      const size_t run = (id * page_step + ((size_t)it.h << a.shift) +
                          (tok & ((1 << a.shift) - 1))) * D;
      unsigned char* st = ring + s * S::kStage + lane * S::kPartBytes;
      sm100::bulk_load(st, a.kc + run, S::kPartBytes, &bars[s]);
      sm100::bulk_load(st + S::kHalf, a.vc + run, S::kPartBytes, &bars[s]);
    }
  };
  auto scale_of = [&](const float* scales, int id) {
    return id >= 0 ? __ldg(scales + (size_t)id * a.H + it.h) : 0.f;
  };
  int id0 = -1, id1 = -1, id2 = -1;                            // a warp's next three tiles
  float ks0 = 0.f, vs0 = 0.f;
  auto load_ids = [&]() {
    const int first = it.t0 + lead;
    id0 = part_id(first);
    id1 = part_id(first + step);
    id2 = part_id(first + 2 * step);
  };
  auto start_copies = [&]() {
    const int first = it.t0 + lead;
    id0 = checked(first, id0);
    id1 = checked(first + step, id1);
    if (!aborted) {
      issue(first, id0, used);
      issue(first + step, id1, used + 1);
    }
    ks0 = scale_of(a.ks, id0);
    vs0 = scale_of(a.vs, id0);
  };
  bool more = find_item(), started = false;
  uint32_t finished = 0;                                       // the counter word before
  auto finish_block = [&]() { return atomicAdd(a.counter, 1u); };
  // q, the in-flight token's key and their angles, eight dims a lane: the next item's are
  // loaded before the merge of the one before it
  const bool turn = a.rope != nullptr, chunk = lane < D / 8;
  const RowChunk rc = row_chunk<8>(lane, D, turn ? a.rd : 0, a.layout);
  float v[8], k[8];
  Turn<8> angles;
  int asked = 0;
  auto fetch_q = [&]() {
    if (turn) asked = few ? __shfl_sync(0xffffffffu, pos_of_lane, it.b) : a.q_pos[it.b];
    if (!chunk) return;
    const size_t row = ((size_t)it.b * a.H + it.h) * D;
    load_chunk<8>(static_cast<const T*>(a.q) + row, rc, v);
    if (a.k_self) load_chunk<8>(static_cast<const T*>(a.k_self) + row, rc, k);
  };
  auto fetch_angles = [&]() {
    if (!chunk || !turn) return;
    const int pos = checked_position(asked, a.rope_max_pos, nullptr, false);
    if (lane == 0 && pos != asked) tell_status(a, LLA_STATUS_POSITION_RANGE);
    if (rc.rotary) angles = load_turn<8>(a.rope + (size_t)pos * (a.rd / 2), rc);
  };
  if (more) {
    load_ids();
    fetch_q();
    fetch_angles();
    start_copies();                                            // while the angles come
  }
  __syncthreads();                                             // abort_word is set
  while (more) {
    started = true;
    const int first = it.t0 + lead;
    const size_t bh = (size_t)it.b * a.H + it.h;

    // q rotated at q_pos, through shared memory, by each warp for itself; the in-flight
    // token's score, which needs no rotation, both sitting at q_pos
    float self = 0.f;
    {
      if (chunk) {
        if (a.k_self) {
#pragma unroll
          for (int j = 0; j < 8; ++j) self = fmaf(v[j], k[j], self);
        }
        if (rc.rotary) rotate_chunk<8>(angles, rc.split, v);
        store_chunk<8>(qs, rc, v);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) self += __shfl_xor_sync(0xffffffffu, self, off);
    self *= a.kappa;
    __syncwarp();

    // q as 24-bit integers, the largest |q| of a lane's dims near 2^23: a lane splits four dims
    // and takes the words of its own through shared memory
    uint32_t q1[W], q2[W], q3[W];
    float score_scale;                                          // of the lane's part of a score
    bool strange = false;                                       // a NaN or an infinity in q
    {
      float v[4] = {0.f, 0.f, 0.f, 0.f}, amax = 0.f;
      if (lane < D / 4) load_run<4>(qs + 4 * lane, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        amax = fmaxf(amax, fabsf(v[j]));
        strange |= !(fabsf(v[j]) <= FLT_MAX);
      }
      strange = __any_sync(0xffffffffu, strange);               // and the values are read
      if constexpr (W == 4) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      } else {
        const float mine = amax;
#pragma unroll
        for (int k = 0; k < W; ++k)
          amax = fmaxf(amax, __shfl_sync(0xffffffffu, mine, lane / W * W + k));
      }
      constexpr float kTop = 8388480.f;                         // a product's rounding below 2^23
      const float inv = amax > kQ8Tiny ? kTop / amax : 0.f;
      // in units of q1 2^8 + q2; strange: pl becomes NaN below
      score_scale = strange ? 0.f : __shfl_sync(0xffffffffu, a.kappa * amax / (kTop / 256.f), col * W);
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = (uint32_t)__float2int_rn(v[j] * inv);
      uint32_t* words = reinterpret_cast<uint32_t*>(qs);
      if (lane < D / 4) {
        const uint32_t y01 = __byte_perm(x[0], x[1], 0x5140), y23 = __byte_perm(x[2], x[3], 0x5140);
        const uint32_t z01 = __byte_perm(x[0], x[1], 0x0062), z23 = __byte_perm(x[2], x[3], 0x0062);
        words[lane] = __byte_perm(z01, z23, 0x5410);            // -128 .. 127
        words[D / 4 + lane] = __byte_perm(y01, y23, 0x7632);    // 0 .. 255
        words[D / 2 + lane] = __byte_perm(y01, y23, 0x5410);
      }
      __syncwarp();
#pragma unroll
      for (int w = 0; w < W; ++w) {
        q1[w] = words[col * W + w];
        q2[w] = words[D / 4 + col * W + w];
        q3[w] = words[D / 2 + col * W + w];
      }
    }

    // Sums are relative to 2^m, m the largest score so far: l of p = 2^(s - m), o of p * scale *
    // code.  A larger score rescales both.
    float m = -INFINITY, l = 0.f;
    float_pair o2[2 * W];                                        // dims 2 j and 2 j + 1
#pragma unroll
    for (int j = 0; j < 2 * W; ++j) o2[j] = 0;

    // Rows r + kRows i of a group are a lane's, i = 0 .. 3; it ends up with the scores of
    // i_own (and i_own + 1 when it has two).
    const int i_own = S::kLanes == 8 ? (((col >> 1) & 1) | ((col >> 1) & 2))
                                     : S::kLanes == 4 ? (((col & 1)) | (col & 2)) : 2 * col;
    uint32_t seq = used;
    for (int t = first; t < it.t1 && !aborted; t += step, ++seq) {
      const int s = seq % kQ8Stages;
      const unsigned live = __ballot_sync(0xffffffffu, id0 >= 0);
      // scales of the next tile, page ids of the one after it
      const float ks1 = scale_of(a.ks, id1), vs1 = scale_of(a.vs, id1);
      id2 = checked(t + 2 * step, id2);
      const int id3 = part_id(t + 3 * step);
      // Each lane looks at the barrier, the abort flag and the timer for itself: near a timeout
      // they may differ, and what follows is the whole warp's.
      if (!__all_sync(0xffffffffu, sm100::mbar_wait(&bars[s], (seq / kQ8Stages) & 1u, abort_flag))) {
        // copies already issued land before the block can end
        for (int k = 0; k < kQ8Stages && t + k * step < it.t1; ++k) {
          const unsigned long long w0 = sm100::global_timer_ns();
          while (!sm100::mbar_try_wait(&bars[(seq + k) % kQ8Stages], ((seq + k) / kQ8Stages) & 1u) &&
                 sm100::global_timer_ns() - w0 < sm100::kWaitTimeoutNs) {
          }
        }
        aborted = true;
        break;
      }
      const unsigned char* st = ring + s * S::kStage + r * D + col * 4 * W;
      const int rows_left = it.n - t * S::kTile - r - S::kRows * i_own;   // of a lane's first score
      if (live) {                                               // else no page of it is there
        // Scores of both groups, then one look at their maxima, then the weights: the groups' long
        // chains of exchanges run side by side.
        constexpr int kFar = S::kLanes / 2, kNear = S::kLanes / 4;
        const bool upper = col & kFar, odd = col & kNear;
        float sc[2][S::kScores], vsc[2][S::kScores];
        bool above = false;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const unsigned char* kp = st + g * S::kSubs * S::kPartBytes;
          float part[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t kw[W];
            load_words<W>(kp + i * S::kRows * D, kw);
            int s1 = 0, s2 = 0, s3 = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) {
              s1 = __dp4a((int)kw[w], (int)q1[w], s1);
              s2 = dp4a_su(kw[w], q2[w], s2);
              s3 = dp4a_su(kw[w], q3[w], s3);
            }
            part[i] = fmaf((float)s3, 1.f / 256.f, (float)(s1 * 256 + s2)) * score_scale;
          }
          // sums over a row's lanes, each exchange halving what a lane holds
          float x[2];
          x[0] = (upper ? part[2] : part[0]) +
                 __shfl_xor_sync(0xffffffffu, upper ? part[0] : part[2], kFar);
          x[1] = (upper ? part[3] : part[1]) +
                 __shfl_xor_sync(0xffffffffu, upper ? part[1] : part[3], kFar);
          if constexpr (S::kLanes >= 4)
            x[0] = (odd ? x[1] : x[0]) + __shfl_xor_sync(0xffffffffu, odd ? x[0] : x[1], kNear);
          if constexpr (S::kLanes == 8) x[0] += __shfl_xor_sync(0xffffffffu, x[0], 1);
#pragma unroll
          for (int k = 0; k < S::kScores; ++k) {
            // the 16-token block of the group that the row lies in
            const int sub = g * S::kSubs + (S::kSubs == 1 ? 0 : S::kSubs == 2 ? i_own >> 1 : i_own + k);
            const float ksc = __shfl_sync(0xffffffffu, ks0, sub);
            vsc[g][k] = __shfl_sync(0xffffffffu, vs0, sub);
            const bool there = rows_left > g * S::kGroup + k * S::kRows && (live >> sub & 1);
            sc[g][k] = there ? x[k] * ksc : -INFINITY;
            above |= sc[g][k] > m;
          }
        }
        if (__any_sync(0xffffffffu, above)) {
          float mt = fmaxf(fmaxf(sc[0][0], sc[0][S::kScores - 1]),
                           fmaxf(sc[1][0], sc[1][S::kScores - 1]));
          mt = warp_largest(mt);
          const float f = exp2_down(m - mt);                      // 0 the first time
          m = mt;
          l *= f;
          const float_pair f2 = pair_of(f, f);
#pragma unroll
          for (int j = 0; j < 2 * W; ++j) o2[j] = mul2(o2[j], f2);
        }
        float_pair weight[2][4];              // of a lane's four rows, twice
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float wt[S::kScores];
#pragma unroll
          for (int k = 0; k < S::kScores; ++k) {
            const float p = exp2_down(sc[g][k] - m);
            l += p;
            wt[k] = p > 0.f ? p * vsc[g][k] : 0.f;                // a row past the end: whatever its scale
          }
          float e0 = wt[0], e1 = wt[S::kScores - 1];
          if constexpr (S::kLanes >= 4) {
            const float other = __shfl_xor_sync(0xffffffffu, wt[0], kNear);
            e0 = odd ? other : wt[0];
            e1 = odd ? wt[0] : other;
          }
          const float f0 = __shfl_xor_sync(0xffffffffu, e0, kFar);
          const float f1 = __shfl_xor_sync(0xffffffffu, e1, kFar);
          const float w4[4] = {upper ? f0 : e0, upper ? f1 : e1, upper ? e0 : f0, upper ? e1 : f1};
#pragma unroll
          for (int i = 0; i < 4; ++i) weight[g][i] = pair_of(w4[i], w4[i]);
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          // a group without a token left weighs nothing, whatever the ring holds there
          const unsigned char* vp = st + S::kHalf + g * S::kSubs * S::kPartBytes;
          uint32_t vw[4][W];
#pragma unroll
          for (int i = 0; i < 4; ++i) load_words<W>(vp + i * S::kRows * D, vw[i]);
#pragma unroll
          for (int w = 0; w < W; ++w) {
            // the four rows' sum by itself: long sums then take a quarter of the roundings
            float_pair lo = 0, hi = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t u = vw[i][w] ^ 0x80808080u;
              const float_pair c0 = codes2<0>(u), c2 = codes2<2>(u);
              lo = i ? fma2(c0, weight[g][i], lo) : mul2(c0, weight[g][i]);
              hi = i ? fma2(c2, weight[g][i], hi) : mul2(c2, weight[g][i]);
            }
            o2[2 * w] = add2(o2[2 * w], lo);
            o2[2 * w + 1] = add2(o2[2 * w + 1], hi);
          }
        }
      }
      __syncwarp();                                             // the stage is read
      issue(t + kQ8Stages * step, id2, seq + kQ8Stages);
      id0 = id1;
      id1 = id2;
      id2 = id3;
      ks0 = ks1;
      vs0 = vs1;
    }
    if (it.t1 > first) used += (it.t1 - first + step - 1) / step;
    if (__any_sync(0xffffffffu, bad) && lane == 0) tell_status(a, LLA_STATUS_PAGE_RANGE);
    bad = false;
    if (aborted && lane == 0) tell_status(a, LLA_STATUS_TIMEOUT);
    // the next item's first tiles are on their way while this one is merged
    const Q8Item now = it;
    more = !aligned && find_item();
    if (more) {
      load_ids();
      fetch_q();
      start_copies();
    }

    // ---------------------------------------------------------------- merge the warps
    float o[4 * W];
#pragma unroll
    for (int j = 0; j < 2 * W; ++j) unpair(o2[j], o[2 * j], o[2 * j + 1]);
    if (S::kLanes == 8) l *= 0.5f;                              // two lanes held every score
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, off);
      if (off < S::kLanes) continue;
#pragma unroll
      for (int j = 0; j < 4 * W; ++j) o[j] += __shfl_xor_sync(0xffffffffu, o[j], off);
    }
    if (more) fetch_angles();
    if (by_warp) {
      float f = 1.f, fs = 0.f;
      if (a.k_self) {
        const float top = fmaxf(m, self);
        f = m > -INFINITY ? exp2f(m - top) : 0.f;
        fs = exp2f(self - top);
      }
      l = fmaf(l, f, fs);
      if (strange && l != 0.f) l = NAN;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (r == 0) {
        const size_t at = bh * D + col * 4 * W;
#pragma unroll
        for (int j = 0; j < 4 * W; j += 4) {
          float v[4] = {0.f, 0.f, 0.f, 0.f};
          if (a.k_self) load_run<4>(static_cast<const T*>(a.v_self) + at + j, v);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = l == 0.f ? 0.f : (a.k_self ? fmaf(o[j + i], f, fs * v[i]) : o[j + i]) * inv;
          store_run<4>(static_cast<T*>(a.out) + at + j, v);
        }
      }
      continue;
    }
    float v_own = 0.f;
    if (a.k_self && tid < D) v_own = as_float(static_cast<const T*>(a.v_self)[bh * D + tid]);
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
    // every status bit of the block is told; the count comes back during the merge
    if (tid == 0 && !more) finished = finish_block();
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
        const float top = fmaxf(pm, self);
        const float f = pm > -INFINITY ? exp2f(pm - top) : 0.f, fs = exp2f(self - top);
        pl = fmaf(pl, f, fs);
        po = fmaf(po, f, fs * v_own);
      }
      if (strange && pl != 0.f) pl = NAN;
      if (tid < D) put(static_cast<T*>(a.out) + bh * D + tid, pl == 0.f ? 0.f : po / pl);
    }
    __syncthreads();                                            // parts and is_last are free
  }
  // the last block to finish publishes the call's status and re-arms the counter
  if (by_warp || !started) {                                   // also a range without a tile
    __syncthreads();
    if (tid == 0) finished = finish_block();
  }
  if (tid == 0 && (finished & ((1u << kQ8StatusShift) - 1)) == blocks - 1) {
    a.status[1] = finished >> kQ8StatusShift;
    *a.counter = 0;
  }
}

// For d > 1, with 2^k < d <= 2^(k + 1) and factor = ceil(2^(32 + k) / d), factor * d exceeds
// 2^(32 + k) by less than 2^(k + 1): too little to carry a quotient of a < 2^31 to the next
// integer.
Q8Divisor divisor(uint32_t d) {
  Q8Divisor r{0, 0};
  if (d == 1) return r;                     // factor 0: divides by one
  while ((2u << r.shift) < d) ++r.shift;
  r.factor = (uint32_t)(((1ull << (32 + r.shift)) + d - 1) / d);
  return r;
}

constexpr int kQ8MostBlocksPerSm = 3;
int q8_max_blocks() { return sm_count() * kQ8MostBlocksPerSm; }

template <typename T, int D>
cudaError_t launch_decode_td(Q8DecodeArgs a, cudaStream_t s) {
  using S = Q8Shape<D>;
  cudaError_t e = cudaFuncSetAttribute(q8_decode_kernel<T, D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != cudaSuccess) return e;
  const long long tiles =
      (((long long)a.max_pages << a.shift) + S::kTile - 1) / S::kTile;
  // at most one block per kQ8MinTiles tiles of every item
  const long long per_item = std::max(1LL, (tiles + kQ8MinTiles - 1) / kQ8MinTiles);
  const long long grid = std::min<long long>((long long)a.B * a.H * per_item,
                                              sm_count() * S::kBlocksPerSm);
  a.by_grid = divisor((uint32_t)grid);
  a.by_warps = divisor((uint32_t)grid * kQ8Warps);
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

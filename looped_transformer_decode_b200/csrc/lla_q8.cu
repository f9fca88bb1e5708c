// Paged 8-bit cache of exact keys and values: the append that quantises and the read
// that gives rows back (decode attention: lla_q8_decode.cu).
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
#include <cuda_pipeline.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "lla_internal.cuh"
#include "lla_rows.cuh"

namespace lla {
namespace {

constexpr float kQ8Grow = 1.25f;

// ---------------------------------------------------------------- append

// Tokens per sequence below which a warp per part is faster, and where there are many parts.
// 8 sequences of 16 heads of 128: 4.3 us either way at 4 tokens, 8.3 against 5.3 by the kernel
// for prompts at 16.  64 of them, in pages of 64: 4.1 against 7.9 at 1 token, 7.4 against 14.8
// at 8, 11.3 against 17.5 at 16, 22.8 against 24.4 at 31.
constexpr int kAppendFew = 8, kAppendFewOfMany = 24;
constexpr int kAppendManyHeads = 512;   // of all sequences
constexpr int kAppendWarps = 8;
constexpr int kAppendBlocksPerSm = 2;
constexpr int kAppendValues = 32;       // of a full page's head, per thread (prompts)
constexpr int kAppendDepth = 2;         // groups in the ring: one in work, the others on their way

// The page that unit u of an append works on: units floor(tok_start[b] / P) + 2 b and
// up belong to sequence b, enough for every page its tokens can touch.
struct AppendUnit {
  const int32_t* entry;       // of the page, in the block table
  int off, count;             // rows [off, off + count) of the page are new
  int tok, row;               // first of their tokens, and its row of k and v
};

// All threads of the block look for the sequence together, blockDim.x starts at a time.
__device__ __forceinline__ bool append_unit(const Q8AppendArgs& a, int u, bool tell,
                                            AppendUnit& r) {
  const int P = 1 << a.shift;
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + blockDim.x - 1) / blockDim.x;
    const int b = lo + threadIdx.x * step;
    const int begun = __syncthreads_count(
        b < hi && (b == lo || (__ldg(a.tok_start + b) >> a.shift) + 2 * b <= u));
    lo += (begun - 1) * step;
    hi = min(hi, lo + step);
  }
  const int s = __ldg(a.tok_start + lo), e = __ldg(a.tok_start + lo + 1);
  const int after = __ldg(a.ctx_len + lo);
  if (s < 0 || e < s || e > a.n_tok || after < e - s ||
      after > (long long)a.max_pages << a.shift) {
    if (tell && a.status) atomicOr(a.status, LLA_STATUS_CTX_RANGE);
    return false;
  }
  const int first_row = a.row_start ? __ldg(a.row_start + lo) : s;
  if (e > s && (first_row < 0 || first_row > a.n_tok - (e - s))) {
    if (tell && a.status) atomicOr(a.status, LLA_STATUS_CTX_RANGE);
    return false;
  }
  const int before = after - (e - s);
  const int j = u - ((s >> a.shift) + 2 * lo);
  const long long page_at = (long long)(before >> a.shift) + j;
  const long long p0 = page_at << a.shift;
  if (j < 0 || e == s || p0 >= after) return false;
  r.entry = a.block_table + (long long)lo * a.max_pages + page_at;
  r.off = before > p0 ? (int)(before - p0) : 0;
  r.count = (int)(after - p0 < P ? after - p0 : P) - r.off;
  r.tok = s + (int)(p0 + r.off - before);
  r.row = first_row + (r.tok - s);
  return true;
}

__device__ __forceinline__ bool known_page(const Q8AppendArgs& a, int page, bool tell) {
  if (page >= 0 && page < a.n_pages) return true;
  if (tell && a.status) atomicOr(a.status, LLA_STATUS_PAGE_RANGE);
  return false;
}

// A page's scale from an earlier append; anything else (damaged, or for values that count as
// zero) is taken for 0, which also bounds what a value is divided by.
__device__ __forceinline__ bool usable_scale(float s) {
  return s >= kQ8Tiny / 128.f && s <= FLT_MAX;
}

// Scale of the page after the append, from the largest new value.  amax / 127 is a product with
// the nearest 1 / 127, as in the definition: in bf16 a quotient value / scale often lies at half a
// step, and one unit in the last place of the scale decides its code.
__device__ __forceinline__ float grown_scale(float amax, float older) {
  const float asked = amax > kQ8Tiny ? __fmul_rn(amax, 1.f / 127.f) : 0.f;
  return asked > older ? fmaxf(asked, __fmul_rn(older, kQ8Grow)) : older;
}

// The codes of four values x with |x inv| < 2^22: adding 1.5 * 2^23 rounds to an integer and
// leaves it in the low bits.
__device__ __forceinline__ uint32_t quantise4(const float* v, float inv) {
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = __float_as_uint(__fadd_rn(__fmul_rn(v[j], inv), 12582912.f));
  return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}

// M codes at p (4 or 8, aligned to them).
template <int M>
__device__ __forceinline__ void store_codes(int8_t* p, const float* v, float inv) {
  if constexpr (M == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(quantise4(v, inv), quantise4(v + 4, inv));
  else
    *reinterpret_cast<uint32_t*>(p) = quantise4(v, inv);
}

// Larger of a and |x|; NaN if either is.
__device__ __forceinline__ float max_or_nan(float a, float x) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(fabsf(x)));
  return y;
}

// Where a thread has met a NaN or an infinity: the larger of a and |x| if x is finite, and
// what is stored for x: 0 for a NaN, the largest code for an infinity.
__device__ __forceinline__ float max_finite(float a, float x) {
  return fabsf(x) <= FLT_MAX ? fmaxf(a, fabsf(x)) : a;
}
__device__ __forceinline__ float stored(float x, float scale) {
  return x != x ? 0.f : fabsf(x) <= FLT_MAX ? x : copysignf(fminf(127.f * scale, FLT_MAX), x);
}

// Largest of the lanes' non-negative values, whose bits order as they do.
__device__ __forceinline__ float warp_max(float x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}

// The page's codes of earlier tokens under the new scale, by `threads` threads.
__device__ __forceinline__ void rescale_codes(int8_t* codes, int n, float ratio, int t,
                                              int threads) {
  uint32_t* words = reinterpret_cast<uint32_t*>(codes);
  for (int i = t; i < n / 4; i += threads) {
    const uint32_t w = words[i];
    const float x[4] = {(float)(int8_t)w, (float)(int8_t)(w >> 8), (float)(int8_t)(w >> 16),
                        (float)(int8_t)(w >> 24)};
    words[i] = quantise4(x, ratio);
  }
}

// Few tokens per sequence (decode steps): blockIdx.x is a page, each warp takes one of its
// parts (a head's keys or its values) by itself, reading the rows twice, for their largest
// magnitude and for their codes.  Latency bounds it: 64 sequences of 16 heads take 3.9 us, by
// the kernel for prompts 7.9.
template <typename T>
__global__ void __launch_bounds__(32 * kAppendWarps) q8_append_kernel(Q8AppendArgs a) {
  constexpr int N = kChunkDims<T>;
  const int lane = threadIdx.x & 31;
  AppendUnit un;
  const bool tell = blockIdx.y == 0 && threadIdx.x == 0;
  if (!append_unit(a, blockIdx.x, tell, un)) return;
  const int page = __ldg(un.entry);
  if (!known_page(a, page, tell)) return;
  const int part = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (part >= 2 * a.H) return;
  const bool is_k = part < a.H;
  const int h = is_k ? part : part - a.H;
  const int tpr = a.d / N, rpp = 32 / tpr;                   // lanes per row, rows per pass
  const int row0 = lane / tpr, c = lane - row0 * tpr;
  const int rows = row0 < rpp ? un.count : 0;
  const bool turn = is_k && a.rope;
  const RowChunk rc = row_chunk<N>(c, a.d, turn ? a.rd : 0, a.layout);
  const long long stride = is_k ? a.k_stride : a.v_stride;
  const T* src = static_cast<const T*>(is_k ? a.k : a.v) + un.row * stride + h * a.d;
  const long long run = (long long)page * a.H + h;
  int8_t* codes = (is_k ? a.kc : a.vc) + (run << a.shift) * a.d;
  float* scale = (is_k ? a.ks : a.vs) + run;

  auto value = [&](int r, float* v) {
    load_chunk<N>(src + r * stride, rc, v);
    if (!turn) return;
    const int pos = checked_position(__ldg(a.positions + un.tok + r), a.rope_max_pos, a.status,
                                     h == 0 && c == 0);
    if (rc.rotary)
      rotate_chunk<N>(load_turn<N>(a.rope + (size_t)pos * (a.rd / 2), rc), rc.split, v);
  };
  float older = un.off > 0 ? *scale : 0.f;
  if (!usable_scale(older)) older = 0.f;
  float amax = 0.f;
  bool strange = false;
#pragma unroll 1
  for (int r = row0; r < rows; r += rpp) {
    float v[N], here = 0.f;
    value(r, v);
#pragma unroll
    for (int j = 0; j < N; ++j) here = max_or_nan(here, v[j]);
    if (!(here <= FLT_MAX)) {
      strange = true;
      here = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) here = max_finite(here, v[j]);
    }
    amax = fmaxf(amax, here);
  }
  if (strange && a.status) atomicOr(a.status, LLA_STATUS_NONFINITE);
  amax = warp_max(amax);
  const float now = grown_scale(amax, older);
  const float inv = now > 0.f ? __frcp_rn(now) : 0.f;
  __syncwarp();                                              // the old scale has been read
  if (lane == 0) *scale = now;
  if (now > older && un.off > 0)
    rescale_codes(codes, un.off * a.d, __fdiv_rn(older, now), lane, 32);
#pragma unroll 1
  for (int r = row0; r < rows; r += rpp) {
    float v[N];
    value(r, v);
    if (strange) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = stored(v[j], now);
    }
    int8_t* row = codes + (un.off + r) * a.d;
    store_codes<N / 2>(row + rc.lo, v, inv);
    store_codes<N / 2>(row + rc.hi, v + N / 2, inv);
  }
}

// Prompts: every block takes an equal run of all pages' groups of heads, keys' before values'
// (a.groups of either; a group is a head for each of the block's teams of a.team threads).  A
// team holds a full page of its head in registers, rotated, between its largest magnitude and
// its codes.  The rows of the next groups are on their way meanwhile, into a ring in shared
// memory of which every thread fills and reads its own part, so that nothing waits for it but
// the thread itself.  20011 tokens of 16 heads of 128: bf16 67 us, fp32 83 (their bytes take 38
// and 63 at the copy rate); without the ring and with a block per page and four heads 128.
template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? kAppendBlocksPerSm : 1)
q8_append_prompts_kernel(Q8AppendArgs a, int units) {
  constexpr int N = kChunkDims<T>, kPasses = kAppendValues / N;
  constexpr int kDepth = kAppendDepth;
  extern __shared__ uint4 ring[];                            // [kDepth][kPasses][2][kThreads]
  __shared__ float red[2][kThreads / 32];
  const int team0 = threadIdx.x / a.team, t = threadIdx.x - team0 * a.team;
  const int teams = kThreads / a.team;
  const int tpr = a.d / N, rpp = a.team / tpr;               // threads per row, rows per pass
  const int row0 = t / tpr, c = t - row0 * tpr;
  uint4* mine = ring + threadIdx.x;

  const long long all = 2LL * units * a.groups;
  long long x = all * blockIdx.x / gridDim.x;
  const long long x1 = all * (blockIdx.x + 1) / gridDim.x;
  int parity = 0;
  while (x < x1) {                                           // a page's keys or values
    const long long part = x / a.groups;
    const int g0 = (int)(x - part * a.groups);
    const int g1 = (int)min((long long)a.groups, g0 + x1 - x);
    x += g1 - g0;
    const bool is_k = !(part & 1);
    const bool tell = is_k && g0 == 0 && threadIdx.x == 0;
    AppendUnit un;
    if (!append_unit(a, (int)(part >> 1), tell, un)) continue;
    const int page = __ldg(un.entry);
    const int rows = row0 < rpp ? un.count : 0;
    const bool turn = is_k && a.rope;
    const RowChunk rc = row_chunk<N>(c, a.d, turn ? a.rd : 0, a.layout);
    const long long stride = is_k ? a.k_stride : a.v_stride, pass = rpp * stride;
    const T* first = static_cast<const T*>(is_k ? a.k : a.v) + (un.row + row0) * stride + rc.lo;
    auto fetch = [&](int g, int stage) {
      const int h = g * teams + team0;
      const T* row = first + h * a.d;
      uint4* to = mine + stage * (kPasses * 2 * kThreads);
#pragma unroll
      for (int i = 0; i < kPasses; ++i, row += pass, to += 2 * kThreads) {
        if (g >= g1 || h >= a.H || row0 + i * rpp >= rows) break;
        __pipeline_memcpy_async(to, row, 16);
        __pipeline_memcpy_async(to + kThreads, row + (rc.hi - rc.lo), 16);
      }
      __pipeline_commit();
    };
#pragma unroll
    for (int s = 0; s < kDepth - 1; ++s) fetch(g0 + s, s);
    Turn<N> turns[kPasses];                                  // of the thread's rows, for all heads
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if (!turn || row0 + i * rpp >= rows) break;
      const int pos = checked_position(__ldg(a.positions + un.tok + row0 + i * rpp),
                                       a.rope_max_pos, a.status, g0 == 0 && c == 0);
      if (rc.rotary) turns[i] = load_turn<N>(a.rope + (size_t)pos * (a.rd / 2), rc);
    }
    const bool known = known_page(a, page, tell);
    const long long run = (long long)page * a.H + g0 * teams + team0;
    int8_t* codes = (is_k ? a.kc : a.vc) + (run << a.shift) * a.d;
    float* scale = (is_k ? a.ks : a.vs) + run;

    int stage = 0;
    for (int g = g0; g < g1 && known; ++g, parity ^= 1) {    // the same for all teams
      const bool mine_too = g * teams + team0 < a.H;          // the last group may have fewer
      const int live = mine_too ? rows : 0;
      fetch(g + kDepth - 1, stage == 0 ? kDepth - 1 : stage - 1);
      float older = un.off > 0 && mine_too ? *scale : 0.f;
      if (!usable_scale(older)) older = 0.f;
      __pipeline_wait_prior(kDepth - 1);
      float v[kPasses][N];
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        if (row0 + i * rpp >= live) break;
        const uint4* from = mine + (stage * kPasses + i) * 2 * kThreads;
        const uint4 lo = from[0], hi = from[kThreads];
        load_run<N / 2>(reinterpret_cast<const T*>(&lo), v[i]);
        load_run<N / 2>(reinterpret_cast<const T*>(&hi), v[i] + N / 2);
        if (rc.rotary) rotate_chunk<N>(turns[i], rc.split, v[i]);
#pragma unroll
        for (int j = 0; j < N; ++j) amax = max_or_nan(amax, v[i][j]);
      }
      stage = stage + 1 == kDepth ? 0 : stage + 1;
      const bool strange = !(amax <= FLT_MAX);
      if (strange) {
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
          if (row0 + i * rpp < live) {
#pragma unroll
            for (int j = 0; j < N; ++j) amax = max_finite(amax, v[i][j]);
          }
        if (a.status) atomicOr(a.status, LLA_STATUS_NONFINITE);
      }
      amax = warp_max(amax);
      if (a.team > 32) {
        const int warps = a.team / 32;                       // 2, 4, 8 or 16
        if ((threadIdx.x & 31) == 0) red[parity][threadIdx.x >> 5] = amax;
        __syncthreads();
        amax = warp_max(red[parity][team0 * warps + (threadIdx.x & (warps - 1))]);
      } else {
        __syncwarp();
      }
      if (mine_too) {
        const float now = grown_scale(amax, older);
        const float inv = now > 0.f ? __frcp_rn(now) : 0.f;
        if (t == 0) *scale = now;       // every thread of the team has read the old one
        if (now > older && un.off > 0)
          rescale_codes(codes, un.off * a.d, __fdiv_rn(older, now), t, a.team);
        if (strange) {
#pragma unroll
          for (int i = 0; i < kPasses; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) v[i][j] = stored(v[i][j], now);
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int r = row0 + i * rpp;
          if (r >= live) break;
          int8_t* row = codes + (un.off + r) * a.d;
          store_codes<N / 2>(row + rc.lo, v[i], inv);
          store_codes<N / 2>(row + rc.hi, v[i] + N / 2, inv);
        }
      }
      scale += teams;
      codes += (long long)(teams << a.shift) * a.d;
    }
    __pipeline_wait_prior(0);
  }
}

// ---------------------------------------------------------------- read

// A thread reads eight keys and eight values of one head in kRows rows and writes 16 bytes of
// each; a.row_block groups of kRows rows a block (one, over gridDim.y blocks, where a row has
// more threads).  20459 rows of 16 heads of 128 take 44.8 us, 86% of the copy rate; one row a
// thread 51.
constexpr int kReadThreads = 256;

template <int kRows>
__global__ void __launch_bounds__(kReadThreads) q8_read_kernel(Q8ReadArgs a) {
  const int per_row = a.H * (a.d / 8);
  const int x = blockIdx.y * kReadThreads + threadIdx.x;
  const int rl = x / per_row, rest = x - rl * per_row;
  const long long row = ((long long)blockIdx.x * a.row_block + rl) * kRows;
  if (rl >= a.row_block) return;
  const int h = rest / (a.d / 8), c = rest - h * (a.d / 8);
  uint2 kw[kRows], vw[kRows];
  float ks[kRows], vs[kRows];
  long long slot[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) slot[i] = row + i < a.n_rows ? __ldg(a.slot + row + i) : -1;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (slot[i] < 0 || slot[i] >= (long long)a.n_pages << a.shift) {
      if (row + i < a.n_rows && rest == 0 && a.status) atomicOr(a.status, LLA_STATUS_SLOT_RANGE);
      slot[i] = -1;
      continue;
    }
    const long long page = (slot[i] >> a.shift) * a.H + h;
    const long long at = ((page << a.shift) + (slot[i] & ((1 << a.shift) - 1))) * a.d + c * 8;
    kw[i] = *reinterpret_cast<const uint2*>(a.kc + at);
    vw[i] = *reinterpret_cast<const uint2*>(a.vc + at);
    ks[i] = a.ks[page];
    vs[i] = a.vs[page];
  }
  auto wide = [](uint2 w, float s) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = s * (float)(int8_t)(w.x >> (8 * j));
      v[4 + j] = s * (float)(int8_t)(w.y >> (8 * j));
    }
    return make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]),
                      bf16x2_bits(v[6], v[7]));
  };
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (slot[i] < 0) continue;
    const long long to = (row + i) * per_row + rest;
    reinterpret_cast<uint4*>(a.k_out)[to] = wide(kw[i], ks[i]);
    reinterpret_cast<uint4*>(a.v_out)[to] = wide(vw[i], vs[i]);
  }
}

template <typename T, int kThreads>
cudaError_t launch_append_prompts(Q8AppendArgs a, int units, cudaStream_t s) {
  constexpr int kBytes = kAppendDepth * kThreads * kAppendValues * (int)sizeof(T);
  cudaError_t e = cudaFuncSetAttribute(q8_append_prompts_kernel<T, kThreads>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  const int teams = kThreads / a.team;
  a.groups = (a.H + teams - 1) / teams;
  const long long blocks = std::min<long long>(
      2LL * units * a.groups, (kThreads == 256 ? kAppendBlocksPerSm : 1) * sm_count());
  q8_append_prompts_kernel<T, kThreads><<<(unsigned)blocks, kThreads, kBytes, s>>>(a, units);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_append(Q8AppendArgs a, cudaStream_t s) {
  const int units = (a.n_tok >> a.shift) + 2 * a.B;
  if (a.n_tok < kAppendFew * a.B ||
      (a.n_tok < kAppendFewOfMany * a.B && a.B * a.H >= kAppendManyHeads)) {
    const int warps = std::min(kAppendWarps, 2 * a.H);
    const dim3 grid(units, (2 * a.H + warps - 1) / warps);
    q8_append_kernel<T><<<grid, 32 * warps, 0, s>>>(a);
    return cudaGetLastError();
  }
  // the threads that hold a full page of one head
  constexpr int N = kChunkDims<T>, kPasses = kAppendValues / N;
  a.team = 32;
  while (a.team / (a.d / N) * kPasses < 1 << a.shift) a.team *= 2;
  return a.team <= 256 ? launch_append_prompts<T, 256>(a, units, s)
                       : launch_append_prompts<T, 512>(a, units, s);
}

}  // namespace

cudaError_t launch_q8_append(const Q8AppendArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_append<__nv_bfloat16>(a, s) : launch_append<float>(a, s);
}

cudaError_t launch_q8_read(Q8ReadArgs a, cudaStream_t s) {
  const int per_row = a.H * (a.d / 8);
  constexpr int kMany = 4;
  const bool many = a.n_rows * per_row >= 2LL * kMany * kReadThreads * sm_count();
  a.row_block = per_row < kReadThreads ? kReadThreads / per_row : 1;
  const int rows = a.row_block * (many ? kMany : 1);
  const dim3 grid((unsigned)((a.n_rows + rows - 1) / rows),
                  (per_row + kReadThreads - 1) / kReadThreads);
  if (many) q8_read_kernel<kMany><<<grid, kReadThreads, 0, s>>>(a);
  else q8_read_kernel<1><<<grid, kReadThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace lla

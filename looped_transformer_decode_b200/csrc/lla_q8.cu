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
#include <cfloat>
#include <cmath>

#include "lla_internal.cuh"
#include "lla_rows.cuh"

namespace lla {
namespace {

constexpr float kQ8Grow = 1.25f;

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

}  // namespace lla

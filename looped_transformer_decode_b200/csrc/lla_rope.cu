// Rotary positions as operators of their own: tables whose frequencies are scaled
// for contexts longer than the trained one, and the rotation of rows of heads (and
// its gradient) by a table, with half-split or interleaved pairs, on the whole head
// or on its first d_rope dims.
//
//   (y_a, y_b) = (x_a c - x_b s, x_a s + x_b c),  (c, s) = table[position][i]
//
// on the pairs (a, b) = (i, i + rd/2) or (2i, 2i + 1), i < rd/2; dims at or past rd
// are copied.  A rotation's transpose is its inverse, so the gradient with respect to
// x is the same kernel with s negated.
#include <cmath>

#include "lla_internal.cuh"
#include "lla_rows.cuh"

namespace lla {
namespace {

// Angles per position of each pair, as base^(-2 i / rd) scaled by kind.  All in fp64
// and rounded once, so that far positions keep fp32 accuracy.
struct RopeScale {
  int kind;
  bool marked;             // frequencies differ from the plain ones: the table says so
  double base, factor, low, span;   // yarn: the ramp over i starts at low, is span wide
};

// A thread walks kRun positions of one pair: one fp64 sincos, then turns by theta, four
// fp64 products a row whose roundings (kRun * 2^-52) stay far below those of far angles
// (position * 2^-53).  A table of 131072 x 64 pairs: 133 us with a power and a sincos per
// entry, 15 us this way; storing it takes 10.
constexpr int kRun = 16;
constexpr int kTableThreads = 256;

__global__ void __launch_bounds__(kTableThreads)
rope_table_scaled_kernel(int max_pos, int half, RopeScale sc, float2* table) {
  __shared__ double2 turn[kTableThreads];
  __shared__ double thetas[kTableThreads];
  if (threadIdx.x < half) {
    const int i = threadIdx.x;
    double theta = pow(sc.base, -2.0 * i / (2.0 * half));
    if (sc.kind == LLA_ROPE_SCALE_LINEAR) theta /= sc.factor;
    if (sc.kind == LLA_ROPE_SCALE_YARN) {
      double ramp = (i - sc.low) / sc.span;
      ramp = ramp < 0.0 ? 0.0 : ramp > 1.0 ? 1.0 : ramp;
      theta = theta * (1.0 - ramp) + theta / sc.factor * ramp;
    }
    double s, c;
    sincos(theta, &s, &c);
    turn[i] = make_double2(c, s);
    thetas[i] = theta;
  }
  __syncthreads();
  const int rows = kTableThreads / half, row = threadIdx.x / half, i = threadIdx.x - row * half;
  const long long pos0 = ((long long)blockIdx.x * rows + row) * kRun;
  if (row >= rows || pos0 >= max_pos) return;
  const int n = max_pos - pos0 < kRun ? (int)(max_pos - pos0) : kRun;
  const double2 t = turn[i];
  double s, c;
  sincos((double)pos0 * thetas[i], &s, &c);
  float2* out = table + pos0 * half + i;
  // the true angle is position * theta; entries are those of its fp64 rounding, as if each had
  // its own sincos: off by the rounding's error, against that at the run's first position
  const double theta = thetas[i], a0 = (double)pos0 * theta, e0 = fma((double)pos0, theta, -a0);
  for (int k = 0;; ++k, out += half) {
    const double p = (double)(pos0 + k), a = p * theta, e = e0 - fma(p, theta, -a);
    *out = make_float2((float)fma(-s, e, c), (float)fma(c, e, s));
    if (k + 1 == n) break;
    const double x = c * t.x - s * t.y;
    s = c * t.y + s * t.x;
    c = x;
  }
  if (sc.marked && pos0 == 0 && i == 0) table[0].y = -0.f;      // see scaled_table
}

// A thread rotates its chunk of kHeads heads of one token, 32 bytes of each in two 16-byte
// accesses, by table entries that it loads once: with one head a thread, the table's reads
// from L1 and L2 are twice the rows' bytes in bf16.
//
// a.tok_block tokens per block (one, over gridDim.y blocks, when a token has more than 256
// threads); a.groups threads share the chunks of a token's heads, neighbours in neighbouring
// heads.
constexpr int kRopeThreads = 256;

template <typename T, int kHeads>
__global__ void __launch_bounds__(kRopeThreads) rope_apply_kernel(RopeApplyArgs a) {
  constexpr int N = kChunkDims<T>;
  const int tpr = a.d / N, per_tok = a.groups * tpr;
  const int x = blockIdx.y * kRopeThreads + threadIdx.x;
  const int tl = x / per_tok, unit = x - tl * per_tok;
  const long long tok = (long long)blockIdx.x * a.tok_block + tl;
  if (tl >= a.tok_block || tok >= a.n_tok) return;
  const int g = unit / tpr, c = unit - g * tpr;
  const RowChunk rc = row_chunk<N>(c, a.d, a.rd, a.layout);
  const T* src = static_cast<const T*>(a.x) + tok * a.x_stride;
  T* dst = static_cast<T*>(a.y) + tok * a.y_stride;
  const int asked = __ldg(a.positions + tok);
  uint4 lo[kHeads], hi[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = j * a.groups + g;
    if (h < a.n_heads) {
      lo[j] = *reinterpret_cast<const uint4*>(src + h * a.d + rc.lo);
      hi[j] = *reinterpret_cast<const uint4*>(src + h * a.d + rc.hi);
    }
  }
  const int pos = checked_position(asked, a.rope_max_pos, a.status, unit == 0);
  Turn<N> turn;
  if (rc.rotary) {
    turn = load_turn<N>(a.rope + (size_t)pos * (a.rd / 2), rc);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) turn.s[j] *= a.sign;
  }
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = j * a.groups + g;
    if (h >= a.n_heads) break;
    T* row = dst + h * a.d;
    if (rc.rotary) {
      float v[N];
      load_run<N / 2>(reinterpret_cast<const T*>(&lo[j]), v);
      load_run<N / 2>(reinterpret_cast<const T*>(&hi[j]), v + N / 2);
      rotate_chunk<N>(turn, rc.split, v);
      store_chunk<N>(row, rc, v);
    } else {
      *reinterpret_cast<uint4*>(row + rc.lo) = lo[j];
      *reinterpret_cast<uint4*>(row + rc.hi) = hi[j];
    }
  }
}

template <typename T>
cudaError_t launch_rope_t(RopeApplyArgs a, cudaStream_t s) {
  constexpr int kHeads = 4;
  const int tpr = a.d / kChunkDims<T>;
  // Four heads a thread where that leaves two blocks per SM: 32768 bf16 tokens of 16 heads of
  // 128, half of each rotated, 48.4 us (87% of the copy rate); small calls want the threads.
  const bool many = a.n_tok * a.n_heads * tpr >= (long long)kHeads * kRopeThreads * 2 * sm_count();
  a.groups = many ? (a.n_heads + kHeads - 1) / kHeads : a.n_heads;
  const int per_tok = a.groups * tpr;
  a.tok_block = per_tok < kRopeThreads ? kRopeThreads / per_tok : 1;
  const int threads =
      per_tok < kRopeThreads ? (a.tok_block * per_tok + 31) / 32 * 32 : kRopeThreads;
  const dim3 grid((unsigned)((a.n_tok + a.tok_block - 1) / a.tok_block),
                  (per_tok + kRopeThreads - 1) / kRopeThreads);
  if (many) rope_apply_kernel<T, kHeads><<<grid, threads, 0, s>>>(a);
  else rope_apply_kernel<T, 1><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_table_scaled(const lla_cfg& c, const lla_rope_scaling& sc, int max_pos,
                                     float2* table, cudaStream_t s) {
  const int rd = rotary_dims(c);
  RopeScale k{};
  k.kind = sc.kind;
  k.marked = sc.kind != LLA_ROPE_SCALE_NONE && sc.factor != 1.0;
  k.base = (double)c.rope_base;
  k.factor = sc.factor;
  if (sc.kind == LLA_ROPE_SCALE_NTK) k.base = k.base * std::pow(sc.factor, rd / (rd - 2.0));
  if (sc.kind == LLA_ROPE_SCALE_YARN) {
    // pair index at which a position turns `turns` times over the trained context
    auto at = [&](double turns) {
      return rd * std::log(sc.orig_len / (2.0 * M_PI * turns)) / (2.0 * std::log(k.base));
    };
    const double lo = std::fmax(std::floor(at(sc.beta_fast > 0 ? sc.beta_fast : 32.0)), 0.0);
    const double hi = std::fmin(std::ceil(at(sc.beta_slow > 0 ? sc.beta_slow : 1.0)), rd - 1.0);
    k.low = lo;
    k.span = std::fmax(hi - lo, 0.001);
  }
  const int per_block = kTableThreads / (rd / 2) * kRun;
  rope_table_scaled_kernel<<<(unsigned)((max_pos - 1LL) / per_block + 1), kTableThreads, 0, s>>>(
      max_pos, rd / 2, k, table);
  return cudaGetLastError();
}

cudaError_t launch_rope_apply(const RopeApplyArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_rope_t<__nv_bfloat16>(a, s) : launch_rope_t<float>(a, s);
}

}  // namespace lla

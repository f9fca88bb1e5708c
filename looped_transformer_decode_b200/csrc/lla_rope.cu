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
  double base, factor, low, span;   // yarn: the ramp over i starts at low, is span wide
};

__global__ void rope_table_scaled_kernel(int max_pos, int half, RopeScale sc, float2* table) {
  const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (idx >= (long long)max_pos * half) return;
  const int pos = (int)(idx / half);
  const int i = (int)(idx % half);
  double theta = pow(sc.base, -2.0 * i / (2.0 * half));
  if (sc.kind == LLA_ROPE_SCALE_LINEAR) theta /= sc.factor;
  if (sc.kind == LLA_ROPE_SCALE_YARN) {
    double ramp = (i - sc.low) / sc.span;
    ramp = ramp < 0.0 ? 0.0 : ramp > 1.0 ? 1.0 : ramp;
    theta = theta * (1.0 - ramp) + theta / sc.factor * ramp;
  }
  double s, c;
  sincos((double)pos * theta, &s, &c);
  table[idx] = make_float2((float)c, (float)s);
}

// One thread per eight dims of one head's row (row_chunk's four pairs, or eight dims
// past the rotary ones).
template <typename T>
__global__ void __launch_bounds__(256) rope_apply_kernel(RopeApplyArgs a) {
  const int tpr = a.d / 8;
  const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long per_tok = (long long)a.n_heads * tpr;
  const long long tok = idx / per_tok;
  if (tok >= a.n_tok) return;
  const int rest = (int)(idx % per_tok);
  const int h = rest / tpr, c = rest % tpr;
  const int pos = checked_position(a.positions[tok], a.rope_max_pos, a.status,
                                   h == 0 && c == 0);
  const RowChunk rc = row_chunk(c, a.d, a.rd, a.layout);
  const T* x = static_cast<const T*>(a.x) + tok * a.x_stride + (long long)h * a.d;
  T* y = static_cast<T*>(a.y) + tok * a.y_stride + (long long)h * a.d;
  float v[8];
  load_chunk(x, rc, v);
  rotate_chunk(a.rope + (size_t)pos * (a.rd / 2), rc, a.sign, v);
  store_chunk(y, rc, v);
}

}  // namespace

cudaError_t launch_rope_table_scaled(const lla_cfg& c, const lla_rope_scaling& sc, int max_pos,
                                     float2* table, cudaStream_t s) {
  const int rd = rotary_dims(c);
  RopeScale k{};
  k.kind = sc.kind;
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
  const long long n = (long long)max_pos * (rd / 2);
  rope_table_scaled_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(max_pos, rd / 2, k, table);
  return cudaGetLastError();
}

cudaError_t launch_rope_apply(const RopeApplyArgs& a, cudaStream_t s) {
  const long long n = a.n_tok * a.n_heads * (a.d / 8);
  const long long blocks = (n + 255) / 256;
  if (a.bf16)
    rope_apply_kernel<__nv_bfloat16><<<(unsigned)blocks, 256, 0, s>>>(a);
  else
    rope_apply_kernel<float><<<(unsigned)blocks, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace lla

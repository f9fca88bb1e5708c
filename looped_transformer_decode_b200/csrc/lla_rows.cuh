// Rows of one head (d dims, fp32 or bf16) cut into chunks of eight dims, one thread
// each, such that both dims of every rotary pair belong to one thread:
//   interleaved pairs, and dims past the rotary ones   eight consecutive dims
//   half-split pairs                                    4 c .. 4 c + 3 and rd/2 above them
// rd and d are multiples of 32, so chunks never straddle the rotary dims' end.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "lla_internal.cuh"

namespace lla {

struct RowChunk {
  int lo, hi;    // first dim of each group of four
  int pair;      // first rotary pair, or -1 past the rotary dims
  bool split;    // half-split: v[j] pairs with v[j + 4]; else v[2 j] with v[2 j + 1]
};

__device__ __forceinline__ RowChunk row_chunk(int c, int d, int rd, int layout) {
  RowChunk r;
  if (c * 8 >= rd) {
    r.lo = c * 8;
    r.hi = r.lo + 4;
    r.pair = -1;
    r.split = false;
  } else if (layout == LLA_ROPE_HALF) {
    r.lo = c * 4;
    r.hi = rd / 2 + c * 4;
    r.pair = c * 4;
    r.split = true;
  } else {
    r.lo = c * 8;
    r.hi = r.lo + 4;
    r.pair = c * 4;
    r.split = false;
  }
  return r;
}

__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  v[0] = f.x;
  v[1] = f.y;
  v[2] = f.z;
  v[3] = f.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* v) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(u.x << 16);
  v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16);
  v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
}

template <typename T>
__device__ __forceinline__ void load_chunk(const T* row, const RowChunk& rc, float* v) {
  load4(row + rc.lo, v);
  load4(row + rc.hi, v + 4);
}
template <typename T>
__device__ __forceinline__ void store_chunk(T* row, const RowChunk& rc, const float* v) {
  store4(row + rc.lo, v);
  store4(row + rc.hi, v + 4);
}

// Rotate a chunk by the table row of its position; sign = -1 rotates back.
__device__ __forceinline__ void rotate_chunk(const float2* table_row, const RowChunk& rc,
                                             float sign, float* v) {
  if (rc.pair < 0) return;
  const float4* t = reinterpret_cast<const float4*>(table_row + rc.pair);
  const float4 t0 = __ldg(t), t1 = __ldg(t + 1);
  const float c[4] = {t0.x, t0.z, t1.x, t1.z};
  const float s[4] = {sign * t0.y, sign * t0.w, sign * t1.y, sign * t1.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int ia = rc.split ? j : 2 * j, ib = rc.split ? j + 4 : 2 * j + 1;
    const float a = v[ia], b = v[ib];
    v[ia] = a * c[j] - b * s[j];
    v[ib] = a * s[j] + b * c[j];
  }
}

// A position clamped into the table; out of range sets the status bit.
__device__ __forceinline__ int checked_position(int pos, int max_pos, int32_t* status, bool tell) {
  if (pos < 0 || pos >= max_pos) {
    if (tell && status) atomicOr(status, LLA_STATUS_POSITION_RANGE);
    pos = pos < 0 ? 0 : max_pos - 1;
  }
  return pos;
}

}  // namespace lla

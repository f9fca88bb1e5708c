// Rows of one head (d dims, fp32 or bf16) cut into chunks of N dims (8 or 16), one thread
// each, such that both dims of every rotary pair belong to one thread: two runs of N / 2
// dims, half of the rotary dims apart (past them: half of the others).  Neighbouring threads
// hold neighbouring runs, so a warp's access to its first runs, or its second, is contiguous.
// The first run holds the first dims of half-split pairs and the second run the second ones;
// interleaved pairs lie within a run.  rd and d are multiples of 32.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "lla_internal.cuh"

namespace lla {

// Dims in two 16-byte accesses.
template <typename T>
constexpr int kChunkDims = 32 / (int)sizeof(T);

struct RowChunk {
  int lo, hi;    // first dim of each run
  bool rotary;   // else past the rotary dims
  bool split;    // half-split pairs (v[j], v[j + N/2]); else (v[2 j], v[2 j + 1])
};

template <int N>
__device__ __forceinline__ RowChunk row_chunk(int c, int d, int rd, int layout) {
  RowChunk r;
  r.rotary = c * N < rd;
  r.split = layout == LLA_ROPE_HALF;
  const int past = r.rotary ? 0 : rd / 2;
  r.lo = past + c * (N / 2);
  r.hi = r.lo + (r.rotary ? rd / 2 : (d - rd) / 2);
  return r;
}

// Four or eight elements to fp32 and back.
template <int M>
__device__ __forceinline__ void load_run(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < M; i += 4) {
    const float4 f = *reinterpret_cast<const float4*>(p + i);
    v[i] = f.x;
    v[i + 1] = f.y;
    v[i + 2] = f.z;
    v[i + 3] = f.w;
  }
}
__device__ __forceinline__ void unpack_bf16x2(uint32_t u, float* v) {
  v[0] = __uint_as_float(u << 16);
  v[1] = __uint_as_float(u & 0xffff0000u);
}
template <int M>
__device__ __forceinline__ void load_run(const __nv_bfloat16* p, float* v) {
  if constexpr (M == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    unpack_bf16x2(u.x, v);
    unpack_bf16x2(u.y, v + 2);
    unpack_bf16x2(u.z, v + 4);
    unpack_bf16x2(u.w, v + 6);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    unpack_bf16x2(u.x, v);
    unpack_bf16x2(u.y, v + 2);
  }
}
__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}
template <int M>
__device__ __forceinline__ void store_run(float* p, const float* v) {
#pragma unroll
  for (int i = 0; i < M; i += 4)
    *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int M>
__device__ __forceinline__ void store_run(__nv_bfloat16* p, const float* v) {
  if constexpr (M == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]),
                                              bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
}

template <int N, typename T>
__device__ __forceinline__ void load_chunk(const T* row, const RowChunk& rc, float* v) {
  load_run<N / 2>(row + rc.lo, v);
  load_run<N / 2>(row + rc.hi, v + N / 2);
}
template <int N, typename T>
__device__ __forceinline__ void store_chunk(T* row, const RowChunk& rc, const float* v) {
  store_run<N / 2>(row + rc.lo, v);
  store_run<N / 2>(row + rc.hi, v + N / 2);
}

// (cos, sin) of a chunk's pairs at a position: its table row.
template <int N>
struct Turn {
  float c[N / 2], s[N / 2];
};
template <int N>
__device__ __forceinline__ Turn<N> load_turn(const float2* table_row, const RowChunk& rc) {
  Turn<N> t;
  const float4* lo = reinterpret_cast<const float4*>(table_row + (rc.split ? rc.lo : rc.lo / 2));
  const float4* hi = rc.split ? lo + N / 8 : reinterpret_cast<const float4*>(table_row + rc.hi / 2);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const float4 f = i < N / 8 ? __ldg(lo + i) : __ldg(hi + i - N / 8);
    t.c[2 * i] = f.x;
    t.s[2 * i] = f.y;
    t.c[2 * i + 1] = f.z;
    t.s[2 * i + 1] = f.w;
  }
  return t;
}

// (a, b) turned by (c, s), every product rounded: fused into the sum, the two outputs would round
// differently from elementary fp32 operations, and a code next to a half step with them.
__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
  a = x;
}

// Rotate a chunk of a head's rotary dims.
template <int N>
__device__ __forceinline__ void rotate_chunk(const Turn<N>& t, bool split, float* v) {
  if (split) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) rotate_pair(v[j], v[j + N / 2], t.c[j], t.s[j]);
  } else {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) rotate_pair(v[2 * j], v[2 * j + 1], t.c[j], t.s[j]);
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

// Rotary positions: the angle arithmetic and the 16-element items that the rotary kernel and the
// index quantiser share.
//
// A rotary part of `rot` dims at `offset` of each head holds rot/2 pairs (a, b); pair i of a token
// at position p turns by the angle p * f[i]:
//     a' = m (a cos - b sin),   b' = m (b cos + a sin)
// (`inverse` turns back: sin -> -sin). The half layout pairs dim i with dim i + rot/2, the
// interleaved layout dims 2i and 2i+1. Dims outside the part are copied.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace dsa {

constexpr int kVec = 8;             // elements per vector
constexpr int kItem = 2 * kVec;     // elements per item: two vectors, a and b

template <int DT>
struct Elem;
template <>
struct Elem<DSA_DTYPE_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float get(T x) { return __bfloat162float(x); }
  static __device__ __forceinline__ T put(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<DSA_DTYPE_F16> {
  using T = __half;
  static __device__ __forceinline__ float get(T x) { return __half2float(x); }
  static __device__ __forceinline__ T put(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<DSA_DTYPE_F32> {
  using T = float;
  static __device__ __forceinline__ float get(T x) { return x; }
  static __device__ __forceinline__ T put(float x) { return x; }
};

// (cos, sin) of p * f, times the magnitude. At position 200000 an angle formed in fp32 would be off
// by up to 200000 * 2^-24 = 0.01 radians, so the number of turns is formed in 64 bits and only its
// fraction, in [-1/2, 1/2], goes on in fp32.
__device__ __forceinline__ float2 rotary_cos_sin(int32_t p, float f, const RotaryArgs& r) {
  constexpr double kInvTwoPi = 0.15915494309189535;
  const double turns = static_cast<double>(p) * (static_cast<double>(f) * kInvTwoPi);
  float s, c;
  sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
  if (r.inverse) s = -s;
  return make_float2(c * r.mscale, s * r.mscale);
}

// One pair turned, with its roundings spelled out, so that every kernel turns it to the same bits.
__device__ __forceinline__ void rotary_pair(float2 cs, float& a, float& b) {
  const float a0 = a, b0 = b;
  a = __fmaf_rn(a0, cs.x, -__fmul_rn(b0, cs.y));
  b = __fmaf_rn(b0, cs.x, __fmul_rn(a0, cs.y));
}

// Eight consecutive elements: as they lie in memory, as fp32, and back. The pointers are 16-byte aligned.
template <int DT>
struct RawVec {
  uint4 w[DT == DSA_DTYPE_F32 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ RawVec<DT> load_raw(const typename Elem<DT>::T* p) {
  RawVec<DT> r;
  r.w[0] = *reinterpret_cast<const uint4*>(p);
  if constexpr (DT == DSA_DTYPE_F32) r.w[1] = *reinterpret_cast<const uint4*>(p + 4);
  return r;
}
template <int DT>
__device__ __forceinline__ void unpack_raw(const RawVec<DT>& r, float (&v)[kVec]) {
  const typename Elem<DT>::T* e = reinterpret_cast<const typename Elem<DT>::T*>(&r);
#pragma unroll
  for (int i = 0; i < kVec; ++i) v[i] = Elem<DT>::get(e[i]);
}
template <int DT>
__device__ __forceinline__ void load_vec(const typename Elem<DT>::T* p, float (&v)[kVec]) {
  unpack_raw<DT>(load_raw<DT>(p), v);
}
template <int DT>
__device__ __forceinline__ void store_vec(typename Elem<DT>::T* p, const float (&v)[kVec]) {
  if constexpr (DT == DSA_DTYPE_F32) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint4 raw;
    typename Elem<DT>::T* e = reinterpret_cast<typename Elem<DT>::T*>(&raw);
#pragma unroll
    for (int i = 0; i < kVec; ++i) e[i] = Elem<DT>::put(v[i]);
    *reinterpret_cast<uint4*>(p) = raw;
  }
}

// Item j of a head of d elements (d / 16 items): the two vectors it covers. The first rot/16 items
// are the rotary part (half layout: vector j and its partner rot/2 further; interleaved: two
// neighbours, each with its own pairs), the others neighbours of what is left.
struct Item {
  int a, b;   // element offsets in the head
  int f;      // first frequency (half: of both vectors; interleaved: of a, b's are f + 4), -1: copied
};
__device__ __forceinline__ Item rotary_item(int j, const RotaryArgs& r) {
  const int n_rot = r.rot / kItem;
  if (j < n_rot) {
    if (r.interleaved) return Item{r.offset + j * kItem, r.offset + j * kItem + kVec, j * kVec};
    return Item{r.offset + j * kVec, r.offset + r.rot / 2 + j * kVec, j * kVec};
  }
  int a = (j - n_rot) * kItem, b = a + kVec;
  if (a >= r.offset) a += r.rot;
  if (b >= r.offset) b += r.rot;
  return Item{a, b, -1};
}

// Turns an item's values; cs: the (cos, sin) of its eight frequencies.
template <bool INTERLEAVED>
__device__ __forceinline__ void rotary_turn(const float2* cs, float (&a)[kVec], float (&b)[kVec]) {
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    if constexpr (INTERLEAVED) {
      float(&v)[kVec] = i < 4 ? a : b;
      rotary_pair(cs[i], v[2 * (i & 3)], v[2 * (i & 3) + 1]);
    } else {
      rotary_pair(cs[i], a[i], b[i]);
    }
  }
}

}  // namespace dsa

// The E4M3 inputs of the indexer for sm_100a: queries and keys rotated and quantised in one pass,
// keys written into the paged cache, and a paged prefix read back.
//
// A row of n values (a token's H x d query values, or its d key values) becomes codes and one scale:
//     scale = max(absmax / 448, FLT_MIN) (1 for an all-zero row),   code = E4M3(x / scale),
// with the row's values in fp32 after the rotation (not rounded to the input's type in between),
// both divisions IEEE fp32 and the code rounded to nearest even. Bound by HBM (long inputs) or by
// one launch (a decode step): each value is read once and kept in registers between the row's
// maximum and its codes.
#include <cfloat>

#include <cuda_fp8.h>

#include "rotary.cuh"

namespace dsa {

constexpr int kQuantThreads = 128;

// Whether a quotient y of magnitude >= 2^-6 lies within four ulps of a border between two codes (their
// middle: the mantissa bits behind E4M3's three are 1000...).
__device__ __forceinline__ bool near_border(float y) {
  const uint32_t u = __float_as_uint(y);
  return ((u + 4u) & 0xFFFFFu) - 0x80000u <= 8u;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// NaN counts as 0 and an infinity as the largest fp32 value of its sign.
__device__ __forceinline__ float finite(float v) {
  if (fabsf(v) <= FLT_MAX) return v;
  return isnan(v) ? 0.0f : copysignf(FLT_MAX, v);
}
// The larger of two non-negative values, NaN if either is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// G threads of a CTA take one row of up to NI * G items, so a CTA takes 128 / G rows: short rows (up to
// 32 items) one item a thread, so that one warp holds whole rows and needs no barrier for their maxima,
// others all 128 threads. The values stay packed as they were loaded (every load of a row is in flight
// at once, and six CTAs fit an SM) and are rotated twice, for the maximum and for the codes. (As fp32
// with 256 threads, two CTAs an SM: 301 us for 16384 x 64 x 128 bf16 values, against a floor of 62.)
template <int DT, int G, int NI>
__global__ void __launch_bounds__(kQuantThreads, G > 32 && NI <= 4 ? 6 : 1) index_quantise_kernel(const QuantParams p) {
  using T = typename Elem<DT>::T;
  constexpr int kRows = kQuantThreads / G;
  extern __shared__ float2 cs_all[];
  __shared__ float warp_max[kQuantThreads / 32];
  const int half = p.r.rot / 2;
  const int g = threadIdx.x / G, l = threadIdx.x % G;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows, t = t0 + g;
  const int per_head = p.d / kItem, n = p.H * per_head;
  int64_t dst = -1;
  if (t < p.T) {
    dst = p.slots ? p.slots[t] : t;
    if (p.slots && (dst < -1 || dst >= p.n_slots)) {
      if (l == 0) record_error(p.hdr, DSA_ERR_DEVICE, DETAIL_BAD_SLOT);
      dst = -1;
    }
  }
  // i / per_head for i < 1024 (per_head_inv = ceil(2^20 / per_head)).
  auto head_of = [&](int i) { return static_cast<int>((static_cast<uint32_t>(i) * p.per_head_inv) >> 20); };
  RawVec<DT> ra[NI], rb[NI];
  const T* row = static_cast<const T*>(p.x) + t * p.xs_t;
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int i = l + k * G;
    if (dst < 0 || i >= n) continue;
    const int head = head_of(i);
    const Item it = rotary_item(i - head * per_head, p.r);
    const T* h = row + head * p.xs_h;
    ra[k] = load_raw<DT>(h + it.a);
    rb[k] = load_raw<DT>(h + it.b);
  }
  for (int i = threadIdx.x; i < kRows * half; i += kQuantThreads) {
    const int64_t tt = t0 + i / half;
    if (tt < p.T) cs_all[i] = rotary_cos_sin(p.r.positions[tt], p.r.inv_freq[i % half], p.r);
  }
  __syncthreads();
  float top = 0.0f;
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int i = l + k * G;
    if (dst < 0 || i >= n) continue;
    float a[kVec], b[kVec];
    unpack_raw<DT>(ra[k], a);
    unpack_raw<DT>(rb[k], b);
    rotary_turn(rotary_item(i - head_of(i) * per_head, p.r), p.r, cs_all + g * half, a, b);
#pragma unroll
    for (int e = 0; e < kVec; ++e) top = max_or_nan(top, max_or_nan(fabsf(a[e]), fabsf(b[e])));
  }
#pragma unroll
  for (int off = (G < 32 ? G : 32) / 2; off > 0; off >>= 1)
    top = max_or_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
  if constexpr (G > 32) {
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < G / 32; ++w) top = max_or_nan(top, warp_max[w]);
  }
  if (dst < 0) return;
  // A row with a value that is not finite: its maximum is not finite either, and is taken over the others.
  const bool mend = !(top <= FLT_MAX);
  if (mend) {
    if (l == 0) record_error(p.hdr, DSA_ERR_DEVICE, DETAIL_NOT_FINITE);
    top = 0.0f;
    for (int i = 0; i < n; ++i) {  // (every thread goes through the whole row: it is a bad one)
      const int head = head_of(i);
      const Item it = rotary_item(i - head * per_head, p.r);
      float a[kVec], b[kVec];
      load_vec<DT>(row + head * p.xs_h + it.a, a);
      load_vec<DT>(row + head * p.xs_h + it.b, b);
      rotary_turn(it, p.r, cs_all + g * half, a, b);
#pragma unroll 1
      for (int e = 0; e < kVec; ++e) top = fmaxf(top, fmaxf(fabsf(finite(a[e])), fabsf(finite(b[e]))));
    }
  }
  const float scale = top > 0.0f ? fmaxf(__fdiv_rn(top, 448.0f), FLT_MIN) : 1.0f;
  // The product with the rounded reciprocal is within two ulps of the quotient. It has the quotient's
  // code unless it is that close to a border between codes or, where the codes' steps no longer scale
  // with the value, below 2^-6: the item is then divided, a few in a hundred.
  const float inv = __fdiv_rn(1.0f, scale);
  uint8_t* out = p.codes + dst * (static_cast<int64_t>(p.H) * p.d);
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int i = l + k * G;
    if (i >= n) continue;
    const int head = head_of(i);
    const Item it = rotary_item(i - head * per_head, p.r);
    float v[2][kVec], y[2][kVec];
    unpack_raw<DT>(ra[k], v[0]);
    unpack_raw<DT>(rb[k], v[1]);
    rotary_turn(it, p.r, cs_all + g * half, v[0], v[1]);
    bool divide = mend;
    float least = INFINITY;
#pragma unroll
    for (int e = 0; e < 2 * kVec; ++e) {
      y[e / kVec][e % kVec] = v[e / kVec][e % kVec] * inv;
      divide |= near_border(y[e / kVec][e % kVec]);
      least = fminf(least, fabsf(y[e / kVec][e % kVec]));
    }
    if (divide || !(least >= 0x1p-6f)) {
#pragma unroll
      for (int e = 0; e < 2 * kVec; ++e)
        y[e / kVec][e % kVec] = __fdiv_rn(mend ? finite(v[e / kVec][e % kVec]) : v[e / kVec][e % kVec], scale);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
      *reinterpret_cast<uint2*>(out + head * p.d + (u ? it.b : it.a)) =
          make_uint2(e4m3x4(y[u][0], y[u][1], y[u][2], y[u][3]), e4m3x4(y[u][4], y[u][5], y[u][6], y[u][7]));
  }
  if (l == 0) p.scale[dst] = scale;
}

template <int DT, int G, int NI>
static dsa_status launch_quantise_g(const QuantParams& p, cudaStream_t stream) {
  constexpr int kRows = kQuantThreads / G;
  const size_t smem = static_cast<size_t>(kRows) * (p.r.rot / 2) * sizeof(float2);
  const int64_t grid = (p.T + kRows - 1) / kRows;
  index_quantise_kernel<DT, G, NI><<<static_cast<unsigned>(grid), kQuantThreads, smem, stream>>>(p);
  return cuda_status(cudaGetLastError());
}

template <int DT>
static dsa_status launch_quantise_t(const QuantParams& p, cudaStream_t stream) {
  const int n = p.H * (p.d / kItem);
  if (n <= 8) return launch_quantise_g<DT, 8, 1>(p, stream);
  if (n <= 16) return launch_quantise_g<DT, 16, 1>(p, stream);
  if (n <= 32) return launch_quantise_g<DT, 32, 1>(p, stream);
  if (n <= 4 * kQuantThreads) return launch_quantise_g<DT, kQuantThreads, 4>(p, stream);
  return launch_quantise_g<DT, kQuantThreads, kQuantMaxRow / kItem / kQuantThreads>(p, stream);
}

dsa_status launch_quantise(const QuantParams& in, int dtype, cudaStream_t stream) {
  QuantParams p = in;
  const uint32_t per_head = p.d / kItem;
  p.per_head_inv = ((1u << 20) + per_head - 1) / per_head;
  if (dtype == DSA_DTYPE_BF16) return launch_quantise_t<DSA_DTYPE_BF16>(p, stream);
  if (dtype == DSA_DTYPE_F16) return launch_quantise_t<DSA_DTYPE_F16>(p, stream);
  return launch_quantise_t<DSA_DTYPE_F32>(p, stream);
}

// ------------------------------------------------------------------------------------------
// Cache read. A CTA takes kReadRows output rows: its first threads find each row's request (a
// binary search over the row offsets) and cache row, then all copy 16 codes at a time.
// ------------------------------------------------------------------------------------------
constexpr int kReadThreads = 256;
constexpr int kReadRows = 64;

template <int VT>  // values' type, or -1 for none
__global__ void __launch_bounds__(kReadThreads) index_cache_read_kernel(const ReadParams p) {
  __shared__ int64_t src[kReadRows];
  __shared__ float scale[kReadRows];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kReadRows;
  if (threadIdx.x < kReadRows) {
    const int64_t r = r0 + threadIdx.x;
    int64_t at = -1;
    if (r < p.total && r >= p.cu[0] && r < p.cu[p.B]) {
      int lo = 0, hi = p.B;  // cu[lo] <= r < cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid] <= r) lo = mid;
        else hi = mid;
      }
      const int64_t pos = r - p.cu[lo] + (p.starts ? p.starts[lo] : 0);
      const int64_t lb = pos / p.block_size;
      int blk = -1;
      if (pos >= 0 && lb < p.max_blocks) blk = p.block_table[static_cast<int64_t>(lo) * p.max_blocks + lb];
      if (blk >= 0 && blk < p.n_blocks) at = static_cast<int64_t>(blk) * p.block_size + pos % p.block_size;
      else record_error(p.hdr, DSA_ERR_DEVICE, DETAIL_BAD_BLOCK_TABLE);
      // a row whose block is bad reads as zeros with scale 1
      const float s = at >= 0 ? p.k_scale_cache[at] : 1.0f;
      scale[threadIdx.x] = s;
      if (p.out_scale) p.out_scale[r] = s;
      if (at < 0) at = -2;
    }
    src[threadIdx.x] = at;
  }
  __syncthreads();
  const int per_row = p.d / 16;
  for (int i = threadIdx.x; i < kReadRows * per_row; i += kReadThreads) {
    const int k = i / per_row, c = (i % per_row) * 16;
    const int64_t at = src[k];
    if (at == -1) continue;
    const uint4 raw = at >= 0 ? *reinterpret_cast<const uint4*>(p.k_cache + at * p.d + c) : make_uint4(0, 0, 0, 0);
    const int64_t o = (r0 + k) * p.d + c;
    if (p.out_codes) *reinterpret_cast<uint4*>(p.out_codes + o) = raw;
    if constexpr (VT >= 0) {
      const float s = scale[k];
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
      float v[2][kVec];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __nv_fp8x2_storage_t two = static_cast<__nv_fp8x2_storage_t>(w[j >> 1] >> ((j & 1) * 16));
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
        v[j >> 2][(j & 3) * 2] = f.x * s;
        v[j >> 2][(j & 3) * 2 + 1] = f.y * s;
      }
      typename Elem<VT>::T* ov = static_cast<typename Elem<VT>::T*>(p.out_values) + o;
      store_vec<VT>(ov, v[0]);
      store_vec<VT>(ov + kVec, v[1]);
    }
  }
}

dsa_status launch_cache_read(const ReadParams& p, int values, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((p.total + kReadRows - 1) / kReadRows);
  if (!p.out_values) index_cache_read_kernel<-1><<<grid, kReadThreads, 0, stream>>>(p);
  else if (values == DSA_DTYPE_BF16) index_cache_read_kernel<DSA_DTYPE_BF16><<<grid, kReadThreads, 0, stream>>>(p);
  else if (values == DSA_DTYPE_F16) index_cache_read_kernel<DSA_DTYPE_F16><<<grid, kReadThreads, 0, stream>>>(p);
  else index_cache_read_kernel<DSA_DTYPE_F32><<<grid, kReadThreads, 0, stream>>>(p);
  return cuda_status(cudaGetLastError());
}

}  // namespace dsa

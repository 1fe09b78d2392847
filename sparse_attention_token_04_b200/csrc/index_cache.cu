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
// The largest of three magnitudes, NaN if any is.
__device__ __forceinline__ float max_or_nan(float a, float b, float c) {
  float m;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return m;
}
// The codes of four quotients from products with the reciprocal, taken a little (2^-21) too small (lo)
// and too large (hi). The rounded reciprocal's product is within 2^-22 of the quotient, so where both
// give the same codes they are the quotients'; else `differ` is set.
__device__ __forceinline__ uint32_t e4m3x4_of(const float* v, float lo, float hi, bool& differ) {
  const uint32_t x = e4m3x4(v[0] * lo, v[1] * lo, v[2] * lo, v[3] * lo);
  differ |= x != e4m3x4(v[0] * hi, v[1] * hi, v[2] * hi, v[3] * hi);
  return x;
}

// Makes the compiler take the values as new: it would keep the first rotation's results, twice the
// registers, for the second.
template <int DT>
__device__ __forceinline__ void keep_packed(RawVec<DT>& r) {
#pragma unroll
  for (uint4& w : r.w) asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w));
}

// The rare paths, out of line so that they hold no registers of the kernel's: the maximum of a row with
// values that are not finite, over the others, and an item's codes by division.
template <int DT, bool INTERLEAVED>
static __device__ __noinline__ float finite_max(const QuantParams* p, const typename Elem<DT>::T* row, const float2* cs) {
  const int per_head = p->d / kItem;
  float top = 0.0f;
#pragma unroll 1
  for (int i = 0; i < p->H * per_head; ++i) {
    const Item it = rotary_item(i % per_head, p->r);
    const typename Elem<DT>::T* h = row + (i / per_head) * p->xs_h;
    float a[kVec], b[kVec];
    load_vec<DT>(h + it.a, a);
    load_vec<DT>(h + it.b, b);
    if (it.f >= 0) rotary_turn<INTERLEAVED>(cs + it.f, a, b);
#pragma unroll
    for (int e = 0; e < kVec; ++e) top = fmaxf(top, fmaxf(fabsf(finite(a[e])), fabsf(finite(b[e]))));
  }
  return top;
}
template <int DT, bool INTERLEAVED>
static __device__ __noinline__ void divided_item(const typename Elem<DT>::T* a, const typename Elem<DT>::T* b,
                                                 const float2* cs, float scale, uint8_t* out_a, uint8_t* out_b) {
  float v[2][kVec];
  load_vec<DT>(a, v[0]);
  load_vec<DT>(b, v[1]);
  if (cs) rotary_turn<INTERLEAVED>(cs, v[0], v[1]);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[u][e] = __fdiv_rn(finite(v[u][e]), scale);
    *reinterpret_cast<uint2*>(u ? out_b : out_a) =
        make_uint2(e4m3x4(v[u][0], v[u][1], v[u][2], v[u][3]), e4m3x4(v[u][4], v[u][5], v[u][6], v[u][7]));
  }
}

// G threads of a CTA take one row, so a CTA takes 128 / G rows: rows of up to 32 items one item a
// thread (one warp then holds whole rows and needs no barrier for their maxima), others all 128
// threads. A thread has the same item of every (128 / items of a head)th head, so that it finds its
// offsets and the eight (cos, sin) that it needs once. The values stay packed as they were loaded (every
// load of a row is in flight at once, and six CTAs fit an SM) and are rotated twice, for the maximum and
// for the codes.
template <int DT, bool INTERLEAVED, int G, int NI>
__global__ void __launch_bounds__(kQuantThreads, G > 32 && NI <= 4 ? 6 : 1) index_quantise_kernel(const __grid_constant__ QuantParams p) {
  using T = typename Elem<DT>::T;
  constexpr int kRows = kQuantThreads / G;
  extern __shared__ __align__(16) float2 cs_all[];
  __shared__ float warp_max[kQuantThreads / 32];
  const int half = p.r.rot / 2;
  const int g = threadIdx.x / G, l = threadIdx.x % G;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows, t = t0 + g;
  const int per_head = p.d / kItem, head0 = l / per_head, heads = G / per_head;
  const Item it = rotary_item(l - head0 * per_head, p.r);
  // The thread's items: heads head0, head0 + heads, ...
  const int last = head0 < heads || NI == 1 ? p.H : 0;
  int64_t dst = -1;
  if (t < p.T) {
    dst = p.slots ? p.slots[t] : t;
    if (p.slots && (dst < -1 || dst >= p.n_slots)) {
      if (l == 0) record_error(p.hdr, DSA_ERR_DEVICE, DETAIL_BAD_SLOT);
      dst = -1;
    }
  }
  RawVec<DT> ra[NI], rb[NI];
  const T* row = static_cast<const T*>(p.x) + t * p.xs_t;
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int head = head0 + k * heads;
    if (dst < 0 || head >= last) continue;
    const T* h = row + head * p.xs_h;
    ra[k] = load_raw<DT>(h + it.a);
    rb[k] = load_raw<DT>(h + it.b);
  }
  for (int i = threadIdx.x; i < kRows * half; i += kQuantThreads) {
    const int64_t tt = t0 + i / half;
    if (tt < p.T) cs_all[i] = rotary_cos_sin(p.r.positions[tt], p.r.inv_freq[i % half], p.r);
  }
  __syncthreads();
  float2 cs[kVec];
  if (it.f >= 0) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) cs[i] = cs_all[g * half + it.f + i];
  }
  auto turned = [&](const RawVec<DT>& xa, const RawVec<DT>& xb, float (&a)[kVec], float (&b)[kVec]) {
    unpack_raw<DT>(xa, a);
    unpack_raw<DT>(xb, b);
    if (it.f >= 0) rotary_turn<INTERLEAVED>(cs, a, b);
  };
  float top = 0.0f;
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    if (dst < 0 || head0 + k * heads >= last) continue;
    float a[kVec], b[kVec];
    turned(ra[k], rb[k], a, b);
#pragma unroll
    for (int e = 0; e < kVec; ++e) top = max_or_nan(top, a[e], b[e]);
  }
#pragma unroll
  for (int off = (G < 32 ? G : 32) / 2; off > 0; off >>= 1)
    top = max_or_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, off), 0.0f);
  if constexpr (G > 32) {
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < G / 32; ++w) top = max_or_nan(top, warp_max[w], 0.0f);
  }
  if (dst < 0) return;
  // A row with a value that is not finite: its maximum is not finite either, and is found anew by every
  // thread from the whole row.
  const bool mend = !(top <= FLT_MAX);
  if (mend) {
    if (l == 0) record_error(p.hdr, DSA_ERR_DEVICE, DETAIL_NOT_FINITE);
    top = finite_max<DT, INTERLEAVED>(&p, row, cs_all + g * half);
  }
  const float scale = top > 0.0f ? fmaxf(__fdiv_rn(top, 448.0f), FLT_MIN) : 1.0f;
  const float inv = __fdiv_rn(1.0f, scale), lo = inv * (1.0f - 0x1p-21f), hi = inv * (1.0f + 0x1p-21f);
  uint8_t* out = p.codes + dst * (static_cast<int64_t>(p.H) * p.d);
  uint32_t again = 0;                           // items to be divided
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int head = head0 + k * heads;
    if (head >= last) continue;
    float v[2][kVec];
    keep_packed(ra[k]);
    keep_packed(rb[k]);
    turned(ra[k], rb[k], v[0], v[1]);
    bool differ = mend;
#pragma unroll
    for (int u = 0; u < 2; ++u)
      *reinterpret_cast<uint2*>(out + head * p.d + (u ? it.b : it.a)) =
          make_uint2(e4m3x4_of(v[u], lo, hi, differ), e4m3x4_of(v[u] + 4, lo, hi, differ));
    again |= static_cast<uint32_t>(differ) << k;
  }
  // A few items in a thousand, or all of a row that is mended, read again.
#pragma unroll 1
  for (int k = 0; again; ++k, again >>= 1) {
    if (!(again & 1u)) continue;
    const int head = head0 + k * heads;
    const T* h = row + head * p.xs_h;
    divided_item<DT, INTERLEAVED>(h + it.a, h + it.b, it.f >= 0 ? cs_all + g * half + it.f : nullptr, scale,
                                  out + head * p.d + it.a, out + head * p.d + it.b);
  }
  if (l == 0) p.scale[dst] = scale;
}

template <int DT, bool INTERLEAVED, int G, int NI>
static dsa_status launch_quantise_g(const QuantParams& p, cudaStream_t stream) {
  constexpr int kRows = kQuantThreads / G;
  const size_t smem = static_cast<size_t>(kRows) * (p.r.rot / 2) * sizeof(float2);
  const int64_t grid = (p.T + kRows - 1) / kRows;
  index_quantise_kernel<DT, INTERLEAVED, G, NI><<<static_cast<unsigned>(grid), kQuantThreads, smem, stream>>>(p);
  return cuda_status(cudaGetLastError());
}

template <int DT, bool INTERLEAVED>
static dsa_status launch_quantise_t(const QuantParams& p, cudaStream_t stream) {
  const int per_head = p.d / kItem, n = p.H * per_head;
  if (n <= 8) return launch_quantise_g<DT, INTERLEAVED, 8, 1>(p, stream);
  if (n <= 16) return launch_quantise_g<DT, INTERLEAVED, 16, 1>(p, stream);
  if (n <= 32) return launch_quantise_g<DT, INTERLEAVED, 32, 1>(p, stream);
  if (p.H <= 4 * (kQuantThreads / per_head)) return launch_quantise_g<DT, INTERLEAVED, kQuantThreads, 4>(p, stream);
  return launch_quantise_g<DT, INTERLEAVED, kQuantThreads, 8>(p, stream);
}

// Rows that a thread can hold: eight items, each of another head (8 * (128 / items of a head) heads).
bool quantise_row_fits(int H, int d) { return d <= kQuantThreads * kItem && H <= 8 * (kQuantThreads * kItem / d); }

dsa_status launch_quantise(const QuantParams& p, int dtype, cudaStream_t stream) {
  if (p.r.interleaved) {
    if (dtype == DSA_DTYPE_BF16) return launch_quantise_t<DSA_DTYPE_BF16, true>(p, stream);
    if (dtype == DSA_DTYPE_F16) return launch_quantise_t<DSA_DTYPE_F16, true>(p, stream);
    return launch_quantise_t<DSA_DTYPE_F32, true>(p, stream);
  }
  if (dtype == DSA_DTYPE_BF16) return launch_quantise_t<DSA_DTYPE_BF16, false>(p, stream);
  if (dtype == DSA_DTYPE_F16) return launch_quantise_t<DSA_DTYPE_F16, false>(p, stream);
  return launch_quantise_t<DSA_DTYPE_F32, false>(p, stream);
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

// The E4M3 inputs of the indexer for sm_100a: queries and keys rotated and quantised in one pass,
// keys written into the paged cache, and a paged prefix read back.
//
// A row of n values (a token's H x d query values, or its d key values) becomes codes and one scale:
//     scale = max(absmax / 448, FLT_MIN) (1 for an all-zero row),   code = E4M3(x / scale),
// with the row's values in fp32 after the rotation (not rounded to the input's type in between),
// both divisions IEEE fp32 and the code rounded to nearest even. Bound by HBM (long inputs) or by
// one launch (a decode step): each value is read once and kept in registers between the row's
// maximum and its codes. 16384 tokens of 64 heads x 128, bf16, half of each head rotated: 89 us,
// 4.5 TB/s, where neither is full (62% of the issue slots, DRAM at 52%): with 20 warps an SM a row's loads,
// its maximum over the CTA and its codes follow one another. 32 keys of 128 into the cache: 2.8 us. The
// instance for rows of more than four passes is far slower (below).
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include <cuda_fp8.h>

#include "rotary.cuh"

namespace dsa {

constexpr int kQuantThreads = 128;
constexpr int kQuantFewRows = 512;               // rows that fill the SMs with 32 threads each

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
// v / scale for inv = 1 / scale, both rounded to nearest: the product's remainder is exact, and with it
// the product is corrected to the rounded quotient (Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990), as long as nothing underflows, which kLeastScale sees to.
// Checked against divisions next to every border between two codes. (Products that were checked against
// the borders and divided where close cost more: bf16 values meet borders exactly often enough that
// every third warp divided. The correction cost the rows of 64 heads above 13%, two values at a time gave
// half of that back; the rotary kernel, bound by HBM, gained nothing from turning two at a time.)
constexpr float kLeastScale = 0x1p-90f;
__device__ __forceinline__ float2 quotient(float2 v, float scale, float inv) {
  const float2 q = mul2(v, make_float2(inv, inv));
  return fma2(fma2(q, make_float2(-scale, -scale), v), make_float2(inv, inv), q);
}

// Makes the compiler take the values as new: it would keep the first rotation's results, twice the
// registers, for the second.
template <int DT>
__device__ __forceinline__ void keep_packed(RawVec<DT>& r) {
#pragma unroll
  for (uint4& w : r.w) asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w));
}

// The rare paths, out of line so that they hold no registers of the kernel's: the maximum of a row with
// values that are not finite, over the others, and an item's codes by division (of such rows and of very small ones).
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

// The absolute maximum of an item that is not rotated, NaN if any value is: 16-bit values are compared
// packed.
template <int DT>
__device__ __forceinline__ float raw_max(float top, const RawVec<DT>& a, const RawVec<DT>& b) {
  if constexpr (DT == DSA_DTYPE_F32) {
    const float *x = reinterpret_cast<const float*>(&a), *y = reinterpret_cast<const float*>(&b);
#pragma unroll
    for (int e = 0; e < kVec; ++e) top = max_or_nan(top, x[e], y[e]);
    return top;
  } else {
    using T2 = std::conditional_t<DT == DSA_DTYPE_BF16, __nv_bfloat162, __half2>;
    const T2 *x = reinterpret_cast<const T2*>(&a), *y = reinterpret_cast<const T2*>(&b);
    T2 m = __habs2(x[0]);
#pragma unroll
    for (int e = 0; e < 4; ++e) m = __hmax2_nan(m, __hmax2_nan(__habs2(x[e]), __habs2(y[e])));
    return max_or_nan(top, Elem<DT>::get(m.x), Elem<DT>::get(m.y));
  }
}

// An item's codes by corrected products.
template <int DT, bool INTERLEAVED>
__device__ __forceinline__ void quotient_item(RawVec<DT>& a, RawVec<DT>& b, const float2* cs, float scale, float inv,
                                              uint8_t* out_a, uint8_t* out_b) {
  float v[2][kVec];
  keep_packed(a);
  keep_packed(b);
  unpack_raw<DT>(a, v[0]);
  unpack_raw<DT>(b, v[1]);
  if (cs) rotary_turn<INTERLEAVED>(cs, v[0], v[1]);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int e = 0; e < kVec; e += 2) {
      const float2 q = quotient(make_float2(v[u][e], v[u][e + 1]), scale, inv);
      v[u][e] = q.x;
      v[u][e + 1] = q.y;
    }
    *reinterpret_cast<uint2*>(u ? out_b : out_a) =
        make_uint2(e4m3x4(v[u][0], v[u][1], v[u][2], v[u][3]), e4m3x4(v[u][4], v[u][5], v[u][6], v[u][7]));
  }
}

// The absolute maximum of `top` and an item's values, turned where cs is given.
template <int DT, bool INTERLEAVED>
__device__ __forceinline__ float item_max(float top, const RawVec<DT>& a, const RawVec<DT>& b, const float2* cs) {
  if (!cs) return raw_max<DT>(top, a, b);
  float x[kVec], y[kVec];
  unpack_raw<DT>(a, x);
  unpack_raw<DT>(b, y);
  rotary_turn<INTERLEAVED>(cs, x, y);
#pragma unroll
  for (int e = 0; e < kVec; ++e) top = max_or_nan(top, x[e], y[e]);
  return top;
}

// A row's place: its number, or its slot in the cache; -1: not written.
__device__ __forceinline__ int64_t row_place(const QuantParams& p, int64_t t) {
  if (t >= p.T) return -1;
  return p.slots ? p.slots[t] : t;
}
__device__ __forceinline__ int64_t checked_place(const QuantParams& p, int64_t dst, bool first) {
  if (!p.slots || (dst >= -1 && dst < p.n_slots)) return dst;
  if (first) record_error(p.hdr, DSA_ERR_DEVICE, DETAIL_BAD_SLOT);
  return -1;
}
__device__ __forceinline__ float row_scale(float top) {
  return top > 0.0f ? fmaxf(__fdiv_rn(top, 448.0f), FLT_MIN) : 1.0f;
}

// Rows of up to 32 items: G threads a row, one item a thread, 128 / G rows a CTA. A warp holds whole rows
// and needs no barrier for their maxima.
template <int DT, bool INTERLEAVED, int G>
__global__ void __launch_bounds__(kQuantThreads) index_quantise_small_kernel(const __grid_constant__ QuantParams p) {
  using T = typename Elem<DT>::T;
  constexpr int kRows = kQuantThreads / G;
  extern __shared__ __align__(16) float2 cs_all[];
  const int half = p.r.rot / 2, per_head = p.d / kItem;
  const int g = threadIdx.x / G, l = threadIdx.x % G;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows, t = t0 + g;
  const int head = l / per_head < p.H ? l / per_head : -1;
  const Item it = rotary_item(l % per_head, p.r);
  const int64_t dst = checked_place(p, row_place(p, t), l == 0);
  const bool mine = dst >= 0 && head >= 0;
  const T* row = static_cast<const T*>(p.x) + t * p.xs_t;
  RawVec<DT> ra, rb;
  if (mine) {
    ra = load_raw<DT>(row + head * p.xs_h + it.a);
    rb = load_raw<DT>(row + head * p.xs_h + it.b);
  }
  for (int i = threadIdx.x; i < kRows * half; i += kQuantThreads) {
    const int64_t tt = t0 + i / half;
    if (tt < p.T) cs_all[i] = rotary_cos_sin(p.r.positions[tt], p.r.inv_freq[i % half], p.r);
  }
  __syncthreads();
  const float2* cs_row = cs_all + g * half;
  float2 cs[kVec];
  if (it.f >= 0) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) cs[i] = cs_row[it.f + i];
  }
  float top = 0.0f;
  if (mine) top = item_max<DT, INTERLEAVED>(top, ra, rb, it.f >= 0 ? cs : nullptr);
#pragma unroll
  for (int off = G / 2; off > 0; off >>= 1) top = max_or_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, off), 0.0f);
  if (dst < 0) return;
  // A row with a value that is not finite: its maximum is not finite either, and is found anew by every
  // thread from the whole row.
  const bool mend = !(top <= FLT_MAX);
  if (mend) {
    if (l == 0) record_error(p.hdr, DSA_ERR_DEVICE, DETAIL_NOT_FINITE);
    top = finite_max<DT, INTERLEAVED>(&p, row, cs_row);
  }
  const float scale = row_scale(top);
  if (mine) {
    uint8_t* out = p.codes + dst * (static_cast<int64_t>(p.H) * p.d) + head * p.d;
    if (mend || scale < kLeastScale)
      divided_item<DT, INTERLEAVED>(row + head * p.xs_h + it.a, row + head * p.xs_h + it.b,
                                    it.f >= 0 ? cs_row + it.f : nullptr, scale, out + it.a, out + it.b);
    else
      quotient_item<DT, INTERLEAVED>(ra, rb, it.f >= 0 ? cs : nullptr, scale, __fdiv_rn(1.0f, scale), out + it.a, out + it.b);
  }
  if (l == 0) p.scale[dst] = scale;
}

// Larger rows: a CTA takes one row after another, in up to NI passes, first over the heads' rotated items
// and then over the copied ones, so that a pass is either for every thread. In every pass a thread has
// the same item of another head: it finds its offsets once. A row's values stay packed as they were
// loaded; rotated ones are rotated twice, for the maximum and for the codes. (With the next row's
// loads on their way while this one's are worked on, which leaves registers for four CTAs an SM instead
// of five, the row of 64 heads above takes 11 to 40% longer.) One barrier a row: in front of it a warp leaves
// its maximum (two buffers) and the first threads the next row's (cos, sin) (three, since the rare paths read
// them behind it).
template <int DT, bool INTERLEAVED, int NI>
__global__ void __launch_bounds__(kQuantThreads, NI <= 4 ? 5 : 1)
    index_quantise_kernel(const __grid_constant__ QuantParams p) {
  using T = typename Elem<DT>::T;
  extern __shared__ __align__(16) float2 cs_all[];  // [3][half]
  __shared__ float warp_max[2][kQuantThreads / 32];
  const int half = p.r.rot / 2, l = threadIdx.x;
  const int n_rot = p.r.rot / kItem, n_copy = p.d / kItem - n_rot;
  // The thread's rotated items: item j_rot of heads h_rot, h_rot + per_rot, ... below end_rot (passes 0 to
  // passes_rot - 1); its copied ones alike.
  int per_rot = 1, per_copy = 1, passes_rot = 0, h_rot = 0, h_copy = 0, j_rot = 0, j_copy = 0, end_rot = 0, end_copy = 0;
  if (n_rot) {
    per_rot = kQuantThreads / n_rot;
    passes_rot = (p.H + per_rot - 1) / per_rot;
    h_rot = l / n_rot;
    j_rot = l - h_rot * n_rot;
    end_rot = h_rot < per_rot ? p.H : 0;
  }
  if (n_copy) {
    per_copy = kQuantThreads / n_copy;
    h_copy = l / n_copy;
    j_copy = l - h_copy * n_copy;
    end_copy = h_copy < per_copy ? p.H : 0;
  }
  const Item ir = rotary_item(j_rot, p.r), ic = rotary_item(n_rot + j_copy, p.r);
  auto head_of = [&](int k) {                   // of pass k, -1: none for this thread
    const int head = k < passes_rot ? h_rot + k * per_rot : h_copy + (k - passes_rot) * per_copy;
    return head < (k < passes_rot ? end_rot : end_copy) ? head : -1;
  };
  auto turns = [&](int64_t t, float2* cs) {
    for (int i = l; i < half; i += kQuantThreads) cs[i] = rotary_cos_sin(p.r.positions[t], p.r.inv_freq[i], p.r);
  };
  RawVec<DT> ra[NI], rb[NI];
  int64_t t = blockIdx.x, place = row_place(p, t);
  turns(t, cs_all);
  __syncthreads();
#pragma unroll 1
  for (int n = 0; t < p.T; ++n, t += gridDim.x) {
    const float2* cs_row = cs_all + n % 3 * half;
    const int64_t next = t + gridDim.x, next_place = row_place(p, next);
    const T* row = static_cast<const T*>(p.x) + t * p.xs_t;
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      const int head = head_of(k);
      if (head < 0) continue;
      const T* h = row + head * p.xs_h;
      ra[k] = load_raw<DT>(h + (k < passes_rot ? ir.a : ic.a));
      rb[k] = load_raw<DT>(h + (k < passes_rot ? ir.b : ic.b));
    }
    const int64_t dst = checked_place(p, place, l == 0);
    place = next_place;
    float2 cs[kVec];
    if (n_rot) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) cs[i] = cs_row[ir.f + i];
    }
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < NI; ++k)
      if (head_of(k) >= 0) top = item_max<DT, INTERLEAVED>(top, ra[k], rb[k], k < passes_rot ? cs : nullptr);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = max_or_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, off), 0.0f);
    if ((l & 31) == 0) warp_max[n & 1][l >> 5] = top;
    if (next < p.T) turns(next, cs_all + (n + 1) % 3 * half);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 32; ++w) top = max_or_nan(top, warp_max[n & 1][w], 0.0f);
    if (dst >= 0) {
      // (A row with a value that is not finite: as above.)
      const bool mend = !(top <= FLT_MAX);
      if (mend) {
        if (l == 0) record_error(p.hdr, DSA_ERR_DEVICE, DETAIL_NOT_FINITE);
        top = finite_max<DT, INTERLEAVED>(&p, row, cs_row);
      }
      const float scale = row_scale(top);
      uint8_t* out = p.codes + dst * (static_cast<int64_t>(p.H) * p.d);
      if (mend || scale < kLeastScale) {
#pragma unroll 1
        for (int k = 0; k < NI; ++k) {
          const int head = head_of(k);
          if (head < 0) continue;
          const Item& it = k < passes_rot ? ir : ic;
          divided_item<DT, INTERLEAVED>(row + head * p.xs_h + it.a, row + head * p.xs_h + it.b,
                                        it.f >= 0 ? cs_row + it.f : nullptr, scale, out + head * p.d + it.a,
                                        out + head * p.d + it.b);
        }
      } else {
        const float inv = __fdiv_rn(1.0f, scale);
#pragma unroll
        for (int k = 0; k < NI; ++k) {
          const int head = head_of(k);
          if (head < 0) continue;
          uint8_t* o = out + head * p.d;
          if (k < passes_rot) quotient_item<DT, INTERLEAVED>(ra[k], rb[k], cs, scale, inv, o + ir.a, o + ir.b);
          else quotient_item<DT, INTERLEAVED>(ra[k], rb[k], nullptr, scale, inv, o + ic.a, o + ic.b);
        }
      }
      if (l == 0) p.scale[dst] = scale;
    }
  }
}

template <int DT, bool INTERLEAVED, int G>
static dsa_status launch_quantise_small(const QuantParams& p, cudaStream_t stream) {
  constexpr int kRows = kQuantThreads / G;
  const size_t smem = static_cast<size_t>(kRows) * (p.r.rot / 2) * sizeof(float2);
  const int64_t grid = (p.T + kRows - 1) / kRows;
  index_quantise_small_kernel<DT, INTERLEAVED, G><<<static_cast<unsigned>(grid), kQuantThreads, smem, stream>>>(p);
  return cuda_status(cudaGetLastError());
}

template <int DT, bool INTERLEAVED, int NI>
static dsa_status launch_quantise_rows(const QuantParams& p, int num_sms, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(3) * (p.r.rot / 2) * sizeof(float2);
  const int grid = static_cast<int>(std::min<int64_t>(p.T, static_cast<int64_t>(num_sms) * (NI <= 4 ? 5 : 2)));
  index_quantise_kernel<DT, INTERLEAVED, NI><<<grid, kQuantThreads, smem, stream>>>(p);
  return cuda_status(cudaGetLastError());
}

// Passes over a row of H heads by all threads; at most 18 with 1024 items (a pass takes more than half of
// the threads).
static int quantise_passes(const QuantParams& p) {
  const int n_rot = p.r.rot / kItem, n_copy = p.d / kItem - n_rot;
  int passes = 0;
  for (const int n : {n_rot, n_copy})
    if (n) passes += (p.H + kQuantThreads / n - 1) / (kQuantThreads / n);
  return passes;
}

template <int DT, bool INTERLEAVED>
static dsa_status launch_quantise_t(const QuantParams& p, int num_sms, cudaStream_t stream) {
  const int n = p.H * (p.d / kItem);
  // As few threads a row as it has items (16384 keys of 128: 6.8 us with 8 threads, 12.6 with 32), but few
  // rows are spread over more CTAs (32 keys of 128: 2.6 us with 32, 3.2 with 8). The instance of 18 passes
  // takes every row of more than four: rows of more than 512 items, and smaller ones whose rotated and
  // copied items each leave a pass part empty (64 heads x 128 with a rotary part of 16, 32, 48, 80, 96 or
  // 112: five or more). Its 255 registers leave two CTAs an SM: 16384 tokens of 64 heads x 128 take 310 us
  // with 32 dims rotated, and 89 in the instance of four with 64.
  if (n <= 32 && p.T <= kQuantFewRows) return launch_quantise_small<DT, INTERLEAVED, 32>(p, stream);
  if (n <= 8) return launch_quantise_small<DT, INTERLEAVED, 8>(p, stream);
  if (n <= 16) return launch_quantise_small<DT, INTERLEAVED, 16>(p, stream);
  if (n <= 32) return launch_quantise_small<DT, INTERLEAVED, 32>(p, stream);
  if (quantise_passes(p) <= 4) return launch_quantise_rows<DT, INTERLEAVED, 4>(p, num_sms, stream);
  return launch_quantise_rows<DT, INTERLEAVED, 18>(p, num_sms, stream);
}

dsa_status launch_quantise(const QuantParams& p, int num_sms, int dtype, cudaStream_t stream) {
  if (p.r.interleaved) {
    if (dtype == DSA_DTYPE_BF16) return launch_quantise_t<DSA_DTYPE_BF16, true>(p, num_sms, stream);
    if (dtype == DSA_DTYPE_F16) return launch_quantise_t<DSA_DTYPE_F16, true>(p, num_sms, stream);
    return launch_quantise_t<DSA_DTYPE_F32, true>(p, num_sms, stream);
  }
  if (dtype == DSA_DTYPE_BF16) return launch_quantise_t<DSA_DTYPE_BF16, false>(p, num_sms, stream);
  if (dtype == DSA_DTYPE_F16) return launch_quantise_t<DSA_DTYPE_F16, false>(p, num_sms, stream);
  return launch_quantise_t<DSA_DTYPE_F32, false>(p, num_sms, stream);
}

// ------------------------------------------------------------------------------------------
// Cache read. A CTA takes kReadRows output rows: its first threads find each row's request (a
// binary search over the row offsets) and cache row, then all copy 16 codes at a time. Bound by HBM:
// 32 requests of 10000 to 200000 keys of 128 dims as bf16 values take 204 us, 5.3 TB/s; three prefixes of
// up to 1500 keys as codes and scales 3.1 us, one launch.
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

// Rotary positions for sm_100a (the arithmetic and its layouts are in rotary.cuh).
//
// The operator moves its bytes once and computes little, so it is bound by HBM (long inputs) or by
// one launch (a decode step). A CTA takes one token: its threads start the loads of their first
// items, then form the token's rot/2 (cos, sin) pairs once in shared memory for all of its heads.
// 16384 tokens of 64 heads x 128, bf16: 97.7 us, 5.5 TB/s. 32 tokens of 128 heads x 64 in rows of 576:
// 2.8 us. A token of few items leaves most of its CTA idle: 16384 tokens of one head x 64 take 27 us, where
// their bytes take 0.6.
#include <cmath>

#include "rotary.cuh"

namespace dsa {

constexpr int kRotThreads = 256;

template <int DT, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(RotaryArgs r, const typename Elem<DT>::T* x, int64_t xs_t,
                                                             int64_t xs_h, typename Elem<DT>::T* out, int64_t os_t,
                                                             int64_t os_h, int32_t H, int32_t d, bool in_place) {
  extern __shared__ __align__(16) float2 cs[];
  const int64_t t = blockIdx.x;
  const int per_head = in_place ? r.rot / kItem : d / kItem;  // in place, copied items stay as they are
  const int n = H * per_head;
  const int i0 = blockIdx.y * kRotThreads + threadIdx.x, step = gridDim.y * kRotThreads;
  float a[kVec], b[kVec];
  const typename Elem<DT>::T* row = x + t * xs_t;
  if (i0 < n) {
    const Item it = rotary_item(i0 % per_head, r);
    const typename Elem<DT>::T* h = row + (i0 / per_head) * xs_h;
    load_vec<DT>(h + it.a, a);
    load_vec<DT>(h + it.b, b);
  }
  const int32_t p = r.positions[t];
  for (int i = threadIdx.x; i < r.rot / 2; i += kRotThreads) cs[i] = rotary_cos_sin(p, r.inv_freq[i], r);
  __syncthreads();
  for (int i = i0; i < n; i += step) {
    const Item it = rotary_item(i % per_head, r);
    const int head = i / per_head;
    if (i != i0) {
      load_vec<DT>(row + head * xs_h + it.a, a);
      load_vec<DT>(row + head * xs_h + it.b, b);
    }
    if (it.f >= 0) rotary_turn<INTERLEAVED>(cs + it.f, a, b);
    typename Elem<DT>::T* o = out + t * os_t + head * os_h;
    store_vec<DT>(o + it.a, a);
    store_vec<DT>(o + it.b, b);
  }
}

// Any even rot, any d, strides and alignment: a thread takes one pair or one copied element. (4096
// tokens of 16 heads x 128, bf16: 18.0 us, the kernel above 10.2.)
template <int DT>
__global__ void __launch_bounds__(kRotThreads) rotary_any_kernel(RotaryArgs r, const typename Elem<DT>::T* x,
                                                                 int64_t xs_t, int64_t xs_h, typename Elem<DT>::T* out,
                                                                 int64_t os_t, int64_t os_h, int32_t H, int32_t d) {
  extern __shared__ __align__(16) float2 cs[];
  const int64_t t = blockIdx.x;
  const int32_t p = r.positions[t];
  const int half = r.rot / 2;
  for (int i = threadIdx.x; i < half; i += kRotThreads) cs[i] = rotary_cos_sin(p, r.inv_freq[i], r);
  __syncthreads();
  const int per_head = d - half;
  for (int i = blockIdx.y * kRotThreads + threadIdx.x; i < H * per_head; i += gridDim.y * kRotThreads) {
    const int head = i / per_head, j = i % per_head;
    const typename Elem<DT>::T* h = x + t * xs_t + head * xs_h;
    typename Elem<DT>::T* o = out + t * os_t + head * os_h;
    if (j < half) {
      const int ia = r.offset + (r.interleaved ? 2 * j : j), ib = r.interleaved ? ia + 1 : ia + half;
      float a = Elem<DT>::get(h[ia]), b = Elem<DT>::get(h[ib]);
      rotary_pair(cs[j], a, b);
      o[ia] = Elem<DT>::put(a);
      o[ib] = Elem<DT>::put(b);
    } else {
      const int e = j - half, ie = e < r.offset ? e : e + r.rot;
      o[ie] = h[ie];
    }
  }
}

template <int DT>
static dsa_status launch_rotary_t(const RotaryLaunch& a) {
  using T = typename Elem<DT>::T;
  const T* x = static_cast<const T*>(a.x);
  T* out = static_cast<T*>(a.out);
  auto vec = [](int64_t n) { return n % kVec == 0; };
  const bool wide = a.r.rot % kItem == 0 && a.d % kItem == 0 && vec(a.r.offset) && vec(a.xs_t) && vec(a.xs_h) &&
                    vec(a.os_t) && vec(a.os_h) && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(out) % 16 == 0;
  const bool in_place = static_cast<const void*>(x) == a.out && a.xs_t == a.os_t && a.xs_h == a.os_h;
  const size_t smem = static_cast<size_t>(a.r.rot / 2) * sizeof(float2);
  const int64_t n = static_cast<int64_t>(a.H) * (wide ? (in_place ? a.r.rot : a.d) / kItem : a.d - a.r.rot / 2);
  // Few tokens: a token's items are spread over CTAs until the GPU has one CTA per SM (32 tokens of 128
  // heads x 64: 7% more time with one CTA a token).
  const int64_t fill = (a.num_sms + a.T - 1) / a.T, need = (n + kRotThreads - 1) / kRotThreads;
  const dim3 grid(a.T, static_cast<unsigned>(need < fill ? need : fill));
  if (wide && a.r.interleaved)
    rotary_kernel<DT, true><<<grid, kRotThreads, smem, a.stream>>>(a.r, x, a.xs_t, a.xs_h, out, a.os_t, a.os_h, a.H, a.d, in_place);
  else if (wide)
    rotary_kernel<DT, false><<<grid, kRotThreads, smem, a.stream>>>(a.r, x, a.xs_t, a.xs_h, out, a.os_t, a.os_h, a.H, a.d, in_place);
  else
    rotary_any_kernel<DT><<<grid, kRotThreads, smem, a.stream>>>(a.r, x, a.xs_t, a.xs_h, out, a.os_t, a.os_h, a.H, a.d);
  return cuda_status(cudaGetLastError());
}

dsa_status launch_rotary(const RotaryLaunch& a) {
  if (a.dtype == DSA_DTYPE_BF16) return launch_rotary_t<DSA_DTYPE_BF16>(a);
  if (a.dtype == DSA_DTYPE_F16) return launch_rotary_t<DSA_DTYPE_F16>(a);
  return launch_rotary_t<DSA_DTYPE_F32>(a);
}

// Frequencies theta^(-2i/rot); with factor > 1 those whose wavelength is longer than the original
// context are divided by it and the ones between beta_fast and beta_slow turns over that context
// are blended linearly (the NTK-by-parts interpolation of the YaRN paper, Peng et al. 2023).
void rotary_frequencies(int rot, double theta, double factor, int original_len, double beta_fast, double beta_slow,
                        float* inv_freq, float* mscale) {
  constexpr double kTwoPi = 6.283185307179586;
  const int half = rot / 2;
  auto dim_of = [&](double turns) { return rot * std::log(original_len / (turns * kTwoPi)) / (2.0 * std::log(theta)); };
  double low = std::floor(dim_of(beta_fast)), high = std::ceil(dim_of(beta_slow));
  low = low < 0.0 ? 0.0 : low;
  high = high > rot - 1 ? rot - 1 : high;
  double width = high - low;
  if (width < 1e-3) width = 1e-3;
  for (int i = 0; i < half; ++i) {
    const double f = std::pow(theta, -static_cast<double>(i) / half);
    double ramp = (i - low) / width;
    ramp = ramp < 0.0 ? 0.0 : (ramp > 1.0 ? 1.0 : ramp);
    inv_freq[i] = static_cast<float>(factor > 1.0 ? f * (1.0 - ramp) + f / factor * ramp : f);
  }
  if (mscale) *mscale = static_cast<float>(factor > 1.0 ? 0.1 * std::log(factor) + 1.0 : 1.0);
}

}  // namespace dsa

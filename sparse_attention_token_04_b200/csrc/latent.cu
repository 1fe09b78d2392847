// Latent attention for sm_100a, plain kernels: a warp takes one query row (token and head), its
// lanes hold the row's dims, and the keys are visited one by one with the running maximum m and
// sum l of the softmax:
//     s = scale q.k,  m' = max(m, s),  o <- o e^(m - m') + e^(s - m') v,  l <- l e^(m - m') + e^(s - m').
// out = o / l and lse = m + log l; a row that sees no key gets zeros and -inf.
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "rotary.cuh"

namespace dsa {

template <int DT, int DK, int DV>
struct RowState {
  float q[DK / 32], o[DV / 32], m = -INFINITY, l = 0.0f;
  __device__ __forceinline__ void step(const float (&k)[DK / 32], const float (&v)[DV / 32], float scale) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < DK / 32; ++i) s += q[i] * k[i];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    s *= scale;
    const float mn = fmaxf(m, s), c = expf(m - mn), p = expf(s - mn);
    m = mn;
    l = l * c + p;
#pragma unroll
    for (int i = 0; i < DV / 32; ++i) o[i] = o[i] * c + p * v[i];
  }
  __device__ __forceinline__ void store(typename Elem<DT>::T* out, float* lse, int lane) {
#pragma unroll
    for (int i = 0; i < DV / 32; ++i) out[lane + 32 * i] = Elem<DT>::put(l > 0.0f ? o[i] / l : 0.0f);
    if (lane == 0 && lse) *lse = l > 0.0f ? m + logf(l) : -INFINITY;
  }
};

template <int DT>
__global__ void __launch_bounds__(256) latent_decode_plain_kernel(const LatentDecodeParams p) {
  using T = typename Elem<DT>::T;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int rows = p.q_len * p.Hq;
  if (row >= static_cast<int64_t>(p.B) * rows) return;
  const int b = static_cast<int>(row / rows), i = static_cast<int>(row % rows) / p.Hq, h = static_cast<int>(row % p.Hq);
  int n = p.seq_lens[b];
  if (n < 0 || n > p.max_blocks * p.block_size) {
    if (lane == 0) record_error(p.hdr, DSA_ERR_DEVICE, DETAIL_BAD_SEQ_LEN);
    n = n < 0 ? 0 : p.max_blocks * p.block_size;
  }
  const int sees = n - p.q_len + 1 + i;
  RowState<DT, 576, 512> st;
  const T* q = static_cast<const T*>(p.q) + (static_cast<int64_t>(b) * p.q_len + i) * p.qs_t + h * p.qs_h;
#pragma unroll
  for (int e = 0; e < 18; ++e) st.q[e] = Elem<DT>::get(q[lane + 32 * e]);
#pragma unroll
  for (int e = 0; e < 16; ++e) st.o[e] = 0.0f;
  for (int s = 0; s < sees; ++s) {
    int blk = p.block_table[static_cast<int64_t>(b) * p.max_blocks + s / p.block_size];
    if (blk < 0 || blk >= p.n_blocks) {
      if (lane == 0) record_error(p.hdr, DSA_ERR_DEVICE, DETAIL_BAD_BLOCK_TABLE);
      blk = 0;
    }
    const T* k = static_cast<const T*>(p.latent) + (static_cast<int64_t>(blk) * p.block_size + s % p.block_size) * 576;
    float kv[18], v[16];
#pragma unroll
    for (int e = 0; e < 18; ++e) kv[e] = Elem<DT>::get(k[lane + 32 * e]);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = kv[e];
    st.step(kv, v, p.scale);
  }
  st.store(static_cast<T*>(p.out) + row * 512, p.lse ? p.lse + row : nullptr, lane);
}

size_t latent_decode_workspace_bytes(int B, int q_len, int Hq) {
  (void)B, (void)q_len, (void)Hq;
  return DSA_WS_HEADER_BYTES;
}

dsa_status launch_latent_decode(const LatentDecodeParams& p, int dtype, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.B) * p.q_len * p.Hq;
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  if (dtype == DSA_DTYPE_BF16) latent_decode_plain_kernel<DSA_DTYPE_BF16><<<grid, 256, 0, stream>>>(p);
  else latent_decode_plain_kernel<DSA_DTYPE_F16><<<grid, 256, 0, stream>>>(p);
  return cuda_status(cudaGetLastError());
}

}  // namespace dsa

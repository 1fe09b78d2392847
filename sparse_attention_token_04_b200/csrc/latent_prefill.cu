// Latent attention of ragged prefills (expanded form) for sm_100a: out = softmax(scale Q K^T) V per
// head, K = (k_nope | k_pe) 192 wide, V 128 wide, causal or not.
//
// A CTA takes 256 queries of one head as two 128-row tiles and walks the request's keys 128 at a
// time. Per key tile and query tile: S = Q K^T (128 x 128 x 192) into TMEM, the softmax of S by 128
// threads (thread = row), P = exp(S - m) back into TMEM over S's columns as 16-bit pairs, and
// O += P V (128 x 128 x 128) with P read from TMEM. The two query tiles alternate: the tensor core
// works for one while the other's softmax runs.
//   warps 0-3, 4-7  softmax of query tile 0, 1: running maximum m and sum l of the row, O rescaled
//                   in TMEM only when m has grown by more than 2^kLazy (so that the accumulator is
//                   touched a few times per row, not every tile); at the end O / l and lse;
//   warp 8          TMA: the query tiles once, K in blocks of 16 KB (three a tile) through a ring of
//                   four, V tiles two deep;
//   warp 9          one thread issues every MMA, in the order PV(0, j), QK(0, j+1), PV(1, j),
//                   QK(1, j+1). QK(w, j+1) overwrites the columns that PV(w, j) reads P from: both go
//                   down the one tensor pipe in issue order.
// Shared memory: 96 KB of Q, 64 KB of K, 64 KB of V, all [128 rows][64 dims] blocks with the 128-byte
// swizzle. (With K two tiles and V one tile deep instead, a V tile came 1000 cycles late every time; in
// one ring of blocks for both, V's two blocks are not neighbours and PV takes twice the MMAs: 12% more time
// on the long prompt below.) TMEM: S (and P) of the two tiles in columns 0-127 and 128-255, O in 256-383 and
// 384-511. P goes over in two halves of 64 keys, so that PV starts behind the first.
//
// Bound: the chain of one query tile. The MMAs of a key tile take 2560 cycles for both query tiles, but
// S and P share columns, so a tile's next QK waits for its PV: from scores to scores its softmax (2200
// cycles: 700 to read S and find the maximum, 1500 for the exponentials, whose unit both tiles share),
// its own products (1280) and some 600 of hand-over follow one another, 4300 cycles in all. A prompt of
// 8192 tokens and 32 heads, bf16: 667 us back to back, which the power limit holds at 1545 MHz: 1030
// TFLOP/s, 75% of the sustained cuBLAS rate (590 us from idle, 71% of the burst rate). The tensor pipe is
// then active in 61% of the cycles, the exponentials' unit in 49%. Measured against it, where it took 578 us
// from idle: two threads a row (614: the pair's exchange and the shared unit take what the shorter rows
// give), a quarter of the exponentials on the FMA pipe (596), P handed over in parts of 96 and 32 keys
// (588), exponentials that start with the maximum so far while the tile's is found (635: more registers than
// there are; the 168 already spill 64 bytes), tiles fetched into L2 ahead of time (598), V in blocks of 64
// keys and K in one ring of eight (579, but 4% more for 2048 tokens behind 6144), a rolled softmax that
// reads S twice (600).
//
// A call with few query blocks (256 queries of one head) would leave SMs idle, so its blocks' key tiles
// are split into parts of `chunk` tiles, which write unnormalised O, m and l, and
// latent_prefill_combine_kernel joins them. lp_plan chooses the chunk. 100 queries behind 8000 keys, 16
// heads: 125 us whole, 31 split; 2500 tokens of one head: 48 and 18; 2048 tokens behind 6144, 16 heads
// (128 blocks, 49 to 64 tiles long): 165 and 162 at the power limit, 169 and 157 from idle. Three requests of
// 1300 tokens at 8 heads, which the rule leaves whole: 30 us, a fifth more split.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace dsa {

constexpr int kLpTile = 128;                 // query rows of a tile, keys of a tile
constexpr int kLpThreads = 320;
constexpr int kLpBlock = kLpTile * 128;      // 16 KB: 128 rows x 64 dims
constexpr int kLpKRing = 4;                  // blocks of the K ring (a tile has three)
constexpr float kLpLazy = 6.0f;              // log2 growth of a row's maximum that is left unscaled
// Splitting: key tiles of a part at least (2500 tokens of one head: with one 35% more time than with two,
// with three 19%), tiles that a split has to save (one, two and three measure alike), parts of a block and
// places for parts per SM (133 KB each) at most.
constexpr int kLpMinTiles = 2, kLpMinGain = 2, kLpMaxSplits = 32, kLpMaxPlaces = 6;

struct LpSmem {
  uint8_t q[2][3][kLpBlock];
  uint8_t k[kLpKRing][kLpBlock];
  uint8_t v[2][2][kLpBlock];
  uint64_t q_full[2], k_full[kLpKRing], k_free[kLpKRing], v_full[2], v_free[2];
  uint64_t s_full[2], p_ready[2][2], o_done[2], drain;
  uint32_t tmem;
  int abort;
};

struct LpParams {
  const int32_t *cu_q, *cu_k;
  int32_t Tq, Tk, max_q, H, causal;
  float scale, scale_log2;
  void* out;
  float* lse;
  int32_t n_blocks;                          // 256-query blocks of a request, at most
  int32_t splits, chunk;                     // CTAs that may share one, key tiles of each but the last
  float* part;                               // [request][block][head][split][32][256][4]: unnormalised O, four
                                             // dims of a row together (lanes have a row each)
  float2* ml;                                // [request][block][head][split][256] m, l
  WsHeader* hdr;
  uint64_t budget_ns;
};

// One 256-query block of a request.
struct LpBlock {
  int q0, nq, k0, nk, i0;
  bool bad, none;                            // bad offsets; no queries in this block
  // Keys that query i of the request sees.
  __device__ __forceinline__ int sees(int i, int causal) const { return causal ? max(0, min(nk, nk - nq + 1 + i)) : nk; }
  // Key tiles of query tile w.
  __device__ __forceinline__ int tiles(int w, int causal) const {
    const int first = i0 + w * kLpTile, last = min(first + kLpTile, nq) - 1;
    return first < nq ? (sees(last, causal) + kLpTile - 1) / kLpTile : 0;
  }
};
__device__ __forceinline__ LpBlock lp_block(const LpParams& p, int b, int qb) {
  const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
  const bool bad = q0 < 0 || q1 < q0 || q1 > p.Tq || k0 < 0 || k1 < k0 || k1 > p.Tk || q1 - q0 > p.max_q;
  const int i0 = qb * 2 * kLpTile;
  return {q0, q1 - q0, k0, k1 - k0, i0, bad, i0 >= q1 - q0};
}
// CTAs that share the n key tiles of a block.
__device__ __forceinline__ int lp_parts(const LpParams& p, int n) { return n <= p.chunk ? 1 : (n + p.chunk - 1) / p.chunk; }

// kSplit: a block's key tiles are shared by up to p.splits CTAs.
template <int DT, bool kSplit>
__global__ void __launch_bounds__(kLpThreads, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_pe, const __grid_constant__ CUtensorMap map_v,
                          const LpParams p) {
  extern __shared__ uint8_t smem_raw[];
  LpSmem& sm = *reinterpret_cast<LpSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                          ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x, n_req = kSplit ? gridDim.z / p.splits : gridDim.z;
  // (The full parts of all blocks come before the rests.)
  const int b = kSplit ? blockIdx.z % n_req : blockIdx.z, split = kSplit ? blockIdx.z / n_req : 0;
  const int qb = gridDim.y - 1 - blockIdx.y;  // the longest rows of a causal call first

  const LpBlock u = lp_block(p, b, qb);
  if (u.bad) {
    if (tid == 0) record_error(p.hdr, DSA_ERR_DEVICE, DETAIL_BAD_SEQ_LEN);
    return;
  }
  if (u.none) return;
  // This CTA's key tiles [j0, j0 + n_tiles); from here on keys are counted from the first of them.
  const int all = max(u.tiles(0, p.causal), u.tiles(1, p.causal)), parts = kSplit ? lp_parts(p, all) : 1;
  if (split >= parts) return;
  const int j0 = kSplit ? split * p.chunk : 0, j1 = kSplit ? min(all, j0 + p.chunk) : all, skip = j0 * kLpTile;
  const int q0 = u.q0, nq = u.nq, i0 = u.i0, k0 = u.k0 + skip, nk = u.nk - skip;
  const int nt[2] = {max(0, min(u.tiles(0, p.causal), j1) - j0), max(0, min(u.tiles(1, p.causal), j1) - j0)};
  const int n_tiles = max(nt[0], nt[1]);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_ready[i][0], 4);
      mbar_init(&sm.p_ready[i][1], 4);
      mbar_init(&sm.o_done[i], 1);
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_free[i], 1);
    }
    for (int i = 0; i < kLpKRing; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_free[i], 1);
    }
    mbar_init(&sm.drain, 1);
    fence_mbar_init();
    sm.abort = 0;
  }
  if (warp == 9) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const WaitCtl ctl{p.hdr, &sm.abort, p.budget_ns};

  if (warp == 8) {
    if (elect_one()) {
      auto load_q = [&](int w) {
        mbar_arrive_expect_tx(&sm.q_full[w], 3 * kLpBlock);
        for (int c = 0; c < 3; ++c)
          tma_load_3d(sm.q[w][c], &map_q, c * 64, h, q0 + i0 + w * kLpTile, &sm.q_full[w]);
      };
      // K blocks g = 3 j + c in their order; V of tile j behind K's first block of the tile (of tile 0:
      // behind its last), which is the order in which their places come free.
      int g = 0, nv = 0;
      bool ok = true;
      auto load_v = [&]() {
        const int st = nv & 1;
        if (!mbar_wait_call(&sm.v_free[st], ((nv >> 1) & 1) ^ 1, ctl, DETAIL_WAIT_KEMPTY)) return false;
        mbar_arrive_expect_tx(&sm.v_full[st], 2 * kLpBlock);
        for (int c = 0; c < 2; ++c) tma_load_3d(sm.v[st][c], &map_v, c * 64, h, k0 + nv * kLpTile, &sm.v_full[st]);
        ++nv;
        return true;
      };
      if (nt[0] > 0) load_q(0);
#pragma unroll 1
      for (; g < 3 * n_tiles; ++g) {
        const int j = g / 3, c = g - 3 * j, slot = g % kLpKRing, key = k0 + j * kLpTile;
        ok = mbar_wait_call(&sm.k_free[slot], ((g / kLpKRing) & 1) ^ 1, ctl, DETAIL_WAIT_KEMPTY);
        if (!ok) break;
        mbar_arrive_expect_tx(&sm.k_full[slot], kLpBlock);
        if (c < 2) tma_load_3d(sm.k[slot], &map_k, c * 64, h, key, &sm.k_full[slot]);
        else tma_load_3d(sm.k[slot], &map_pe, 0, 0, key, &sm.k_full[slot]);
        if (g == 2) {
          if (nt[1] > 0) load_q(1);
          ok = load_v();
        } else if (g > 2 && c == 0) {
          ok = load_v();
        }
        if (!ok) {
          ++g;
          break;
        }
      }
      // Let every copy land before the CTA exits (bounded).
      for (int w = 0; w < 2; ++w)
        if (nt[w] > 0 && (w == 0 || g > 2)) mbar_drain_call(&sm.q_full[w], 0, p.budget_ns);
#pragma unroll 1
      for (int i = max(0, g - kLpKRing); i < g; ++i) mbar_drain_call(&sm.k_full[i % kLpKRing], (i / kLpKRing) & 1, p.budget_ns);
#pragma unroll 1
      for (int i = max(0, nv - 2); i < nv; ++i) mbar_drain_call(&sm.v_full[i & 1], (i >> 1) & 1, p.budget_ns);
    }
    __syncwarp();
  } else if (warp == 9) {
    if (n_tiles > 0 && elect_one()) {
      constexpr uint32_t bf16 = DT == DSA_DTYPE_BF16 ? 1u : 0u;
      constexpr uint32_t idesc_qk = make_idesc_16(bf16, kLpTile, kLpTile);
      constexpr uint32_t idesc_pv = make_idesc_16(bf16, kLpTile, 128) | kIdescBMnMajor;
      const uint64_t dk = make_smem_desc(smem_u32(sm.k[0]), 128);
      const uint64_t dv = make_smem_desc_mn(smem_u32(sm.v[0][0]), kLpBlock, 1024);
      // `first`, `last`: whether this query tile is the first or the last to use the key tile.
      auto qk = [&](int w, int j, bool first, bool last) {
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const int g = 3 * j + c, slot = g % kLpKRing;
          if (first) {
            if (!mbar_wait_call(&sm.k_full[slot], (g / kLpKRing) & 1, ctl, DETAIL_WAIT_KFULL)) return false;
            tc_fence_after();
          }
          const uint64_t da = make_smem_desc(smem_u32(sm.q[w][c]), 128), db = dk + slot * (kLpBlock >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_16(tmem + w * 128, da + 2ull * kk, db + 2ull * kk, idesc_qk, (c > 0 || kk > 0) ? 1u : 0u);
          if (last) tc_commit(&sm.k_free[slot]);
        }
        tc_commit(&sm.s_full[w]);
        return true;
      };
      // The PV of 64 keys: P comes in two halves.
      auto pv = [&](int w, int j, int half) {
        if (!mbar_wait_call(&sm.p_ready[w][half], j & 1, ctl, DETAIL_WAIT_SCORES)) return false;
        tc_fence_after();
        const uint64_t db = dv + (j & 1) * (2 * kLpBlock >> 4);
#pragma unroll
        for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
          tc_mma_16_ts(tmem + 256 + w * 128, tmem + w * 128 + kk * 8, db + (kk * 2048 >> 4), idesc_pv,
                       (j > 0 || kk > 0) ? 1u : 0u);
        return true;
      };
      const bool both = nt[0] > 0 && nt[1] > 0;
      bool ok = true;
      for (int w = 0; w < 2 && ok; ++w) {
        if (nt[w] == 0) continue;
        ok = mbar_wait_call(&sm.q_full[w], 0, ctl, DETAIL_WAIT_QFULL) && qk(w, 0, w == 0 || !both, w == 1 || !both);
      }
#pragma unroll 1
      for (int j = 0; j < n_tiles && ok; ++j) {
        ok = mbar_wait_call(&sm.v_full[j & 1], (j >> 1) & 1, ctl, DETAIL_WAIT_KFULL);
        const bool two = j < nt[0] && j < nt[1], two_next = j + 1 < nt[0] && j + 1 < nt[1];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (ok && j < nt[w]) {
            ok = pv(w, j, 0) && pv(w, j, 1);
            if (!ok) break;
            tc_commit(&sm.o_done[w]);
            if (w == 1 || !two) tc_commit(&sm.v_free[j & 1]);
          }
          if (ok && j + 1 < nt[w]) ok = qk(w, j + 1, w == 0 || !two_next, w == 1 || !two_next);
        }
      }
      tc_commit(&sm.drain);
      mbar_drain_call(&sm.drain, 0, p.budget_ns);
    }
    __syncwarp();
  } else {
    const int w = warp >> 2;
    const int row = (warp & 3) * 32 + lane, first = i0 + w * kLpTile + (warp & 3) * 32, i = first + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + w * 128 + lanes, tO = tmem + 256 + w * 128 + lanes;
    const int n_row = u.sees(i, p.causal) - skip, n_warp = u.sees(first, p.causal) - skip;
    constexpr float kShift = kNumeratorShift<DT>;
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < nt[w]; ++j) {
      ok = mbar_wait_warp(&sm.s_full[w], j & 1, ctl, DETAIL_WAIT_ACCFULL);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[4][32];
      tmem_ld_32x32b_x32(tS, s[0]);
      tmem_ld_32x32b_x32(tS + 32, s[1]);
      tmem_wait_ld_regs(s[0]);
      tmem_wait_ld_regs(s[1]);
      tmem_ld_32x32b_x32(tS + 64, s[2]);
      tmem_ld_32x32b_x32(tS + 96, s[3]);
      const bool masked = (j + 1) * kLpTile > n_warp;
      const int left = n_row - j * kLpTile;  // visible keys of this tile
      auto mask = [&](int c) {
        if (!masked) return;
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (c * 32 + e >= left) s[c][e] = 0xFF800000u;  // -inf
      };
      float mx[4] = {m, -INFINITY, -INFINITY, -INFINITY};
      auto row_max = [&](int c) {
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          mx[(e >> 1) & 3] = fmaxf(fmaxf(mx[(e >> 1) & 3], __uint_as_float(s[c][e])), __uint_as_float(s[c][e + 1]));
      };
      mask(0);
      mask(1);
      row_max(0);
      row_max(1);
      tmem_wait_ld_regs(s[2]);
      tmem_wait_ld_regs(s[3]);
      mask(2);
      mask(3);
      row_max(2);
      row_max(3);
      const float mn = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (j == 0) {
        m = mn;
      } else if (__any_sync(0xFFFFFFFFu, (mn - m) * p.scale_log2 > kLpLazy)) {
        // (-inf - -inf is NaN and compares false; the row's O is 0 then and stays so)
        ok = mbar_wait_warp(&sm.o_done[w], (j - 1) & 1, ctl, DETAIL_WAIT_ACCFULL);
        if (!ok) break;
        tc_fence_after();
        const float f = mn == -INFINITY ? 1.0f : exp2_fast((m - mn) * p.scale_log2);
        m = mn;
        l *= f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tO + c * 32, o);
          tmem_wait_ld_regs(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tmem_st_32x32b_x32(tO + c * 32, o);
        }
        tmem_wait_st();
      }
      if ((j + 1) * kLpTile > nk) {
        // Rows of V behind the request's last key belong to others: zero weights must meet zeros.
        ok = mbar_wait_warp(&sm.v_full[j & 1], (j >> 1) & 1, ctl, DETAIL_WAIT_KFULL);
        if (!ok) break;
        if (row >= nk - j * kLpTile)
#pragma unroll 1
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<uint4*>(sm.v[j & 1][c] + row * 128 + u * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      const float base = m == -INFINITY ? 0.0f : kShift - m * p.scale_log2;
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      // The numerators of 32 keys, rounded into P.
      auto numerators = [&](int c) {
        uint32_t packed[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x = fma2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])),
                                make_float2(p.scale_log2, p.scale_log2), make_float2(base, base));
          const float p0 = exp2_fast(x.x), p1 = exp2_fast(x.y);
          sum[e & 2] += p0;
          sum[(e & 2) + 1] += p1;
          packed[e >> 1] = pack_16<DT>(p0, p1);
        }
        tmem_st_32x32b_x16(tS + c * 16, packed);
      };
      auto hand_over = [&](int part) {
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready[w][part]);
      };
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        numerators(c);
        if (c == 1) hand_over(0);
        // (Nothing of a chunk is computed before the one in front of it is on its way.)
        if (c < 3) {
#pragma unroll
          for (int e = 0; e < 32; ++e) asm volatile("" : "+r"(s[c + 1][e]));
        }
      }
      hand_over(1);
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
    if (ok && nt[w] > 0) ok = mbar_wait_warp(&sm.o_done[w], (nt[w] - 1) & 1, ctl, DETAIL_WAIT_ACCFULL);
    tc_fence_after();
    if (ok && first < nq) {
      // A row that has seen nothing (l = 0) gets zeros; one that met a NaN keeps it.
      const float inv = l != 0.0f ? 1.0f / l : 0.0f;
      const int64_t at = static_cast<int64_t>(q0 + i) * p.H + h;
      const int64_t unit = ((static_cast<int64_t>(b) * p.n_blocks + qb) * p.H + h) * p.splits + split;
      float* part = p.part + unit * 2 * kLpTile * 128 + (i - i0) * 4;
      uint16_t* o_row = static_cast<uint16_t*>(p.out) + at * 128;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (nt[w] > 0) {
          tmem_ld_32x32b_x32(tO + c * 32, o);
          tmem_wait_ld_regs(o);
        }
        if (kSplit && i < nq && parts > 1) {
          if (l != 0.0f)
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part + (c * 32 + e) * 2 * kLpTile) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        } else if (i < nq) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              r[k] = l != 0.0f ? pack_16<DT>(__uint_as_float(o[e + 2 * k]) * inv, __uint_as_float(o[e + 2 * k + 1]) * inv)
                               : 0u;
            *reinterpret_cast<uint4*>(o_row + c * 32 + e) = make_uint4(r[0], r[1], r[2], r[3]);
          }
        }
      }
      if (kSplit && i < nq && parts > 1)
        p.ml[unit * 2 * kLpTile + (i - i0)] = make_float2(m, l);
      else if (i < nq && p.lse)
        p.lse[at] = l != 0.0f ? m * p.scale + (logf(l) - kShift * 0.69314718055994531f) : -INFINITY;
    }
    tc_fence_before();
  }
  __syncthreads();
  if constexpr (kSplit) grid_launch_dependents();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the split blocks: with M the largest m of a row, out = sum_c 2^((m_c - M) scale log2 e) O_c / L,
// L the same sum of the l_c, lse = scale M + ln L. A CTA takes 32 rows of a block, a warp 16 of the
// dims, a lane one row.
template <int DT>
__global__ void __launch_bounds__(256) latent_prefill_combine_kernel(const LpParams p) {
  constexpr int kRows = 2 * kLpTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.x, b = blockIdx.z;
  const int qb = blockIdx.y / (kRows / 32), row = blockIdx.y % (kRows / 32) * 32 + lane;
  const LpBlock u = lp_block(p, b, qb);
  // Every CTA waits before it exits, also where there is nothing to join: what comes behind this grid on the
  // stream waits for this grid only, and the grid in front has results of its own to write.
  grid_dependency_wait();
  if (u.bad || u.i0 + row - lane >= u.nq) return;
  const int parts = lp_parts(p, max(u.tiles(0, p.causal), u.tiles(1, p.causal)));
  if (parts == 1) return;                     // (its CTA has written the results)
  if (u.i0 + row >= u.nq) return;
  const int64_t unit = ((static_cast<int64_t>(b) * p.n_blocks + qb) * p.H + h) * p.splits * kRows;
  const float2* ml = p.ml + unit + row;
  float M = -INFINITY, L = 0.0f;
  uint32_t live = 0;                          // parts that have seen something of this row (others write no O)
#pragma unroll 8
  for (int c = 0; c < parts; ++c) {
    const float2 v = ml[c * kRows];
    M = fmaxf(M, v.x);
    live |= (v.y != 0.0f ? 1u : 0u) << c;
  }
  float acc[16] = {};
  const float* src = p.part + unit * 128 + (warp * 4 * kRows + row) * 4;
#pragma unroll 4
  for (int c = 0; c < parts; ++c) {
    const bool seen = live >> c & 1;
    float4 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = seen ? __ldcs(reinterpret_cast<const float4*>(src + (static_cast<int64_t>(c) * 32 + k) * kRows * 4))
                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float2 v = ml[c * kRows];
    const float f = seen ? exp2f((v.x - M) * p.scale_log2) : 0.0f;
    L += f * v.y;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      acc[4 * k] = fmaf(f, o[k].x, acc[4 * k]);
      acc[4 * k + 1] = fmaf(f, o[k].y, acc[4 * k + 1]);
      acc[4 * k + 2] = fmaf(f, o[k].z, acc[4 * k + 2]);
      acc[4 * k + 3] = fmaf(f, o[k].w, acc[4 * k + 3]);
    }
  }
  const float inv = L != 0.0f ? 1.0f / L : 0.0f;
  const int64_t at = static_cast<int64_t>(u.q0 + u.i0 + row) * p.H + h;
  uint32_t out[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = pack_16<DT>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * 128 + warp * 16);
  dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
  dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
  if (warp == 0 && p.lse)
    p.lse[at] = L != 0.0f ? M * p.scale + (logf(L) - kNumeratorShift<DT> * 0.69314718055994531f) : -INFINITY;
}

static int64_t lp_blocks(int max_q, int Tq) { return (static_cast<int64_t>(std::min(max_q, Tq)) + 2 * kLpTile - 1) / (2 * kLpTile); }

// How the key tiles of the blocks are split: parts of `chunk` tiles, `splits` of them at most.
struct LpPlan {
  int chunk, splits;
};
// The chunk with the shortest estimated run, in tiles, of a call with no more blocks than SMs, taken from
// the average request: SMs that have no full part take the rests, each of which costs two tiles more for
// its start and end, the join costs two for every part an SM and an empty CTA half of one. The call stays
// whole unless that saves kLpMinGain tiles of its longest block.
static LpPlan lp_plan(int B, int Tq, int Tk, int max_q, int H, bool causal, int num_sms) {
  const int64_t units = lp_blocks(max_q, Tq) * B * H;
  if (units < 1 || units > num_sms) return {0, 1};
  // (Rows outside the requests count towards Tq and Tk; max_q bounds what they can add.)
  const int64_t nq = std::min<int64_t>((static_cast<int64_t>(Tq) + B - 1) / B, max_q);
  const int64_t nk = (static_cast<int64_t>(Tk) + B - 1) / B, key_tiles = (static_cast<int64_t>(Tk) + kLpTile - 1) / kLpTile;
  auto tiles = [&](int64_t i) {                 // of the block of query i
    const int64_t sees = causal ? std::max<int64_t>(0, nk - nq + std::min(i + 2 * kLpTile, nq)) : nk;
    return (sees + kLpTile - 1) / kLpTile;
  };
  int64_t total = 0, longest = 0;
  for (int64_t i = 0; i < nq; i += 2 * kLpTile) {
    longest = std::max(longest, tiles(i));
    total += tiles(i);
  }
  // The partial sums have places for as many parts a block as the longest request could have.
  const int64_t most = std::min<int64_t>(kLpMaxSplits, kLpMaxPlaces * num_sms / units);
  const int64_t lo = std::max<int64_t>({kLpMinTiles, (total * B * H + num_sms - 1) / num_sms, (key_tiles + most - 1) / most});
  int64_t best = 0, best_run = longest - kLpMinGain + 1;
  for (int64_t chunk = lo; chunk < best_run; chunk += std::max<int64_t>(1, lo / 32)) {
    int64_t full = 0, rests = 0, rest_tiles = 0, parts = 0;
    for (int64_t i = 0; i < nq; i += 2 * kLpTile) {
      const int64_t n = tiles(i);
      full += n / chunk;
      rests += n % chunk ? 1 : 0;
      rest_tiles += n % chunk;
      parts += n > chunk ? (n + chunk - 1) / chunk : 0;
    }
    const int64_t free = num_sms - full * B * H;
    if (free < 0 || (free == 0 && rests > 0)) continue;
    const int64_t run = std::max(chunk, rests == 0 ? 0 : (rest_tiles + 2 * rests) * B * H / free - 2) +
                        (2 * parts * B * H + (key_tiles + chunk - 1) / chunk * units / 2) / num_sms;
    if (run < best_run) best = chunk, best_run = run;
  }
  if (best == 0) return {0, 1};
  return {static_cast<int>(best), static_cast<int>((key_tiles + best - 1) / best)};
}

size_t latent_prefill_workspace_bytes(int B, int Tq, int Tk, int max_q, int H, bool causal, int num_sms) {
  const int splits = lp_plan(B, Tq, Tk, max_q, H, causal, num_sms).splits;
  if (splits <= 1) return DSA_WS_HEADER_BYTES;
  const size_t rows = static_cast<size_t>(lp_blocks(max_q, Tq)) * B * H * splits * 2 * kLpTile;
  return DSA_WS_HEADER_BYTES + rows * (128 + 2) * sizeof(float);
}

template <int DT>
static dsa_status launch_prefill_dt(const LatentPrefillParams& a, LpPlan plan, cudaStream_t stream) {
  CUtensorMap mq, mk, mpe, mv;
  // With no keys at all no key box is loaded: any valid map does.
  const bool none = a.Tk == 0;
  const uint64_t Tk = none ? 1 : a.Tk;
  if (!encode_tmap_3d_16(&mq, a.q, 192, a.H, a.qs_h, a.Tq, a.qs_t, 64, 1, kLpTile) ||
      !encode_tmap_3d_16(&mk, none ? a.q : a.k_nope, 128, a.H, a.ks_h, Tk, a.ks_t, 64, 1, kLpTile) ||
      !encode_tmap_3d_16(&mpe, none ? a.q : a.k_pe, 64, 1, 64, Tk, a.pes_t, 64, 1, kLpTile) ||
      !encode_tmap_3d_16(&mv, none ? a.q : a.v, 128, a.H, a.vs_h, Tk, a.vs_t, 64, 1, kLpTile))
    return DSA_ERR_CUDA;
  const int blocks = static_cast<int>(lp_blocks(a.max_q, a.Tq)), splits = plan.splits;
  float* part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.hdr) + DSA_WS_HEADER_BYTES);
  float* ml = part + static_cast<size_t>(blocks) * a.B * a.H * splits * 2 * kLpTile * 128;
  const LpParams p{a.cu_q, a.cu_k, a.Tq, a.Tk, a.max_q, a.H, a.causal, a.scale, a.scale * 1.4426950408889634f,
                   a.out, a.lse, blocks, splits, plan.chunk, part, reinterpret_cast<float2*>(ml), a.hdr, a.budget_ns};
  const size_t smem = sizeof(LpSmem) + 1024;
  static_assert(sizeof(LpSmem) + 1024 <= 227 * 1024, "shared memory");
  const auto kernel = splits > 1 ? latent_prefill_kernel<DT, true> : latent_prefill_kernel<DT, false>;
  if (!allow_shared<latent_prefill_kernel<DT, true>>(smem) || !allow_shared<latent_prefill_kernel<DT, false>>(smem))
    return DSA_ERR_CUDA;
  kernel<<<dim3(a.H, blocks, a.B * splits), kLpThreads, smem, stream>>>(mq, mk, mpe, mv, p);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  if (splits == 1) return DSA_OK;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.H, blocks * (2 * kLpTile / 32), a.B);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, latent_prefill_combine_kernel<DT>, p));
}

dsa_status launch_latent_prefill(const LatentPrefillParams& a, size_t workspace_bytes, int dtype, cudaStream_t stream) {
  if (lp_blocks(a.max_q, a.Tq) > 65535) return DSA_ERR_UNSUPPORTED;
  // A workspace without room for the parts leaves the blocks whole.
  LpPlan plan{0, 1};
  if (workspace_bytes >= latent_prefill_workspace_bytes(a.B, a.Tq, a.Tk, a.max_q, a.H, a.causal, a.num_sms))
    plan = lp_plan(a.B, a.Tq, a.Tk, a.max_q, a.H, a.causal, a.num_sms);
  return dtype == DSA_DTYPE_BF16 ? launch_prefill_dt<DSA_DTYPE_BF16>(a, plan, stream)
                                 : launch_prefill_dt<DSA_DTYPE_F16>(a, plan, stream);
}

}  // namespace dsa

// Dense latent attention of decode queries (absorbed form) for sm_100a: 1 to 8 new tokens a request
// against all of the request's paged 576-wide latents, whose first 512 entries are the values.
//
// A request's query rows are its q_len * Hq (token, head) pairs, taken HT (16, 32 or 64) at a time.
// For one row tile the requests' key tiles (32 keys each), laid end to end, are split into equal
// contiguous ranges, one per CTA, so that every CTA streams the same number of tiles whatever the
// lengths; the part of a range inside one request is a segment. A segment that is a whole request
// writes its outputs, any other its unnormalised sums with m and l, and latent_combine_kernel joins
// those of a request. The grid is one CTA per SM over all row tiles, so row tiles of the same
// request run side by side and the second one finds the latents in L2.
//
// Per key tile: S = Q K^T (rows x 32 keys x 576) into TMEM, softmax numerators P to shared memory,
// and O^T += V^T P^T (4 x 128 dims x rows x 32 keys). The latent tile in shared memory serves both
// products: as K (dims contiguous, K-major) and as V^T (the same bytes, M-major), so every latent is
// fetched once. O^T has the dims on TMEM lanes and the rows on columns: 4 * HT columns, which is what
// leaves room beside it (512 dims of 64 rows in 32 bits are half of TMEM).
//   warps 0-3  softmax of 16 rows each (S of a 64-row MMA lies on the first 16 lanes of each TMEM
//              quarter), as many of them as the row tile needs;
//   warps 4-7  the queries of each segment into shared memory, O^T rescaled (thread = dim) only when
//              some row's maximum has grown by more than 2^kLdLazy, the segment's results;
//   warp 8     TMA: a tile as one box of nine 64-dim chunks of 4 KB, into a ring of four or five tiles;
//   warp 9     one thread issues the QK products, up to three tiles ahead of the softmax;
//   warp 10    one thread issues the PV products. (With both in one thread the tensor core idled while
//              that thread looked at its barriers: 1.4% more time on the long case below.)
//
// Row tiles of 16, 32 or 64 rows: the fewest rows that hold a request's. 16 requests of 8000 keys: 36.5 us
// at 16 rows and 39.6 at 32, where tiles of 64 rows take 48 for both; 4 requests of 900 keys, 16 rows:
// 13.4, and 18.8 in tiles of 64. More than 64 rows are several tiles: O^T of 128 would fill TMEM.
//
// Bound: for up to 64 rows a request the bytes, 1152 a key (24 requests of 8000 to 16000 keys, 8 heads:
// 62 us, 5.0 TB/s). With more, the products of each row tile: a QK of 64 rows and 32 keys reads 3 KB of
// operands from shared memory in 25 cycles, three times what its FLOPs need, so a tile's 36 take 900
// cycles and its PV 260 more, of the 1550 that a tile takes: 32 requests of 10000 to 40000 keys at 128
// heads, 335 us back to back, which the power limit holds at 1700 MHz (300 to 320 from idle). 4 requests of
// up to 900 keys at 16 heads: 13 us, which is two launches and the latency of one tile's chain, TMA to
// result. Measured against it on the long case, where it took 292 us from idle: two softmax groups 300, the
// queries in TMEM 298, the tiles fetched into L2 ahead of time 304, QKs of two key tiles at once, which
// read the queries half as often, 331 (a ring of four tiles then leaves nothing to look ahead to).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace dsa {

constexpr int kLdDqk = 576, kLdDv = 512;
constexpr int kLdKeys = 32;                     // keys of a tile
constexpr int kLdChunks = kLdDqk / 64;          // 9
constexpr int kLdScores = 3;                    // S buffers: two QK products ahead of the PV
constexpr int kLdSlotBytes = kLdKeys * 128;     // 4 KB: one chunk
constexpr int kLdTileBytes = kLdChunks * kLdSlotBytes;
constexpr int kLdThreads = 352;
// Tiles whose barriers and rescale factors are kept apart. One of warps 4-7 may be two tiles ahead of
// another (the softmax hands over the maxima of tile t + 2 before it waits for the PV of tile t): with
// p_ready of two tiles its arrival there would count for the slow one's at tile t.
constexpr int kLdLead = 4;
// Cost of a segment's start and end, in tiles: CTAs that pass from one request to the next get fewer tiles.
// (20 requests of 100 to 600 keys, 64 rows: 21.2 us with 4, 24.8 with 0; 300 of 1 to 300, 16 rows: 42.8 and
// 49.7; 12 of 300 to 5000, 128 rows: 35.9 and 36.9; 2, 6 and 9 are within 5% of 4.)
constexpr int kLdSegment = 4;
constexpr float kLdLazy = 6.0f;

template <int HT>
struct LdSmem {
  static constexpr int kStages = HT == 64 ? 4 : 5;
  uint8_t q[kLdChunks][HT * 128];               // the MMA reads 64 rows from each: into what follows
  uint8_t p[HT * 128];                          // P of two tiles side by side
  uint8_t ring[kStages][kLdTileBytes];
  float fac[kLdLead][HT], inv[HT];
  int grow[kLdLead][4];                         // whether a softmax warp's factors are to be applied
  uint64_t full[kStages], empty[kStages];       // empty: the tile's PV is done
  uint64_t q_full, s_full[kLdScores], m_ready[kLdLead], p_ready[kLdLead], seg_ready, seg_done, drain[2];
  uint32_t tmem;
  int abort;
  int b0, tile0, ntiles;                        // this CTA's range
};

struct LdParams {
  const uint16_t* q;
  int64_t qs_t, qs_h;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int32_t n_blocks, block_size, max_blocks, B, q_len, Hq;
  int32_t box_rows;                             // latent rows of one TMA box
  float scale, scale_log2;
  uint16_t* out;
  float* lse;
  float* part;                                  // [row tiles][CTAs][2][HT / 4][512][4] unnormalised O^T
  float* ml;                                    // [row tiles][CTAs][2][2][HT] m, l
  WsHeader* hdr;
  uint64_t budget_ns;
};

__device__ __forceinline__ int ld_len(const LdParams& p, int b) {
  return max(0, min(__ldg(&p.seq_lens[b]), p.max_blocks * p.block_size));
}
__device__ __forceinline__ int ld_tiles(const LdParams& p, int b) { return (ld_len(p, b) + kLdKeys - 1) / kLdKeys; }

// A request's work in units of a tile: its tiles, and kLdSegment for the segment that begins with it.
__device__ __forceinline__ int ld_work(int tiles) { return tiles > 0 ? tiles + kLdSegment : 0; }

// The work of requests [0, n), by one warp.
__device__ __forceinline__ int64_t ld_work_before(const LdParams& p, int n, int lane) {
  int64_t sum = 0;
  for (int b = lane; b < n; b += 32) sum += ld_work(ld_tiles(p, b));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
  return sum;
}

// CTAs of a row tile that share work T: no more than its units. (One whose range is all kLdSegment has
// nothing to do.)
__device__ __forceinline__ int64_t ld_sharers(int64_t T, int n_cta) { return T < n_cta ? (T > 0 ? T : 1) : n_cta; }

template <int DT>
__device__ __forceinline__ uint16_t ld_round(float x) {
  return static_cast<uint16_t>(pack_16<DT>(x, 0.0f));
}

// Two values with zeros for those that are not finite.
template <int DT>
__device__ __forceinline__ uint32_t ld_finite(uint32_t two) {
  constexpr uint32_t kExp = DT == DSA_DTYPE_BF16 ? 0x7F80u : 0x7C00u;
  if ((two & kExp) == kExp) two &= 0xFFFF0000u;
  if ((two >> 16 & kExp) == kExp) two &= 0x0000FFFFu;
  return two;
}

template <int DT, int HT>
__global__ void __launch_bounds__(kLdThreads, 1)
    latent_decode_kernel(const __grid_constant__ CUtensorMap map_latent, const LdParams p) {
  extern __shared__ uint8_t smem_raw[];
  LdSmem<HT>& sm = *reinterpret_cast<LdSmem<HT>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                  ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ht = blockIdx.x, cta = blockIdx.y;  // row tiles fastest: those of one range run together
  const int R = p.q_len * p.Hq;

  constexpr int kStages = LdSmem<HT>::kStages, kSoft = HT / 16;
  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.q_full, 4);
    for (int i = 0; i < kLdScores; ++i) mbar_init(&sm.s_full[i], 1);
    for (int i = 0; i < kLdLead; ++i) {
      mbar_init(&sm.m_ready[i], kSoft);
      mbar_init(&sm.p_ready[i], kSoft + 4);
    }
    mbar_init(&sm.seg_ready, kSoft);
    mbar_init(&sm.seg_done, 4);
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    // This CTA's range [lo, hi) of all key tiles, and the request holding lo.
    if (cta == 0 && ht == 0)
      for (int b = lane; b < p.B; b += 32) {
        const int n = __ldg(&p.seq_lens[b]);
        if (n < 0 || n > p.max_blocks * p.block_size) record_error(p.hdr, DSA_ERR_DEVICE, DETAIL_BAD_SEQ_LEN);
      }
    const int nt0 = lane < p.B ? ld_tiles(p, lane) : 0;  // (of the first 32 requests)
    int64_t T = ld_work(nt0);
#pragma unroll 1
    for (int b = lane + 32; b < p.B; b += 32) T += ld_work(ld_tiles(p, b));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) T += __shfl_xor_sync(0xFFFFFFFFu, T, off);
    const int64_t G = ld_sharers(T, gridDim.y);
    const int64_t lo = cta < G ? T * cta / G : T, hi = cta < G ? T * (cta + 1) / G : T;
    int64_t carry = 0;
    int mine = 0;                               // key tiles of the lane's requests inside the range
#pragma unroll 1
    for (int base = 0; base < p.B && carry < hi; base += 32) {
      const int bb = base + lane;
      const int nt = base == 0 ? nt0 : bb < p.B ? ld_tiles(p, bb) : 0, work = ld_work(nt);
      uint32_t incl = work;                     // (32 requests of 2^31 keys stay below 2^32)
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += o;
      }
      const int64_t first = carry + incl - work + kLdSegment;  // its first tile's place
      if (nt > 0) {
        const int64_t from = max(lo, first), to = min(hi, first + nt);
        if (from < to) mine += static_cast<int>(to - from);
        if (first - kLdSegment <= lo && lo < first + nt) {
          sm.b0 = bb;
          sm.tile0 = static_cast<int>(from - first);
        }
      }
      carry += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, off);
    if (lane == 0) sm.ntiles = mine;
  }
  if (warp == 9) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem, tO = tmem + kLdScores * kLdKeys;
  const WaitCtl ctl{p.hdr, &sm.abort, p.budget_ns};
  const int total = sm.ntiles;
  // Waits (as a warp) for the PV of the CTA's tile i.
  auto pv_done = [&](int i) {
    return mbar_wait_warp(&sm.empty[i % kStages], (i / kStages) & 1, ctl, DETAIL_WAIT_ACCFULL);
  };

  // Each of the two issuing roles runs in one thread that elect picks: the compiler then knows that the
  // operands of its instructions are uniform (an MMA takes 29 cycles to issue instead of 54, a box of a
  // TMA load 32 instead of 70; measured alone).
  if (warp == 8) {
    if (total > 0 && elect_one()) {
      const int n_box = kLdKeys / p.box_rows;
      // First latent row of box i of request b's key tile t, -1 at or behind the request's end.
      auto box_row = [&](int b, int t, int n, int i) {
        const int s = t * kLdKeys + i * p.box_rows;
        if (s >= n) return -1;
        int blk = __ldg(&p.block_table[static_cast<int64_t>(b) * p.max_blocks + s / p.block_size]);
        if (blk < 0 || blk >= p.n_blocks) {
          record_error(p.hdr, DSA_ERR_DEVICE, DETAIL_BAD_BLOCK_TABLE);
          blk = 0;
        }
        return blk * p.block_size + s % p.block_size;
      };
      int b = sm.b0, t = sm.tile0, n = ld_len(p, b), row = box_row(b, t, n, 0), done = 0, st = 0, ph = 0;
      bool ok = true;
      for (; done < total && ok; ++done) {
        const int cb = b, ct = t, cn = n, cur = row;
        if (done + 1 < total) {                 // the next tile's first table entry, a tile ahead
          if (++t >= (n + kLdKeys - 1) / kLdKeys) {
            t = 0;
#pragma unroll 1
            do n = ld_len(p, ++b);
            while (n == 0);
          }
          row = box_row(b, t, n, 0);
        }
        uint8_t* ring = sm.ring[st];
        ok = mbar_wait_call(&sm.empty[st], ph ^ 1, ctl, DETAIL_WAIT_KEMPTY);
        if (!ok) break;
        if (n_box == 1) {
          mbar_arrive_expect_tx(&sm.full[st], kLdTileBytes);
          tma_load_3d(ring, &map_latent, 0, cur, 0, &sm.full[st]);
        } else {
          const int boxes = min(n_box, (cn - ct * kLdKeys + p.box_rows - 1) / p.box_rows);
          mbar_arrive_expect_tx(&sm.full[st], kLdChunks * boxes * p.box_rows * 128);
#pragma unroll 1
          for (int i = 0; i < boxes; ++i) {
            const int first = i == 0 ? cur : box_row(cb, ct, cn, i);
#pragma unroll 1
            for (int c = 0; c < kLdChunks; ++c)
              tma_load_3d(ring + c * kLdSlotBytes + i * p.box_rows * 128, &map_latent, 0, first, c, &sm.full[st]);
          }
        }
        if (++st == kStages) st = 0, ph ^= 1;
      }
      // Let every copy land before the CTA exits (bounded).
#pragma unroll 1
      for (int i = max(0, done - kStages); i < done; ++i)
        mbar_drain_call(&sm.full[i % kStages], (i / kStages) & 1, p.budget_ns);
    }
    __syncwarp();
  } else if (warp == 9) {
    if (total > 0 && elect_one()) {
      constexpr uint32_t idesc = make_idesc_16(DT == DSA_DTYPE_BF16 ? 1u : 0u, 64, kLdKeys);
      int b = sm.b0, left = min(ld_tiles(p, b) - sm.tile0, total), seg = 0, st = 0, ph = 0, buf = 0;
      const uint64_t dq = make_smem_desc(smem_u32(sm.q[0]), 128), dk0 = make_smem_desc(smem_u32(sm.ring[0]), 128);
      bool ok = mbar_wait_call(&sm.q_full, 0, ctl, DETAIL_WAIT_QFULL);
#pragma unroll 1
      for (int t = 0; t < total && ok; ++t) {
        if (left == 0) {                        // the next segment, once its queries are there
#pragma unroll 1
          do left = min(ld_tiles(p, ++b), total - t);
          while (left == 0);
          ++seg;
          ok = mbar_wait_call(&sm.q_full, seg & 1, ctl, DETAIL_WAIT_QFULL);
        }
        // An S buffer is free once the scores of the tile that had it have been read.
        const int u = t - kLdScores;
        if (ok && u >= 0) ok = mbar_wait_call(&sm.m_ready[u % kLdLead], (u / kLdLead) & 1, ctl, DETAIL_WAIT_SCORES);
        ok = ok && mbar_wait_call(&sm.full[st], ph, ctl, DETAIL_WAIT_KFULL);
        if (!ok) break;
        tc_fence_after();
        const uint64_t dk = dk0 + st * (kLdTileBytes >> 4);
#pragma unroll
        for (int c = 0; c < kLdChunks; ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_16(tmem + buf * kLdKeys, dq + (c * HT * 128 >> 4) + 2ull * kk,
                        dk + (c * kLdSlotBytes >> 4) + 2ull * kk, idesc, c > 0 || kk > 0 ? 1u : 0u);
        tc_commit(&sm.s_full[buf]);
        --left;
        if (++buf == kLdScores) buf = 0;
        if (++st == kStages) st = 0, ph ^= 1;
      }
      tc_commit(&sm.drain[0]);
      mbar_drain_call(&sm.drain[0], 0, p.budget_ns);
    }
    __syncwarp();
  } else if (warp == 10) {
    if (total > 0 && elect_one()) {
      constexpr uint32_t idesc = make_idesc_16(DT == DSA_DTYPE_BF16 ? 1u : 0u, 128, HT) | kIdescAMnMajor;
      int b = sm.b0, left = min(ld_tiles(p, b) - sm.tile0, total), st = 0;
      uint32_t acc = 0;                         // 0: the segment's first tile
      const uint64_t dv0 = make_smem_desc_mn(smem_u32(sm.ring[0]), kLdSlotBytes, 1024);
      const uint64_t dp0 = make_smem_desc(smem_u32(sm.p), 128);
#pragma unroll 1
      for (int t = 0; t < total; ++t) {
        if (left == 0) {
#pragma unroll 1
          do left = min(ld_tiles(p, ++b), total - t);
          while (left == 0);
          acc = 0;
        }
        // (A tile whose P is there has landed: its scores came from it.)
        if (!mbar_wait_call(&sm.p_ready[t % kLdLead], (t / kLdLead) & 1, ctl, DETAIL_WAIT_SCORES)) break;
        tc_fence_after();
        const uint64_t dv = dv0 + st * (kLdTileBytes >> 4), dp = dp0 + (t & 1) * (kLdKeys * 2 >> 4);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int kk = 0; kk < kLdKeys / 16; ++kk)
            tc_mma_16(tO + mt * HT, dv + (mt * 2 * kLdSlotBytes + kk * 2048 >> 4), dp + 2ull * kk, idesc,
                        kk > 0 ? 1u : acc);
        tc_commit(&sm.empty[st]);
        --left;
        acc = 1;
        if (++st == kStages) st = 0;
      }
      tc_commit(&sm.drain[1]);
      mbar_drain_call(&sm.drain[1], 0, p.budget_ns);
    }
    __syncwarp();
  } else if (warp < 4) {
    // Softmax. S of a 64-row MMA has rows 16 w .. 16 w + 15 on the first 16 TMEM lanes of warp w's
    // quarter: the other half of the warp idles along.
    if (warp < kSoft && total > 0) {
      const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
      const int row = warp * 16 + (lane & 15), r = ht * HT + row;  // row of the tile, of the request
      const bool mine = lane < 16;
      int b = sm.b0, t = sm.tile0, left = total, done = 0, seg = 0, s_buf = 0, s_ph = 0;
      bool ok = true, have = false;             // have: s holds the tile's scores already
      uint32_t s[32], s_next[32];
      while (left > 0 && ok) {
        const int n = ld_len(p, b), nt = (n + kLdKeys - 1) / kLdKeys, te = min(nt, t + left), t_first = t;
        if (te <= t) {                          // a request without keys
          ++b;
          continue;
        }
        left -= te - t;
        const int sees = r < R ? max(0, n - p.q_len + 1 + r / p.Hq) : n;
        float m = -INFINITY, l = 0.0f;
#pragma unroll 1
        for (; t < te; ++t, ++done) {
          if (!have) {
            ok = mbar_wait_warp(&sm.s_full[s_buf], s_ph, ctl, DETAIL_WAIT_ACCFULL);
            if (!ok) break;
            tc_fence_after();
            tmem_ld_32x32b_x32(tmem + s_buf * kLdKeys + lanes, s);
            tmem_wait_ld_regs(s);
          }
          if (++s_buf == kLdScores) s_buf = 0, s_ph ^= 1;
          const int seen = sees - t * kLdKeys;  // visible keys of this tile
          if (__any_sync(0xFFFFFFFFu, seen < kLdKeys)) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= seen) s[e] = 0xFF800000u;  // -inf
          }
          float mx[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(s[e]));
          const float mn = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          // Rows whose maximum has grown by more than 2^kLdLazy have what they summed so far scaled down;
          // a segment's first tile has nothing yet. (-inf - -inf is NaN and compares false.)
          bool grow = mine && (mn - m) * p.scale_log2 > kLdLazy;
          if (t == t_first) {
            m = mn;
            grow = false;
          }
          const bool any = __any_sync(0xFFFFFFFFu, grow);
          if (any && mine) {
            const float f = grow ? exp2_fast((m - mn) * p.scale_log2) : 1.0f;
            if (grow) m = mn;
            l *= f;
            sm.fac[done % kLdLead][row] = f;
          }
          if (lane == 0) sm.grow[done % kLdLead][warp] = any;
          tc_fence_before();                    // (the QK issuer takes this as leave to overwrite S)
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.m_ready[done % kLdLead]);
          // The next tile's scores, where they are there already; they arrive behind the exponentials.
          have = done + 1 < total && __all_sync(0xFFFFFFFFu, mbar_test(&sm.s_full[s_buf], s_ph));
          if (have) {
            tc_fence_after();
            tmem_ld_32x32b_x32(tmem + s_buf * kLdKeys + lanes, s_next);
          }
          if (done >= 2) ok = pv_done(done - 2);  // P's half of the buffer is free
          if (mine) {
            const float base = m == -INFINITY ? 0.0f : kNumeratorShift<DT> - m * p.scale_log2;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t w4[4];
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const float p0 = exp2_fast(fmaf(__uint_as_float(s[u * 8 + e]), p.scale_log2, base));
                const float p1 = exp2_fast(fmaf(__uint_as_float(s[u * 8 + e + 1]), p.scale_log2, base));
                sum[e & 2] += p0;
                sum[(e & 2) + 1] += p1;
                w4[e >> 1] = pack_16<DT>(p0, p1);
              }
              *reinterpret_cast<uint4*>(sm.p + sw128(row, (done & 1) * 4 + u)) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_ready[done % kLdLead]);
          if (have) {
            tmem_wait_ld_regs(s_next);
#pragma unroll
            for (int e = 0; e < 32; ++e) s[e] = s_next[e];
          }
          if (!ok) break;
        }
        if (!ok) break;
        // The segment's sums, once the results of the one before are out.
        if (seg > 0) ok = mbar_wait_warp(&sm.seg_done, (seg - 1) & 1, ctl, DETAIL_WAIT_ACCEMPTY);
        if (mine) {
          if (t_first == 0 && te == nt) {
            sm.inv[row] = l != 0.0f ? 1.0f / l : 0.0f;
            if (p.lse && r < R)
              p.lse[static_cast<int64_t>(b) * R + r] =
                  l != 0.0f ? m * p.scale + (logf(l) - kNumeratorShift<DT> * 0.69314718055994531f) : -INFINITY;
          } else {
            float* ml = p.ml + ((static_cast<int64_t>(ht) * gridDim.y + cta) * 2 + (t_first == 0)) * 2 * HT;
            ml[row] = m;
            ml[HT + row] = l;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.seg_ready);
        ++seg;
        ++b;
        t = 0;
      }
    }
    __syncwarp();
  } else if (total > 0) {
    // Queries, O^T's scaling and the results (warps 4-7; TMEM quarter warp - 4).
    const int quarter = warp - 4, ctid = tid - 128;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    int b = sm.b0, t = sm.tile0, left = total, done = 0, seg = 0;
    bool ok = true;
    // A request's queries into shared memory (zeros behind the last row). A warp takes every fourth row;
    // a lane finds one of the warp's rows (16 at most) for the others.
    auto load_q = [&](int b) {
      const uint16_t* base = p.q + static_cast<int64_t>(b) * p.q_len * p.qs_t;
      const int rl = ht * HT + quarter + 4 * (lane & 15);
      const int64_t off = rl < R ? (rl / p.Hq) * p.qs_t + (rl % p.Hq) * p.qs_h : -1;
#pragma unroll 1
      for (int k = 0; k < HT / 4; ++k) {
        const int64_t o = __shfl_sync(0xFFFFFFFFu, off, k);
        const uint16_t* src = base + (o < 0 ? 0 : o);
#pragma unroll
        for (int x = lane; x < kLdDqk / 8; x += 32)
          cp_async_16(sm.q[x / 8] + sw128(quarter + 4 * k, x & 7), src + (o < 0 ? 0 : x * 8), o < 0 ? 0u : 16u);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full);
    };
    load_q(b);
    while (left > 0 && ok) {
      const int n = ld_len(p, b), nt = (n + kLdKeys - 1) / kLdKeys, te = min(nt, t + left), t_first = t;
      left -= te - t;
      int next = b;                             // the request of the segment after this one
      if (left > 0) {
#pragma unroll 1
        do ++next;
        while (ld_len(p, next) == 0);
      }
#pragma unroll 1
      for (; t < te; ++t, ++done) {
        // The tile's scores are complete and read, its rescale factors written.
        ok = mbar_wait_warp(&sm.m_ready[done % kLdLead], (done / kLdLead) & 1, ctl, DETAIL_WAIT_SCORES);
        if (!ok) break;
        const int* grow = sm.grow[done % kLdLead];
        bool any = false;
#pragma unroll
        for (int w = 0; w < kSoft; ++w) any |= grow[w] != 0;
        if (any) {
          ok = pv_done(done - 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4 * HT; c += 16) {
            const int w = (c & (HT - 1)) / 16;  // the softmax warp of these 16 rows
            if (!grow[w]) continue;
            uint32_t o[16];
            tmem_ld_32x32b_x16(tO + lanes + c, o);
            tmem_wait_ld_regs16(o);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * sm.fac[done % kLdLead][w * 16 + e]);
            tmem_st_32x32b_x16(tO + lanes + c, o);
          }
          tmem_wait_st();
        }
        if ((t + 1) * kLdKeys > n - p.q_len + 1) {
          // Zero weights must meet finite values: rows behind the request's last key hold anything, and
          // those of the new tokens are hidden from the tokens in front of them. (A token that sees a
          // latent which is not finite has it in its score.)
          ok = mbar_wait_warp(&sm.full[done % kStages], (done / kStages) & 1, ctl, DETAIL_WAIT_KFULL);
          if (!ok) break;
          const int key = ctid >> 2, pos = t * kLdKeys + key;
          if (pos > n - p.q_len) {
#pragma unroll 1
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int u = 0; u < 8; ++u) {
                uint4* v = reinterpret_cast<uint4*>(sm.ring[done % kStages] + (2 * (ctid & 3) + c) * kLdSlotBytes +
                                                    key * 128 + u * 16);
                if (pos >= n) {
                  *v = make_uint4(0, 0, 0, 0);
                } else {
                  const uint4 x = *v;
                  *v = make_uint4(ld_finite<DT>(x.x), ld_finite<DT>(x.y), ld_finite<DT>(x.z), ld_finite<DT>(x.w));
                }
              }
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready[done % kLdLead]);
      }
      if (!ok) break;
      // Every QK of the segment is done, so the next one's queries may come.
      if (left > 0) load_q(next);
      ok = mbar_wait_warp(&sm.seg_ready, seg & 1, ctl, DETAIL_WAIT_SCORES) && pv_done(done - 1);
      if (!ok) break;
      tc_fence_after();
      const bool whole = t_first == 0 && te == nt;
      float* part = p.part + ((static_cast<int64_t>(ht) * gridDim.y + cta) * 2 + (t_first == 0)) * kLdDv * HT;
#pragma unroll 1
      for (int c = 0; c < 4 * HT; c += 32) {    // 16 columns at a time, two loads in flight
        uint32_t o[2][16];
        tmem_ld_32x32b_x16(tO + lanes + c, o[0]);
        tmem_ld_32x32b_x16(tO + lanes + c + 16, o[1]);
        tmem_wait_ld_regs16(o[0]);
        tmem_wait_ld_regs16(o[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int col = c + 16 * k, dim = col / HT * 128 + quarter * 32 + lane, h0 = col & (HT - 1);
          if (whole) {
            uint16_t* out = p.out + (static_cast<int64_t>(b) * R + ht * HT + h0) * kLdDv + dim;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float f = sm.inv[h0 + e];
              if (ht * HT + h0 + e < R)
                out[e * kLdDv] = f != 0.0f ? ld_round<DT>(__uint_as_float(o[k][e]) * f) : static_cast<uint16_t>(0);
            }
          } else {
            float* dst = part + (static_cast<int64_t>(h0 / 4) * kLdDv + dim) * 4;
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<uint4*>(dst + e * kLdDv) = make_uint4(o[k][e], o[k][e + 1], o[k][e + 2], o[k][e + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.seg_done);
      ++seg;
      b = next;
      t = 0;
    }
  }
  __syncthreads();
  grid_launch_dependents();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the split requests: with M the largest m_c of a row, out = sum_c 2^((m_c - M) scale log2 e) O_c
// / L, L the same sum of the l_c, lse = scale M + ln L. A request without keys gets zeros and -inf.
// Block (x, ht, z) takes kLcDims of the dims of a run of requests, four rows of one dim a thread; the
// partial sums are read along the dims and turned in shared memory, so that out is written along them
// too.
template <int HT>
struct Lc {
  static constexpr int kDims = 256 * 4 / HT;    // 16 (HT = 64) to 64 (HT = 16): a vector a thread
  static constexpr int kPitch = kDims + 2;
};
template <int DT, int HT>
__global__ void __launch_bounds__(256) latent_combine_kernel(const LdParams p, int n_cta) {
  constexpr int kDims = Lc<HT>::kDims, kPitch = Lc<HT>::kPitch, kPer = 256 / HT;  // kPer: threads of a row
  extern __shared__ __align__(16) float lc_smem[];
  float* wt = lc_smem;                          // [splits][HT] weights
  float* tile = lc_smem + n_cta * HT;           // [HT][kPitch]
  __shared__ int64_t sh[2];
  const int tid = threadIdx.x, ht = blockIdx.y, d0 = blockIdx.z * kDims;
  const int R = p.q_len * p.Hq, rows = min(HT, R - ht * HT);
  const int b_lo = static_cast<int>(static_cast<int64_t>(p.B) * blockIdx.x / gridDim.x);
  const int b_hi = static_cast<int>(static_cast<int64_t>(p.B) * (blockIdx.x + 1) / gridDim.x);
  if (tid < 64) {
    const int64_t n = ld_work_before(p, tid < 32 ? p.B : b_lo, tid & 31);
    if ((tid & 31) == 0) sh[tid >> 5] = n;
  }
  __syncthreads();
  const int64_t T = sh[0], G = ld_sharers(T, n_cta);
  int64_t start = sh[1];
  grid_dependency_wait();
  for (int b = b_lo; b < b_hi; ++b) {
    const int nt = ld_tiles(p, b);
    const int64_t first = start + kLdSegment;
    start += ld_work(nt);
    uint16_t* out = p.out + (static_cast<int64_t>(b) * R + ht * HT) * kLdDv + d0;
    float* lse = p.lse ? p.lse + static_cast<int64_t>(b) * R + ht * HT : nullptr;
    if (nt == 0) {
      for (int i = tid; i < rows * kDims; i += 256) out[(i / kDims) * kLdDv + i % kDims] = 0;
      if (lse && blockIdx.z == 0 && tid < rows) lse[tid] = -INFINITY;
      continue;
    }
    // CTA c holds the places [T c / G, T (c + 1) / G): the holder of place x is ceil((x + 1) G / T) - 1.
    const int c0 = static_cast<int>(((first + 1) * G - 1) / T), c1 = static_cast<int>(((first + nt) * G - 1) / T);
    if (c0 == c1) continue;
    const int ns = c1 - c0 + 1;
    // The request's first CTA holds its beginning (slot 1), every other one begins inside it (slot 0).
    const int64_t slot0 = (static_cast<int64_t>(ht) * n_cta + c0) * 2;
    auto slot = [&](int c) { return slot0 + 2 * c + (c == 0 ? 1 : 0); };
    // The thread's vector of the first eight splits is on its way while the weights are formed.
    const int dim = tid % kDims, h = tid / kDims * 4;
    const float* src = p.part + (static_cast<int64_t>(h / 4) * kLdDv + d0 + dim) * 4;
    auto load = [&](int c) { return __ldcs(reinterpret_cast<const float4*>(src + slot(c) * kLdDv * HT)); };
    float4 o[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = c < ns ? load(c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    {
      const int row = tid / kPer, c_first = tid % kPer;
      float M = -INFINITY, L = 0.0f;
#pragma unroll 4
      for (int c = c_first; c < ns; c += kPer) {
        const float mc = p.ml[slot(c) * 2 * HT + row];
        wt[c * HT + row] = mc;
        M = fmaxf(M, mc);
      }
#pragma unroll
      for (int off = 1; off < kPer; off *= 2) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
#pragma unroll 4
      for (int c = c_first; c < ns; c += kPer) {
        const float mc = wt[c * HT + row], w = mc == -INFINITY ? 0.0f : exp2f((mc - M) * p.scale_log2);
        wt[c * HT + row] = w;
        L += w * p.ml[slot(c) * 2 * HT + HT + row];
      }
#pragma unroll
      for (int off = 1; off < kPer; off *= 2) L += __shfl_xor_sync(0xFFFFFFFFu, L, off);
      const float inv = L != 0.0f ? 1.0f / L : 0.0f;
      for (int c = c_first; c < ns; c += kPer) wt[c * HT + row] *= inv;
      if (lse && blockIdx.z == 0 && c_first == 0 && row < rows)
        lse[row] = L != 0.0f ? M * p.scale + (logf(L) - kNumeratorShift<DT> * 0.69314718055994531f) : -INFINITY;
    }
    __syncthreads();
    {
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
      for (int c0 = 0; c0 < ns; c0 += 8) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (c0 + c >= ns) break;
          const float4 w = *reinterpret_cast<const float4*>(wt + (c0 + c) * HT + h);
          acc.x += w.x * o[c].x;
          acc.y += w.y * o[c].y;
          acc.z += w.z * o[c].z;
          acc.w += w.w * o[c].w;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c0 + 8 + c < ns) o[c] = load(c0 + 8 + c);
      }
      tile[(h + 0) * kPitch + dim] = acc.x;
      tile[(h + 1) * kPitch + dim] = acc.y;
      tile[(h + 2) * kPitch + dim] = acc.z;
      tile[(h + 3) * kPitch + dim] = acc.w;
    }
    __syncthreads();
    for (int i = tid; i < rows * kDims / 2; i += 256) {
      const int h = i / (kDims / 2), d = i % (kDims / 2) * 2;
      *reinterpret_cast<uint32_t*>(out + h * kLdDv + d) = pack_16<DT>(tile[h * kPitch + d], tile[h * kPitch + d + 1]);
    }
    __syncthreads();
  }
}

// Rows of a row tile: the fewest that take all rows of a request, 64 at most.
static int ld_row_tile(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
// CTAs of one row tile: all row tiles together fill the SMs once.
static int ld_ctas(int row_tiles, int num_sms) { return std::max(1, num_sms / row_tiles); }

size_t latent_decode_workspace_bytes(int B, int q_len, int Hq, int num_sms) {
  (void)B;
  const int rows = q_len * Hq, ht = ld_row_tile(rows), tiles = (rows + ht - 1) / ht;
  const size_t segments = static_cast<size_t>(tiles) * ld_ctas(tiles, num_sms) * 2;
  return DSA_WS_HEADER_BYTES + segments * ht * (kLdDv + 2) * sizeof(float);
}

template <int DT, int HT>
static dsa_status launch_decode_ht(const LatentDecodeParams& a, cudaStream_t stream) {
  const int R = a.q_len * a.Hq, row_tiles = (R + HT - 1) / HT, n_cta = ld_ctas(row_tiles, a.num_sms);
  int box = kLdKeys;                            // the largest box that divides tiles and blocks
  while (a.block_size % box) box /= 2;
  CUtensorMap map;
  // A latent as nine chunks of 64 dims: one load brings a whole tile, chunk by chunk, where it is one box.
  if (!encode_tmap_3d_16(&map, a.latent, 64, static_cast<uint64_t>(a.n_blocks) * a.block_size, kLdDqk, kLdChunks, 64,
                         64, box, box == kLdKeys ? kLdChunks : 1))
    return DSA_ERR_CUDA;
  float* part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.hdr) + DSA_WS_HEADER_BYTES);
  const LdParams p{static_cast<const uint16_t*>(a.q), a.qs_t, a.qs_h, a.block_table, a.seq_lens, a.n_blocks,
                   a.block_size, a.max_blocks, a.B, a.q_len, a.Hq, box, a.scale, a.scale * 1.4426950408889634f,
                   static_cast<uint16_t*>(a.out), a.lse, part,
                   part + static_cast<size_t>(row_tiles) * n_cta * 2 * kLdDv * HT, a.hdr, a.budget_ns};
  const size_t smem = sizeof(LdSmem<HT>) + 1024;
  static_assert(sizeof(LdSmem<HT>) + 1024 <= 227 * 1024, "shared memory");
  // (At most one CTA a row tile and SM.)
  const size_t csmem = (static_cast<size_t>(a.num_sms) * HT + HT * Lc<HT>::kPitch) * sizeof(float);
  if (!allow_shared<latent_decode_kernel<DT, HT>>(smem) || !allow_shared<latent_combine_kernel<DT, HT>>(csmem))
    return DSA_ERR_CUDA;
  latent_decode_kernel<DT, HT><<<dim3(row_tiles, n_cta), kLdThreads, smem, stream>>>(map, p);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min(a.B, 128), row_tiles, kLdDv / Lc<HT>::kDims);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = csmem;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, latent_combine_kernel<DT, HT>, p, n_cta));
}

template <int DT>
static dsa_status launch_decode_dt(const LatentDecodeParams& a, cudaStream_t stream) {
  switch (ld_row_tile(a.q_len * a.Hq)) {
    case 16: return launch_decode_ht<DT, 16>(a, stream);
    case 32: return launch_decode_ht<DT, 32>(a, stream);
    default: return launch_decode_ht<DT, 64>(a, stream);
  }
}

dsa_status launch_latent_decode(const LatentDecodeParams& a, int dtype, cudaStream_t stream) {
  return dtype == DSA_DTYPE_BF16 ? launch_decode_dt<DSA_DTYPE_BF16>(a, stream)
                                 : launch_decode_dt<DSA_DTYPE_F16>(a, stream);
}

}  // namespace dsa

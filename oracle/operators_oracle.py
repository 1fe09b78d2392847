"""Oracle of the operators around the indexer: rotary positions, the E4M3 quantisation of index
queries and keys, the paged cache read, and dense latent attention in both forms.

TEST INFRASTRUCTURE ONLY. Nothing on the product path imports this module, and it shares no code
with the CUDA path. Plain fp64 numpy, one row or request at a time. The attention functions also
return sum_s p_s |v_s| / l of every output, which the tests' error bounds are built from.
"""

from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

E4M3_MAX = 448.0
F32_MIN_NORMAL = 2.0 ** -126


def rotary(x: np.ndarray, positions: np.ndarray, inv_freq: np.ndarray, interleaved: bool = False,
           offset: int = 0, mscale: float = 1.0, inverse: bool = False) -> np.ndarray:
    """x [T][H][d] with the 2 * len(inv_freq) dims from `offset` on turned by positions * inv_freq."""
    out = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    angle = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)[None, :]
    turn = mscale * np.exp((-1j if inverse else 1j) * angle)
    for i in range(half):
        a = offset + (2 * i if interleaved else i)
        b = a + (1 if interleaved else half)
        z = (x[:, :, a].astype(np.float64) + 1j * x[:, :, b]) * turn[:, i][:, None]
        out[:, :, a], out[:, :, b] = z.real, z.imag
    return out


def e4m3_values() -> np.ndarray:
    """The non-negative finite E4M3 values, by code 0 .. 126."""
    e, m = np.divmod(np.arange(127), 8)
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def e4m3_code(y: np.ndarray) -> np.ndarray:
    """Codes of the E4M3 values nearest to y (ties to the even code, saturated at 448)."""
    table = e4m3_values()
    mag = np.minimum(np.abs(y), E4M3_MAX)
    hi = np.searchsorted(table, mag)                   # table[hi - 1] < mag <= table[hi]
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - mag, mag - table[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantise(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """Rows x [T][n] (fp32 values) -> (codes [T][n], scale [T] f32); both quotients are fp32 numbers."""
    x = np.asarray(x, dtype=np.float32)
    top = np.abs(x).max(axis=1)
    scale = np.where(top > 0, np.maximum(top / np.float32(E4M3_MAX), np.float32(F32_MIN_NORMAL)), np.float32(1))
    scale = scale.astype(np.float32)
    return e4m3_code(x / scale[:, None]), scale


def cache_rows(block_table: np.ndarray, starts: Optional[np.ndarray], cu: np.ndarray, block_size: int) -> np.ndarray:
    """Cache row of every output row of a paged read."""
    rows = []
    for b in range(len(cu) - 1):
        first = 0 if starts is None else int(starts[b])
        for pos in range(first, first + int(cu[b + 1] - cu[b])):
            rows.append(int(block_table[b][pos // block_size]) * block_size + pos % block_size)
    return np.array(rows, dtype=np.int64)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float):
    """One query row q [dk] over k [n][dk], v [n][dv]: (out, lse, sum p |v| / l)."""
    if len(k) == 0:
        zero = np.zeros(v.shape[1])
        return zero, -np.inf, zero
    s = scale * (k @ q)
    p = np.exp(s - s.max())
    l = p.sum()
    return p @ v / l, s.max() + np.log(l), p @ np.abs(v) / l


def latent_decode(q, latent, block_table, seq_lens, scale: float, block_size: int, dv: int = 512):
    """q [B][q_len][Hq][dqk] over the paged latents: (out, lse, absolute sums), in float64."""
    B, q_len, Hq, _ = q.shape
    out, lse, mag = np.zeros((B, q_len, Hq, dv)), np.zeros((B, q_len, Hq)), np.zeros((B, q_len, Hq, dv))
    for b in range(B):
        n = int(seq_lens[b])
        pos = np.arange(n)
        k = latent[block_table[b][pos // block_size].astype(np.int64) * block_size + pos % block_size] if n else latent[:0]
        k = k.astype(np.float64)
        for i in range(q_len):
            sees = max(0, n - q_len + 1 + i)
            for h in range(Hq):
                out[b, i, h], lse[b, i, h], mag[b, i, h] = attend(q[b, i, h].astype(np.float64), k[:sees],
                                                                  k[:sees, :dv], scale)
    return out, lse, mag


def latent_prefill(q, k_nope, k_pe, v, cu_q, cu_k, scale: float, causal: bool = True):
    """Ragged prefill rows: (out [Tq][H][dv], lse [Tq][H], absolute sums), in float64; rows outside
    every request are NaN."""
    Tq, H, _ = q.shape
    out, lse = np.full((Tq, H, v.shape[2]), np.nan), np.full((Tq, H), np.nan)
    mag = np.full(out.shape, np.nan)
    for b in range(len(cu_q) - 1):
        nq, nk = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        ks = slice(int(cu_k[b]), int(cu_k[b + 1]))
        for h in range(H):
            k = np.concatenate([k_nope[ks, h], k_pe[ks]], axis=1).astype(np.float64)
            vv = v[ks, h].astype(np.float64)
            for i in range(nq):
                sees = max(0, nk - nq + 1 + i) if causal else nk
                t = int(cu_q[b]) + i
                out[t, h], lse[t, h], mag[t, h] = attend(q[t, h].astype(np.float64), k[:sees], vv[:sees], scale)
    return out, lse, mag

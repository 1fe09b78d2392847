"""Dense latent attention (absorbed decode form, expanded prefill form) through the C-ABI against the
fp64 oracle (GPU).

Tolerances, per output. A score is scale * q.k over dk terms accumulated in fp32 16 terms at a time
(dk / 16 roundings of a sum that never passes sum |q k|; half a step each, doubled for an accumulator
that truncates), plus the product with scale log2 e and the exponent's argument (2 more): ds = scale
sum |q k| (dk / 16 + 2) 2^-23. An exponential is off by ds + 2^-21 relatively (ex2.approx 2 ulp, or a
polynomial as good) and a softmax numerator is rounded to half a step u (eps / 2) before the value
product, so with A = sum p |v| / l an output is off by at most A (u + 2 ds + 2^-20) for that, A times
2^-16 for the fp32 sums over up to 2^8 blocks of keys and their joins, and u |out| for the last
rounding. lse is off by ds + 2^-20 + |lse| 2^-22. In f16 a numerator below 2^-24 of the row's largest
(after the kernel's scaling) may vanish: n 2^-24 max |v| more."""

import math

import numpy as np
import pytest
import torch

import oracle.operators_oracle as O
from sparse_attention_token_04_b200 import binding as B
from synth import latent_decode_inputs

pytestmark = pytest.mark.gpu

NOPE, PE, DV, LATENT, LV = 128, 64, 128, 576, 512


def _num(t):
    return t.detach().cpu().double().numpy()


def _close(out, lse, ref, ref_lse, mag, ds, dtype, n_keys, vmax):
    u = torch.finfo(dtype).eps / 2
    tol = mag * (u + 2 * ds[..., None] + 2.0 ** -20 + 2.0 ** -16) + u * np.abs(ref) * (1 + 2.0 ** -6) + 1e-30
    if dtype == torch.float16:
        tol = tol + n_keys * 2.0 ** -24 * vmax + 2.0 ** -25
    err = np.abs(_num(out) - ref)
    assert (err <= tol).all(), (err - tol).max()
    if lse is not None:
        got = _num(lse)
        none = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(got), none)
        assert (np.abs(got[~none] - ref_lse[~none]) <= ds[~none] + 2.0 ** -20 + np.abs(ref_lse[~none]) * 2.0 ** -22).all()


def _paged(lens, block_size, seed, dtype, poison=True):
    """Latents of requests in shuffled pages; rows behind a request's last position are NaN."""
    g = torch.Generator().manual_seed(seed)
    nb = [(n + block_size - 1) // block_size for n in lens]
    perm = torch.randperm(sum(nb) + 1, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(max(nb), 1)), -1, dtype=torch.int32)
    latent = torch.randn((sum(nb) + 1) * block_size, LATENT, generator=g).to(dtype)
    at = 0
    for b, n in enumerate(lens):
        table[b, :nb[b]] = perm[at:at + nb[b]]
        at += nb[b]
        if poison and n % block_size:
            last = int(table[b, nb[b] - 1]) * block_size
            latent[last + n % block_size:last + block_size] = float("nan")
    if poison:
        latent[int(perm[-1]) * block_size:(int(perm[-1]) + 1) * block_size] = float("inf")
    return latent, table, torch.tensor(lens, dtype=torch.int32)


def _decode_case(lens, q_len, Hq, block_size, dtype, seed, scale=0.08, **kw):
    latent, table, seq = _paged(lens, block_size, seed, dtype)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(len(lens), q_len, Hq, LATENT, generator=g).to(dtype)
    return q, latent, table, seq, scale


def _check_decode(q, latent, table, seq, scale, block_size, out, lse):
    nq, nl = _num(q), _num(latent)
    ref, ref_lse, mag = O.latent_decode(nq, nl, table.numpy(), seq.numpy(), scale, block_size)
    n = max(1, int(seq.max()))
    top = np.nan_to_num(np.abs(nl), nan=0.0, posinf=0.0)
    ds = scale * np.abs(nq).sum(-1) * top.max() * 0.5 * (LATENT / 16 + 2) * 2.0 ** -23
    _close(out, lse, ref, ref_lse, mag, ds, q.dtype, n, top[:, :LV].max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,q_len,Hq,block_size", [
    ([1], 1, 1, 64), ([64], 1, 128, 64), ([65, 63, 1, 0, 128], 1, 16, 64), ([700, 3, 129], 1, 128, 64),
    ([300, 2, 1, 0], 3, 5, 64), ([1000, 40], 8, 16, 64), ([500, 77], 2, 64, 16), ([200, 9], 1, 33, 8),
    ([900, 130], 1, 20, 128), ([90], 8, 128, 64), ([513, 250], 1, 8, 24)])
def test_decode_matches_oracle(dtype, lens, q_len, Hq, block_size):
    q, latent, table, seq, scale = _decode_case(lens, q_len, Hq, block_size, dtype, sum(lens) + Hq)
    ws = torch.zeros(B.dsa_latent_attention_decode_workspace_bytes(len(lens), q_len, Hq), dtype=torch.uint8,
                     device="cuda")
    out, lse = B.dsa_latent_attention_decode(q.cuda(), latent.cuda(), table.cuda(), seq.cuda(), scale,
                                             block_size=block_size, workspace=ws)
    assert B.dsa_read_device_status(ws) == (0, 0)
    _check_decode(q, latent, table, seq, scale, block_size, out, lse)


@pytest.mark.parametrize("B_,lo,hi,Hq", [(1, 9000, 9000, 16), (300, 1, 200, 8), (7, 1, 3000, 64), (2, 20000, 20001, 128)])
def test_decode_many_requests_and_long_ones(B_, lo, hi, Hq):
    """Requests split over many CTAs and CTAs that hold many requests, checked on a few heads; a
    rising score makes every later key tile the new maximum of some heads."""
    g = torch.Generator().manual_seed(Hq)
    lens = [int(x) for x in torch.randint(lo, hi + 1, (B_,), generator=g)]
    q, latent, table, seq, scale = _decode_case(lens, 1, Hq, 64, torch.bfloat16, 3)
    for b in range(0, B_, 2):                     # keys of the even requests grow along the request
        n = lens[b]
        pos = torch.arange(n)
        rows = table[b][pos // 64].long() * 64 + pos % 64
        latent[rows] = (latent[rows].float() * (0.1 + 2.0 * pos / n)[:, None]).to(torch.bfloat16)
    out, lse = B.dsa_latent_attention_decode(q.cuda(), latent.cuda(), table.cuda(), seq.cuda(), scale)
    heads = [0, Hq // 2, Hq - 1]
    some = list(range(B_)) if B_ < 10 else [0, 1, 2, 77, 150, 298, 299]
    _check_decode(q[some][:, :, heads], latent, table[some], seq[some], scale, 64, out[some][:, :, heads],
                  lse[some][:, :, heads])
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_decode_fewer_tiles_than_sms_with_a_dirty_workspace():
    """47 key tiles, fewer than there are SMs, with a workspace full of large numbers behind its header:
    nothing is joined that the call has not written."""
    q, latent, table, seq, scale = _decode_case([3000 - 129, 0, 129], 1, 16, 64, torch.bfloat16, 3)
    ws = torch.full((B.dsa_latent_attention_decode_workspace_bytes(3, 1, 16),), 0x7E, dtype=torch.uint8, device="cuda")
    B.dsa_workspace_init(ws)
    out, lse = B.dsa_latent_attention_decode(q.cuda(), latent.cuda(), table.cuda(), seq.cuda(), scale, workspace=ws)
    _check_decode(q, latent, table, seq, scale, 64, out, lse)


def test_decode_strided_queries_and_no_lse():
    q, latent, table, seq, scale = _decode_case([100, 257], 2, 6, 64, torch.bfloat16, 5)
    wide = torch.full((4, 9, 600), float("nan"), dtype=torch.bfloat16)
    wide[:, 2:8, 16:592] = q.reshape(4, 6, LATENT)
    out, lse = B.dsa_latent_attention_decode(wide.cuda()[:, 2:8, 16:592].view(2, 2, 6, LATENT), latent.cuda(),
                                             table.cuda(), seq.cuda(), scale, want_lse=False)
    assert lse is None
    _check_decode(q, latent, table, seq, scale, 64, out, None)
    one, _ = B.dsa_latent_attention_decode(q[:, 1].cuda(), latent.cuda(), table.cuda(), seq.cuda(), scale)
    assert one.shape == (2, 6, LV)
    assert (one.float() - out[:, 1].float()).abs().max() <= 2.0 ** -7 * out.float().abs().max()


def test_decode_large_scores_and_equal_scores():
    """Scores far apart (a one-hot softmax, exponents past the type's range) and all equal."""
    q, latent, table, seq, _ = _decode_case([300, 65], 1, 16, 64, torch.bfloat16, 6)
    for scale in (30.0, 1e-6):
        out, lse = B.dsa_latent_attention_decode(q.cuda(), latent.cuda(), table.cuda(), seq.cuda(), scale)
        if scale == 30.0:
            # gaps between scores are large against ds: the argmax row comes out
            ref, ref_lse, _ = O.latent_decode(_num(q), _num(latent), table.numpy(), seq.numpy(), scale, 64)
            assert np.abs(_num(out) - ref).max() <= 0.02 * np.abs(ref).max()
            assert (np.abs(_num(lse) - ref_lse) <= np.abs(ref_lse) * 2.0 ** -12).all()
        else:
            _check_decode(q, latent, table, seq, scale, 64, out, lse)


def test_decode_device_side_checks():
    q, latent, table, seq, scale = _decode_case([130, 70], 1, 8, 64, torch.bfloat16, 8)
    latent = torch.nan_to_num(latent, nan=0.0, posinf=0.0)
    ws = torch.zeros(B.dsa_latent_attention_decode_workspace_bytes(2, 1, 8), dtype=torch.uint8, device="cuda")
    bad = table.clone()
    bad[1, 0] = 10_000
    out, _ = B.dsa_latent_attention_decode(q.cuda(), latent.cuda(), bad.cuda(), seq.cuda(), scale, workspace=ws)
    assert B.dsa_read_device_status(ws) == (B.DSA_ERR_DEVICE, 16)
    bad[1, 0] = 0
    _check_decode(q, latent, bad, seq, scale, 64, out, None)
    for n, used in ((-5, 0), (10_000, 192)):
        wrong = torch.tensor([130, n], dtype=torch.int32)
        full = table.clamp_min(0)
        out, lse = B.dsa_latent_attention_decode(q.cuda(), latent.cuda(), full.cuda(), wrong.cuda(), scale, workspace=ws)
        assert B.dsa_read_device_status(ws) == (B.DSA_ERR_DEVICE, 17)
        wrong[1] = used
        _check_decode(q, latent, full, wrong, scale, 64, out, lse)


def test_decode_agrees_with_sparse_attention_over_everything():
    """A context no longer than top-k: the dense form equals dsa_sparse_attention_decode over all its
    positions (both within the bf16 rounding of their numerators and, here, of the output)."""
    x = latent_decode_inputs([256, 100, 7], 256, seed=2)
    scale = 0.05
    sparse = B.dsa_sparse_attention_decode(x.q.cuda(), x.latent.cuda(), x.block_table.cuda(), x.seq_lens.cuda(),
                                           x.idx.cuda(), scale)
    dense, _ = B.dsa_latent_attention_decode(x.q.cuda(), x.latent.cuda(), x.block_table.cuda(), x.seq_lens.cuda(), scale)
    assert (sparse - dense.float()).abs().max() <= 4 * 2.0 ** -8 * float(x.latent.float().abs().max())


def test_decode_repeats_bit_for_bit_on_streams_and_in_graphs():
    q, latent, table, seq, scale = _decode_case([700, 3, 1500], 1, 64, 64, torch.bfloat16, 11)
    q, latent, table, seq = q.cuda(), latent.cuda(), table.cuda(), seq.cuda()
    want, lse = B.dsa_latent_attention_decode(q, latent, table, seq, scale)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    two, lse2 = B.dsa_latent_attention_decode(q, latent, table, seq, scale, stream=side)
    side.synchronize()
    assert torch.equal(two, want) and torch.equal(lse2, lse)
    ws = torch.zeros(B.dsa_latent_attention_decode_workspace_bytes(3, 1, 64), dtype=torch.uint8, device="cuda")
    qin = torch.zeros_like(q)
    lens = torch.zeros_like(seq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        three, lse3 = B.dsa_latent_attention_decode(qin, latent, table, lens, scale, workspace=ws)
    graph.replay()                                   # empty requests
    torch.cuda.synchronize()
    assert not three.any() and torch.isneginf(lse3).all()
    qin.copy_(q)
    lens.copy_(seq)                                  # longer ones than were captured
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(three, want) and torch.equal(lse3, lse)


def _prefill_case(nq, nk, H, dtype, seed, extra=3):
    """Ragged requests with `extra` rows before the first and after the last that belong to none (NaN)."""
    g = torch.Generator().manual_seed(seed)
    Tq, Tk = sum(nq) + 2 * extra, sum(nk) + 2 * extra
    q = torch.randn(Tq, H, NOPE + PE, generator=g).to(dtype)
    kv = torch.randn(Tk, H, NOPE + DV, generator=g).to(dtype)
    pe = torch.randn(Tk, PE, generator=g).to(dtype)
    for t, n in ((kv, sum(nk)), (pe, sum(nk))):
        t[:extra] = float("nan")
        t[extra + n:] = float("nan")
    cu_q = torch.tensor([extra] + nq).cumsum(0).to(torch.int32)
    cu_k = torch.tensor([extra] + nk).cumsum(0).to(torch.int32)
    return q, kv, pe, cu_q, cu_k


def _check_prefill(q, kv, pe, cu_q, cu_k, scale, causal, out, lse, rows=None):
    nq, nkv, npe = _num(q), _num(kv), _num(pe)
    ref, ref_lse, mag = O.latent_prefill(nq, nkv[..., :NOPE], npe, nkv[..., NOPE:], cu_q.numpy(), cu_k.numpy(), scale,
                                         causal)
    inside = ~np.isnan(ref_lse)[:, 0]
    top = max(np.nan_to_num(np.abs(nkv)).max(), np.nan_to_num(np.abs(npe)).max())
    ds = scale * np.abs(nq).sum(-1) * top * 0.5 * (192 / 16 + 2) * 2.0 ** -23
    n = int((cu_k[1:] - cu_k[:-1]).max()) if len(cu_k) > 1 else 1
    _close(out[torch.from_numpy(inside)], lse[torch.from_numpy(inside)] if lse is not None else None, ref[inside],
           ref_lse[inside], mag[inside], ds[inside], q.dtype, n, top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nq,nk,H,causal", [
    ([1], [1], 1, True), ([128], [128], 2, True), ([129, 1, 255], [129, 1, 255], 2, True),
    ([3, 100], [200, 100], 3, True), ([256], [700], 1, True), ([300], [300], 1, True), ([5, 40], [0, 17], 2, True),
    ([0, 7, 0], [0, 7, 3], 2, True), ([130, 20], [300, 1], 2, False), ([64], [0], 1, False), ([600], [611], 1, True)])
def test_prefill_matches_oracle(dtype, nq, nk, H, causal):
    q, kv, pe, cu_q, cu_k = _prefill_case(nq, nk, H, dtype, sum(nq) + H)
    scale = 2.0 / math.sqrt(192.0)
    kvd = kv.cuda()
    out = torch.full((q.shape[0], H, DV), 77.0, dtype=dtype, device="cuda")
    lse = torch.full((q.shape[0], H), 77.0, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.dsa_latent_attention_prefill(q.cuda(), kvd[..., :NOPE], pe.cuda(), kvd[..., NOPE:], cu_q.cuda(), cu_k.cuda(),
                                   max(nq), scale, causal=causal, out=out, lse=lse, workspace=ws)
    assert B.dsa_read_device_status(ws) == (0, 0)
    _check_prefill(q, kv, pe, cu_q, cu_k, scale, causal, out, lse)
    outside = torch.ones(q.shape[0], dtype=torch.bool)
    outside[3:3 + sum(nq)] = False
    assert (out.cpu()[outside] == 77).all() and (lse.cpu()[outside] == 77).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nq,nk,H,causal", [
    ([1], [4000], 1, True), ([900], [900], 1, True), ([300, 0, 5], [2500, 90, 1000], 3, True),
    ([130], [1037], 2, False), ([700], [500], 1, True), ([257, 256], [700, 3000], 2, True), ([64], [9000], 1, True)])
def test_prefill_of_few_queries_splits_the_keys(dtype, nq, nk, H, causal):
    q, kv, pe, cu_q, cu_k = _prefill_case(nq, nk, H, dtype, sum(nq) + H + 1)
    need = B.dsa_latent_attention_prefill_workspace_bytes(len(nq), q.shape[0], pe.shape[0], max(nq), H, causal)
    assert need > 256
    scale, kvd = 2.0 / math.sqrt(192.0), kv.cuda()
    out = torch.full((q.shape[0], H, DV), 77.0, dtype=dtype, device="cuda")
    lse = torch.full((q.shape[0], H), 77.0, device="cuda")
    ws = torch.full((need,), 0x7F, dtype=torch.uint8, device="cuda")     # partial sums of 0x7F7F7F7F, but
    ws[:256] = 0                                                        # for the header
    args = (q.cuda(), kvd[..., :NOPE], pe.cuda(), kvd[..., NOPE:], cu_q.cuda(), cu_k.cuda(), max(nq), scale)
    B.dsa_latent_attention_prefill(*args, causal=causal, out=out, lse=lse, workspace=ws)
    assert B.dsa_read_device_status(ws) == (0, 0)
    _check_prefill(q, kv, pe, cu_q, cu_k, scale, causal, out, lse)
    outside = torch.ones(q.shape[0], dtype=torch.bool)
    outside[3:3 + sum(nq)] = False
    assert (out.cpu()[outside] == 77).all() and (lse.cpu()[outside] == 77).all()
    again, lse2 = B.dsa_latent_attention_prefill(*args, causal=causal)
    assert torch.equal(again[3:3 + sum(nq)], out[3:3 + sum(nq)]) and torch.equal(lse2[3:3 + sum(nq)], lse[3:3 + sum(nq)])


def test_a_visible_nan_stays_one():
    """A query that meets a NaN or infinite score gets NaN, not zeros; the others of the call are unharmed."""
    q, kv, pe, cu_q, cu_k = _prefill_case([600], [600], 1, torch.bfloat16, 3, extra=0)
    q[7, 0, 5] = float("nan")
    q[300, 0, 150] = float("inf")
    for ws in (torch.zeros(256, dtype=torch.uint8, device="cuda"), None):
        out, lse = B.dsa_latent_attention_prefill(q.cuda(), kv.cuda()[..., :NOPE], pe.cuda(), kv.cuda()[..., NOPE:],
                                                  cu_q.cuda(), cu_k.cuda(), 600, 0.1, workspace=ws)
        bad = out.isnan().all(-1).flatten().cpu()
        assert bad.nonzero().flatten().tolist() == [7, 300] and not out[~bad].isnan().any()
        assert torch.equal(lse.isnan().flatten().cpu(), bad)
    qd, latent, table, seq, scale = _decode_case([700, 3], 1, 20, 64, torch.bfloat16, 11)
    qd[0, 0, 4, 570], qd[1, 0, 19, 0] = float("nan"), float("nan")
    out, lse = B.dsa_latent_attention_decode(qd.cuda(), latent.cuda(), table.cuda(), seq.cuda(), scale)
    bad = out.isnan().all(-1).cpu()
    assert bad.nonzero().tolist() == [[0, 0, 4], [1, 0, 19]] and not out.cpu()[~bad].isnan().any()
    assert torch.equal(lse.isnan().cpu(), bad)


def test_prefill_longer_rising_scores():
    """1500 tokens whose keys grow, so that the running maximum moves many times."""
    q, kv, pe, cu_q, cu_k = _prefill_case([1500], [1500], 2, torch.bfloat16, 4)
    grow = (0.05 + 1.5 * torch.arange(1506) / 1506)[:, None]
    kv[..., :NOPE] = (kv[..., :NOPE].float() * grow[:, None]).to(torch.bfloat16)
    pe = (pe.float() * grow).to(torch.bfloat16)
    kvd = kv.cuda()
    out, lse = B.dsa_latent_attention_prefill(q.cuda(), kvd[..., :NOPE], pe.cuda(), kvd[..., NOPE:], cu_q.cuda(),
                                              cu_k.cuda(), 1500, 0.2)
    _check_prefill(q, kv, pe, cu_q, cu_k, 0.2, True, out, lse)


def test_prefill_chunks_equal_the_whole_and_join():
    """The last 300 of 900 tokens as a chunk of their own equal their rows of the whole call bit for bit
    up to the tiling (within the bound), and two parts of the keys joined by lse equal the whole."""
    q, kv, pe, cu_q, cu_k = _prefill_case([900], [900], 2, torch.bfloat16, 6, extra=0)
    qd, kvd, ped = q.cuda(), kv.cuda(), pe.cuda()
    whole, lse = B.dsa_latent_attention_prefill(qd, kvd[..., :NOPE], ped, kvd[..., NOPE:], cu_q.cuda(), cu_k.cuda(),
                                                900, 0.1)
    cq = torch.tensor([0, 300], dtype=torch.int32).cuda()
    part, plse = B.dsa_latent_attention_prefill(qd[600:], kvd[..., :NOPE], ped, kvd[..., NOPE:], cq, cu_k.cuda(), 300, 0.1)
    tol = 4 * 2.0 ** -8 * float(kv[..., NOPE:].float().abs().max())
    assert (part.float() - whole[600:].float()).abs().max() <= tol and (plse - lse[600:]).abs().max() <= 1e-4
    a, la = B.dsa_latent_attention_prefill(qd[600:], kvd[:600, :, :NOPE], ped[:600], kvd[:600, :, NOPE:], cq,
                                           torch.tensor([0, 600], dtype=torch.int32).cuda(), 300, 0.1, causal=False)
    b, lb = B.dsa_latent_attention_prefill(qd[600:], kvd[600:, :, :NOPE], ped[600:], kvd[600:, :, NOPE:], cq, cq, 300, 0.1)
    both = torch.logaddexp(la, lb)
    o = a.float() * torch.exp(la - both)[..., None] + b.float() * torch.exp(lb - both)[..., None]
    assert (o - part.float()).abs().max() <= tol and (both - plse).abs().max() <= 1e-4


def test_prefill_device_side_checks():
    q, kv, pe, cu_q, cu_k = _prefill_case([10, 20], [10, 20], 1, torch.bfloat16, 6, extra=0)
    kvd = kv.cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def call(cq, ck, max_q):
        out = torch.full((30, 1, DV), 77.0, dtype=torch.bfloat16, device="cuda")
        B.dsa_latent_attention_prefill(q.cuda(), kvd[..., :NOPE], pe.cuda(), kvd[..., NOPE:],
                                       torch.tensor(cq, dtype=torch.int32).cuda(),
                                       torch.tensor(ck, dtype=torch.int32).cuda(), max_q, 0.1, out=out, workspace=ws)
        return out.cpu(), B.dsa_read_device_status(ws)

    good, status = call([0, 10, 30], [0, 10, 30], 20)
    assert status == (0, 0)
    for cq, ck, max_q in (([0, 10, 31], [0, 10, 30], 21), ([0, 10, 30], [0, 10, 31], 20), ([0, 10, 30], [0, 10, 5], 20),
                          ([0, 10, 30], [0, 10, 30], 15)):
        out, status = call(cq, ck, max_q)
        assert status == (B.DSA_ERR_DEVICE, 17)
        assert torch.equal(out[:10], good[:10]) and (out[10:] == 77).all()   # request 1 is left out
    out, status = call([-1, 10, 30], [0, 10, 30], 20)
    assert status == (B.DSA_ERR_DEVICE, 17) and (out[:10] == 77).all() and torch.equal(out[10:], good[10:])


def test_prefill_streams_graphs_and_shapes():
    q, kv, pe, cu_q, cu_k = _prefill_case([200, 31], [260, 31], 3, torch.bfloat16, 9, extra=0)
    q, kv, pe, cu_q, cu_k = q.cuda(), kv.cuda(), pe.cuda(), cu_q.cuda(), cu_k.cuda()
    args = (kv[..., :NOPE], pe, kv[..., NOPE:], cu_q, cu_k, 200, 0.1)
    want, lse = B.dsa_latent_attention_prefill(q, *args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    two, _ = B.dsa_latent_attention_prefill(q, *args, stream=side)
    side.synchronize()
    assert torch.equal(two, want)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    qin = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        three, lse3 = B.dsa_latent_attention_prefill(qin, *args, workspace=ws)
    qin.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(three, want) and torch.equal(lse3, lse)
    with pytest.raises(ValueError):
        B.dsa_latent_attention_prefill(q, kv[..., :64], pe, kv[..., NOPE:], cu_q, cu_k, 200, 0.1)
    with pytest.raises(ValueError):
        B.dsa_latent_attention_prefill(q, kv[..., :NOPE].half(), pe, kv[..., NOPE:], cu_q, cu_k, 200, 0.1)
    none, none_lse = B.dsa_latent_attention_prefill(q[:0], *args[:5], 0, 0.1)
    assert none.shape == (0, 3, DV) and none_lse.shape == (0, 3)

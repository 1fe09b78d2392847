"""Latent attention where a call meets its edges: replayed on other sizes than it was captured with, with a
consumer right behind it, under load (GPU). Tolerances are those of test_gpu_latent_attention.py, derived
there; results of the same arithmetic are compared bit for bit."""

import math
import random

import pytest
import torch

from sparse_attention_token_04_b200 import binding as B

pytestmark = pytest.mark.gpu

NOPE, PE, DV = 128, 64, 128


def test_consumer_behind_a_planned_split_that_joins_nothing():
    """A key buffer sized for a long context has the call planned as a split one, and the request in it is so
    short that every block is one part: a consumer captured behind the call reads finished results, on every
    replay. (The one part of 90 key tiles runs long after a join without work could end.)"""
    g = torch.Generator().manual_seed(1)
    Tq, Tk, nk, H = 200, 400_000, 90 * 128 - 5, 1
    kv = torch.zeros(Tk, H, NOPE + DV, dtype=torch.bfloat16, device="cuda")
    pe = torch.zeros(Tk, PE, dtype=torch.bfloat16, device="cuda")
    kv[:nk] = torch.randn(nk, H, NOPE + DV, generator=g).to(torch.bfloat16).cuda()
    pe[:nk] = torch.randn(nk, PE, generator=g).to(torch.bfloat16).cuda()
    queries = torch.randn(6, Tq, H, NOPE + PE, generator=g).to(torch.bfloat16).cuda()
    cu_q, cu_k = (torch.tensor(v, dtype=torch.int32).cuda() for v in ([0, Tq], [0, nk]))
    args = (kv[..., :NOPE], pe, kv[..., NOPE:], cu_q, cu_k, Tq, 1.0 / math.sqrt(NOPE + PE))
    need = B.dsa_latent_attention_prefill_workspace_bytes(1, Tq, Tk, Tq, H)
    assert need > B.DSA_WS_HEADER_BYTES
    whole = torch.zeros(B.DSA_WS_HEADER_BYTES, dtype=torch.uint8, device="cuda")   # no room for a split
    want = [B.dsa_latent_attention_prefill(q, *args, workspace=whole) for q in queries]
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    q = torch.zeros_like(queries[0])
    out = torch.empty(Tq, H, DV, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(Tq, H, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.dsa_latent_attention_prefill(q, *args, out=out, lse=lse, workspace=ws)
        seen, seen_lse = out.clone(), lse.clone()
    for x, (o, l) in zip(queries, want):
        q.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(seen, o) and torch.equal(seen_lse, l)
    assert B.dsa_read_device_status(ws) == (0, 0)
    # and the same request in a buffer of its own size, which splits it and joins the parts, within the
    # rounding of the other order of sums
    part, _ = B.dsa_latent_attention_prefill(queries[0], kv[:nk, :, :NOPE], pe[:nk], kv[:nk, :, NOPE:], *args[3:])
    assert (part.float() - want[0][0].float()).abs().max() <= 4 * 2.0 ** -8 * float(kv.float().abs().max())


@pytest.mark.parametrize("Hq,q_len,dtype", [(128, 1, torch.bfloat16), (16, 2, torch.float16), (20, 1, torch.bfloat16)])
def test_decode_under_load_repeats_bit_for_bit(Hq, q_len, dtype):
    """Calls beside copies that keep the memory busy, so that some of the kernel's waits are short and others
    long: many requests of many lengths, the same bits every time."""
    g = torch.Generator().manual_seed(Hq)
    lens = [int(x) for x in torch.randint(1, 2500, (40,), generator=g)]
    blocks = [(n + 63) // 64 for n in lens]
    table = torch.zeros(len(lens), max(blocks), dtype=torch.int32)
    perm = torch.randperm(sum(blocks), generator=g).to(torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    latent = torch.randn(sum(blocks) * 64, 576, generator=g).to(dtype).cuda()
    q = torch.randn(len(lens), q_len, Hq, 576, generator=g).to(dtype).cuda()
    args = (q, latent, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.08)
    ws = torch.zeros(B.dsa_latent_attention_decode_workspace_bytes(len(lens), q_len, Hq), dtype=torch.uint8, device="cuda")
    want, want_lse = B.dsa_latent_attention_decode(*args, workspace=ws)
    src = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    dst = torch.empty_like(src)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(40):
            dst.copy_(src)
    outs = [B.dsa_latent_attention_decode(*args, workspace=ws) for _ in range(30)]
    torch.cuda.synchronize()
    for out, lse in outs:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert B.dsa_read_device_status(ws) == (0, 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,q_len,Hq,block_size", [([70, 130], 3, 8, 64), ([33, 5, 100], 8, 5, 64), ([4000, 9], 4, 16, 64),
                                                      ([64, 2, 40], 3, 40, 8), ([2000], 2, 128, 64)])
def test_decode_latents_of_new_tokens_that_are_not_finite(dtype, lens, q_len, Hq, block_size):
    """A new token whose latent is not finite harms the tokens that see it; the ones in front of it, and the
    other requests, get the bits that they get with a finite one in its place (their weight on it is 0)."""
    g = torch.Generator().manual_seed(sum(lens))
    blocks = [(n + block_size - 1) // block_size for n in lens]
    table = torch.zeros(len(lens), max(blocks), dtype=torch.int32)
    for b, n in enumerate(blocks):
        table[b, :n] = torch.arange(sum(blocks[:b]), sum(blocks[:b]) + n)
    latent = torch.randn(sum(blocks) * block_size, 576, generator=g).to(dtype)
    q = torch.randn(len(lens), q_len, Hq, 576, generator=g).to(dtype).cuda()
    rest = (table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.08)
    clean, clean_lse = B.dsa_latent_attention_decode(q, latent.cuda(), *rest, block_size=block_size)
    row = lambda pos: int(table[0, pos // block_size]) * block_size + pos % block_size
    for first in range(1, q_len):                   # the first of request 0's new tokens that is not finite
        bad = latent.clone()
        for i in range(first, q_len):
            bad[row(lens[0] - q_len + i), [0, 77, 300, 511, 575]] = torch.tensor(
                [float("nan"), float("inf"), -float("inf"), float("nan"), float("inf")], dtype=dtype)
        out, lse = B.dsa_latent_attention_decode(q, bad.cuda(), *rest, block_size=block_size)
        assert torch.equal(out[0, :first], clean[0, :first]) and torch.equal(lse[0, :first], clean_lse[0, :first])
        assert out[0, first:].isnan().all() and lse[0, first:].isnan().all()
        assert torch.equal(out[1:], clean[1:]) and torch.equal(lse[1:], clean_lse[1:])
    # one that is not finite among the values only: NaN scores for those who see it all the same
    bad = latent.clone()
    bad[row(lens[0] - 1), 200] = float("nan")
    out, _ = B.dsa_latent_attention_decode(q, bad.cuda(), *rest, block_size=block_size)
    assert torch.equal(out[0, :-1], clean[0, :-1]) and out[0, -1].isnan().all()


def test_decode_random_calls():
    """Calls of random shapes one after another: few and many requests of very uneven lengths, drafted tokens
    over tile borders, pages of all sizes, so that the kernel's warps meet in ever new orders."""
    from test_gpu_latent_attention import _check_decode, _decode_case

    rng = random.Random(7)
    for n in range(120):
        size = lambda: max(0, int(round(math.exp(rng.uniform(0, math.log(700))))) - rng.choice([0, 0, 1]))
        lens = [size() for _ in range(rng.choice([1, 2, 3, 7, 33]))]
        q_len, Hq, block = rng.randint(1, 8), rng.choice([1, 3, 8, 16, 17, 32, 40, 64, 100, 128]), rng.choice([8, 16, 24, 40, 64, 128])
        q, latent, table, seq, scale = _decode_case(lens, q_len, Hq, block, rng.choice([torch.bfloat16, torch.float16]), n)
        ws = torch.zeros(B.dsa_latent_attention_decode_workspace_bytes(len(lens), q_len, Hq), dtype=torch.uint8, device="cuda")
        out, lse = B.dsa_latent_attention_decode(q.cuda(), latent.cuda(), table.cuda(), seq.cuda(), scale,
                                                 block_size=block, workspace=ws)
        assert B.dsa_read_device_status(ws) == (0, 0), (lens, q_len, Hq, block)
        heads, some = sorted({0, Hq // 2, Hq - 1}), sorted(rng.sample(range(len(lens)), min(3, len(lens))))
        _check_decode(q[some][:, :, heads], latent, table[some], seq[some], scale, block, out[some][:, :, heads],
                      lse[some][:, :, heads])

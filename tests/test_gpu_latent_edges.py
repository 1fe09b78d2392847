"""Latent attention where a call meets its edges: replayed on other sizes than it was captured with, with a
consumer right behind it, under load (GPU). Tolerances are those of test_gpu_latent_attention.py, derived
there; results of the same arithmetic are compared bit for bit."""

import math

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

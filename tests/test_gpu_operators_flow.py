"""The operators around the indexer run together as one attention layer would (GPU): rotary positions,
index queries and keys quantised, keys into and out of the paged cache, the indexer over both, latent
attention of the prompt in its expanded form and of the next token in its absorbed form, dense and over
the indexer's selection. Every stage is held to fp64 on that stage's own inputs; the tolerances of the
attention stages are those of test_gpu_latent_attention.py, derived there."""

import math

import numpy as np
import pytest
import torch

import oracle.operators_oracle as O
from sparse_attention_token_04_b200 import binding as B

from test_gpu_latent_attention import (LATENT, LV, NOPE, PE, _check_decode, _check_prefill, _decode_case,
                                       _prefill_case)

pytestmark = pytest.mark.gpu

H, HI, D, BLOCK, TOPK = 128, 64, 128, 64, 256
N = [150, 70]                                     # prompt tokens of two requests, whose last is the "next" token


class Layer:
    """Inputs and buffers of one layer for two prompts of N tokens in shuffled pages."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)

        def rand(*shape, dtype=torch.bfloat16):
            return torch.randn(*shape, generator=g).to(dtype).cuda()

        T = self.T = sum(N)
        self.q = rand(T, H, NOPE + PE)
        self.rows = rand(T, LATENT)               # the tokens' latents: 512 compressed dims | 64 rotary ones
        self.qi, self.ki, self.w = rand(T, HI, D), rand(T, D), rand(T, HI, dtype=torch.float32)
        self.pos = torch.cat([torch.arange(n) for n in N]).to(torch.int32).cuda()
        self.cu = torch.tensor([0] + N).cumsum(0).to(torch.int32).cuda()
        self.freq, self.mscale = B.dsa_rotary_frequencies(PE, device="cuda")
        self.ifreq, _ = B.dsa_rotary_frequencies(32, device="cuda")
        nb = [(n + BLOCK - 1) // BLOCK for n in N]
        table = torch.full((2, max(nb)), -1, dtype=torch.int32)
        perm = torch.randperm(sum(nb), generator=g).to(torch.int32)
        table[0, :nb[0]], table[1, :nb[1]] = perm[:nb[0]], perm[nb[0]:]
        self.table = table.cuda()
        slots = [int(table[b, p // BLOCK]) * BLOCK + p % BLOCK for b in range(2) for p in range(N[b])]
        self.slots = torch.tensor(slots, dtype=torch.int64).cuda()
        self.k_cache = torch.zeros(sum(nb), BLOCK, D, dtype=torch.uint8, device="cuda")
        self.k_scale = torch.zeros(sum(nb), BLOCK, device="cuda")
        self.latent = torch.zeros(sum(nb) * BLOCK, LATENT, dtype=torch.bfloat16, device="cuda")
        self.lens = torch.tensor(N, dtype=torch.int32).cuda()
        self.last = (self.cu[1:] - 1).long()

    def run(self, scale):
        """Everything on the current stream; the heads' up-projections pick 128 of the 512 dims (head h
        those from 3 h on), which makes the expanded and the absorbed form the same sums."""
        r = {}
        r["q"] = torch.cat((self.q[..., :NOPE], B.dsa_rotary(self.q[..., NOPE:], self.pos, self.freq, interleaved=True)), -1)
        kpe = B.dsa_rotary(self.rows[:, None, LV:], self.pos, self.freq, interleaved=True)[:, 0]
        r["lat"] = torch.cat((self.rows[:, :LV], kpe), -1)
        self.latent.index_copy_(0, self.slots, r["lat"])
        r["qc"], r["qs"] = B.dsa_index_quantise(self.qi, self.pos, self.ifreq)
        B.dsa_index_cache_write(self.ki, self.slots, self.k_cache, self.k_scale, self.pos, self.ifreq)
        r["kc"], r["ks"], _ = B.dsa_index_cache_read(self.k_cache, self.k_scale, self.table, self.cu, self.T)
        r["sel"] = [B.dsa_indexer_prefill(r["qc"][a:e], r["qs"][a:e], self.w[a:e], r["kc"][a:e], r["ks"][a:e], TOPK)
                    for a, e in ((0, N[0]), (N[0], self.T))]
        ql = [t[self.last].contiguous() for t in (r["qc"], r["qs"], self.w)]
        r["idx"], r["score"] = B.dsa_indexer_decode(*ql, self.k_cache, self.k_scale, self.table, self.lens, TOPK)
        cols = (torch.arange(H, device="cuda")[:, None] * 3 + torch.arange(NOPE, device="cuda")).flatten()
        up = r["lat"][:, cols].view(self.T, H, NOPE)
        r["kv"] = torch.cat((up, up), -1)
        r["out"], r["lse"] = B.dsa_latent_attention_prefill(r["q"], r["kv"][..., :NOPE], r["lat"][:, LV:],
                                                            r["kv"][..., NOPE:], self.cu, self.cu, max(N), scale)
        r["qa"] = torch.zeros(2, H, LATENT, dtype=torch.bfloat16, device="cuda")
        r["qa"].scatter_(2, cols.view(1, H, NOPE).expand(2, -1, -1), r["q"][self.last][..., :NOPE])
        r["qa"][..., LV:] = r["q"][self.last][..., NOPE:]
        r["dense"], r["dlse"] = B.dsa_latent_attention_decode(r["qa"], self.latent, self.table, self.lens, scale)
        r["sparse"] = B.dsa_sparse_attention_decode(r["qa"], self.latent, self.table, self.lens, r["idx"], scale)
        r["head"] = r["dense"].gather(2, cols.view(1, H, NOPE).expand(2, -1, -1))   # the value up-projection
        return r


def test_one_layer():
    x, scale = Layer(5), 1.0 / math.sqrt(NOPE + PE)
    r = x.run(scale)
    num = lambda t: t.detach().cpu().double().numpy()
    pos, freq, ifreq = x.pos.cpu().numpy(), x.freq.cpu().numpy(), x.ifreq.cpu().numpy()
    # rotated parts: bf16's half step of the result and the angle's share of the pair
    for got, src in ((r["q"][..., NOPE:], x.q[..., NOPE:]), (r["lat"][:, None, LV:], x.rows[:, None, LV:])):
        ref = O.rotary(num(src), pos, freq, True)
        assert (np.abs(num(got) - ref) <= np.abs(ref) * 2.0 ** -8 * 1.001 + np.abs(num(src)).max() * 2.0 ** -19).all()
    # the cache holds what quantising the keys gives, and reads back the same rows
    kc, ks = B.dsa_index_quantise(x.ki, x.pos, x.ifreq)
    assert torch.equal(r["kc"], kc) and torch.equal(r["ks"], ks)
    # index scores of the last tokens, from the codes; every visible position is selected
    dec = lambda c: num(c.view(torch.float8_e4m3fn).float())
    for b, (a, e) in enumerate(((0, N[0]), (N[0], x.T))):
        k = dec(r["kc"][a:e]) * num(r["ks"][a:e])[:, None]
        q = dec(r["qc"][e - 1]) * num(r["qs"][e - 1])
        want = (np.maximum(q @ k.T, 0) * num(x.w[e - 1])[:, None]).sum(0)
        idx, score = r["idx"][b].cpu().numpy(), num(r["score"][b])
        assert sorted(idx[:N[b]].tolist()) == list(range(N[b])) and (idx[N[b]:] == -1).all()
        assert (np.abs(score[:N[b]] - want[idx[:N[b]]]) <= 1e-5 * np.abs(want).max()).all()
        rows, _ = r["sel"][b]
        assert sorted(rows[-1, :N[b]].tolist()) == list(range(N[b])) and (rows[-1, N[b]:] == -1).all()
    # attention: heads 0, 77 and 127 of each form against fp64, and the forms against each other
    some = [0, 77, 127]
    _check_prefill(r["q"][:, some], r["kv"][:, some], r["lat"][:, LV:], x.cu.cpu(), x.cu.cpu(), scale, True,
                   r["out"][:, some].cpu(), r["lse"][:, some].cpu())
    _check_decode(r["qa"][:, None, some], x.latent.cpu(), x.table.cpu(), x.lens.cpu(), scale, BLOCK,
                  r["dense"][:, None, some], r["dlse"][:, None, some])
    tol = 4 * 2.0 ** -8 * float(r["lat"].float().abs().max())
    assert (r["sparse"] - r["dense"].float()).abs().max() <= tol
    assert (r["head"].float() - r["out"][x.last].float()).abs().max() <= tol


def test_one_layer_captured_and_replayed():
    """The calls from the rotation to the decode's result in one graph (each with its own workspace, as it
    allocates it), replayed on other inputs than it was captured with."""
    scale = 1.0 / math.sqrt(NOPE + PE)
    x, y = Layer(5), Layer(6)
    want = y.run(scale)
    x.run(scale)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = x.run(scale)
    for name in ("q", "rows", "qi", "ki", "w", "table", "slots"):
        getattr(x, name).copy_(getattr(y, name))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for name in ("kc", "ks", "qc", "qs", "idx", "out", "lse", "dense", "dlse"):
        assert torch.equal(got[name], want[name]), name


def test_two_calls_at_once():
    """A decode and a prefill on two streams at once give what each gives alone."""
    q, latent, table, seq, scale = _decode_case([2000, 900, 5], 1, 128, 64, torch.bfloat16, 4)
    dec = [t.cuda() for t in (q, latent, table, seq)]
    pq, kv, pe, cu_q, cu_k = (t.cuda() for t in _prefill_case([700, 300], [700, 900], 4, torch.bfloat16, 5, extra=0))
    pre = (pq, kv[..., :NOPE], pe, kv[..., NOPE:], cu_q, cu_k, 700, 0.1)
    a, la = B.dsa_latent_attention_decode(*dec, scale)
    b, lb = B.dsa_latent_attention_prefill(*pre)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(10):
        outs.append(B.dsa_latent_attention_decode(*dec, scale, stream=streams[i & 1]))
        outs.append(B.dsa_latent_attention_prefill(*pre, stream=streams[~i & 1]))
    torch.cuda.synchronize()
    for k, (o, l) in enumerate(outs):
        assert torch.equal(o, b if k & 1 else a) and torch.equal(l, lb if k & 1 else la)


def test_prefill_of_heads_major_tensors():
    """Queries, keys and values whose heads lie outermost, as views."""
    q, kv, pe, cu_q, cu_k = _prefill_case([140, 9], [140, 300], 3, torch.float16, 8)
    major = lambda t: t.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    out, lse = B.dsa_latent_attention_prefill(major(q), major(kv[..., :NOPE]), pe.cuda(), major(kv[..., NOPE:]),
                                              cu_q.cuda(), cu_k.cuda(), 140, 0.1)
    _check_prefill(q, kv, pe, cu_q, cu_k, 0.1, True, out, lse)


def test_very_many_short_requests():
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 3, (3000,), generator=g).tolist()
    lens[0], lens[2999] = 0, 2
    q, latent, table, seq, scale = _decode_case(lens, 1, 3, 8, torch.bfloat16, 9)
    out, lse = B.dsa_latent_attention_decode(q.cuda(), latent.cuda(), table.cuda(), seq.cuda(), scale, block_size=8)
    _check_decode(q, latent, table, seq, scale, 8, out, lse)
    nk = torch.randint(0, 4, (3000,), generator=g).tolist()
    q, kv, pe, cu_q, cu_k = _prefill_case([1] * 3000, nk, 1, torch.bfloat16, 9)
    kvd = kv.cuda()
    out, lse = B.dsa_latent_attention_prefill(q.cuda(), kvd[..., :NOPE], pe.cuda(), kvd[..., NOPE:], cu_q.cuda(),
                                              cu_k.cuda(), 1, 0.1)
    _check_prefill(q, kv, pe, cu_q, cu_k, 0.1, True, out, lse)


def test_the_same_latent_block_in_several_requests():
    """Requests that share a prefix share its pages."""
    q, latent, table, seq, scale = _decode_case([300, 300, 190], 2, 16, 64, torch.bfloat16, 4)
    table[1, :4] = table[0, :4]
    table[2, :2] = table[0, :2]
    out, lse = B.dsa_latent_attention_decode(q.cuda(), latent.cuda(), table.cuda(), seq.cuda(), scale)
    _check_decode(q, latent, table, seq, scale, 64, out, lse)


def test_offsets_past_32_bits():
    """Rows whose offsets, in elements and in bytes, pass 2^31 and 2^32, against the same rows in small
    tensors: the key cache and the latents of long contexts, the index queries of a long prefill, the
    prefill's keys."""
    g = torch.Generator().manual_seed(1)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    # 2^32 + some bytes of key codes; slots at both ends
    blocks = (1 << 32) // (64 * 128) + 4
    cache = torch.empty(blocks, 64, 128, dtype=torch.uint8, device="cuda")
    scale = torch.empty(blocks, 64, device="cuda")
    x = torch.randn(6, 128, generator=g).to(torch.bfloat16).cuda()
    slots = torch.tensor([0, blocks * 64 - 1, blocks * 64 - 64, (1 << 24), (1 << 25) - 1, (1 << 25)]).cuda()
    B.dsa_index_cache_write(x, slots, cache, scale, workspace=ws)
    codes, s = B.dsa_index_quantise(x, workspace=ws)
    assert torch.equal(cache.view(-1, 128)[slots], codes) and torch.equal(scale.flatten()[slots], s)
    table = torch.tensor([[blocks - 1], [1 << 19]], dtype=torch.int32, device="cuda")
    got, gs, _ = B.dsa_index_cache_read(cache, scale, table, torch.tensor([0, 64, 65], dtype=torch.int32).cuda(), 65,
                                        workspace=ws)
    assert torch.equal(got[0], codes[2]) and torch.equal(got[63], codes[1]) and torch.equal(got[64], codes[5])
    assert B.dsa_read_device_status(ws) == (0, 0)
    del cache, scale, got
    # latents past 2^32 bytes
    n = (1 << 32) // (LATENT * 2) // 64 + 3
    latent = torch.empty(n * 64, LATENT, dtype=torch.bfloat16, device="cuda")
    small = torch.randn(128, LATENT, generator=g).to(torch.bfloat16).cuda()
    latent[-64:], latent[:64] = small[:64], small[64:]
    q = torch.randn(1, 1, 16, LATENT, generator=g).to(torch.bfloat16).cuda()
    lens = torch.tensor([100], dtype=torch.int32).cuda()
    far = torch.tensor([[n - 1, 0]], dtype=torch.int32).cuda()
    a = B.dsa_latent_attention_decode(q, latent, far, lens, 0.05)
    b = B.dsa_latent_attention_decode(q, small, torch.tensor([[0, 1]], dtype=torch.int32).cuda(), lens, 0.05)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    del latent
    # queries past 2^32 bytes, the last tokens against a call of their own
    T = (1 << 32) // (64 * 128 * 2) + 5
    x = torch.zeros(T, 64, 128, dtype=torch.bfloat16, device="cuda")
    x[-5:] = torch.randn(5, 64, 128, generator=g).to(torch.bfloat16).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freq, _ = B.dsa_rotary_frequencies(64, device="cuda")
    codes, s = B.dsa_index_quantise(x, pos, freq, workspace=ws)
    c5, s5 = B.dsa_index_quantise(x[-5:], pos[-5:], freq, workspace=ws)
    assert torch.equal(codes[-5:], c5) and torch.equal(s[-5:], s5)
    y5 = B.dsa_rotary(x[-5:], pos[-5:], freq)
    assert torch.equal(B.dsa_rotary(x, pos, freq, out=x)[-5:], y5)
    del x, codes
    # keys and values of a prefill in the last rows of a long tensor
    Tk = (1 << 31) // (16 * 256) + 300
    kv = torch.empty(Tk, 16, 256, dtype=torch.bfloat16, device="cuda")
    pe = torch.empty(Tk, PE, dtype=torch.bfloat16, device="cuda")
    kv[-300:] = torch.randn(300, 16, 256, generator=g).to(torch.bfloat16).cuda()
    pe[-300:] = torch.randn(300, PE, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(40, 16, NOPE + PE, generator=g).to(torch.bfloat16).cuda()
    cu = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    a = B.dsa_latent_attention_prefill(q, kv[..., :NOPE], pe, kv[..., NOPE:], cu(0, 40), cu(Tk - 300, Tk), 40, 0.1,
                                       workspace=ws)
    b = B.dsa_latent_attention_prefill(q, kv[-300:, :, :NOPE], pe[-300:], kv[-300:, :, NOPE:], cu(0, 40), cu(0, 300), 40,
                                       0.1, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_prefill_workspace_of_rows_outside_requests():
    """Rows that belong to no request cost the plan nothing: max_q bounds a request."""
    need = B.dsa_latent_attention_prefill_workspace_bytes
    assert need(1, 2 ** 31 - 1, 5000, 1, 1) == need(1, 1, 5000, 1, 1) > 256
    assert need(1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 1) == 256
    assert need(1, 1, 2 ** 31 - 1, 1, 1) < 2 ** 30

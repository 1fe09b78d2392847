"""The README's lines for a layer, run as they stand for a chunk behind a cached prefix and checked against
the fp64 oracle (GPU). Tolerances are those of the operators' own tests, derived there."""

import math
import os
import re

import numpy as np
import pytest
import torch

import oracle.operators_oracle as O
from sparse_attention_token_04_b200 import binding as B

from test_gpu_latent_attention import LATENT, NOPE, PE, _check_decode, _check_prefill

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _sample() -> str:
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    found = [b for b in blocks if "dsa_rotary(" in b]
    assert len(found) == 1
    return found[0]


def test_the_readmes_layer():
    g = torch.Generator().manual_seed(3)
    past, n, H, block = 100, 70, 3, 64
    total = past + n
    rand = lambda *shape: torch.randn(*shape, generator=g).to(torch.bfloat16)
    num = lambda t: t.detach().cpu().double().numpy()
    q, kv, pe, rows = rand(n, H, NOPE + PE), rand(total, H, 2 * NOPE), rand(total, PE), rand(192, LATENT)
    keys, index_q, qa = rand(total, 128), rand(n, 64, 128), rand(1, H, LATENT)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    place = torch.tensor([int(table[0, p // block]) * block + p % block for p in range(total)]).cuda()
    freq, _ = B.dsa_rotary_frequencies(PE, device="cuda")
    cache, scales = torch.zeros(3, block, 128, dtype=torch.uint8, device="cuda"), torch.zeros(3, block, device="cuda")
    old = torch.arange(past, dtype=torch.int32, device="cuda")
    B.dsa_index_cache_write(keys[:past].cuda(), place[:past], cache, scales, old, freq)
    k_pe = pe.cuda()
    k_pe[:past] = B.dsa_rotary(k_pe[:past, None], old, freq, interleaved=True)[:, 0]
    dev = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    kvd = kv.cuda()
    names = dict(q=q.cuda(), k_pe=k_pe, k_nope=kvd[..., :NOPE], v=kvd[..., NOPE:], past=past,
                 pos=torch.arange(past, total, dtype=torch.int32, device="cuda"), index_q=index_q.cuda(),
                 index_k=keys[past:].cuda(), slots=place[past:], k_cache=cache, k_scale=scales, block_table=table.cuda(),
                 cu_q=dev(0, n), cu_k=dev(0, total), total=total, max_q=n, scale=1.0 / math.sqrt(NOPE + PE),
                 w=torch.randn(n, 64, generator=g).cuda(), q_absorbed=qa.cuda(), latent=rows.cuda(), seq_lens=dev(total))
    exec(_sample(), names)
    # the rotations happened, in place
    pos, f = np.arange(total), num(freq)
    for got, src, at in ((names["q"][..., NOPE:], q[..., NOPE:], pos[past:]), (k_pe[:, None], pe[:, None], pos)):
        ref = O.rotary(num(src), at, f, True)
        assert (np.abs(num(got) - ref) <= np.abs(ref) * 2.0 ** -8 * 1.001 + np.abs(num(src)).max() * 2.0 ** -19).all()
    assert torch.equal(names["q"][..., :NOPE].cpu(), q[..., :NOPE])
    # the cache holds every token's key, and each query selects all that it sees
    codes, s = B.dsa_index_quantise(keys.cuda(), torch.arange(total, dtype=torch.int32, device="cuda"), freq)
    assert torch.equal(names["k"], codes) and torch.equal(names["k_s"], s)
    for i, row in enumerate(names["idx"].tolist()):
        assert sorted(row[:past + i + 1]) == list(range(past + i + 1)) and set(row[past + i + 1:]) == {-1}
    _check_prefill(names["q"].cpu(), kv, k_pe.cpu(), names["cu_q"].cpu(), names["cu_k"].cpu(), names["scale"], True,
                   names["out"].cpu(), names["lse"].cpu())
    _check_decode(qa[:, None], rows, table, names["seq_lens"].cpu(), names["scale"], block, names["out_1"][:, None],
                  names["lse_1"][:, None])

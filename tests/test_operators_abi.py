"""Host-side refusals of the operators around the indexer, and the rotary frequencies (no GPU)."""

import ctypes
import math
import os

import pytest
import torch

from sparse_attention_token_04_b200 import binding as B
from sparse_attention_token_04_b200.build import LIB_PATH, build

P = ctypes.c_void_p(1 << 20)      # never dereferenced: every call below is refused first
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB_PATH):
        build()
    return B.lib()


def _caller(fn, **defaults):
    def call(**kw):
        assert not set(kw) - set(defaults)
        return fn(*{**defaults, **kw}.values())
    return call


def test_rotary_refusals(lib):
    call = _caller(lib.dsa_rotary, x=P, xt=64, xh=64, pos=P, f=P, T=4, H=2, d=64, rot=64, off=0, inter=0, inv=0,
                   m=1.0, dtype=B.DSA_DTYPE_BF16, out=P, ot=64, oh=64, stream=None)
    for bad in (dict(rot=63), dict(rot=0), dict(rot=128), dict(off=2), dict(off=-1), dict(T=-1), dict(H=0),
                dict(dtype=3), dict(m=float("nan")), dict(x=None), dict(out=None), dict(pos=None), dict(f=None),
                dict(x=ctypes.c_void_p((1 << 20) + 1)), dict(ot=0), dict(xt=-8)):
        assert call(**bad) == B.DSA_ERR_INVALID, bad
    assert call(d=2048, rot=1026) == B.DSA_ERR_UNSUPPORTED
    assert call(H=1 << 15) == B.DSA_ERR_UNSUPPORTED
    assert call(T=0, x=None, out=None) == B.DSA_OK            # nothing to do


def test_rotary_frequencies(lib):
    f, m = B.dsa_rotary_frequencies(64)
    assert m == 1.0 and f.shape == (32,)
    want = [10000.0 ** (-i / 32) for i in range(32)]
    assert torch.equal(f, torch.tensor(want, dtype=torch.float64).float())
    g, m = B.dsa_rotary_frequencies(64, factor=40.0)
    assert abs(m - (0.1 * math.log(40.0) + 1.0)) < 1e-7
    # at least 32 turns over 4096 tokens: kept; at most one: divided; in between: in between
    for i, (a, b) in enumerate(zip(f.tolist(), g.tolist())):
        turns = 4096 * a / (2 * math.pi)
        if turns > 45:
            assert b == a, i
        elif turns < 0.8:
            assert abs(b - a / 40) <= 1e-7 * a, i
        else:
            assert a / 40 * (1 - 1e-6) <= b <= a, i
    assert all(x >= y for x, y in zip(g.tolist(), g.tolist()[1:]))
    for bad in (dict(rot=0), dict(rot=7), dict(rot=64, theta=1.0), dict(rot=64, factor=0.5), dict(rot=64, original_len=0),
                dict(rot=64, beta_slow=0.0), dict(rot=64, beta_fast=0.5), dict(rot=64, theta=float("nan"))):
        with pytest.raises(B.DsaError) as e:
            B.dsa_rotary_frequencies(**bad)
        assert e.value.status == B.DSA_ERR_INVALID


def test_quantise_and_write_refusals(lib):
    call = _caller(lib.dsa_index_quantise, x=P, xt=8192, xh=128, T=4, H=64, d=128, dtype=0, pos=P, f=P, rot=64, off=0,
                   inter=0, m=1.0, codes=P, scale=P, ws=P, nb=256, stream=None)
    for bad in (dict(x=None), dict(x=ODD), dict(xt=8190), dict(xh=4), dict(T=-1), dict(H=0), dict(dtype=5), dict(f=None),
                dict(rot=65), dict(rot=130), dict(off=72), dict(codes=None), dict(scale=None), dict(ws=None),
                dict(nb=255), dict(ws=ctypes.c_void_p((1 << 20) + 16)), dict(m=float("inf"))):
        assert call(**bad) == B.DSA_ERR_INVALID, bad
    for bad in (dict(d=120, pos=None), dict(H=256), dict(rot=24), dict(off=4)):
        assert call(**bad) == B.DSA_ERR_UNSUPPORTED, bad
    assert call(T=0, x=None, codes=None, scale=None) == B.DSA_OK
    write = _caller(lib.dsa_index_cache_write, x=P, xt=128, T=4, d=128, dtype=0, slots=P, pos=None, f=None, rot=0, off=0,
                    inter=0, m=1.0, k=P, ks=P, n_blocks=4, bs=64, ws=P, nb=256, stream=None)
    for bad in (dict(slots=None), dict(n_blocks=0), dict(bs=0), dict(n_blocks=1 << 26, bs=64), dict(k=None),
                dict(ks=None), dict(ws=None)):
        assert write(**bad) == B.DSA_ERR_INVALID, bad


def test_cache_read_refusals(lib):
    call = _caller(lib.dsa_index_cache_read, k=P, ks=P, n_blocks=4, bs=64, d=128, table=P, mb=4, starts=None, cu=P, B=2,
                   total=10, codes=P, scale=P, values=None, vt=0, ws=P, nb=256, stream=None)
    for bad in (dict(k=None), dict(ks=None), dict(table=None), dict(cu=None), dict(B=0), dict(total=-1), dict(mb=0),
                dict(vt=3), dict(k=ODD), dict(codes=ODD), dict(values=ODD), dict(ws=None), dict(nb=8),
                dict(mb=1 << 26)):
        assert call(**bad) == B.DSA_ERR_INVALID, bad
    assert call(d=72) == B.DSA_ERR_UNSUPPORTED
    assert call(total=0) == B.DSA_OK and call(codes=None, scale=None) == B.DSA_OK


def test_latent_decode_refusals(lib):
    need = lib.dsa_latent_attention_decode_workspace_bytes(2, 1, 16)
    call = _caller(lib.dsa_latent_attention_decode, q=P, qt=9216, qh=576, latent=P, n_blocks=4, bs=64, table=P, mb=4,
                   seq=P, B=2, q_len=1, Hq=16, dqk=576, dv=512, dtype=0, scale=0.1, out=P, lse=None, ws=P, nb=need,
                   stream=None)
    for bad in (dict(q=None), dict(latent=None), dict(table=None), dict(seq=None), dict(out=None), dict(B=0),
                dict(q_len=0), dict(Hq=0), dict(scale=0.0), dict(scale=float("nan")), dict(qt=9220), dict(qh=0),
                dict(q=ODD), dict(latent=ODD), dict(out=ODD), dict(ws=None), dict(mb=1 << 26), dict(n_blocks=1 << 26),
                dict(ws=ctypes.c_void_p((1 << 20) + 128))):
        assert call(**bad) == B.DSA_ERR_INVALID, bad
    for bad in (dict(q_len=9), dict(Hq=129), dict(dqk=512), dict(dv=576), dict(dtype=2), dict(bs=4), dict(B=65536)):
        assert call(**bad) == B.DSA_ERR_UNSUPPORTED, bad
    for sizes in ((0, 1, 16), (1, 0, 16), (1, 9, 16), (1, 1, 129), (65536, 1, 16)):
        assert lib.dsa_latent_attention_decode_workspace_bytes(*sizes) == 0


def test_latent_prefill_refusals(lib):
    call = _caller(lib.dsa_latent_attention_prefill, q=P, qt=384, qh=192, kn=P, kt=512, kh=256, pe=P, pt=64, v=P, vt=512,
                   vh=256, cq=P, ck=P, B=1, Tq=4, Tk=4, max_q=4, H=2, nope=128, pe_d=64, dv=128, dtype=0, causal=1,
                   scale=0.1, out=P, lse=None, ws=P, nb=256, stream=None)
    for bad in (dict(q=None), dict(kn=None), dict(pe=None), dict(v=None), dict(cq=None), dict(ck=None), dict(out=None),
                dict(B=0), dict(H=0), dict(Tq=-1), dict(Tk=-1), dict(max_q=-1), dict(scale=-1.0), dict(qt=388),
                dict(kh=0), dict(vt=4), dict(pt=2), dict(q=ODD), dict(v=ODD), dict(ws=None), dict(nb=0)):
        assert call(**bad) == B.DSA_ERR_INVALID, bad
    for bad in (dict(nope=64), dict(pe_d=32), dict(dv=64), dict(dtype=2), dict(H=65536), dict(B=65536)):
        assert call(**bad) == B.DSA_ERR_UNSUPPORTED, bad
    assert call(Tq=0, q=None, out=None) == B.DSA_OK and call(max_q=0) == B.DSA_OK


def test_latent_prefill_workspace(lib):
    """0 for sizes that the call refuses, else the header at least."""
    for sizes in ((0, 1, 1, 1, 1, 1), (1, -1, 1, 1, 1, 1), (1, 1, -1, 1, 1, 1), (1, 1, 1, -1, 1, 1), (1, 1, 1, 1, 0, 1),
                  (65536, 1, 1, 1, 1, 1), (1, 1, 1, 1, 65536, 1)):
        assert lib.dsa_latent_attention_prefill_workspace_bytes(*sizes) == 0
    assert lib.dsa_latent_attention_prefill_workspace_bytes(1, 0, 0, 0, 1, 1) in (0, 256)   # (0 without a GPU)

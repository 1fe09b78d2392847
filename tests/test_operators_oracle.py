"""The oracle of the operators around the indexer against independent statements of the same things
(no GPU): torch's own float8 conversion, closed forms of the rotation, and attention by hand."""

import math

import numpy as np
import torch

import oracle.operators_oracle as O
from synth import quantize_e4m3_per_token


def test_e4m3_codes_match_torch_over_every_boundary():
    v = O.e4m3_values()
    mid = (v[1:] + v[:-1]) / 2
    y = np.concatenate([v, mid, np.nextafter(mid.astype(np.float32), np.float32(0)),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9))]).astype(np.float32)
    y = np.concatenate([y, -y])
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.e4m3_code(y), want)


def test_quantise_matches_the_generator():
    x = torch.randn(40, 256, generator=torch.Generator().manual_seed(1))
    x[3] = 0
    codes, scale = quantize_e4m3_per_token(x)
    c, s = O.quantise(x.numpy())
    assert np.array_equal(c, codes.numpy()) and np.array_equal(s, scale.numpy())


def test_rotary_closed_forms():
    x = np.random.RandomState(0).randn(3, 2, 8)
    f = np.array([math.pi / 2, math.pi])
    y = O.rotary(x, np.array([0, 1, 2]), f, offset=2)
    assert np.allclose(y[0], x[0])                                        # position 0 turns nothing
    assert np.allclose(y[1, :, 2], -x[1, :, 4]) and np.allclose(y[1, :, 4], x[1, :, 2])   # a quarter turn
    assert np.allclose(y[1, :, 3], -x[1, :, 3])                           # half a turn
    assert np.array_equal(y[:, :, :2], x[:, :, :2]) and np.array_equal(y[:, :, 6:], x[:, :, 6:])
    z = O.rotary(O.rotary(x, np.arange(3), f, interleaved=True), np.arange(3), f, interleaved=True, inverse=True)
    assert np.allclose(z, x)
    a, b = np.random.RandomState(1).randn(2, 1, 1, 4)                     # products depend on distances only
    dot = lambda p, r: (O.rotary(a, np.array([p]), f) * O.rotary(b, np.array([r]), f)).sum()  # noqa: E731
    assert abs(dot(17, 3) - dot(114, 100)) < 1e-9


def test_attention_by_hand():
    q = np.array([1.0, 0.0])
    k = np.array([[0.0, 5.0], [math.log(3.0), 1.0]])
    out, lse, mag = O.attend(q, k, np.array([[4.0], [-8.0]]), 1.0)
    assert np.allclose(out, [(4 - 24) / 4]) and np.allclose(lse, math.log(4.0)) and np.allclose(mag, [7.0])
    out, lse, _ = O.attend(q, k[:0], np.zeros((0, 1)), 1.0)
    assert out.tolist() == [0.0] and lse == -np.inf


def test_prefill_and_decode_forms_agree():
    """The absorbed form on latents c equals the expanded form with k_nope = W_k c, v = W_v c, where the
    absorbed query is W_k^T q_nope and W_v is applied to the absorbed output."""
    r = np.random.RandomState(3)
    n, rank, nope, pe, dv = 7, 6, 4, 2, 3
    c, kpe, wk, wv = r.randn(n, rank), r.randn(n, pe), r.randn(nope, rank), r.randn(dv, rank)
    qn, qp = r.randn(nope), r.randn(pe)
    lat = np.concatenate([c, kpe], axis=1)
    q = np.concatenate([qn @ wk, qp])[None, None, None]
    out, lse, _ = O.latent_decode(q, lat, np.zeros((1, 1), dtype=np.int64), [n], 0.3, n, dv=rank)
    full = np.concatenate([qn, qp])[None, None]
    exp, lse2, _ = O.latent_prefill(full, (c @ wk.T)[:, None], kpe, (c @ wv.T)[:, None], [0, 1], [0, n], 0.3)
    assert np.allclose(out[0, 0, 0] @ wv.T, exp[0, 0]) and np.allclose(lse[0, 0, 0], lse2[0, 0])

"""Rotary positions and the indexer's E4M3 inputs (quantisation, paged cache write and read) through
the C-ABI against the fp64 oracle (GPU).

Tolerances. A rotated value is m (a c - b s): c and s come from an angle whose fraction of a turn is
rounded to fp32 once (at most 2 pi 2^-26 < 2^-23 radians off) and from sincospif (2 ulp, 2^-22 at
most), and the two products, the sum and the magnitude's product round four times (2^-22 together),
so it is within m (|a| + |b|) 2^-20 of the exact one before the final rounding of half a step
(eps / 2 of the type). Codes of unrotated rows are exact: every step of their definition is one
IEEE operation. A pair's rotated maximum is at least its norm / sqrt 2 and |a| + |b| at most sqrt 2
norms, so a rotated row's scale is within 2^-19 relatively; its codes are within half an E4M3 step
(2^-4 of the value, or 2^-10 of the scale among the subnormals) of the value, plus that."""

import numpy as np
import pytest
import torch

import oracle.operators_oracle as O
from oracle.dsa_oracle import e4m3_decode
from sparse_attention_token_04_b200 import binding as B

pytestmark = pytest.mark.gpu

HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}


def _randn(shape, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(torch.randn((shape[0],) + (1,) * (len(shape) - 1), generator=g))
    return x.to(dtype)


def _positions(T, seed):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, 200001, (T,), generator=g).to(torch.int32)
    p[:2] = torch.tensor([0, 200000])[:T]
    if T > 3:
        p[3] = -7
    return p


def _check_rotary(y, x, ref, rot_dims, mscale=1.0):
    x, y = x.double().numpy(), y.cpu()
    step = HALF_STEP[y.dtype]
    y = y.double().numpy()
    lo, hi = rot_dims
    mag = np.abs(x[..., lo:hi]).max(axis=-1, keepdims=True) * 2 * mscale      # >= m (|a| + |b|) of any pair
    tol = mag * 2.0 ** -20 + np.abs(ref[..., lo:hi]) * step * (1 + 2.0 ** -10) + (6e-8 if step == 2.0 ** -11 else 0)
    assert (np.abs(y - ref)[..., lo:hi] <= tol).all()
    assert np.array_equal(y[..., :lo], x[..., :lo]) and np.array_equal(y[..., hi:], x[..., hi:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,d,rot,offset", [(1, 1, 64, 64, 0), (5, 128, 64, 64, 0), (33, 64, 128, 64, 64),
                                              (7, 3, 192, 64, 128), (2, 5, 96, 32, 8), (9, 2, 7, 6, 1),
                                              (300, 1, 10, 2, 3), (4, 2, 130, 130, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_matches_oracle(dtype, T, H, d, rot, offset, interleaved):
    x, pos = _randn((T, H, d), T + d, dtype), _positions(T, T)
    f, m = B.dsa_rotary_frequencies(rot, factor=4.0)
    ref = O.rotary(x.double().numpy(), pos.numpy(), f.double().numpy(), interleaved, offset, m)
    y = B.dsa_rotary(x.cuda(), pos.cuda(), f.cuda(), interleaved=interleaved, rot_offset=offset, mscale=m)
    _check_rotary(y, x, ref, (offset, offset + rot), m)


@pytest.mark.parametrize("shift", [0, 1])
def test_rotary_strided_in_place_and_inverse(shift):
    """A view inside wider rows (also one element off the 16-byte boundary), turned in place: the rows
    around the view stay, and the inverse of the fp32 result gives x back."""
    T, H, d, row = 11, 6, 64, 200
    base = _randn((T, H, row), 5).cuda()
    f, _ = B.dsa_rotary_frequencies(64, device="cuda")
    pos = _positions(T, 2).cuda()
    keep = base.clone()
    view = base[..., 100 + shift:100 + shift + d]
    x = view.cpu().clone()
    out = B.dsa_rotary(view, pos, f, out=view)
    assert out.data_ptr() == view.data_ptr()
    ref = O.rotary(x.double().numpy(), pos.cpu().numpy(), f.cpu().double().numpy())
    _check_rotary(view.contiguous(), x, ref, (0, d))
    keep[..., 100 + shift:100 + shift + d] = view
    assert torch.equal(base, keep)
    fresh = B.dsa_rotary(x.cuda(), pos, f)
    assert torch.equal(fresh, view.contiguous())
    back = B.dsa_rotary(fresh, pos, f, inverse=True).cpu().double().numpy()
    mag = 2 * np.abs(x.double().numpy()).max(axis=-1, keepdims=True)
    assert (np.abs(back - x.double().numpy()) <= mag * 2.0 ** -18).all()


def test_rotary_gradient_against_differences():
    """The inverse rotation is the gradient: <g, R(x + h e) - R(x - h e)> / 2h = (R^-1 g)[e]."""
    T, H, d = 2, 1, 32
    x, g = _randn((T, H, d), 1).cuda(), _randn((T, H, d), 2).cuda()
    f, _ = B.dsa_rotary_frequencies(16, device="cuda")
    pos = torch.tensor([3, 1000], dtype=torch.int32, device="cuda")
    grad = B.dsa_rotary(g, pos, f, rot_offset=8, mscale=1.5, inverse=True)
    h = 0.5                                                    # linear: any step, large against rounding
    for e in range(d):
        up, dn = x.clone(), x.clone()
        up[..., e] += h
        dn[..., e] -= h
        r = [B.dsa_rotary(v, pos, f, rot_offset=8, mscale=1.5).double() for v in (up, dn)]
        num = (g.double() * (r[0] - r[1])).sum(dim=(1, 2)) / (2 * h)
        # each of d terms: |g| (|x| + h) 1.5 2^-19 from each side, over 2h
        tol = float(d * g.abs().max() * (x.abs().max() + h) * 1.5 * 2.0 ** -18)
        assert (num - grad[:, 0, e].double()).abs().max() <= tol


def test_rotary_no_tokens_and_bad_shapes():
    f, _ = B.dsa_rotary_frequencies(64, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert B.dsa_rotary(torch.empty(0, 4, 64, device="cuda"), none, f).shape == (0, 4, 64)
    x = torch.zeros(2, 1, 32, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(B.DsaError):
        B.dsa_rotary(x, pos, f)                                # rot > d
    with pytest.raises(ValueError):
        B.dsa_rotary(x.transpose(0, 2), pos, f)
    with pytest.raises(ValueError):
        B.dsa_rotary(x, pos.long(), f)
    with pytest.raises(ValueError):
        B.dsa_rotary(x, pos.cpu(), f)


def _check_codes(codes, scale, values, rel=2.0 ** -19):
    top = np.abs(values).max(axis=1)
    want = np.where(top > 0, top / 448.0, 1.0)
    scale = scale.cpu().double().numpy()
    assert (np.abs(scale - want) <= want * rel).all()
    got = e4m3_decode(codes.cpu().numpy()) * scale[:, None]
    tol = np.maximum(np.abs(values) * 2.0 ** -4, scale[:, None] * 2.0 ** -10) + top[:, None] * 2 * rel
    assert (np.abs(got - values) <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,d", [(1, 1, 128), (37, 1, 128), (5, 64, 128), (19, 8, 64), (3, 1, 16), (4, 128, 128),
                                   (2, 5, 48), (40, 1, 256)])
def test_quantise_without_rotation_is_exact(dtype, T, H, d):
    x = _randn((T, H, d), T * d, dtype)
    x[T // 2] = 0
    if T > 3:
        x[1] *= 1e-4
    codes, scale = B.dsa_index_quantise(x.cuda())
    c, s = O.quantise(x.float().numpy().reshape(T, -1))
    assert np.array_equal(scale.cpu().numpy(), s)
    got = codes.cpu().numpy().reshape(T, -1)
    assert np.array_equal(e4m3_decode(got), e4m3_decode(c))   # -0 and 0 are the same value


def test_quantise_next_to_every_border_between_codes():
    """fp32 rows whose quotients lie within a few ulps of the middle of two neighbouring codes, for rows of
    many magnitudes, and all codes' own values: each code is that of the fp32 quotient."""
    v = O.e4m3_values()
    mids = np.concatenate([(v[1:] + v[:-1]) / 2, v[:-1]])
    g = np.random.RandomState(5)
    rows = []
    for k in range(60):
        top = np.float32(448.0 * 2.0 ** g.randint(-100, 100) * (1 + g.rand()))
        scale = np.float32(top) / np.float32(448.0)
        x = (mids * np.float64(scale)).astype(np.float32)
        x = np.maximum(x.view(np.int32) + g.randint(-4, 5, x.shape), 0).astype(np.int32).view(np.float32)
        x = np.clip(x, 0, top) * g.choice([-1, 1], x.shape).astype(np.float32)
        rows.append(np.concatenate([x, np.zeros(255 - len(x), np.float32), [top]]))
    x = np.stack(rows).astype(np.float32)
    assert x.shape == (60, 256)
    codes, scale = B.dsa_index_quantise(torch.from_numpy(x).cuda())
    c, s = O.quantise(x)
    assert np.array_equal(scale.cpu().numpy(), s)
    assert np.array_equal(e4m3_decode(codes.cpu().numpy()), e4m3_decode(c))


def test_quantise_smallest_and_largest_rows():
    x = torch.zeros(4, 128)
    x[0, 5] = 1e-45
    x[1, 7] = -3e38
    x[2, :3] = torch.tensor([2.0 ** -126, -2.0 ** -130, 2.0 ** -140])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    codes, scale = B.dsa_index_quantise(x.cuda(), workspace=ws)
    c, s = O.quantise(x.numpy())
    assert np.array_equal(scale.cpu().numpy(), s) and (s > 0).all()
    assert np.array_equal(e4m3_decode(codes.cpu().numpy()), e4m3_decode(c))
    assert B.dsa_read_device_status(ws) == (0, 0)


def test_quantise_not_finite_is_reported_and_yields_valid_codes():
    x = _randn((6, 2, 64), 3)
    x[1, 0, 3], x[2, 1, 5], x[4, 0, 0] = float("nan"), float("inf"), -float("inf")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    codes, scale = B.dsa_index_quantise(x.cuda(), workspace=ws)
    assert B.dsa_read_device_status(ws) == (B.DSA_ERR_DEVICE, 21)
    clean = torch.nan_to_num(x, nan=0.0)                      # infinities as the largest fp32 value
    c, s = O.quantise(clean.numpy().reshape(6, -1))
    assert np.array_equal(scale.cpu().numpy(), s)
    assert np.array_equal(e4m3_decode(codes.cpu().numpy().reshape(6, -1)), e4m3_decode(c))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,d,rot,offset", [(50, 64, 128, 64, 0), (3, 8, 64, 32, 8), (70, 1, 128, 64, 64),
                                              (1, 1, 64, 64, 0), (2, 128, 128, 32, 16), (3, 7, 1040, 1024, 8),
                                              (2, 64, 128, 128, 0), (2, 9, 144, 48, 40), (2, 4, 48, 16, 24)])
def test_quantise_with_rotation(T, H, d, rot, offset, interleaved):
    x, pos = _randn((T, H, d), 7, torch.bfloat16), _positions(T, 3)
    f, m = B.dsa_rotary_frequencies(rot, factor=40.0)
    ref = O.rotary(x.double().numpy(), pos.numpy(), f.double().numpy(), interleaved, offset, m)
    wide = torch.zeros(T, H + 1, d + 8, dtype=torch.bfloat16, device="cuda")   # strided rows
    wide[:, 1:, :d] = x.cuda()
    codes, scale = B.dsa_index_quantise(wide[:, 1:, :d], pos.cuda(), f.cuda(), interleaved=interleaved,
                                        rot_offset=offset, mscale=m)
    _check_codes(codes.reshape(T, -1), scale, ref.reshape(T, -1))


@pytest.mark.parametrize("T,block_size", [(1, 64), (130, 64), (45, 16), (9, 7)])
def test_cache_write_and_read_back(T, block_size):
    """Keys written at scattered slots (some skipped), the rest of the cache untouched, then read back
    through a block table with ranges that start and end inside pages."""
    d, blocks = 128, max(24, 3 * T // block_size + 3)
    x, pos = _randn((T, d), 4, torch.bfloat16), _positions(T, 9)
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(blocks * block_size, generator=g)[:T]
    slots[T // 2] = -1 if T > 1 else slots[0]
    k_cache = torch.randint(0, 120, (blocks, block_size, d), generator=g).to(torch.uint8)
    k_scale = torch.rand(blocks, block_size, generator=g) + 0.5
    f, _ = B.dsa_rotary_frequencies(64)
    kc, ks = k_cache.cuda(), k_scale.cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.dsa_index_cache_write(x.cuda(), slots.cuda(), kc, ks, pos.cuda(), f.cuda(), interleaved=True, workspace=ws)
    assert B.dsa_read_device_status(ws) == (0, 0)
    keep = slots >= 0
    same = torch.ones(blocks * block_size, dtype=torch.bool)
    same[slots[keep]] = False
    flat, fs = kc.cpu().view(-1, d), ks.cpu().view(-1)
    assert torch.equal(flat[same], k_cache.view(-1, d)[same]) and torch.equal(fs[same], k_scale.view(-1)[same])
    ref = O.rotary(x[:, None].double().numpy(), pos.numpy(), f.double().numpy(), True)[:, 0]
    _check_codes(flat[slots[keep]], fs[slots[keep]], ref[keep.numpy()])
    one, one_scale = B.dsa_index_quantise(x.cuda(), pos.cuda(), f.cuda(), interleaved=True)
    assert torch.equal(one.cpu()[keep], flat[slots[keep]]) and torch.equal(one_scale.cpu()[keep], fs[slots[keep]])

    lens = [3 * block_size // 2, 0, block_size, 1]
    starts = torch.tensor([block_size // 2, 5, 0, block_size], dtype=torch.int32)
    table = torch.randperm(blocks, generator=g)[:8].view(4, 2).to(torch.int32)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    total = int(cu[-1])
    rows = O.cache_rows(table.numpy(), starts.numpy(), cu.numpy(), block_size)
    for values in (None, torch.bfloat16, torch.float16, torch.float32):
        codes, scale, vals = B.dsa_index_cache_read(kc, ks, table.cuda(), cu.cuda(), total, starts=starts.cuda(),
                                                    values=values, workspace=ws)
        assert B.dsa_read_device_status(ws) == (0, 0)
        assert torch.equal(codes.cpu(), flat[rows]) and torch.equal(scale.cpu(), fs[rows])
        if values is not None:
            want = (flat[rows].view(torch.float8_e4m3fn).float() * fs[rows][:, None]).to(values)
            assert torch.equal(vals.cpu(), want)


def test_cache_write_bad_slots_are_reported_and_left_out():
    x = _randn((3, 128), 8, torch.float16).cuda()
    for bad in (4 * 64, -2, 1 << 40):
        kc = torch.zeros(4, 64, 128, dtype=torch.uint8, device="cuda")
        ks = torch.zeros(4, 64, device="cuda")
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        B.dsa_index_cache_write(x, torch.tensor([5, bad, 255], device="cuda"), kc, ks, workspace=ws)
        assert B.dsa_read_device_status(ws) == (B.DSA_ERR_DEVICE, 20)
        assert ks.view(-1).nonzero().flatten().tolist() == [5, 255]


def test_cache_read_bad_blocks_and_rows_outside():
    kc = torch.full((2, 16, 32), 9, dtype=torch.uint8, device="cuda")
    ks = torch.full((2, 16), 3.0, device="cuda")
    table = torch.tensor([[1, 5], [0, -1]], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    cu = torch.tensor([2, 22, 30], dtype=torch.int32, device="cuda")   # rows 0, 1 and 30.. are no request's
    codes = torch.full((34, 32), 77, dtype=torch.uint8, device="cuda")
    scale = torch.full((34,), 7.0, device="cuda")
    B.dsa_index_cache_read(kc, ks, table, cu, 34, out_codes=codes, out_scale=scale, workspace=ws)
    assert B.dsa_read_device_status(ws) == (B.DSA_ERR_DEVICE, 16)
    want = [7.0] * 2 + [3.0] * 16 + [1.0] * 4 + [3.0] * 8 + [7.0] * 4
    assert scale.tolist() == want
    code_of = {7.0: 77, 3.0: 9, 1.0: 0}
    assert codes[:, 0].tolist() == [code_of[w] for w in want] and codes[:, 31].tolist() == codes[:, 0].tolist()
    # a position past the table is reported as well; outputs shorter than the offsets are not passed
    B.dsa_index_cache_read(kc, ks, table[:, :1].contiguous(), torch.tensor([0, 17, 17], dtype=torch.int32, device="cuda"),
                           10, workspace=ws)
    assert B.dsa_read_device_status(ws) == (0, 0)
    B.dsa_index_cache_read(kc, ks, table[:, :1].contiguous(), torch.tensor([0, 17, 17], dtype=torch.int32, device="cuda"),
                           17, workspace=ws)
    assert B.dsa_read_device_status(ws) == (B.DSA_ERR_DEVICE, 16)


def test_streams_and_graphs():
    """A call on a given stream, and one captured and replayed on new inputs, write what a plain call
    writes."""
    x, pos = _randn((20, 64, 128), 1, torch.bfloat16).cuda(), _positions(20, 1).cuda()
    f, _ = B.dsa_rotary_frequencies(64, device="cuda")
    want, scale = B.dsa_index_quantise(x, pos, f)
    rot = B.dsa_rotary(x, pos, f)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c2, s2 = B.dsa_index_quantise(x, pos, f, stream=side)
    r2 = B.dsa_rotary(x, pos, f, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(c2, want) and torch.equal(s2, scale) and torch.equal(r2, rot)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    xin = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c3, s3 = B.dsa_index_quantise(xin, pos, f, workspace=ws)
        r3 = B.dsa_rotary(xin, pos, f)
    xin.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c3, want) and torch.equal(s3, scale) and torch.equal(r3, rot)


@pytest.mark.parametrize("dtype,H,d,rot,interleaved", [
    (torch.bfloat16, 64, 128, 64, False), (torch.float16, 64, 128, 64, True), (torch.float32, 33, 64, 32, False),
    (torch.bfloat16, 9, 64, 0, False), (torch.float32, 128, 128, 128, True), (torch.bfloat16, 100, 48, 16, False)])
def test_quantise_many_large_rows(dtype, H, d, rot, interleaved):
    """More rows than there are CTAs for, among them zero, tiny and non-finite ones: the same bits as in calls
    of few rows, and the finite rows within the oracle's bound."""
    T = 3100
    x = _randn((T, H, d), H + d, dtype)
    x[5::97] = 0
    x[6::97] *= 2.0 ** -14
    if dtype != torch.float16:
        x[7::97] *= 1e-30
    x[1000, H - 1, d - 1], x[1001, 0, 0], x[2999, H // 2, 1] = float("nan"), float("inf"), -float("inf")
    pos = _positions(T, 3)
    f, _ = B.dsa_rotary_frequencies(rot, device="cuda") if rot else (None, 1.0)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def call(a, e):
        kw = dict(positions=pos[a:e].cuda(), inv_freq=f, interleaved=interleaved) if rot else {}
        return B.dsa_index_quantise(x[a:e].cuda(), workspace=ws, **kw)

    codes, scale = call(0, T)
    assert B.dsa_read_device_status(ws) == (B.DSA_ERR_DEVICE, 21)
    parts = [call(a, min(a + 100, T)) for a in range(0, T, 100)]
    assert torch.equal(codes, torch.cat([c for c, _ in parts])) and torch.equal(scale, torch.cat([s for _, s in parts]))
    some = [0, 1, 5, 6, 7, 739, 740, 741, 1480, 2220, 2221, 3099]
    values = x[some].double().numpy()
    if rot:
        values = O.rotary(values, pos[some].numpy(), f.cpu().numpy(), interleaved)
    _check_codes(codes[some].flatten(1), scale[some], values.reshape(len(some), -1))

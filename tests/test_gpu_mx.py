"""GPU parity of the MX calls with the fp64 oracle.

Quantization, decoding and the norm's sum are exact and compared bit for bit. A
norm's codes may differ from the oracle's only where its y lies within the
kernel's error of a rounding boundary. Products are compared bit for bit on
inputs whose sums are exact in fp32, and otherwise within the bound of an fp32
sum and one bf16 rounding."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_nf4_quantized_absmax_b200 import binding as b
from oracle import mx
from oracle.merge import f64_to_bf16_bits_rn
from tests.helpers import bf16_bits_np, require_gpu

pytestmark = pytest.mark.gpu

FORMATS = [b.MX_E4M3, b.MX_E2M1]


def _f64(t):
    return t.detach().double().cpu().numpy()


def _done():
    torch.cuda.synchronize()
    assert b.qlora_device_error() == 0


def _rand(shape, seed, spread=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if spread:
        x = x * torch.exp2(torch.randint(-spread, spread + 1, shape, generator=g).float())
    return x.to(torch.bfloat16)


def _all_bf16():
    """Every bf16 pattern, the non-finite ones alone in blocks of their own rows' end, and shuffled into blocks."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    perm = torch.randperm(65536, generator=torch.Generator().manual_seed(5))
    finite = bits.view(torch.bfloat16)
    near = finite.clone().view(-1, 32)  # neighbouring patterns: blocks of one binade
    return torch.cat([near, finite[perm].view(-1, 32)])


def _check_storage(q, X):
    codes, sc = mx.quantize(_f64(X), q.format)
    data, scales = mx.pack(codes, sc, q.format)
    assert np.array_equal(q.scales.cpu().numpy().reshape(scales.shape), scales)
    got = q.data.cpu().numpy().reshape(data.shape)
    assert np.array_equal(got, data), np.argwhere(got != data)[:4]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", [(1, 32), (1, 4096), (3, 160), (5, 96), (257, 320), (333, 11040), (1000, 128)])
def test_quantize_bits(shape, fmt):
    dev = require_gpu()
    X = _rand(shape, shape[0] * 7 + shape[1], spread=12)
    q = b.qlora_quantize_mx(X.to(dev), fmt)
    _done()
    _check_storage(q, X)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_every_bf16_value(fmt):
    dev = require_gpu()
    X = _all_bf16()
    q = b.qlora_quantize_mx(X.to(dev), fmt)
    _done()
    _check_storage(q, X)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_rounding_boundaries(fmt):
    """Blocks whose first element fixes the scale and whose others sit on and next to every midpoint."""
    dev = require_gpu()
    t = mx.MAGNITUDES[fmt]
    mid = (t[:-1] + t[1:]) / 2
    vals = torch.tensor(np.concatenate([t, mid]), dtype=torch.float64).to(torch.bfloat16)
    assert torch.equal(vals.double(), torch.tensor(np.concatenate([t, mid])))
    up = (vals.view(torch.int16) + 1).view(torch.bfloat16)
    dn = (vals.view(torch.int16) - (vals != 0).to(torch.int16)).view(torch.bfloat16)
    allv = torch.cat([vals, up, dn])
    allv = allv[allv.float() <= 480]
    allv = torch.cat([allv, -allv])
    rows = -(-allv.numel() // 31)
    X = torch.zeros(rows, 32, dtype=torch.bfloat16)
    X[:, 0] = float(t[-1])
    X[:, 1:] = torch.cat([allv, torch.zeros(rows * 31 - allv.numel(), dtype=torch.bfloat16)]).view(rows, 31)
    for scale in (1.0, 2.0 ** -40, 2.0 ** 60):
        Xs = (X.float() * scale).to(torch.bfloat16)
        q = b.qlora_quantize_mx(Xs.to(dev), fmt)
        _done()
        _check_storage(q, Xs)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_from_16_byte_aligned_base(fmt):
    dev = require_gpu()
    X = _rand((9, 288), 3, spread=3)
    buf = torch.zeros(X.numel() + 8, dtype=torch.bfloat16, device=dev)
    view = buf[8:].view(X.shape)
    assert view.data_ptr() % 32 == 16
    view.copy_(X)
    q = b.qlora_quantize_mx(view, fmt)
    out = torch.zeros(X.numel() + 8, dtype=torch.bfloat16, device=dev)
    v = b.qlora_dequantize_mx(q, out=out[8:].view(X.shape))
    _done()
    _check_storage(q, X)
    ref = mx.dequantize(*mx.quantize(_f64(X), fmt), fmt)
    assert np.array_equal(_f64(v), ref) and not out[:8].any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_dequantize_every_code_and_scale(fmt):
    dev = require_gpu()
    n = 256 if fmt == b.MX_E4M3 else 16
    codes = np.tile(np.arange(n, dtype=np.uint8), (256, 256 // n)).reshape(256, 256)
    sc = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, 1)
    data, scales = mx.pack(codes, sc, fmt)
    q = b.MXTensor(torch.tensor(data).to(dev), torch.tensor(scales).to(dev), 256, 256, fmt)
    got = b.qlora_dequantize_mx(q)
    _done()
    with np.errstate(over="ignore"):
        ref = mx.dequantize(codes, sc, fmt)
    bits, want = bf16_bits_np(got), np.zeros(ref.shape, np.uint16)
    fine = np.isfinite(ref)
    want[fine] = f64_to_bf16_bits_rn(ref[fine])
    assert np.array_equal(bits[fine], want[fine])
    assert np.isnan(_f64(got)[~fine]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_dequantize_past_the_largest_bf16_value(fmt):
    """Scale bytes that only imported storage has: results of 2^128 or more are infinities, those below are exact."""
    dev = require_gpu()
    table = mx.MAGNITUDES[fmt]
    codes = np.zeros((16, 256), np.uint8)
    codes[:, :len(table)] = np.arange(len(table))
    codes[:, 128:128 + len(table)] = np.arange(len(table)) + mx.SIGN[fmt]
    sc = np.repeat(np.arange(239, 255, dtype=np.uint8)[:, None], 8, 1)
    data, scales = mx.pack(codes, sc, fmt)
    got = b.qlora_dequantize_mx(b.MXTensor(torch.tensor(data).to(dev), torch.tensor(scales).to(dev), 16, 256, fmt))
    _done()
    ref = mx.dequantize(codes, sc, fmt)
    big = np.abs(ref) >= 2.0 ** 128
    assert big.any(1).tolist() == [byte >= (253 if fmt == b.MX_E2M1 else 247) for byte in range(239, 255)]
    assert np.array_equal(_f64(got), np.where(big, np.copysign(np.inf, ref), ref))


def test_rows_beyond_32_bit_offsets():
    """2.2e9 elements: the last rows are those of a small call."""
    dev = require_gpu()
    rows, cols = 540_000, 4096
    X = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
    X.normal_(generator=torch.Generator(device=dev).manual_seed(1))
    q = b.qlora_quantize_mx(X, b.MX_E4M3)
    t = b.qlora_quantize_mx(X[-7:].contiguous(), b.MX_E4M3)
    assert torch.equal(q.data[-7:], t.data) and torch.equal(q.scales[:, -7:], t.scales)
    v = b.qlora_dequantize_mx(q)
    assert torch.equal(v[-7:], b.qlora_dequantize_mx(t))
    del v
    gamma = torch.ones(cols, dtype=torch.bfloat16, device=dev)
    n, _ = b.qlora_rmsnorm_mx(X, gamma, 1e-5, out=q)
    m, _ = b.qlora_rmsnorm_mx(X[-7:].contiguous(), gamma, 1e-5)
    _done()
    assert torch.equal(n.data[-7:], m.data) and torch.equal(n.scales[:, -7:], m.scales)


# ---- RMS norm ----
# (The kernel's sums are fp64, so the bound that follows, of sums in fp32, holds with room to spare; the narrow one stands at
# test_rmsnorm_codes_of_the_exact_value.)
# A thread adds at most 32 squares in fp32 (each addition off by 2^-24 of the partial sum, all terms positive: the sum
# within 32 * 2^-24 relative), which the root halves; the fp64 steps and the tail of rstd add less than 2^-40, and y is
# rounded once to fp32 (2^-24): 17 * 2^-24 covers it.
NORM_TOL = 17 * 2.0 ** -24


def _check_norm(q, y):
    """q's values lie between those of y (1 - tol) and y (1 + tol), block by block with the scale that q chose, which is
    the scale of one of the two."""
    rows, cols = y.shape
    codes, sc = mx.unpack(q.data.cpu().numpy(), q.scales.cpu().numpy(), rows, cols, q.format)
    blocks = y.reshape(rows, -1, 32)
    lo, hi = np.abs(blocks).max(-1) * (1 - NORM_TOL), np.abs(blocks).max(-1) * (1 + NORM_TOL)
    byte = lambda a: np.where(a > 0, np.maximum(np.frexp(a)[1] - 1 - mx.EMAX[q.format], -127), -127) + 127  # noqa: E731
    assert np.all((sc == byte(lo)) | (sc == byte(hi)))
    e = sc.astype(np.int64)[..., None] - 127
    got = mx.decode(codes, q.format).reshape(blocks.shape)
    a = mx.decode(mx.encode(np.ldexp(blocks * (1 - NORM_TOL), -e), q.format), q.format)
    c = mx.decode(mx.encode(np.ldexp(blocks * (1 + NORM_TOL), -e), q.format), q.format)
    bad = (got < np.minimum(a, c)) | (got > np.maximum(a, c))
    assert not bad.any(), np.argwhere(bad)[:4]
    assert np.mean(a != c) < 0.01  # the bracket means something


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("shape", [(1, 32), (1, 4096), (3, 160), (517, 5152), (64, 8192), (5, 8224), (3, 16384),
                                   (2, 32768), (2, 32736)])
def test_rmsnorm(shape, residual, fmt):
    dev = require_gpu()
    X, R = _rand(shape, 11, spread=4), _rand(shape, 12, spread=4)
    g = (1 + 0.1 * _rand((shape[1],), 13).float()).to(torch.bfloat16)
    q, h = b.qlora_rmsnorm_mx(X.to(dev), g.to(dev), 1e-5, fmt, residual=R.to(dev) if residual else None)
    _done()
    ref_h = (X.float() + R.float()).to(torch.bfloat16) if residual else X
    if residual:
        assert torch.equal(h.cpu().view(torch.int16), ref_h.view(torch.int16))
    else:
        assert h is None
    _check_norm(q, mx.rmsnorm(_f64(ref_h), _f64(g), float(np.float32(1e-5))))
    if shape[1] % 128:  # the padding is what the products expect
        kp = (shape[1] + 127) // 128 * 128
        d = q.data.view(shape[0], -1).cpu()
        assert not d[:, shape[1] if fmt == b.MX_E4M3 else shape[1] // 2:].any()
        s = q.scales.view(kp // 128, shape[0], 4).cpu()
        assert torch.all(s[-1, :, (shape[1] % 128) // 32:] == 127)


@pytest.mark.parametrize("fmt", FORMATS)
def test_rmsnorm_is_not_rounded_twice(fmt):
    """The squares of whole numbers up to 255 add up exactly in a thread's fp32, so rstd is good to 2^-40 and every code is that of the
    exact y: an fp32 y that is a tie of the element type only by its own rounding does not decide for the even one."""
    dev = require_gpu()
    shape = (4096, 4096)
    gen = torch.Generator().manual_seed(77)
    X = torch.randint(-255, 256, shape, generator=gen).to(torch.bfloat16)
    g = (1 + torch.rand(shape[1], generator=gen)).to(torch.bfloat16)
    q, _ = b.qlora_rmsnorm_mx(X.to(dev), g.to(dev), 1e-5, fmt)
    _done()
    y = mx.rmsnorm(_f64(X), _f64(g), float(np.float32(1e-5)))
    codes, sc = mx.unpack(q.data.cpu().numpy(), q.scales.cpu().numpy(), *shape, fmt)
    near = []
    for sign in (-1, 1):  # what values 2^-38 off would give: no statement where they differ
        near.append(mx.quantize(y * (1 + sign * 2.0 ** -38), fmt))
    sure = (near[0][0] == near[1][0])
    assert np.array_equal(sc, near[0][1]) and np.array_equal(sc, near[1][1])
    assert sure.mean() > 0.9999
    bad = (codes != near[0][0]) & sure
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])


# The squares are added up in fp64 (some 45 additions one after another: 2^-47), the root is a 2-ulp fp32 estimate, within
# 2^-22, after one Newton step (1.5 * 2^-44), and its head and tail hold 48 bits: y is known to within 2^-43.
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("shape", [(1500, 288), (2000, 4096), (517, 5152), (300, 16416)])
def test_rmsnorm_codes_of_the_exact_value(shape, residual, fmt):
    """Rows of any bf16 numbers: every code is that of the exact y, wherever it is one for all y within 2^-42. (Partial sums in
    fp32 would leave 2 or 3 codes of 16 million off.)"""
    dev = require_gpu()
    X, R = _rand(shape, 31, spread=3), _rand(shape, 32, spread=3)
    g = (1 + 0.1 * _rand((shape[1],), 33).float()).to(torch.bfloat16)
    q, _ = b.qlora_rmsnorm_mx(X.to(dev), g.to(dev), 1e-5, fmt, residual=R.to(dev) if residual else None)
    _done()
    h = (X.float() + R.float()).to(torch.bfloat16) if residual else X
    y = mx.rmsnorm(_f64(h), _f64(g), float(np.float32(1e-5)))
    codes, sc = mx.unpack(q.data.cpu().numpy(), q.scales.cpu().numpy(), *shape, fmt)
    (c0, s0), (c1, s1) = (mx.quantize(y * (1 + sign * 2.0 ** -42), fmt) for sign in (-1, 1))
    sure, sure_scale = c0 == c1, s0 == s1
    assert sure.mean() > 0.99999 and sure_scale.all()
    assert np.array_equal(sc, s0)
    bad = (codes != c0) & sure
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])


@pytest.mark.parametrize("fmt", FORMATS)
def test_rmsnorm_of_large_and_small_rows(fmt):
    """Scaled by a power of two, with eps = 0, a row has the codes of the row itself: the squares overflow or vanish in fp32,
    not in fp64."""
    dev = require_gpu()
    X = _rand((40, 4128), 34)
    g = (1 + 0.1 * _rand((4128,), 35).float()).to(torch.bfloat16)
    q, _ = b.qlora_rmsnorm_mx(X.to(dev), g.to(dev), 0.0, fmt)
    for e in (-110, -75, 66, 100):
        Xs = torch.ldexp(X.float(), torch.tensor(e)).to(torch.bfloat16)
        assert torch.equal(torch.ldexp(Xs.double(), torch.tensor(-e)), X.double())
        t, _ = b.qlora_rmsnorm_mx(Xs.to(dev), g.to(dev), 0.0, fmt)
        _done()
        assert torch.equal(q.scales, t.scales) and torch.equal(q.data, t.data), e


@pytest.mark.parametrize("fmt", FORMATS)
def test_rmsnorm_exact_ties_and_zeros(fmt):
    """Where rstd is a power of two, y is exact and its ties go to even; zeros stay zeros, alone in a block or among
    others."""
    dev = require_gpu()
    X = torch.full((4, 1024), 4.0, dtype=torch.bfloat16)
    X[1] = -0.5
    X[2, 1::2] = 0          # the mean of the squares is 8: rstd is no binary fraction
    X[2, 64:128] = 0
    X[3] = 0
    g = ((torch.arange(1024) % 256 + 1).float() / 64).to(torch.bfloat16)
    for e in (0.0, 2.0 ** -40):
        rows = 3 if e == 0.0 else 4
        q, _ = b.qlora_rmsnorm_mx(X[:rows].to(dev), g.to(dev), e, fmt)
        _done()
        y = mx.rmsnorm(_f64(X[:rows]), _f64(g), e)
        codes, sc = mx.unpack(q.data.cpu().numpy(), q.scales.cpu().numpy(), rows, 1024, fmt)
        want, scales = mx.quantize(y, fmt)
        exact = [0, 1] if e == 0.0 else [3]
        assert np.array_equal(sc[exact], scales[exact])
        v, w = mx.decode(codes, fmt), mx.decode(want, fmt)
        assert np.array_equal(v[exact], w[exact])
        assert np.array_equal(v[2] == 0, w[2] == 0) and not v[2, 64:128].any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("cols,ones,eps,p,k", [
    (288, 128, 0.0, 3, 1), (288, 92, 0.125, 3, 1), (800, 512, 0.0, 5, 2), (1568, 128, 0.0, 7, 1), (9248, 2048, 0.0, 17, 3),
    (30752, 8192, 0.0, 31, 4), (1024, 256, 0.0, 1, -1)])
def test_rmsnorm_ties_where_rstd_is_a_fraction(cols, ones, eps, p, k, fmt):
    """rstd = p / 2^k exactly, which column counts with an odd square factor allow: y is exact and its ties go to even. With
    one more, tiny element rstd is just below it, and no y is a tie any longer."""
    dev = require_gpu()
    rstd = p / 2.0 ** k
    assert (ones + eps * cols) * rstd * rstd == cols
    X = torch.zeros(3, cols, dtype=torch.bfloat16)
    X[:, :ones] = 1.0
    X[1] *= -1
    X[2, -1] = 2.0 ** -11 if ones < cols - 32 else 0.0
    g = torch.ones(cols, dtype=torch.bfloat16)
    g[:ones] = (torch.arange(ones) % 256 + 1).float().to(torch.bfloat16)  # y: odd multiples of p / 2^k among them
    q, _ = b.qlora_rmsnorm_mx(X.to(dev), g.to(dev), eps, fmt)
    _done()
    codes, sc = mx.unpack(q.data.cpu().numpy(), q.scales.cpu().numpy(), 3, cols, fmt)
    exact = np.stack([_f64(X[i]) * _f64(g) * rstd for i in (0, 1)])
    want, scales = mx.quantize(exact, fmt)
    assert np.array_equal(sc[:2], scales)
    assert np.array_equal(mx.decode(codes[:2], fmt), mx.decode(want, fmt))
    table = mx.MAGNITUDES[fmt]
    u = np.abs(np.ldexp(exact.reshape(2, -1, 32), 127 - scales.astype(np.int64)[..., None]))
    # There are ties where they can be: a midpoint is an odd number of 5 (e4m3) or 3 bits (e2m1) times a power of two, and a
    # multiple of p is such a number for p up to 31 or 7 alone.
    assert np.isin(u, (table[:-1] + table[1:]) / 2).any() == (p <= (31 if fmt == b.MX_E4M3 else 7))
    below, bscale = mx.quantize(mx.rmsnorm(_f64(X[2:]), _f64(g), eps), fmt)  # 2^-22 / (2 * 8192) below at least: 2^-36
    assert np.array_equal(sc[2:], bscale) and np.array_equal(mx.decode(codes[2:], fmt), mx.decode(below, fmt))


def test_rmsnorm_in_place_and_edges():
    dev = require_gpu()
    X, R = _rand((6, 256), 21), _rand((6, 256), 22)
    R[1] = -X[1]                      # the sum is zero: y = 0 with eps > 0
    X[2, 5] = float("inf")
    X[3, 40] = float("nan")
    X[4] = X[4] * 2.0 ** 50
    g = torch.ones(256, dtype=torch.bfloat16)
    r = R.to(dev)
    q, h = b.qlora_rmsnorm_mx(X.to(dev), g.to(dev), 1e-6, residual=r, residual_out=r)
    v = b.qlora_dequantize_mx(q)
    _done()
    assert h.data_ptr() == r.data_ptr()
    ref = (X.float() + R.float()).to(torch.bfloat16)
    ok = [0, 1, 4, 5]
    assert torch.equal(r.cpu()[ok], ref[ok])
    assert not v[1].any() and torch.isfinite(v[ok]).all()
    assert torch.isnan(v[3]).all()    # NaN spreads through the mean
    assert torch.isnan(v[2, :32]).all() and not v[2, 32:].any()  # inf * 0 in its block, finite * 0 elsewhere
    # eps = 0 and a row of zeros: 0 / 0
    z = torch.zeros(1, 64, dtype=torch.bfloat16, device=dev)
    q, _ = b.qlora_rmsnorm_mx(z, g.to(dev)[:64], 0.0)
    assert torch.isnan(b.qlora_dequantize_mx(q)).all()
    _done()


# ---- products ----

def _exact_operand(rows, cols, fmt, seed, spread):
    """Storage whose values are small multiples of a power of two: sums over k are exact in fp32."""
    rng = np.random.default_rng(seed)
    if fmt == b.MX_E2M1:
        codes = rng.integers(0, 16, size=(rows, cols)).astype(np.uint8)
    else:
        codes = mx.encode(rng.integers(-8, 9, size=(rows, cols)) / 2.0, fmt)
    sc = (127 + rng.integers(-spread, spread + 1, size=(rows, cols // 32))).astype(np.uint8)
    data, scales = mx.pack(codes, sc, fmt)
    return mx.dequantize(codes, sc, fmt), (data, scales)


def _to(dev, storage, rows, cols, fmt):
    return b.MXTensor(torch.tensor(storage[0]).to(dev), torch.tensor(storage[1]).to(dev), rows, cols, fmt)


def _bits(ref):
    return f64_to_bf16_bits_rn(ref.ravel()).reshape(ref.shape)


# Products are multiples of 2^-2 (times 2^-2s) of magnitude at most 36 (times 2^2s): with s = 2 and K <= 11040 sums stay
# below 2^24 units of 2^-6 for the random signs used (checked), so fp32 holds every partial sum.
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 128, 128), (2, 130, 160), (7, 64, 96), (16, 256, 4096), (1, 11008, 512),
                                   (17, 200, 288), (32, 129, 1024), (33, 384, 640), (64, 77, 2080), (65, 512, 256),
                                   (100, 1000, 1056), (128, 128, 4096), (129, 257, 384), (300, 4100, 544),
                                   (256, 256, 1024), (700, 520, 1184), (1025, 770, 256), (2048, 1024, 512),
                                   # more tiles of 128 x 128 than SMs: CTA pairs, whole and narrow tiles, odd N
                                   (1200, 2100, 288), (700, 4100, 544), (2049, 1283, 1184), (4096, 1024, 160), (1057, 2560, 96),
                                   (520, 5000, 2144)])
def test_product_bits(M, N, K, fmt):
    dev = require_gpu()
    x, xs = _exact_operand(M, K, fmt, 100 + M, 2)
    w, ws = _exact_operand(N, K, b.MX_E2M1, 200 + N, 2)
    ref = x @ w.T
    assert np.abs(ref).max() < 2.0 ** 17
    Y = b.qlora_mx_linear_fwd(_to(dev, xs, M, K, fmt), _to(dev, ws, N, K, b.MX_E2M1))
    _done()
    got, want = bf16_bits_np(Y), _bits(ref)
    same = (got == want) | ((got | want) & 0x7FFF == 0)  # +0 and -0
    assert same.all(), (np.argwhere(~same)[:4], (~same).mean())


# fp32 sums: the MMA of 32 products, and each addition to the accumulator, keep at least 23 bits of the largest term
# (truncating at worst): (K / 32 + 32) * 2^-23 of the sum of magnitudes covers any order; then one bf16 rounding, 2^-8.
def _check_product(Y, x, w):
    ref = x @ w.T
    tol = 2.0 ** -8 * np.abs(ref) + (x.shape[1] / 32 + 32) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    bad = ~(np.abs(_f64(Y) - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], bad.mean())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (4, 300, 11008), (16, 4096, 11040), (50, 700, 4128), (333, 1100, 4128),
                                   (512, 2048, 4096)])
def test_product_of_real_values(M, N, K, fmt):
    """bf16 activations with loud channels against a normal weight, through the quantizing form of the call."""
    dev = require_gpu()
    X = _rand((M, K), M + N)
    X[:, ::97] *= 20
    W = (0.02 * _rand((N, K), M + K).float()).to(torch.bfloat16)
    w = b.qlora_quantize_mx(W.to(dev), b.MX_E2M1)
    Y = b.qlora_mx_linear_fwd(X.to(dev), w, x_format=fmt)
    Yq = b.qlora_mx_linear_fwd(b.qlora_quantize_mx(X.to(dev), fmt), w)
    _done()
    assert torch.equal(Y, Yq)
    xv = mx.dequantize(*mx.quantize(_f64(X), fmt), fmt)
    wv = mx.dequantize(*mx.quantize(_f64(W), b.MX_E2M1), b.MX_E2M1)
    _check_product(Y, xv, wv)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_product_extreme_scales_and_nan(M):
    """Scale bytes from one end to the other, zero blocks, and NaN blocks, which reach their own row or column only."""
    dev = require_gpu()
    N, K = 200, 512
    x, xs = _exact_operand(M, K, b.MX_E4M3, 1, 0)
    w, ws = _exact_operand(N, K, b.MX_E2M1, 2, 0)
    xs[1][:, 1, :], ws[1][:, 5, :] = 0, 254    # 2^-127 and 2^127: their product is 1
    xs[1][:, 2, :], ws[1][:, 6, :] = 90, 250
    x[1] *= 2.0 ** -127
    x[2] *= 2.0 ** -37
    w[5] *= 2.0 ** 127
    w[6] *= 2.0 ** 123
    xs[1][3, 0, 2] = 255
    ws[1][0, 9, 1] = 255
    Y = b.qlora_mx_linear_fwd(_to(dev, xs, M, K, b.MX_E4M3), _to(dev, ws, N, K, b.MX_E2M1))
    _done()
    ref = x @ w.T
    nan = np.zeros_like(ref, bool)
    nan[0], nan[:, 9] = True, True
    got = _f64(Y)
    # An fp32 sum may pass through any partial sum: they are at most the sum of the magnitudes, and only where that is
    # below fp32's largest value (3.4e38) does a finite total say that none overflowed (2^127 * (4 - 3) can: 4 * 2^127
    # is infinite). Totals below 2^-100 may lose bits below fp32's smallest.
    mag = np.abs(x) @ np.abs(w).T
    fine = ~nan & (mag < 3e38) & ((np.abs(ref) > 2.0 ** -100) | (ref == 0))
    assert fine[1, 6] and fine[0 if M < 3 else 2].sum() > 100
    assert np.isnan(got[nan]).all()
    assert np.array_equal(got[fine], _f64(torch.tensor(ref[fine]).to(torch.bfloat16)))


def test_product_into_more_than_2_31_outputs():
    dev = require_gpu()
    M, N, K = 70_000, 32_768, 128
    X = torch.empty(M, K, dtype=torch.bfloat16, device=dev).normal_(generator=torch.Generator(device=dev).manual_seed(1))
    W = torch.empty(N, K, dtype=torch.bfloat16, device=dev).normal_(generator=torch.Generator(device=dev).manual_seed(2))
    w, x = b.qlora_quantize_mx(W, b.MX_E2M1), b.qlora_quantize_mx(X, b.MX_E4M3)
    Y = b.qlora_mx_linear_fwd(x, w)
    T = b.qlora_mx_linear_fwd(X[-300:].contiguous(), w)
    _done()
    assert torch.equal(Y[-300:], T)
    assert torch.equal(Y[:300], b.qlora_mx_linear_fwd(X[:300].contiguous(), w))


# ---- grouped ----

GROUPS = [
    ([1], 128, 128),
    ([0, 3, 0, 0, 5, 1, 0], 200, 160),
    ([0, 0, 0], 64, 64),
    ([16, 17, 1, 0, 15], 130, 288),
    ([40, 0, 33, 129, 2], 96, 544),
    ([300, 1, 0, 700, 128, 127], 260, 256),
    ([0] * 33 + [2] + [0] * 29 + [1], 128, 256),
    ([1] * 40, 257, 96),
    ([1000, 3], 513, 384),
    ([5] * 300, 16, 64),
    # CTA pairs
    ([602, 30, 87, 67, 134, 14, 39, 27], 1300, 416),
    ([2000], 1200, 256),
    ([5, 900, 0, 260], 2051, 160),
    ([257] * 6, 1281, 1184),
    ([0] * 40 + [1500] + [33] * 3, 1284, 1056),
    ([0] * 33 + [4000, 0, 600], 516, 96),
    # one CTA from tile to tile
    ([(i * 37) % 90 for i in range(64)], 1600, 160),
    ([300, 0, 1, 127, 128, 129], 4100, 1184),
    ([200 if i % 3 == 0 else i % 7 for i in range(70)], 300, 96),
    ([0] * 65 + [5500] + [0] * 14 + [1], 130, 1056),
    ([17, 0, 40, 9] * 64, 400, 64),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_grouped_bits(case, fmt):
    """Bit equality with the oracle, rows before the first offset and behind the last left as they were."""
    dev = require_gpu()
    sizes, N, K = GROUPS[case]
    E, lead, tail = len(sizes), 5, 9
    off = np.concatenate([[0], np.cumsum(sizes)]) + lead
    M = int(off[-1]) + tail
    x, xs = _exact_operand(M, K, fmt, case, 2)
    w, ws = _exact_operand(E * N, K, b.MX_E2M1, 50 + case, 2)
    Y = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device=dev)
    out = b.qlora_mx_grouped_fwd(_to(dev, xs, M, K, fmt), _to(dev, ws, E * N, K, b.MX_E2M1),
                                 torch.tensor(off, dtype=torch.int32, device=dev), Y=Y[:M])
    _done()
    assert out.data_ptr() == Y.data_ptr()
    ref = mx.grouped(x, w.reshape(E, N, K), off)
    rows = slice(lead, M - tail)
    got, want = bf16_bits_np(Y)[rows], _bits(ref[rows])
    same = (got == want) | ((got | want) & 0x7FFF == 0)
    assert same.all(), np.argwhere(~same)[:4]
    assert torch.all(Y[:lead] == 7) and torch.all(Y[M - tail:] == 7)


@pytest.mark.parametrize("off", [[0, 30, 10, 40], [-5, 8, 20, 1000], [50, 40, 30, 20], [2**31 - 1, -2**31, 3, 4],
                                 [0, 64, 64, 64]])
def test_grouped_with_bad_offsets_stays_in_bounds(off):
    """Offsets are clamped to [0, M] and to their running maximum; rows that no group has are untouched."""
    dev = require_gpu()
    M, N, K, E = 64, 144, 128, 3
    x, xs = _exact_operand(M, K, b.MX_E4M3, 3, 1)
    w, ws = _exact_operand(E * N, K, b.MX_E2M1, 4, 1)
    Y = torch.full((M + 8, N), 7.0, dtype=torch.bfloat16, device=dev)
    b.qlora_mx_grouped_fwd(_to(dev, xs, M, K, b.MX_E4M3), _to(dev, ws, E * N, K, b.MX_E2M1),
                           torch.tensor(off, dtype=torch.int32, device=dev), Y=Y[4:4 + M])
    _done()
    mended = np.minimum(np.maximum.accumulate(np.maximum(np.array(off, dtype=np.int64), 0)), M)
    ref = mx.grouped(x, w.reshape(E, N, K), mended)
    want = np.where(np.isnan(ref), 7.0, ref)
    assert np.array_equal(_f64(Y[4:4 + M]), _f64(torch.tensor(want).to(torch.bfloat16)))
    assert torch.all(Y[:4] == 7) and torch.all(Y[4 + M:] == 7)


@pytest.mark.parametrize("sizes", [[2, 0, 7, 3, 8], [1] * 30, [40, 0, 0, 1, 2, 0, 1, 1], [9, 20, 3], [16]])
def test_grouped_from_bf16(sizes):
    """bf16 activations quantized in the product's kernel or before it: the bits of the two separate calls."""
    dev = require_gpu()
    N, K, E, M = 200, 1184, len(sizes), sum(sizes)
    w = b.qlora_quantize_mx((0.02 * _rand((E * N, K), 2).float()).to(torch.bfloat16).to(dev), b.MX_E2M1)
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=dev)
    X = _rand((M, K), M, spread=3).to(dev)
    X[0, 40] = float("nan")
    for fmt in FORMATS:
        x = b.qlora_quantize_mx(X, fmt)
        Y, Q = b.qlora_mx_grouped_fwd(X, w, off, x_format=fmt), b.qlora_mx_grouped_fwd(x, w, off)
        _done()
        assert torch.isnan(Y[0]).all() and torch.isnan(Q[0]).all()
        assert torch.equal(Y[1:], Q[1:])
        xv, wv = _f64(b.qlora_dequantize_mx(x)), _f64(b.qlora_dequantize_mx(w))
        for e in range(E):
            a, c = max(1, int(off[e])), int(off[e + 1])
            if c > a:
                _check_product(Y[a:c], xv[a:c], wv[e * N:(e + 1) * N])


def test_grouped_equals_dense_by_group():
    dev = require_gpu()
    sizes, N, K = [3, 0, 70, 257], 384, 1056
    E, M = len(sizes), sum(sizes)
    X = _rand((M, K), 1).to(dev)
    W = (0.02 * _rand((E * N, K), 2).float()).to(torch.bfloat16).to(dev)
    w = b.qlora_quantize_mx(W, b.MX_E2M1)
    off = torch.tensor([0, 3, 3, 73, 330], dtype=torch.int32, device=dev)
    Y = b.qlora_mx_grouped_fwd(X, w, off)
    _done()
    Xv, Wv = _f64(b.qlora_dequantize_mx(b.qlora_quantize_mx(X, b.MX_E4M3))), _f64(b.qlora_dequantize_mx(w))
    for e in range(E):
        a, c = int(off[e]), int(off[e + 1])
        if c > a:
            _check_product(Y[a:c], Xv[a:c], Wv[e * N:(e + 1) * N])


# ---- together ----

def test_merged_weight_to_mx_serving():
    """NF4 base and adapter merged, the result quantized to MX, a norm in front: the path of a served layer."""
    dev = require_gpu()
    N, K, r, M = 384, 512, 16, 21
    W = (0.02 * _rand((N, K), 1).float()).to(torch.bfloat16).to(dev)
    A, B = (0.02 * _rand((r, K), 2).float()).to(torch.bfloat16), (0.02 * _rand((N, r), 3).float()).to(torch.bfloat16)
    merged = b.qlora_merge_lora(b.qlora_quantize_nf4_dq(W), [(A.to(dev), B.to(dev), 16.0, 1.0)])
    w = b.qlora_quantize_mx(merged, b.MX_E2M1)
    X, R, g = _rand((M, K), 4).to(dev), _rand((M, K), 5).to(dev), torch.ones(K, dtype=torch.bfloat16, device=dev)
    x, h = b.qlora_rmsnorm_mx(X, g, 1e-5, residual=R)
    Y = b.qlora_mx_linear_fwd(x, w)
    off = torch.tensor([0, 9, 9, M], dtype=torch.int32, device=dev)
    w3 = b.qlora_quantize_mx(merged[:384].contiguous(), b.MX_E2M1)   # 3 experts of 128
    G = b.qlora_mx_grouped_fwd(x, w3, off)
    _done()
    xv, wv = _f64(b.qlora_dequantize_mx(x)), _f64(b.qlora_dequantize_mx(w))
    _check_norm(x, mx.rmsnorm(_f64(h), np.ones(K), float(np.float32(1e-5))))
    _check_product(Y, xv, wv)
    _check_product(G[:9], xv[:9], wv[:128])
    _check_product(G[9:], xv[9:], wv[256:])


def test_another_stream_and_repeatability():
    dev = require_gpu()
    X = _rand((70, 1056), 1).to(dev)
    w = b.qlora_quantize_mx((0.02 * _rand((3 * 130, 1056), 2).float()).to(torch.bfloat16).to(dev), b.MX_E2M1)
    g = torch.ones(1056, dtype=torch.bfloat16, device=dev)
    off = torch.tensor([0, 20, 21, 70], dtype=torch.int32, device=dev)

    def chain(stream=None):
        n, h = b.qlora_rmsnorm_mx(X, g, 1e-5, residual=X, stream=stream)
        return (b.qlora_mx_linear_fwd(n, w, stream=stream), b.qlora_mx_grouped_fwd(X, w, off, stream=stream),
                b.qlora_dequantize_mx(n, stream=stream), h)

    want = chain()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    many = [(chain(s1), chain(s2)) for _ in range(10)]  # two streams at once
    _done()
    for pair in many:
        for got in pair:
            assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_captured_and_replayed_with_new_inputs():
    dev = require_gpu()
    M, K, N, E = 48, 640, 130, 4
    X = torch.zeros(M, K, dtype=torch.bfloat16, device=dev)
    R = torch.zeros_like(X)
    g = (1 + 0.1 * _rand((K,), 9).float()).to(torch.bfloat16).to(dev)
    w = b.qlora_quantize_mx((0.02 * _rand((E * N, K), 2).float()).to(torch.bfloat16).to(dev), b.MX_E2M1)
    off = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    Y = torch.zeros(M, N, dtype=torch.bfloat16, device=dev)
    D = torch.zeros(M, E * N, dtype=torch.bfloat16, device=dev)
    F = torch.zeros(8, E * N, dtype=torch.bfloat16, device=dev)

    def step():
        x, h = b.qlora_rmsnorm_mx(X, g, 1e-5, residual=R)
        b.qlora_mx_grouped_fwd(x, w, off, Y=Y)
        b.qlora_mx_linear_fwd(h, w, Y=D)          # quantized into a workspace of the graph
        b.qlora_mx_linear_fwd(h[:8], w, Y=F)      # quantized in the product's kernel
        return x, h

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, sizes in ((1, [10, 0, 30, 8]), (2, [0, 0, 48, 0]), (3, [1, 1, 1, 1])):
        X.copy_(_rand((M, K), seed))
        R.copy_(_rand((M, K), seed + 10))
        off.copy_(torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32))
        Y.fill_(3.0)
        graph.replay()
        _done()
        gotY, gotD, gotF = Y.clone(), D.clone(), F.clone()
        Y.fill_(3.0)
        step()
        _done()
        assert torch.equal(gotY, Y) and torch.equal(gotD, D) and torch.equal(gotF, F)
        assert torch.all(Y[sum(sizes):] == 3)
    del graph


def test_persistent_tiles_on_two_streams_and_replayed():
    """Grids of one CTA (or pair) per SM, twice at once, and in a graph whose offsets change between replays, to ones
    that leave most CTAs without a tile too."""
    dev = require_gpu()
    M, N, K, E = 900, 2600, 288, 8
    W = (0.02 * _rand((E * N, K), 2).float()).to(torch.bfloat16).to(dev)
    X, X2 = _rand((M, K), 3).to(dev), _rand((3 * M, K), 4).to(dev)
    w = b.qlora_quantize_mx(W, b.MX_E2M1)
    x = b.qlora_quantize_mx(X, b.MX_E4M3)    # 113 rows a group: single CTAs
    x2 = b.qlora_quantize_mx(X2, b.MX_E4M3)  # 338: pairs
    cuts = [[100, 100, 100, 100, 200, 100, 100, 100], [900, 0, 0, 0, 0, 0, 0, 0], [0] * 8, [1, 0, 500, 3, 0, 0, 0, 300]]
    offs = [torch.tensor(np.concatenate([[0], np.cumsum(c)]), dtype=torch.int32, device=dev) for c in cuts]
    fill = lambda m: torch.full((m, N), 5.0, dtype=torch.bfloat16, device=dev)  # noqa: E731
    want = []
    for off, c in zip(offs, cuts):
        y, y2 = fill(M), fill(3 * M)
        for e in range(E):  # the dense product of the group's rows: other tiles and orders of the sum
            r = slice(int(off[e]), int(off[e + 1]))
            if c[e]:
                we = b.qlora_quantize_mx(W[e * N:(e + 1) * N], b.MX_E2M1)
                y[r] = b.qlora_mx_linear_fwd(b.qlora_quantize_mx(X[r], b.MX_E4M3), we)
                y2[r] = b.qlora_mx_linear_fwd(b.qlora_quantize_mx(X2[r], b.MX_E4M3), we)
        want.append((y, y2))
    _done()
    # the fp32 sums of 288 terms, sum of magnitudes under 12, differ by at most 2 * 288 * 2^-24 * 12; a step of bf16 more
    close = lambda a, c: torch.allclose(a.float(), c.float(), rtol=2.0 ** -7, atol=576 * 12 * 2.0 ** -24)  # noqa: E731
    got = []
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for off in offs:
        ys = fill(M), fill(3 * M), fill(M), fill(3 * M)
        torch.cuda.synchronize()
        for s, (p, p2) in ((s1, ys[:2]), (s2, ys[2:])):
            b.qlora_mx_grouped_fwd(x, w, off, Y=p, stream=s)
            b.qlora_mx_grouped_fwd(x2, w, off, Y=p2, stream=s)
        _done()
        assert torch.equal(ys[0], ys[2]) and torch.equal(ys[1], ys[3])
        got.append(ys[:2])
    for (a, a2), (c, c2) in zip(got, want):
        assert close(a, c) and close(a2, c2)
    off, y, y2 = offs[0].clone(), fill(M), fill(3 * M)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.qlora_mx_grouped_fwd(x, w, off, Y=y)
        b.qlora_mx_grouped_fwd(x2, w, off, Y=y2)
    for o, (a, a2) in zip(offs, got):
        off.copy_(o)
        y.fill_(5.0)
        y2.fill_(5.0)
        graph.replay()
        _done()
        assert torch.equal(y, a) and torch.equal(y2, a2)
    del graph


def test_empty_calls():
    dev = require_gpu()
    w = b.qlora_quantize_mx(torch.zeros(64, 64, dtype=torch.bfloat16, device=dev), b.MX_E2M1)
    X = torch.zeros(0, 64, dtype=torch.bfloat16, device=dev)
    assert b.qlora_mx_linear_fwd(X, w).shape == (0, 64)
    off = torch.zeros(3, dtype=torch.int32, device=dev)
    assert b.qlora_mx_grouped_fwd(X, w, off).shape == (0, 32)
    q, h = b.qlora_rmsnorm_mx(X, torch.zeros(64, dtype=torch.bfloat16, device=dev), 1e-5, residual=X)
    assert b.qlora_dequantize_mx(q).shape == (0, 64) and h.shape == (0, 64)
    _done()

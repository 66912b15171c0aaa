"""CPU checks of the MX calls: the oracle against its definition, storage sizes,
and every refusal of the C entry points and of the binding. Nothing is launched."""
from __future__ import annotations

import ctypes
import sys
import threading

import numpy as np
import pytest
import torch

from bit_nf4_quantized_absmax_b200 import binding as b
from oracle import mx


def test_oracle_element_values():
    assert mx.MAGNITUDES[mx.E2M1].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    t = mx.MAGNITUDES[mx.E4M3]
    assert t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and t[-1] == 448 and len(t) == 127
    ours = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ours)


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
def test_oracle_rounding(fmt):
    """Every element value encodes to itself, midpoints go to the even code, and random values to a nearest one."""
    t = mx.MAGNITUDES[fmt]
    assert np.array_equal(mx.encode(t, fmt), np.arange(len(t)))
    mid = (t[:-1] + t[1:]) / 2
    assert np.all(mx.encode(mid, fmt) % 2 == 0)
    rng = np.random.default_rng(0)
    v = rng.normal(size=2000) * t[-1] / 2
    got = mx.decode(mx.encode(v, fmt), fmt)
    both = np.concatenate([-t, t])
    best = np.abs(np.clip(v, -t[-1], t[-1])[:, None] - both).min(1)
    assert np.array_equal(np.abs(np.clip(v, -t[-1], t[-1]) - got), best)
    assert mx.encode(np.array([1e9, -1e9]), fmt).tolist() == [len(t) - 1, len(t) - 1 + mx.SIGN[fmt]]


@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E2M1])
def test_oracle_blocks(fmt):
    """Quantizing decoded values gives them back, a block's largest value keeps its binade, a zero block has byte 0 and
    a block with an infinity or NaN decodes to NaN."""
    rng = np.random.default_rng(1)
    x = rng.normal(size=(4, 96)) * 2.0 ** rng.integers(-30, 30, size=(4, 96))
    x[0, :32] = 0.0
    codes, sc = mx.quantize(x, fmt)
    v = mx.dequantize(codes, sc, fmt)
    assert sc[0, 0] == 0 and not v[0, :32].any()
    c2, s2 = mx.quantize(v, fmt)
    assert np.array_equal(mx.dequantize(c2, s2, fmt), v)
    big = np.abs(x).reshape(4, 3, 32).max(-1)
    kept = np.abs(v).reshape(4, 3, 32).max(-1)
    assert np.all(kept <= 2 * big) and np.all(kept >= big * 0.75 - 1e-300)  # 6 / 8: saturation takes a quarter at most
    x[1, 33], x[2, 64] = np.nan, -np.inf
    v = mx.dequantize(*mx.quantize(x, fmt), fmt)
    assert np.isnan(v[1, 32:64]).all() and np.isnan(v[2, 64:]).all() and np.isfinite(v[0]).all()
    d, s = mx.pack(codes, sc, fmt)
    got = mx.unpack(d, s, 4, 96, fmt)
    assert np.array_equal(got[0], codes) and np.array_equal(got[1], sc)
    assert s.shape == (1, 4, 4) and np.all(s[0, :, 3] == 127)


def test_storage_bytes():
    assert b.qlora_mx_storage_bytes(b.MX_E2M1, 11008, 4096) == (11008 * 2048, 11008 * 128)
    assert b.qlora_mx_storage_bytes(b.MX_E4M3, 3, 160) == (3 * 256, 3 * 8)  # rows padded to 256 columns
    assert b.qlora_mx_storage_bytes(b.MX_E4M3, 0, 32) == (0, 0)
    for args, status in (((7, 4, 64), 2), ((0, 4, 48), 2), ((0, -1, 64), 1), ((0, 4, 0), 1), ((0, 1 << 31, 64), 2),
                         ((0, 4, (1 << 30) + 32), 2)):
        with pytest.raises(b.QloraError) as e:
            b.qlora_mx_storage_bytes(*args)
        assert e.value.status == status, args
    assert b.load_library().qlora_mx_storage_bytes(0, 4, 64, None) == 1


P = 1 << 20  # an aligned non-null dummy


def _mx(rows=8, cols=128, fmt=b.MX_E4M3, data=P, scales=P):
    return b._MX(data, scales, rows, cols, fmt)


def test_refusals_of_the_c_calls():
    """Each returns its status before anything is launched (there is no device here: a call that got further would
    return QLORA_ERR_CUDA)."""
    lib = b.load_library()
    ok = _mx()
    bad = [(_mx(rows=-1), 1), (_mx(cols=0), 1), (_mx(cols=48), 2), (_mx(fmt=2), 2), (_mx(fmt=-1), 2),
           (_mx(rows=1 << 31), 2), (_mx(data=None), 1), (_mx(scales=None), 1), (_mx(data=P + 16), 3),
           (_mx(scales=P + 2), 3)]
    w = _mx(rows=64, fmt=b.MX_E2M1)
    for q, status in bad:
        r = ctypes.byref(q)
        assert lib.qlora_quantize_mx(P, r, None) == status
        assert lib.qlora_dequantize_mx(r, P, None) == status
        assert lib.qlora_rmsnorm_mx(P, None, P, 1e-5, r, None, None) == status
        assert lib.qlora_mx_linear_fwd(r, ctypes.byref(w), P, None) == status
        assert lib.qlora_mx_grouped_fwd(r, ctypes.byref(w), P, 4, P, None) == status
        if q.format != b.MX_E4M3 or status != 2:
            continue
        assert lib.qlora_mx_linear_fwd(ctypes.byref(ok), r, P, None) == status
    r, rw = ctypes.byref(ok), ctypes.byref(w)
    assert lib.qlora_quantize_mx(P, None, None) == 1
    assert lib.qlora_quantize_mx(None, r, None) == 1
    assert lib.qlora_quantize_mx(P + 8, r, None) == 3
    assert lib.qlora_dequantize_mx(r, None, None) == 1
    assert lib.qlora_dequantize_mx(r, P + 2, None) == 3
    norm = lib.qlora_rmsnorm_mx
    assert norm(P, None, P, -1e-5, r, None, None) == 1
    assert norm(P, None, P, float("nan"), r, None, None) == 1
    assert norm(None, None, P, 1e-5, r, None, None) == 1
    assert norm(P, None, None, 1e-5, r, None, None) == 1
    assert norm(P, P, P, 1e-5, r, None, None) == 1             # a residual needs residual_out
    assert norm(P, P, P, 1e-5, r, P + 8, None) == 3
    assert norm(P, P + 4, P, 1e-5, r, P, None) == 3
    assert norm(P, None, P, 1e-5, ctypes.byref(_mx(cols=32768 + 32)), None, None) == 2
    fwd, grp = lib.qlora_mx_linear_fwd, lib.qlora_mx_grouped_fwd
    assert fwd(r, r, P, None) == 2                              # the weight has to be E2M1
    assert fwd(r, ctypes.byref(_mx(rows=64, cols=256, fmt=b.MX_E2M1)), P, None) == 1
    assert fwd(r, ctypes.byref(_mx(rows=0, fmt=b.MX_E2M1)), P, None) == 1
    assert fwd(None, rw, P, None) == 1 and fwd(r, None, P, None) == 1
    assert fwd(r, rw, None, None) == 1 and fwd(r, rw, P + 2, None) == 3
    assert grp(r, rw, None, 4, P, None) == 1
    assert grp(r, rw, P, 0, P, None) == 1
    assert grp(r, rw, P + 1, 4, P, None) == 3
    assert grp(r, rw, P, 4097, P, None) == 2
    assert grp(r, rw, P, 5, P, None) == 1                       # 64 rows are not 5 experts
    deep = (1 << 20) + 32
    assert fwd(ctypes.byref(_mx(cols=deep)), ctypes.byref(_mx(rows=64, cols=deep, fmt=b.MX_E2M1)), P, None) == 2
    many = _mx(rows=(1 << 31) - 1)
    assert fwd(ctypes.byref(many), ctypes.byref(_mx(rows=(1 << 31) - 1, fmt=b.MX_E2M1)), P, None) == 2
    # no rows: nothing to do, and the pointers are not looked at
    none = ctypes.byref(_mx(rows=0, data=None, scales=None))
    assert lib.qlora_quantize_mx(None, none, None) == 0 and lib.qlora_dequantize_mx(none, None, None) == 0
    assert norm(None, None, None, 1e-5, none, None, None) == 0
    assert fwd(none, rw, None, None) == 0 and grp(none, rw, P, 4, None, None) == 0


def test_refusals_and_workspace_of_the_quantizing_products():
    lib = b.load_library()
    w = _mx(rows=64, fmt=b.MX_E2M1)
    rw = ctypes.byref(w)

    def size(v=0):
        return ctypes.byref(ctypes.c_size_t(v))

    def need(M, fmt, groups=None):
        n = ctypes.c_size_t(0)
        st = lib.qlora_mx_linear_fwd_bf16(None, M, fmt, rw, None, None, ctypes.byref(n), None) if groups is None else \
            lib.qlora_mx_grouped_fwd_bf16(None, M, fmt, rw, P, groups, None, None, ctypes.byref(n), None)
        assert st == 0
        return n.value

    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    assert need(0, b.MX_E4M3) == 256 and need(16, b.MX_E4M3) == 256 and need(32, b.MX_E4M3, groups=4) == 256
    assert need(16, b.MX_E4M3, groups=1) == 256
    assert need(17, b.MX_E4M3) == up(17 * 128) + up(17 * 4)
    assert need(33, b.MX_E2M1, groups=4) == up(33 * 64) + up(33 * 4)
    lin, grp = lib.qlora_mx_linear_fwd_bf16, lib.qlora_mx_grouped_fwd_bf16
    big = 1 << 20
    assert lin(P, 4, 7, rw, P, P, size(big), None) == 2
    assert lin(P, -1, 0, rw, P, P, size(big), None) == 1
    assert lin(P, 1 << 31, 0, rw, P, P, size(big), None) == 2
    assert lin(P, 4, 0, None, P, P, size(big), None) == 1
    assert lin(P, 4, 0, ctypes.byref(_mx(rows=64)), P, P, size(big), None) == 2
    assert lin(P, 4, 0, ctypes.byref(_mx(rows=0, fmt=b.MX_E2M1)), P, P, size(big), None) == 1
    assert lin(None, 4, 0, rw, P, P, size(big), None) == 1
    assert lin(P, 4, 0, rw, None, P, size(big), None) == 1
    assert lin(P + 8, 4, 0, rw, P, P, size(big), None) == 3
    assert lin(P, 4, 0, rw, P + 8, P, size(big), None) == 3
    assert lin(P, 40, 0, rw, P, P + 128, size(big), None) == 3
    assert lin(P, 40, 0, rw, P, P, size(100), None) == 5
    assert lin(P, 40, 0, rw, P, P, None, None) == 1
    assert lin(None, 0, 0, rw, None, P, size(big), None) == 0
    assert grp(P, 4, 0, rw, None, 4, P, P, size(big), None) == 1
    assert grp(P, 4, 0, rw, P, 0, P, P, size(big), None) == 1
    assert grp(P, 4, 0, rw, P, 4097, P, P, size(big), None) == 2
    assert grp(P, 4, 0, rw, P + 2, 4, P, P, size(big), None) == 3
    assert grp(P, 4, 0, rw, P, 5, P, P, size(big), None) == 1
    assert grp(None, 0, 0, rw, P, 4, None, P, size(big), None) == 0


def _tensors(rows, cols, fmt, device="cpu"):
    return b.MXTensor.empty(rows, cols, fmt, device)


def test_refusals_of_the_binding():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError):
        b.MXTensor.empty(4, 48, b.MX_E4M3, "cpu")
    with pytest.raises(ValueError):
        b.MXTensor.empty(4, 64, 5, "cpu")
    d, s = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8)
    b.MXTensor(d, s, 4, 64, b.MX_E4M3)
    for bad in ((d[:, :64], s), (d.to(torch.int8), s), (d, s[:, :2].contiguous()), (d[:3], s), (d.t(), s)):
        with pytest.raises(ValueError):
            b.MXTensor(*bad, 4, 64, b.MX_E4M3)
    w = _tensors(64, 128, b.MX_E2M1)
    x = _tensors(4, 128, b.MX_E4M3)
    calls = [
        lambda: b.qlora_quantize_mx(bf(4, 128).float(), b.MX_E4M3),
        lambda: b.qlora_quantize_mx(bf(4, 256)[:, ::2], b.MX_E4M3),
        lambda: b.qlora_quantize_mx(bf(128), b.MX_E4M3),
        lambda: b.qlora_quantize_mx(bf(4, 100), b.MX_E4M3),
        lambda: b.qlora_quantize_mx(bf(4, 128), b.MX_E4M3, out=w),
        lambda: b.qlora_quantize_mx(bf(4, 128), b.MX_E4M3),                    # not on a GPU
        lambda: b.qlora_dequantize_mx(x, out=bf(4, 64)),
        lambda: b.qlora_dequantize_mx(x),
        lambda: b.qlora_rmsnorm_mx(bf(4, 128), bf(64), 1e-5),
        lambda: b.qlora_rmsnorm_mx(bf(4, 128), bf(128), 1e-5, residual=bf(3, 128)),
        lambda: b.qlora_rmsnorm_mx(bf(4, 128), bf(128), 1e-5, residual=bf(4, 128), residual_out=bf(4, 64)),
        lambda: b.qlora_rmsnorm_mx(bf(4, 128), bf(128), 1e-5, out=w),
        lambda: b.qlora_mx_linear_fwd(_tensors(4, 64, b.MX_E4M3), w),
        lambda: b.qlora_mx_linear_fwd(x, w, Y=bf(4, 32)),
        lambda: b.qlora_mx_linear_fwd(x, w),
        lambda: b.qlora_mx_grouped_fwd(x, w, torch.zeros(5)),
        lambda: b.qlora_mx_grouped_fwd(x, w, torch.zeros(1, dtype=torch.int32)),
        lambda: b.qlora_mx_grouped_fwd(x, w, torch.zeros(6, dtype=torch.int32)),
        lambda: b.qlora_mx_grouped_fwd(x, w, torch.zeros(10, dtype=torch.int32)[::2]),
    ]
    class OtherStream:
        device = torch.device("cuda:7")

    other = OtherStream()
    calls += [  # a stream of another device than the tensors'
        lambda: b.qlora_quantize_mx(bf(4, 128), b.MX_E4M3, stream=other),
        lambda: b.qlora_dequantize_mx(x, stream=other),
        lambda: b.qlora_rmsnorm_mx(bf(4, 128), bf(128), 1e-5, stream=other),
        lambda: b.qlora_mx_linear_fwd(x, w, stream=other),
        lambda: b.qlora_mx_grouped_fwd(x, w, torch.zeros(5, dtype=torch.int32), stream=other),
    ]
    for k, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was not refused")


def test_storage_views_asked_for_by_several_threads():
    """`data` and `scales` of a result are views that the first access makes; any thread may be that one."""
    failures = []

    def look(q, at, start):
        start.wait()
        try:
            assert q.data.shape == (2, 128) and q.scales.shape == (1, 2, 4)
            assert q.data.data_ptr() == at and q.scales.data_ptr() == at + 256
        except BaseException as e:  # noqa: BLE001
            failures.append(repr(e))

    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for _ in range(400):
            q = _tensors(2, 32, b.MX_E4M3)
            start = threading.Barrier(4)
            threads = [threading.Thread(target=look, args=(q, q.as_c().data, start)) for _ in range(4)]
            for t in threads:
                t.start()
            for t in threads:
                t.join()
    finally:
        sys.setswitchinterval(interval)
    assert not failures, (len(failures), failures[0])


class _Reached(Exception):
    """A call got past the binding's checks."""


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _offsets(*v):
    return torch.tensor(v, dtype=torch.int32)


class _StreamOfAnotherDevice:
    device = torch.device("cuda:7")


def _accepted():
    """Calls that pass every check of the binding but that of the device's type."""
    w, x = _tensors(64, 128, b.MX_E2M1), _tensors(4, 128, b.MX_E4M3)
    return {
        "quantize": lambda **k: b.qlora_quantize_mx(**{"X": _bf(4, 128), "format": b.MX_E4M3, **k}),
        "dequantize": lambda **k: b.qlora_dequantize_mx(**{"q": x, **k}),
        "norm": lambda **k: b.qlora_rmsnorm_mx(**{"X": _bf(4, 128), "gamma": _bf(128), "eps": 1e-5, **k}),
        "linear": lambda **k: b.qlora_mx_linear_fwd(**{"x": x, "w": w, **k}),
        "grouped": lambda **k: b.qlora_mx_grouped_fwd(**{"x": x, "w": w, "offsets": _offsets(0, 1, 2, 3, 4), **k}),
    }


_MATRIX, _OTHER = "contiguous bfloat16 matrix", "out has another shape, format or device"
_REFUSED = [
    ("quantize", lambda: {"X": _bf(4, 128).float()}, "X has to be a " + _MATRIX),
    ("quantize", lambda: {"X": _bf(4, 256)[:, ::2]}, "X has to be a " + _MATRIX),
    ("quantize", lambda: {"X": _bf(128, 4).t()}, "X has to be a " + _MATRIX),
    ("quantize", lambda: {"X": _bf(128)}, "X has to be a " + _MATRIX),
    ("quantize", lambda: {"X": _bf(1, 4, 128)}, "X has to be a " + _MATRIX),
    ("quantize", lambda: {"X": _bf(4, 100)}, "cols % 32 == 0"),
    ("quantize", lambda: {"format": 5}, "unknown MX format"),
    ("quantize", lambda: {"out": _tensors(3, 128, b.MX_E4M3)}, _OTHER),
    ("quantize", lambda: {"out": _tensors(4, 96, b.MX_E4M3)}, _OTHER),
    ("quantize", lambda: {"out": _tensors(4, 128, b.MX_E2M1)}, _OTHER),
    ("quantize", lambda: {"out": _tensors(4, 128, b.MX_E4M3, "meta")}, _OTHER),
    ("dequantize", lambda: {"out": _bf(4, 64)}, "out has to be a contiguous bfloat16 tensor of shape"),
    ("dequantize", lambda: {"out": _bf(3, 128)}, "out has to be"),
    ("dequantize", lambda: {"out": _bf(4, 128).half()}, "out has to be"),
    ("dequantize", lambda: {"out": _bf(4, 256)[:, ::2]}, "out has to be"),
    ("dequantize", lambda: {"out": _bf(4, 128).to("meta")}, "out has to be"),
    ("norm", lambda: {"X": _bf(4, 256)[:, ::2]}, "X has to be a " + _MATRIX),
    ("norm", lambda: {"gamma": _bf(64)}, "gamma has to be"),
    ("norm", lambda: {"gamma": _bf(1, 128)}, "gamma has to be"),
    ("norm", lambda: {"gamma": _bf(128).float()}, "gamma has to be"),
    ("norm", lambda: {"gamma": _bf(256)[::2]}, "gamma has to be"),
    ("norm", lambda: {"gamma": _bf(128).to("meta")}, "gamma has to be"),
    ("norm", lambda: {"residual": _bf(3, 128)}, "residual has to be"),
    ("norm", lambda: {"residual": _bf(4, 128).float()}, "residual has to be"),
    ("norm", lambda: {"residual": _bf(4, 128), "residual_out": _bf(4, 64)}, "residual_out has to be"),
    ("norm", lambda: {"residual": _bf(4, 128), "residual_out": _bf(4, 128).float()}, "residual_out has to be"),
    ("norm", lambda: {"out": _tensors(64, 128, b.MX_E4M3)}, _OTHER),
    ("norm", lambda: {"out": _tensors(4, 128, b.MX_E2M1)}, _OTHER),
    ("norm", lambda: {"X": _bf(4, 100), "gamma": _bf(100)}, "cols % 32 == 0"),
]
for _op in ("linear", "grouped"):
    _REFUSED += [
        (_op, lambda: {"x": _tensors(4, 64, b.MX_E4M3)}, "do not match a weight"),
        (_op, lambda: {"x": _tensors(4, 128, b.MX_E4M3, "meta")}, "do not match a weight"),
        (_op, lambda: {"x": _bf(4, 96)}, "do not match a weight"),
        (_op, lambda: {"x": _bf(4, 128).to("meta")}, "do not match a weight"),
        (_op, lambda: {"x": _bf(128)}, "x, where it is no MXTensor, has to be a " + _MATRIX),
        (_op, lambda: {"x": _bf(4, 128).float()}, "has to be a " + _MATRIX),
        (_op, lambda: {"x": _bf(4, 256)[:, ::2]}, "has to be a " + _MATRIX),
        (_op, lambda: {"Y": _bf(3, 64)}, "Y has to be"),
        (_op, lambda: {"Y": _bf(4, 32)}, "Y has to be"),
        (_op, lambda: {"Y": _bf(4, 16).float()}, "Y has to be"),
        (_op, lambda: {"Y": _bf(4, 128)[:, ::2]}, "Y has to be"),
    ]
_REFUSED += [
    ("linear", lambda: {"Y": _bf(4, 64).to("meta")}, "Y has to be"),
    ("grouped", lambda: {"Y": _bf(4, 16).to("meta")}, "Y has to be"),
    ("grouped", lambda: {"Y": _bf(4, 64)}, "Y has to be"),
    ("grouped", lambda: {"offsets": torch.zeros(5)}, "offsets have to be"),
    ("grouped", lambda: {"offsets": torch.zeros(5, dtype=torch.int64)}, "offsets have to be"),
    ("grouped", lambda: {"offsets": _offsets(0)}, "offsets have to be"),
    ("grouped", lambda: {"offsets": _offsets(0, 1, 2, 3, 4).view(1, 5)}, "offsets have to be"),
    ("grouped", lambda: {"offsets": _offsets(*range(10))[::2]}, "offsets have to be"),
    ("grouped", lambda: {"offsets": _offsets(0, 1, 2, 3, 4).to("meta")}, "offsets have to be"),
    ("grouped", lambda: {"offsets": _offsets(0, 1, 2, 3, 4, 4)}, "is not 5 experts of equal size"),
    ("grouped", lambda: {"w": _tensors(0, 128, b.MX_E2M1)}, "is not 4 experts of equal size"),
]
_REFUSED += [(_op, lambda: {"stream": _StreamOfAnotherDevice()}, "the stream is of cuda:7")
             for _op in ("quantize", "dequantize", "norm", "linear", "grouped")]


@pytest.mark.parametrize("k", range(len(_REFUSED)))
def test_each_refusal_of_the_binding_by_its_message(k, monkeypatch):
    """The C calls get bare addresses, so the binding's checks are all that keeps a wrong shape from being read or written
    out of range. Each is met with its own message, before anything reaches the library."""
    def reached(*a):
        raise _Reached()

    monkeypatch.setattr(b, "_mx_run", reached)
    op, args, message = _REFUSED[k]
    with pytest.raises(ValueError, match=message):
        _accepted()[op](**args())


@pytest.mark.parametrize("op", ["quantize", "dequantize", "norm", "linear", "grouped"])
def test_calls_without_a_fault_reach_the_library(op, monkeypatch):
    """The calls that the refusals start from are refused for the device's type alone."""
    with pytest.raises(ValueError, match="have to be on a CUDA device, not cpu"):
        _accepted()[op]()

    def reached(*a):
        raise _Reached()

    monkeypatch.setattr(b, "_mx_run", reached)
    with pytest.raises(_Reached):
        _accepted()[op]()
    more = {"quantize": {"out": _tensors(4, 128, b.MX_E4M3)}, "dequantize": {"out": _bf(4, 128)},
            "norm": {"residual": _bf(4, 128), "residual_out": _bf(4, 128), "out": _tensors(4, 128, b.MX_E4M3)},
            "linear": {"x": _bf(4, 128), "Y": _bf(4, 64)}, "grouped": {"x": _bf(4, 128), "Y": _bf(4, 16)}}
    with pytest.raises(_Reached):
        _accepted()[op](**more[op])

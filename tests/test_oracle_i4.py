"""Pins of the 4-bit oracle, and the refusals of the decode entry points (no GPU)."""
import ctypes
import os
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

import mixture_experts_layer_02_amd as moe
import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
G = 1 << 20  # an aligned address; nothing is launched


def test_codes_are_the_exact_quotients():
    rng = np.random.default_rng(0)
    rows = [rng.normal(0, 1, 64).astype(np.float32) for _ in range(40)]
    for m in (np.float32(14.0), np.float32(7 * 2.0 ** -20), np.float32(1.7), np.float32(3e-39), np.float32(3e38)):
        n = rng.integers(-6, 6, 20)
        v = ((n + 0.5) / 7.0 * np.float64(m)).astype(np.float32)          # at, just below and just above a tie
        rows.append(np.concatenate([v, np.nextafter(v, np.float32(-3e38)), np.nextafter(v, np.float32(3e38)),
                                    [m, -m, 0, 0]]).astype(np.float32))
    w = np.stack(rows)
    codes, scale = oracle.i4_quantize(w, 32)
    for r in range(len(rows)):
        for j in range(2):
            v = w[r, 32 * j:32 * j + 32]
            m = np.abs(v).max()
            assert scale[r, j] == np.float32(m) / np.float32(7)
            for c in range(32):
                assert codes[r, 32 * j + c] == round(Fraction(float(v[c])) * 7 / Fraction(float(m))), (r, j, c)


def test_error_is_half_a_step_and_short_groups_are_their_own():
    rng = np.random.default_rng(1)
    w = rng.normal(0, 3, (50, 200)).astype(np.float32)
    codes, scale = oracle.i4_quantize(w, 64)
    assert scale.shape == (50, 4)
    assert (np.abs(codes[:, 192:].astype(int)).max(axis=1) == 7).all()
    err = np.abs(oracle.i4_dequantize(codes, scale, 64) - w.astype(np.float64))
    step = np.repeat(scale.astype(np.float64), 64, axis=1)[:, :200]
    assert (err <= step * (0.5 + 7 * 2.0 ** -23)).all()


def test_zero_and_not_finite_groups():
    w = np.zeros((4, 64), np.float32)
    w[1, 3], w[2, 40], w[3, 10], w[3, 50] = np.inf, np.nan, 2.0, -1.0
    codes, scale = oracle.i4_quantize(w, 32)
    assert scale[0].tolist() == [0, 0] and np.isnan(scale[1, 0]) and scale[1, 1] == 0 and np.isnan(scale[2, 1])
    assert (codes[:3] == 0).all() and codes[3, 10] == 7 and codes[3, 50] == -7


def test_packing_by_hand_and_back():
    q = oracle.i4_pack(np.array([[-8, -7, -6, -5, -4, -3, -2, -1]]))
    assert q.tolist() == [[0x20, 0x64, 0x31, 0x75]]          # nibbles 0 2 | 4 6 | 1 3 | 5 7, low ones first
    rng = np.random.default_rng(2)
    c = rng.integers(-8, 8, (5, 72))
    assert (oracle.i4_unpack(oracle.i4_pack(c)) == c).all()


def test_linear_by_hand():
    codes = np.zeros((2, 40), int)
    codes[0, 0], codes[0, 33], codes[1, 39] = 3, -2, 7
    x = np.zeros((1, 40))
    x[0, 0], x[0, 33], x[0, 39] = 2.0, 5.0, -1.0
    y = oracle.i4_linear(x, codes, [[0.5, 2.0], [1.0, 0.25]], 32, [1.0, -1.0])
    np.testing.assert_array_equal(y, [[3.0 - 20.0 + 1.0, -1.75 - 1.0]])


def test_library_exports_every_declared_symbol():
    with open(os.path.join(ROOT, "include", "moe_decode.h")) as fh:
        names = sorted(set(re.findall(r"^\s*int\s+(moe_\w+)\s*\(", fh.read(), re.M)))
    assert names == moe.EXPORTS_DECODE
    for n in names:
        assert hasattr(moe.lib(), n), n


def _quant(**kw):
    a = dict(w=G, dtype=moe.MOE_BF16, rows=4, cols=64, ldw=64, group=32, q=G, ldq=32, scale=G, lds=2)
    a.update(kw)
    l = moe.lib()
    back = l.moe_i4_dequantize(a["q"], a["ldq"], a["scale"], a["lds"], a["rows"], a["cols"], a["group"], a["w"],
                               a["dtype"], a["ldw"], None)
    there = l.moe_i4_quantize(a["w"], a["dtype"], a["rows"], a["cols"], a["ldw"], a["group"], a["q"], a["ldq"],
                              a["scale"], a["lds"], None)
    assert there == back
    return there


BAD, NOT = -1, -2


@pytest.mark.parametrize("kw,rc", [
    (dict(w=None), BAD), (dict(w=G + 8), BAD), (dict(q=None), BAD), (dict(q=G + 4), BAD), (dict(scale=None), BAD),
    (dict(scale=G + 2), BAD), (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(cols=60, ldw=60), BAD),
    (dict(ldw=63), BAD), (dict(ldq=28), BAD), (dict(ldq=34), BAD), (dict(lds=1), BAD), (dict(group=16), NOT),
    (dict(group=0), NOT), (dict(group=-32), NOT), (dict(dtype=2), NOT), (dict(cols=2 ** 28 + 8, ldw=2 ** 29, ldq=2 ** 28), NOT),
    (dict(rows=0), 0)])
def test_quantiser_refusals(kw, rc):
    assert _quant(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), BAD), (dict(x=G + 2), BAD), (dict(wq=None), BAD), (dict(wq=G + 8), BAD), (dict(ws=None), BAD),
    (dict(ws=G + 1), BAD), (dict(bias=G + 4), BAD), (dict(y=None), BAD), (dict(M=-1), BAD), (dict(N=0), BAD), (dict(K=0), BAD),
    (dict(K=60), BAD), (dict(ldx=56), BAD), (dict(ldx=68), BAD), (dict(ldw=16), BAD), (dict(ldw=40), BAD), (dict(lds=1), BAD),
    (dict(ldy=15), BAD), (dict(group=256), NOT), (dict(group=0), NOT), (dict(dtype=3), NOT),
    (dict(K=2 ** 20 + 8, ldx=2 ** 21, ldw=2 ** 20, lds=2 ** 16), NOT), (dict(ldx=2 ** 21 + 8), NOT), (dict(ldw=2 ** 21 + 16), NOT),
    (dict(lds=2 ** 21 + 1), NOT), (dict(M=2 ** 31 - 256), NOT), (dict(N=2 ** 31 - 256, ldy=2 ** 31), NOT), (dict(M=0), 0)])
def test_linear_refusals(kw, rc):
    a = dict(M=3, N=16, K=64, group=32, x=G, ldx=64, wq=G, ldw=32, ws=G, lds=2, bias=None, y=G, ldy=16, dtype=moe.MOE_F32)
    a.update(kw)
    assert moe.lib().moe_i4_linear(*[a[n] for n in ("M", "N", "K", "group", "x", "ldx", "wq", "ldw", "ws", "lds", "bias",
                                                    "y", "ldy", "dtype")], None) == rc


def _desc(**kw):
    return moe.make_desc(**{**dict(T=4, d=128, f=64, E=8, k=2, dtype=moe.MOE_BF16), **kw})


DECODE = ("n_groups", "x", "wr", "bias", "w1", "w3", "w2", "idx", "w", "y", "ws", "n")
DECODE_I4 = ("group", "n_groups", "x", "wr", "bias", "w1", "s1", "w3", "s3", "w2", "s2", "idx", "w", "y", "ws", "n")


def _decode(desc, i4, **kw):
    a = {n: G for n in DECODE_I4}
    a.update(group=32, n_groups=1, bias=None, n=1 << 30)
    a.update(kw)
    name, args = ("moe_decode_i4", DECODE_I4) if i4 else ("moe_decode", DECODE)
    return getattr(moe.lib(), name)(ctypes.byref(desc), *[a[n] for n in args], None)


@pytest.mark.parametrize("i4", [False, True])
@pytest.mark.parametrize("kw,rc", [
    (dict(T=65), NOT), (dict(dtype=moe.MOE_F32), NOT), (dict(d=2 ** 20 + 64), NOT), (dict(f=2 ** 20 + 64), NOT), (dict(T=0), BAD),
    (dict(d=96), NOT), (dict(k=9), BAD)])
def test_decode_refuses_descriptors(i4, kw, rc):
    d = _desc(**kw)
    assert _decode(d, i4) == rc
    assert moe.lib().moe_decode_workspace_size(ctypes.byref(d), ctypes.byref(ctypes.c_size_t())) == rc
    with pytest.raises(moe.MoeError):
        moe.decode_workspace_size(d)


@pytest.mark.parametrize("i4", [False, True])
@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), BAD), (dict(x=G + 8), BAD), (dict(wr=G + 8), BAD), (dict(bias=G + 4), BAD), (dict(w1=None), BAD), (dict(w3=G + 2), BAD),
    (dict(w2=None), BAD), (dict(idx=None), BAD), (dict(w=G + 4), BAD), (dict(y=None), BAD), (dict(ws=None), BAD), (dict(ws=G + 8), -3),
    (dict(n=0), -3), (dict(n_groups=0), BAD), (dict(n_groups=3), BAD), (dict(n_groups=4), BAD), (dict(wr=None, bias=G), BAD),
    (dict(wr=None, n_groups=2), BAD)])
def test_decode_refuses_arguments(i4, kw, rc):
    assert _decode(_desc(), i4, **kw) == rc


def test_decode_i4_refuses_groups_and_scales():
    for kw, rc in ((dict(group=16), NOT), (dict(group=0), NOT), (dict(s1=None), BAD), (dict(s3=G + 8), BAD), (dict(s2=None), BAD)):
        assert _decode(_desc(), True, **kw) == rc
    assert moe.lib().moe_decode_workspace_size(ctypes.byref(_desc()), None) == BAD


def test_python_refuses_groups_and_host_tensors():
    w, q, s = torch.zeros(2, 64), torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 1)
    for group in (0, 16, -128):
        with pytest.raises(ValueError):
            moe.i4_linear(w.bfloat16(), q, s, w, group=group)
    with pytest.raises(ValueError):
        moe.i4_quantize(w, q, s)
    with pytest.raises(ValueError):
        moe.i4_linear(w.bfloat16(), q, s, torch.zeros(2, 2))

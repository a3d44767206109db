"""The 4-bit operators and the decode step of the layer on the GPU against the oracle in float64.

4-bit codes and scales match bit for bit.  With u = 2^-24 (float32) and U = 2^-8
(bf16, 0 for float32), and c(K) = K/8 + 64 + 128 the longest chain of additions of a
product over K (a wave's share, the waves, a group of 128), each off by at most
2 u of the terms' magnitudes:
  linear  the codes are multiplied as 24 + q and 24 times the row's sum taken off, so
          the terms of k are |x| s (|24 + q| + 24) <= 56 |x| s:
          2 c u sum(56 |x| s) + 4 u |b| + U |y|.  Where x, scales and bias are whole
          numbers times powers of two, every sum is exact, and so is y up to U.
  decode  G and U': 2 c u sum(|x||W|) (4 bits: 56 |x| s in place of |x||W|), E_G and E_U;
          h: silu is 1.1-Lipschitz: E_h = 1.1 |U'| E_G + |silu(G)| E_U + (13 + 4 |G|) 2 u |h|
          and U |h| for its rounding; y: the sum over the slots of w (|W2| (E_h + U |h|) +
          2 c u |W2||h|), 8 u w for the weights' rounding and their E_w, and U |y|.
  topk_w  the logits are off by E_L = 2 c u sum(|x||Wr|) + u |b|, a weight by w (2 max E_L + 16 u).
Bounds are on each value, doubled in their float32 part for second-order terms.
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_02_amd as moe
import oracle
import synth
from gpu_util import to_host
from launched import kernels

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8


def _chain(K):
    return K / 8 + 64 + 128


def _bf(a):
    """a rounded to bf16, as float32."""
    return synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(np.asarray(a, np.float32)))


def _dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)


def _dev_rows(a, ld, dtype, fill):
    """Rows of a on the GPU, ld elements apart, `fill` in between."""
    t = torch.full((a.shape[0], ld), fill, dtype=dtype, device="cuda")
    t[:, :a.shape[1]] = torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)
    return t


def _within(got, want, f32_part, bf16):
    got = np.asarray(got, np.float64)
    assert np.isfinite(got).all()
    bound = 2 * f32_part + (UBF if bf16 else U32) * np.abs(want) + 2.0 ** -120
    bad = np.abs(got - want) > bound
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - want) / bound).max()), np.argwhere(bad)[:4].tolist())


# ---------------------------------------------------------------- quantiser

def _special_rows(cols, dtype, seed):
    rng = np.random.default_rng(seed)
    w = rng.normal(0, 1, (20, cols)).astype(np.float32)
    w[1] = 0.0
    w[2] = -0.0
    w[3] = 0.0
    w[3, cols // 2] = -0.25
    w[4] *= 1e-38                                     # 7 / max overflows; subnormal values among them
    w[5] *= 1e-41
    w[6] *= 1e38 / 5
    w[7, cols - 1] = np.inf
    w[8, 0] = np.nan
    w[9, cols // 3] = -np.inf
    for r, m in ((10, 14.0), (11, 7 * 2.0 ** -30), (12, 1.7), (13, 3e-39), (14, 3e38), (15, 255.0), (16, 1.9921875)):
        n = rng.integers(-6, 6, cols)
        v = ((n + 0.5) / 7.0 * m).astype(np.float32)            # ties and their neighbours
        v = np.where(np.arange(cols) % 3 == 1, np.nextafter(v, np.float32(-3.4e38)), v)
        v = np.where(np.arange(cols) % 3 == 2, np.nextafter(v, np.float32(3.4e38)), v)
        w[r] = np.clip(v, -m, m)
        w[r, ::32] = m
    return _bf(w) if dtype == "bf16" else w


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("cols,ldw,ldq,lds", [(8, 8, 4, 1), (40, 41, 20, 2), (128, 128, 64, 4), (200, 208, 112, 9),
                                              (1000, 1004, 500, 32), (1792, 1792, 896, 56), (2056, 2056, 1028, 70)])
def test_quantise_and_back_match_the_oracle(gpu, dtype, group, cols, ldw, ldq, lds):
    w = _special_rows(cols, dtype, cols + group)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    wd = _dev_rows(w, ldw, tdt, 1e30)
    groups = -(-cols // group)
    q = torch.full((20, ldq), 77, dtype=torch.uint8, device=gpu)
    s = torch.full((20, lds), -1.0, device=gpu)
    moe.i4_quantize(wd[:, :cols], q[:, :cols // 2], s[:, :groups], group)
    codes, scale = oracle.i4_quantize(w, group)
    np.testing.assert_array_equal(s[:, :groups].cpu().numpy(), scale)
    np.testing.assert_array_equal(q[:, :cols // 2].cpu().numpy(), oracle.i4_pack(codes))
    assert (q[:, cols // 2:] == 77).all() and (s[:, groups:] == -1).all()
    for odt in (torch.float32, torch.bfloat16):
        out = torch.full((20, ldw), 5.0, dtype=odt, device=gpu)
        moe.i4_dequantize(q[:, :cols // 2], s[:, :groups], out[:, :cols], group)
        want = (codes.astype(np.float32) * np.repeat(scale, group, axis=1)[:, :cols]).astype(np.float32)
        np.testing.assert_array_equal(to_host(out[:, :cols].contiguous()), want if odt == torch.float32 else _bf(want))
        assert (out[:, cols:] == 5.0).all()


@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 6144), (70000, 136), (17, 100000)])
def test_quantise_of_many_and_long_rows(gpu, rows, cols):
    g = torch.Generator(device="cuda").manual_seed(rows)
    w = torch.randn(rows, cols, generator=g, device=gpu).bfloat16()
    q = torch.empty(rows, cols // 2, dtype=torch.uint8, device=gpu)
    s = torch.empty(rows, -(-cols // 128), device=gpu)
    moe.i4_quantize(w, q, s)
    pick = sorted({0, rows // 2, rows - 1})
    codes, scale = oracle.i4_quantize(to_host(w[pick]), 128)
    np.testing.assert_array_equal(s[pick].cpu().numpy(), scale)
    np.testing.assert_array_equal(q[pick].cpu().numpy(), oracle.i4_pack(codes))


def test_quantise_no_rows_and_past_32_bit_offsets(gpu):
    e = torch.empty(0, 64, device=gpu)
    moe.i4_quantize(e, torch.empty(0, 32, dtype=torch.uint8, device=gpu), torch.empty(0, 1, device=gpu))
    rows, cols = 40000, 65536  # 5 GiB of weights, 1.3 GiB of codes
    w = torch.zeros(rows, cols, dtype=torch.bfloat16, device=gpu)
    for r in (0, 17000, rows - 1):
        w[r].normal_(generator=torch.Generator(device="cuda").manual_seed(r))
    q = torch.empty(rows, cols // 2, dtype=torch.uint8, device=gpu)
    s = torch.empty(rows, cols // 64, device=gpu)
    moe.i4_quantize(w, q, s, 64)
    back = torch.empty_like(w)
    moe.i4_dequantize(q, s, back, 64)
    for r in (0, 1, 17000, rows - 1):
        codes, scale = oracle.i4_quantize(to_host(w[r:r + 1]), 64)
        np.testing.assert_array_equal(q[r:r + 1].cpu().numpy(), oracle.i4_pack(codes))
        np.testing.assert_array_equal(to_host(back[r:r + 1]), _bf(codes * np.repeat(scale, 64, axis=1)))


# ------------------------------------------------------------------- linear

LINEAR = [(1, 16, 8, 32), (1, 1, 64, 64), (2, 33, 40, 32), (3, 16, 128, 128), (5, 1003, 1992, 32), (7, 40, 264, 128), (8, 24, 520, 64),
          (9, 100, 2048, 128), (16, 64, 1024, 64), (17, 17, 136, 32), (33, 48, 448, 128), (64, 96, 832, 32), (100, 256, 1792, 128),
          (1, 6144, 1792, 128), (2, 300, 6144, 64), (257, 72, 96, 64)]


def _linear_case(M, N, K, group, whole):
    rng = np.random.default_rng(M * 7 + N + K + group)
    codes = rng.integers(-8, 8, (N, K))
    if whole:
        x = rng.integers(-4, 5, (M, K)).astype(np.float32)
        scale = 2.0 ** rng.integers(-3, 2, (N, -(-K // group)))
        bias = rng.integers(-50, 50, N).astype(np.float32)
    else:
        x = _bf(rng.normal(0, 1, (M, K)) * np.exp(0.5 * rng.normal(0, 1, (M, 1))))
        scale = rng.uniform(1e-3, 1e-2, (N, -(-K // group)))
        bias = rng.normal(0, 1, N).astype(np.float32)
    return x, codes, scale.astype(np.float32), bias


def _run_linear(gpu, x, codes, scale, bias, group, odt, pad=1):
    """The product with rows of every operand apart, and what lies behind them unfit to use."""
    (M, K), N = x.shape, codes.shape[0]
    ldw = (K // 2 + 15) // 16 * 16 + 16 * pad
    xd = _dev_rows(x, (K + 7) // 8 * 8 + 8 * pad, torch.bfloat16, float("nan"))
    wd = _dev_rows(oracle.i4_pack(codes), ldw, torch.uint8, 0xFF)
    sd = _dev_rows(scale, scale.shape[1] + 3 * pad, torch.float32, float("nan"))
    y = torch.full((M, N + 5 * pad), 9.0, dtype=odt, device=gpu)
    moe.i4_linear(xd[:, :K], wd[:, :K // 2], sd[:, :scale.shape[1]], y[:, :N], None if bias is None else _dev(bias), group)
    assert (y[:, N:] == 9.0).all()
    return to_host(y[:, :N].contiguous())


@pytest.mark.parametrize("M,N,K,group", LINEAR)
def test_linear_of_whole_numbers_is_exact(gpu, M, N, K, group):
    x, codes, scale, bias = _linear_case(M, N, K, group, True)
    want = oracle.i4_linear(x, codes, scale, group, bias)
    np.testing.assert_array_equal(_run_linear(gpu, x, codes, scale, bias, group, torch.float32), want)
    np.testing.assert_array_equal(_run_linear(gpu, x, codes, scale, bias, group, torch.bfloat16, 0), _bf(want))


@pytest.mark.parametrize("M,N,K,group", LINEAR)
def test_linear_against_the_oracle(gpu, M, N, K, group):
    x, codes, scale, bias = _linear_case(M, N, K, group, False)
    for b, odt in ((bias, torch.float32), (None, torch.bfloat16)):
        want = oracle.i4_linear(x, codes, scale, group, b)
        mag = 56 * np.abs(x).astype(np.float64) @ np.repeat(scale.astype(np.float64), group, axis=1)[:, :K].T
        part = 2 * _chain(K) * U32 * mag + (4 * U32 * np.abs(b) if b is not None else 0)
        _within(_run_linear(gpu, x, codes, scale, b, group, odt), want, part, odt == torch.bfloat16)


def test_linear_of_no_rows_and_of_not_finite_rows(gpu):
    x, codes, scale, _ = _linear_case(6, 40, 256, 128, True)
    assert _run_linear(gpu, x[:0], codes, scale, None, 128, torch.float32).shape == (0, 40)
    want = oracle.i4_linear(x, codes, scale, 128)
    x[2, 5], x[4, 200] = np.inf, np.nan
    scale[7, 1] = np.nan
    got = _run_linear(gpu, x, codes, scale, None, 128, torch.float32)
    ok = np.ones((6, 40), bool)
    ok[[2, 4]], ok[:, 7] = False, False
    np.testing.assert_array_equal(got[ok], want[ok])  # a row, or a channel, is its own affair
    assert not np.isfinite(got[~ok]).any()


def test_linear_past_32_bit_offsets(gpu):
    """Weights of 4.3 GB of codes: first, middle and last channels."""
    N, K, group = 540672, 16384, 128
    wq = torch.zeros(N, K // 2, dtype=torch.uint8, device=gpu)
    ws = torch.zeros(N, K // group, device=gpu)
    x, codes, scale, _ = _linear_case(2, 48, K, group, True)
    rows = np.r_[0:16, 270000:270016, N - 16:N]
    wq[rows] = _dev(oracle.i4_pack(codes), torch.uint8)
    ws[rows] = _dev(scale)
    y = torch.empty(2, N, device=gpu)
    moe.i4_linear(_dev(x, torch.bfloat16), wq, ws, y, group=group)
    np.testing.assert_array_equal(y[:, rows].cpu().numpy(), oracle.i4_linear(x, codes, scale, group))
    y[:, rows] = 0
    assert (y == 0).all()


# ------------------------------------------------------------------- decode

class Case:
    """A layer's inputs on the GPU and their float64 reference with its bounds."""

    def __init__(self, T, d, f, E, k, e0=0, NL=None, n_groups=1, renorm=1, group=0, seed=0, bias=True, routing=None, skew=0.0,
                 apart=False):
        rng = np.random.default_rng(seed + 1000 * T + d)
        NL = E if NL is None else NL
        self.D = moe.make_desc(T, d, f, E, k, e0, NL, "bf16", renormalize=renorm)
        self.group, self.n_groups, self.e0, self.NL = group, n_groups, e0, NL
        self.x = _bf(rng.normal(0, 1, (T, d)) * np.exp(0.3 * rng.normal(0, 1, (T, 1))))
        self.wr = _bf(rng.normal(0, d ** -0.5, (E, d)))
        if apart:  # (token t's logits are Wr's column t: a permutation of 0 .. E - 1, in 32nds)
            self.x = np.eye(T, d, dtype=np.float32)
            self.wr = np.zeros((E, d), np.float32)
            self.wr[:, :T] = np.stack([rng.permutation(E) / 32.0 for _ in range(T)], axis=1)
        self.bias = (0.3 * rng.normal(0, 1, E) - skew * np.log(1 + np.arange(E))).astype(np.float32) if bias else None
        self.routing = routing
        self.dev = dict(x=_dev(self.x, torch.bfloat16), wr=_dev(self.wr, torch.bfloat16),
                        bias=None if self.bias is None else _dev(self.bias))
        w, mag = {}, {}
        for name, rows, cols in (("w1", f, d), ("w3", f, d), ("w2", d, f)):
            if group:
                codes = rng.integers(-8, 8, (NL * rows, cols), dtype=np.int8)
                scale = rng.uniform(2e-3, 8e-3, (NL * rows, -(-cols // group))).astype(np.float32)
                w[name] = oracle.i4_dequantize(codes, scale, group).reshape(NL, rows, cols)
                mag[name] = 56 * np.repeat(scale.astype(np.float64), group, axis=1)[:, :cols].reshape(NL, rows, cols)
                self.dev[name + "q"] = _dev(oracle.i4_pack(codes), torch.uint8).view(NL, rows, cols // 2)
                self.dev[name + "s"] = _dev(scale).view(NL, rows, -1)
            else:
                v = _bf(rng.normal(0, 0.02, (NL, rows, cols)))
                self.dev[name] = _dev(v, torch.bfloat16)
                w[name] = v.astype(np.float64)
                mag[name] = np.abs(w[name])
        if group:
            self.experts = moe.Int4Experts.from_codes(*[self.dev[n + s] for n in ("w1", "w3", "w2") for s in "qs"], group=group)
        self._reference(w, mag, rng)

    def _reference(self, w, mag, rng):
        T, d, f, E, k = self.D.T, self.D.d, self.D.f, self.D.E, self.D.k
        x = self.x.astype(np.float64)
        EL = np.zeros(T)
        if self.routing is None:
            L = x @ self.wr.astype(np.float64).T + (0 if self.bias is None else self.bias.astype(np.float64))
            el = 2 * _chain(d) * U32 * (np.abs(x) @ np.abs(self.wr.astype(np.float64)).T) + (
                0 if self.bias is None else U32 * np.abs(self.bias))
            EL = el.max(axis=1)
            if self.n_groups > 1:
                self.idx, self.w = oracle.topk_route_grouped(L, k, self.n_groups, self.D.renormalize)
            else:
                self.idx, self.w = oracle.topk_route(L, k, self.D.renormalize)
            # tokens whose selection the bound decides (slot order too) are not compared
            S = np.sort(L.reshape(T, self.n_groups, -1), axis=2)[:, :, ::-1]
            kg = k // self.n_groups
            gap = np.abs(np.diff(np.sort(np.take_along_axis(L, self.idx.astype(int), 1), axis=1), axis=1)).min(axis=1, initial=9.0)
            if kg < S.shape[2]:
                gap = np.minimum(gap, (S[:, :, kg - 1] - S[:, :, kg]).min(axis=1))
            self.sure = gap > 2 * EL
            self.Ew = self.w * (2 * EL + 16 * U32)[:, None]
        else:
            self.idx, self.w = (np.asarray(a) for a in self.routing)
            self.sure, self.Ew = np.ones(T, bool), np.zeros((T, k))
        self.y, part = np.zeros((T, d)), np.zeros((T, d))
        for e in range(self.NL):
            t, j = np.nonzero(self.idx - self.e0 == e)
            if len(t) == 0:
                continue
            xe, c1, c2 = x[t], 2 * _chain(d) * U32, 2 * _chain(f) * U32
            G, Uv = xe @ w["w1"][e].T, xe @ w["w3"][e].T
            EG, EU = c1 * np.abs(xe) @ mag["w1"][e].T, c1 * np.abs(xe) @ mag["w3"][e].T
            sl = G / (1 + np.exp(-G))
            h = sl * Uv
            Eh = 1.1 * np.abs(Uv) * EG + np.abs(sl) * EU + (13 + 4 * np.abs(G)) * 2 * U32 * np.abs(h)
            out = h @ w["w2"][e].T
            a2 = np.abs(w["w2"][e]).T
            # (h's rounding to bf16 is not a float32 part: halved here, as _within doubles)
            Eo = Eh @ a2 + 0.5 * UBF * (np.abs(h) @ a2) + c2 * (np.abs(h) @ mag["w2"][e].T)
            ww, Ew = np.abs(self.w[t, j])[:, None], (self.Ew[t, j] + 8 * U32 * np.abs(self.w[t, j]))[:, None]
            np.add.at(self.y, t, self.w[t, j][:, None] * out)
            np.add.at(part, t, ww * Eo + Ew * np.abs(out))
        self.part = part

    def run(self, b=None):
        b = b or moe.DecodeBuffers(self.D)
        routing = None
        if self.routing is not None:
            routing = (_dev(self.idx, torch.int32), _dev(self.w))
        kw = dict(bias=self.dev["bias"] if routing is None else None, n_groups=self.n_groups, routing=routing)
        if self.group:
            moe.decode_i4(b, self.dev["x"], self.dev["wr"], self.experts, **kw)
        else:
            moe.decode(b, self.dev["x"], self.dev["wr"], self.dev["w1"], self.dev["w3"], self.dev["w2"], **kw)
        return b

    def check(self, b):
        assert 2 * self.sure.sum() >= len(self.sure)  # (how many tokens the logits' bound leaves decided)
        if self.routing is None:
            np.testing.assert_array_equal(b.topk_idx.cpu().numpy()[self.sure], self.idx[self.sure])
            got = b.topk_w.cpu().numpy().astype(np.float64)
            assert (np.abs(got - self.w)[self.sure] <= 2 * self.Ew[self.sure]).all()
        _within(to_host(b.y)[self.sure], self.y[self.sure], self.part[self.sure], True)


# T, d, f, E, k, expert_begin, local experts, router groups, renormalised
LAYERS = [(1, 64, 64, 8, 1, 0, 8, 1, 1), (1, 128, 64, 8, 8, 0, 8, 1, 1), (1, 2048, 1024, 64, 8, 0, 64, 1, 1), (2, 832, 448, 24, 3, 0, 24, 1, 0),
          (3, 192, 320, 16, 4, 5, 7, 1, 1), (5, 832, 448, 24, 3, 0, 24, 1, 1), (8, 256, 128, 64, 8, 16, 16, 4, 1), (9, 128, 192, 8, 2, 0, 8, 1, 0),
          (12, 1024, 512, 96, 8, 0, 24, 4, 1), (16, 512, 256, 16, 4, 0, 16, 1, 1), (17, 320, 64, 8, 3, 0, 8, 1, 1),
          (31, 64, 128, 1024, 8, 1000, 24, 1, 1), (33, 448, 832, 40, 5, 0, 40, 1, 0), (64, 256, 128, 8, 8, 0, 8, 1, 1),
          (64, 512, 192, 64, 32, 0, 64, 1, 1), (64, 640, 320, 384, 8, 96, 96, 4, 1), (64, 128, 64, 128, 2, 3, 1, 1, 1)]


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("shape", LAYERS, ids=lambda s: "-".join(map(str, s)))
def test_decode_against_the_oracle(gpu, shape, group):
    T, d, f, E, k, e0, NL, n_groups, renorm = shape
    c = Case(T, d, f, E, k, e0, NL, n_groups, renorm, group, seed=3, bias=(T % 2 == 1))
    b = moe.DecodeBuffers(c.D)
    b.ws.fill_(0xFF)  # the workspace needs no preparation
    b.y.fill_(float("nan"))
    c.check(c.run(b))


@pytest.mark.parametrize("group", [0, 128])
def test_decode_at_the_1t_widths(gpu, group):
    c = Case(3, 6144, 1792, 24, 4, 4, 12, 1, 1, group, seed=5)
    c.check(c.run())


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 9, 30])
def test_decode_with_a_short_last_item(gpu, T, group):
    """d of 24 channels an item and 8 in the last; f of less than a stage and of odd stages; one token per wave and more."""
    c = Case(T, 6080, 64 if T < 9 else 192, 8, 2, 0, 8, 1, 1, group, seed=6)
    c.check(c.run())


@pytest.mark.parametrize("n_groups", [2, 3, 6, 8, 16, 32])
def test_decode_with_any_number_of_router_groups(gpu, n_groups):
    E, k = (192, 12) if n_groups in (3, 6) else (256, 32)
    for T, renorm in ((1, 1), (9, 0), (20, 1)):
        c = Case(T, 128, 64, E, k, 0, 16, n_groups, renorm, 0, seed=n_groups, bias=False, apart=True)
        assert c.sure.all()
        c.check(c.run())


@pytest.mark.parametrize("group", [0, 64])
def test_decode_with_busy_experts(gpu, group):
    """Nearly all of 60 tokens at the same experts: more rows than one tile of them holds."""
    c = Case(60, 384, 192, 16, 3, 0, 16, 1, 1, group, seed=7, skew=4.0)
    assert np.bincount(c.idx.ravel(), minlength=16).max() > 48
    c.check(c.run())


@pytest.mark.parametrize("group", [0, 32])
def test_decode_with_a_given_routing(gpu, group):
    """Experts named twice by a token, experts outside the local ones and outside any, weights of zero and below it."""
    rng = np.random.default_rng(9)
    T, E, k = 20, 16, 6
    idx = rng.integers(-2, E + 2, (T, k)).astype(np.int32)
    idx[3], idx[4], idx[5], idx[6] = 5, [4, 4, 9, 9, 4, 2 ** 31 - 1], -(2 ** 31), 0
    w = _bf(rng.normal(0, 1, (T, k)))
    w[7] = 0
    c = Case(T, 256, 128, E, k, 4, 8, 1, 1, group, seed=9, routing=(idx, w))
    b = c.run()
    c.check(b)
    y = to_host(b.y)
    assert (y[5] == 0).all() and (y[6] == 0).all() and (y[7] == 0).all()  # nothing local; weight zero
    c1 = Case(2, 256, 128, E, k, 4, 8, 1, 1, group, seed=9, routing=(np.full((2, k), 99, np.int32), w[:2]))
    assert (to_host(c1.run().y) == 0).all()


@pytest.mark.parametrize("T,group", [(64, 0), (64, 32), (64, 64), (64, 128), (16, 0), (16, 128)])
def test_decode_with_the_longest_lists(gpu, T, group):
    """32 picks a token: half of the tokens name every expert once, the others all the same 32."""
    E, k = 16 * T, 32
    idx = np.concatenate([np.arange(E).reshape(T // 2, k), np.tile(np.arange(k)[::-1], (T // 2, 1))]).astype(np.int32)
    w = _bf(np.random.default_rng(T).uniform(0.01, 0.1, (T, k)))
    c = Case(T, 64, 128, E, k, 0, E, 1, 1, group, seed=T, routing=(idx, w))
    c.check(c.run())


@pytest.mark.parametrize("n_groups", [1, 4])
def test_decode_gives_ties_to_the_lower_expert(gpu, n_groups):
    """Logits of small whole numbers, equal by the dozen."""
    rng = np.random.default_rng(11)
    T, d, E, k = 40, 64, 64, 8
    D = moe.make_desc(T, d, 64, E, k, 0, E, "bf16")
    x, wr = rng.integers(-1, 2, (T, d)).astype(np.float32), rng.integers(-1, 2, (E, d)).astype(np.float32)
    wr[:, 8:] = 0
    x[0], x[1, :8] = 0, 1  # (all equal)
    L = x.astype(np.float64) @ wr.T
    idx = (oracle.topk_route_grouped(L, k, n_groups) if n_groups > 1 else oracle.topk_route(L, k))[0]
    b = moe.DecodeBuffers(D)
    w = torch.zeros(E, 64, 64, dtype=torch.bfloat16, device=gpu)
    moe.decode(b, _dev(x, torch.bfloat16), _dev(wr, torch.bfloat16), w, w, w, n_groups=n_groups)
    np.testing.assert_array_equal(b.topk_idx.cpu().numpy(), idx)
    assert (b.y == 0).all()


@pytest.mark.parametrize("group", [0, 64])
def test_decode_keeps_a_token_that_is_not_finite_to_itself(gpu, group):
    c = Case(6, 256, 128, 16, 4, 0, 16, 1, 1, group, seed=13)
    c.dev["x"][2, 7] = float("nan")
    c.dev["x"][4, 9] = float("inf")
    b = c.run()
    ok = np.array([t for t in range(6) if t not in (2, 4) and c.sure[t]])
    _within(to_host(b.y)[ok], c.y[ok], c.part[ok], True)
    np.testing.assert_array_equal(b.topk_idx.cpu().numpy()[ok], c.idx[ok])


def test_decode_is_two_kernels_and_the_same_on_every_call(gpu):
    for T, group in ((1, 0), (64, 0), (1, 32), (20, 128)):
        c = Case(T, 256, 128, 32, 4, 0, 32, 1, 1, group, seed=15)
        b = c.run()
        first = [t.clone() for t in (b.y, b.topk_idx, b.topk_w)]
        assert 1 <= len(kernels(lambda: c.run(b))) <= 2
        for _ in range(20):
            b.ws.random_(0, 256)
            c.run(b)
            assert all(torch.equal(p, q) for p, q in zip(first, (b.y, b.topk_idx, b.topk_w)))


@pytest.mark.parametrize("group", [0, 128])
def test_decode_captured_shared_and_on_two_streams(gpu, group):
    """Two graphs that share buffers, replayed on new inputs between eager work, and two calls at once on two streams with
    buffers of their own, give bitwise what one eager call gives."""
    cs = [Case(T, 512, 256, 32, 4, 0, 32, 1, 1, group, seed=17) for T in (7, 7)]
    c = cs[0]
    xs = [_dev(_bf(np.random.default_rng(i).normal(0, 1, (7, 512))), torch.bfloat16) for i in range(3)]
    b = moe.DecodeBuffers(c.D)
    want = []
    for x in xs:
        c.dev["x"] = x
        want.append(c.run(b).y.clone())
    a = [xs[0].clone(), xs[0].clone()]
    graphs = []
    for i in range(2):
        c.dev["x"] = a[i]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(b)
        graphs.append(g)
    for i in range(6):
        a[i % 2].copy_(xs[i % 3])
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(b.y, want[i % 3])
        c.dev["x"] = xs[(i + 1) % 3]
        assert torch.equal(c.run(b).y, want[(i + 1) % 3])
    sets = [moe.DecodeBuffers(c.D) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                c.dev["x"] = xs[j]
                c.run(sets[j])
    torch.cuda.synchronize()
    for j in range(2):
        assert torch.equal(sets[j].y, want[j])


@pytest.mark.parametrize("T,group", [(3, 0), (3, 128), (64, 0), (64, 32)])
def test_decode_beside_a_kernel_that_holds_compute_units(gpu, T, group):
    c = Case(T, 1024, 512, 16, 4, 0, 16, 1, 1, group, seed=19)
    b = c.run()
    want = b.y.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for held in (64, 200, 250):
        moe.hold_cus(held, 3000, stream=side)
        b.y.zero_()
        c.run(b)
        torch.cuda.synchronize()
        assert torch.equal(b.y, want)


@pytest.mark.parametrize("group", [0, 128])
def test_decode_past_32_bit_offsets(gpu, group):
    """Experts of 33 M weights, 96 of them: 6.4 GB a matrix (4 bits: 1.6 GB); the first and the last one are taken."""
    E, d, f, T = 96, 6144, 5440, 3
    g = torch.Generator(device="cuda").manual_seed(25)
    D = moe.make_desc(T, d, f, E, 2, 0, E, "bf16")
    b = moe.DecodeBuffers(D)
    x = torch.randn(T, d, generator=g, device=gpu).bfloat16()
    idx = torch.tensor([[0, E - 1]] * T, dtype=torch.int32, device=gpu)
    w = torch.tensor([[0.75, 0.25], [1.0, -0.5], [0.0, 1.0]], device=gpu)
    host = {}
    args = []
    for name, rows, cols in (("w1", f, d), ("w3", f, d), ("w2", d, f)):
        if group:
            q = torch.empty(E, rows, cols // 2, dtype=torch.uint8, device=gpu).random_(0, 256, generator=g)
            s = torch.rand(E, rows, -(-cols // group), generator=g, device=gpu) * 4e-3 + 2e-3
            args += [q, s]
            host[name] = [oracle.i4_dequantize(oracle.i4_unpack(q[e].cpu().numpy()), s[e].cpu().numpy(), group) for e in (0, E - 1)]
        else:
            v = torch.empty(E, rows, cols, dtype=torch.bfloat16, device=gpu)
            for e in (0, E - 1):
                v[e].normal_(0, 0.02, generator=g)
            args.append(v)
            host[name] = [to_host(v[e]).astype(np.float64) for e in (0, E - 1)]
    if group:
        moe.decode_i4(b, x, None, moe.Int4Experts.from_codes(*args, group=group), routing=(idx, w))
    else:
        moe.decode(b, x, None, *args, routing=(idx, w))
    xh, want = to_host(x).astype(np.float64), np.zeros((T, d))
    for i in range(2):
        G, Uv = xh @ host["w1"][i].T, xh @ host["w3"][i].T
        want += w.cpu().numpy().astype(np.float64)[:, i:i + 1] * ((G / (1 + np.exp(-G)) * Uv) @ host["w2"][i].T)
    assert np.abs(to_host(b.y) - want).max() <= 2e-2 * np.abs(want).max()


def test_a_decode_step_in_4_bits_from_bf16_weights(gpu):
    """Experts quantised, a projection quantised, and a step of both as a server runs it: the projection's output is the
    layer's input."""
    rng = np.random.default_rng(21)
    T, K, d, f, E, k = 4, 192, 256, 128, 16, 4
    wp, x0 = _bf(rng.normal(0, K ** -0.5, (d, K))), _bf(rng.normal(0, 1, (T, K)))
    w = {n: _bf(rng.normal(0, 0.05, s)) for n, s in (("w1", (E, f, d)), ("w3", (E, f, d)), ("w2", (E, d, f)))}
    wr = _bf(rng.normal(0, d ** -0.5, (E, d)))
    dev = {n: _dev(v, torch.bfloat16) for n, v in w.items()}
    ex = moe.Int4Experts(dev["w1"], dev["w3"], dev["w2"], group=64)
    q, s = torch.empty(d, K // 2, dtype=torch.uint8, device=gpu), torch.empty(d, K // 64, device=gpu)
    moe.i4_quantize(_dev(wp, torch.bfloat16), q, s, group=64)
    x = torch.empty(T, d, dtype=torch.bfloat16, device=gpu)
    moe.i4_linear(_dev(x0, torch.bfloat16), q, s, x, group=64)
    D = moe.make_desc(T, d, f, E, k, 0, E, "bf16")
    b = moe.DecodeBuffers(D)
    moe.decode_i4(b, x, _dev(wr, torch.bfloat16), ex)
    codes, scale = oracle.i4_quantize(wp, 64)
    want = oracle.i4_linear(x0, codes, scale, 64)
    mag = 56 * np.abs(x0).astype(np.float64) @ np.repeat(scale.astype(np.float64), 64, axis=1).T
    _within(to_host(x), want, 2 * _chain(K) * U32 * mag, True)
    deq = {}
    for n, v in w.items():
        cc, sc = oracle.i4_quantize(v.reshape(-1, v.shape[2]), 64)
        deq[n] = oracle.i4_dequantize(cc, sc, 64).reshape(v.shape)
    # the layer on the values that the codes stand for, and forward() on those values in bf16 beside it
    ref = oracle.layer_forward(to_host(x), wr, deq["w1"], deq["w3"], deq["w2"], k, 0, E,
                               routing=(b.topk_idx.cpu().numpy(), b.topk_w.cpu().numpy()))
    assert np.abs(to_host(b.y) - ref["y"]).max() <= 2e-2 * np.abs(ref["y"]).max()
    for n, (rows, cols) in (("w1", (f, d)), ("w3", (f, d)), ("w2", (d, f))):
        moe.i4_dequantize(getattr(ex, n + "q").view(E * rows, cols // 2), getattr(ex, n + "s").view(E * rows, -1),
                          dev[n].view(E * rows, cols), group=64)
    buf = moe.Buffers(D)
    y = moe.forward(buf, x, _dev(wr, torch.bfloat16), dev["w1"], dev["w3"], dev["w2"])
    assert torch.equal(buf.topk_idx, b.topk_idx)
    assert np.abs(to_host(b.y) - to_host(y)).max() <= 2e-2 * np.abs(ref["y"]).max()


def test_python_checks_of_the_decode_calls(gpu):
    c = Case(4, 128, 64, 8, 2, 0, 8, 1, 1, 32, seed=23)
    b = moe.DecodeBuffers(c.D)
    dev, bf = c.dev, torch.bfloat16
    for bad in (dict(x=dev["x"][:3]), dict(x=dev["x"].float()), dict(x=dev["x"].t()), dict(wr=dev["wr"][:4]), dict(x=dev["x"].cpu()),
                dict(bias=torch.zeros(7, device=gpu)), dict(routing=(torch.zeros(4, 2, device=gpu), torch.zeros(4, 2, device=gpu)))):
        with pytest.raises(ValueError):
            moe.decode_i4(b, **{**dict(x=dev["x"], wr=dev["wr"], experts=c.experts), **bad})
    ex = moe.Int4Experts.from_codes(dev["w1q"][:-1], dev["w1s"], dev["w3q"], dev["w3s"], dev["w2q"], dev["w2s"], 32)
    with pytest.raises(ValueError):
        moe.decode_i4(b, dev["x"], dev["wr"], ex)
    w = torch.zeros(8, 64, 128, dtype=bf, device=gpu)
    with pytest.raises(ValueError):
        moe.decode(b, dev["x"], dev["wr"], w, w, w[:, :, :120])
    small = moe.DecodeBuffers(c.D)
    small.ws = small.ws[:64]
    with pytest.raises(moe.MoeError):
        moe.decode(small, dev["x"], dev["wr"], w, w, w)
    q, s, y = dev["w1q"][0], dev["w1s"][0], torch.zeros(4, 64, device=gpu)
    for bad in (dict(x=dev["x"][:, :120]), dict(wq=q[:, :56]), dict(ws=s[:, :3]), dict(ws=s.double()), dict(y=y[:3]), dict(y=y.half()),
                dict(bias=torch.zeros(63, device=gpu)), dict(wq=q.to(torch.int8))):
        with pytest.raises(ValueError):
            moe.i4_linear(**{**dict(x=dev["x"], wq=q, ws=s, y=y, group=32), **bad})
    with pytest.raises(moe.MoeError):  # (rows of x start at multiples of 16 bytes)
        moe.i4_linear(torch.zeros(4, 132, dtype=bf, device=gpu)[:, :128], q, s, y, group=32)

"""Every form of the INT8 kernels, each at a size for which it is the one launched.

The name of the launched kernel is part of each test, so a moved limit between
the forms cannot leave one of them without its test.  Outputs that the header
gives as a sequence of float32 operations are compared bit for bit:
  linear     fl(fl(fl(fl(S) xs) ws) + b), then one rounding to the output type;
  G, U       fl(fl(fl(S) xs) ws), then one rounding to bf16; down likewise;
with S the whole-number sum, taken here in float64, where it is exact.  h goes
by the bound of silu(G) U in float32 (see test_gpu_i8).
"""
import re

import numpy as np
import pytest
import torch

import mixture_experts_layer_02_amd as moe
import oracle
from gpu_util import to_host
from launched import kernels
from test_gpu_i8 import SENTINEL, U32, _special_rows, _within

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


def _form(fn):
    """The one kernel of a product and its sizes: (few, row blocks, channel blocks, waves), (mid, rows, channels,
    wave rows) or (tiles, dynamic)."""
    (name,) = kernels(fn)
    ints = [int(v) for v in re.findall(r"Li(\d+)E", name)]
    if "i8_few_rows_kernel" in name:
        return ("few", *ints[:3])
    if "i8_mid_rows_kernel" in name:
        return ("mid", *ints[:3])
    assert "gemm_dma_kernel" in name, name
    flags = [int(v) for v in re.findall(r"Lb(\d)E", name)]  # DUAL, CF32, DYN, BQ8, F8, I8
    assert flags[3:] == [0, 0, 1], name
    return "tiles", flags[2]


def _codes(g, rows, cols, ld=None, fill=127):
    """Random codes [rows][cols], rows ld bytes apart (a multiple of 16), `fill` in between."""
    q = torch.full((rows, ld or (cols + 15) // 16 * 16), fill, dtype=torch.int8, device="cuda")[:, :cols]
    q.copy_(torch.randint(-127, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8))
    return q


def _scales(g, *shape):
    return torch.rand(shape, generator=g, device="cuda") * 1e-3 + 1e-4


def _scaled(xq, xs, wq, ws):
    """fl(fl(fl(S) xs) ws) as float32."""
    s = torch.mm(xq.double(), wq.double().t().contiguous())
    return s.float() * xs[:, None] * ws


def _same(got, want):
    """Bit for bit, but for the sign of zero."""
    bad = got != want
    assert not bad.any(), (int(bad.sum()), got[bad][:4].tolist(), want[bad][:4].tolist())


LINEAR = [  # M, N, K, the form
    (1, 1003, 1990, ("few", 1, 2, 4)), (3, 999, 4100, ("few", 1, 2, 8)),
    (5, 24577, 203, ("few", 1, 4, 4)), (1, 49153, 203, ("few", 1, 8, 4)), (8, 49153, 203, ("few", 1, 8, 4)),
    (32, 9999, 203, ("few", 2, 2, 4)), (17, 24577, 203, ("few", 2, 4, 4)), (20, 49153, 203, ("few", 2, 8, 4)),
    (40, 24577, 203, ("few", 4, 4, 4)), (20, 153601, 203, ("mid", 64, 128, 1)), (40, 51300, 203, ("mid", 64, 128, 1)),
    (300, 11000, 203, ("mid", 64, 128, 1)), (100, 51300, 203, ("mid", 128, 128, 2)),
    (150, 46100, 203, ("mid", 192, 128, 2)), (200, 44801, 203, ("mid", 192, 128, 2)), (500, 24568, 2048, ("tiles", 0)),
]


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("M,N,K,form", LINEAR)
def test_linear_rounds_as_the_header_says(gpu, M, N, K, form, dtype, bias):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    xq, wq, xs, ws = _codes(g, M, K), _codes(g, N, K, fill=-127), _scales(g, M), _scales(g, N)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    y = torch.full((M, N), float(SENTINEL), dtype=dtype, device=gpu)
    assert _form(lambda: moe.i8_linear(xq, xs, wq, ws, y, bias=b)) == form
    moe.i8_linear(xq, xs, wq, ws, y, bias=b)
    want = _scaled(xq, xs, wq, ws)
    if bias:
        want = want + b
    _same(y, want.to(dtype))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_linear_of_a_row_alone_and_among_many(gpu, dtype):
    """A row's outputs do not depend on the rows beside it, although other kernels take them."""
    g = torch.Generator(device="cuda").manual_seed(1)
    M, N, K = 500, 24568, 2048
    xq, wq, xs, ws = _codes(g, M, K), _codes(g, N, K), _scales(g, M), _scales(g, N)
    b = torch.randn(N, generator=g, device="cuda")
    y = torch.empty(M, N, dtype=dtype, device=gpu)
    moe.i8_linear(xq, xs, wq, ws, y, bias=b)
    for n in (1, 12, 40, 64, 200, 300):
        part = torch.empty(n, N, dtype=dtype, device=gpu)
        assert _form(lambda: moe.i8_linear(xq[:n], xs, wq, ws, part, bias=b)) != ("tiles", 0)
        moe.i8_linear(xq[:n], xs, wq, ws, part, bias=b)
        assert torch.equal(part, y[:n])


@pytest.mark.parametrize("M,N,ldw,form", [(1100, 2900, 1 << 22, ("mid", 64, 128, 1)), (1500, 4300, 1 << 22, ("mid", 128, 128, 2)),
                                          (1100, 14950, 1 << 19, ("mid", 192, 128, 2))])
def test_linear_of_rows_far_apart_on_shared_tiles(gpu, M, N, ldw, form):
    """Codes and outputs past 32-bit offsets through the shared-operand kernel's three forms."""
    K, g = 300, torch.Generator(device="cuda").manual_seed(M)
    xq, wq, xs, ws = _codes(g, M, K, 1 << 22), _codes(g, N, K, ldw, -127), _scales(g, M), _scales(g, N)
    b = torch.randn(N, generator=g, device="cuda")
    y = torch.full((M, 1 << 21), float(SENTINEL), dtype=BF, device=gpu)
    assert _form(lambda: moe.i8_linear(xq, xs, wq, ws, y[:, :N], bias=b)) == form
    moe.i8_linear(xq, xs, wq, ws, y[:, :N], bias=b)
    _same(y[:, :N], (_scaled(xq, xs, wq, ws) + b).to(BF))
    assert (y[:, N:N + 256] == SENTINEL).all()


EXPERTS = [  # T, d, f, E, k, experts here, the forms of gate/up and of down
    (1, 4096, 64, 8, 1, 8, ("few", 1, 2, 8), ("few", 1, 2, 4)),
    (1, 6144, 1792, 384, 8, 96, ("few", 1, 2, 8), ("few", 1, 2, 4)),
    (2, 6144, 1792, 384, 8, 96, ("few", 1, 2, 8), ("few", 1, 4, 4)),
    (5, 64, 4160, 8, 1, 8, ("few", 1, 8, 4), ("few", 1, 2, 8)),
    (3, 832, 448, 24, 8, 24, ("few", 1, 4, 4), ("few", 1, 4, 4)),
    (60, 576, 1024, 64, 1, 64, ("few", 1, 8, 4), ("few", 1, 8, 4)),
    (100, 512, 192, 24, 2, 24, ("few", 1, 2, 4), ("few", 2, 2, 4)),
    (100, 192, 64, 96, 8, 96, ("few", 2, 2, 4), ("few", 2, 2, 4)),
    (100, 832, 448, 24, 2, 24, ("few", 2, 4, 4), ("few", 2, 4, 4)),
    (300, 576, 1024, 64, 2, 64, ("few", 2, 8, 4), ("few", 2, 8, 4)),
    (100, 832, 448, 24, 8, 24, ("few", 4, 4, 4), ("few", 4, 4, 4)),
    (120, 832, 448, 192, 8, 192, ("mid", 64, 128, 1), ("mid", 64, 128, 1)),
    (600, 192, 448, 64, 8, 64, ("mid", 128, 128, 2), ("mid", 64, 128, 1)),
    (400, 832, 448, 64, 8, 64, ("mid", 128, 128, 2), ("mid", 128, 128, 2)),
    (1300, 576, 448, 96, 8, 96, ("mid", 256, 256, 4), ("mid", 192, 128, 2)),
    # four k-tiles, the fewest that the large tiles take: the next tile is not loaded ahead
    (1000, 512, 1792, 32, 8, 32, "tiles", ("mid", 64, 128, 1)),
    (1300, 512, 1792, 32, 8, 32, "tiles", ("mid", 64, 128, 1)),
    (1000, 4096, 512, 64, 4, 64, ("mid", 128, 128, 2), "tiles"),
]


def _routed(T, d, f, E, k, NL, dyn):
    """The routed rows of T tokens with k random picks each, the first token's first pick an expert that is here."""
    D = moe.make_desc(T, d, f, E, k, 0, NL, "bf16", tile_counters=moe.new_tile_counters() if dyn else None)
    g = torch.Generator(device="cuda").manual_seed(T + d + f)
    score = torch.rand(T, E, generator=g, device="cuda")
    score[0, NL - 1] = 2.0
    idx = score.topk(k, dim=1).indices.to(torch.int32)
    b = moe.Buffers(D, gather=True)
    moe.permute(D, idx, None, b.counts, b.offsets, b.row_token, b.slot_row, None, b.ws_permute)
    return D, b, b.offsets.tolist(), g


def _per_expert(off, rows, rs, wq, ws):
    out = torch.zeros(off[-1], wq.shape[1], device="cuda")
    for n in range(len(off) - 1):
        a, z = off[n], off[n + 1]
        if z > a:
            out[a:z] = _scaled(rows[a:z], rs[a:z], wq[n], ws[n])
    return out


def _as_form(form, dyn):
    return ("tiles", int(dyn)) if form == "tiles" else form


CASES = [(*c, dyn) for c in EXPERTS for dyn in ((False, True) if "tiles" in c else (False,))]


@pytest.mark.parametrize("T,d,f,E,k,NL,form,_,dyn", CASES)
def test_gate_up_in_each_form(gpu, T, d, f, E, k, NL, form, _, dyn):
    D, b, off, g = _routed(T, d, f, E, k, NL, dyn)
    R = off[-1]
    xq, xs = _codes(g, T, d), _scales(g, T)
    w = [(_codes(g, NL * f, d).view(NL, f, d), _scales(g, NL, f)) for _ in range(2)]
    gu = torch.full((D.R_cap, 2 * f), float(SENTINEL), dtype=BF, device=gpu)
    h = torch.full((D.R_cap, f), float(SENTINEL), dtype=BF, device=gpu)

    def call(gu):
        moe.expert_gate_up_i8(D, b.offsets, b.row_token, xq, xs, *w[0], *w[1], gu, h)

    assert R > 0 and _form(lambda: call(gu)) == _as_form(form, dyn)
    call(gu)
    tok = b.row_token[:R].long()
    G, U = (_per_expert(off, xq[tok], xs[tok], *v) for v in w)
    _same(gu[:R], torch.cat([G, U], 1).to(BF))
    G, U = G.double().cpu().numpy(), U.double().cpu().numpy()
    H = G / (1 + np.exp(-G)) * U
    _within(to_host(h[:R]), H, U32 * (13 + 4 * np.abs(G)) * np.abs(H), True)
    assert (gu[R:] == SENTINEL).all() and (h[R:] == SENTINEL).all()
    kept = h.clone()
    h.fill_(SENTINEL)
    call(None)
    assert torch.equal(h, kept)


@pytest.mark.parametrize("T,d,f,E,k,NL,_,form,dyn", CASES)
def test_down_in_each_form(gpu, T, d, f, E, k, NL, _, form, dyn):
    D, b, off, g = _routed(T, d, f, E, k, NL, dyn)
    R = off[-1]
    hq, hs = _codes(g, D.R_cap, f), _scales(g, D.R_cap)
    hs[R:] = float("nan")
    wq, ws = _codes(g, NL * d, f).view(NL, d, f), _scales(g, NL, d)
    y = torch.full((D.R_cap, d), float(SENTINEL), dtype=BF, device=gpu)
    assert R > 0 and _form(lambda: moe.expert_down_i8(D, b.offsets, hq, hs, wq, ws, y)) == _as_form(form, dyn)
    moe.expert_down_i8(D, b.offsets, hq, hs, wq, ws, y)
    _same(y[:R], _per_expert(off, hq, hs, wq, ws).to(BF))
    assert (y[R:] == SENTINEL).all()


@pytest.mark.parametrize("rows", [24, 1032])
@pytest.mark.parametrize("dtype,cols,ldw,ldq", [("bf16", 1, 8, 16), ("bf16", 7, 8, 16), ("bf16", 63, 72, 64), ("bf16", 257, 264, 288),
                                                ("bf16", 1000, 1000, 1008), ("bf16", 1791, 1792, 1792), ("bf16", 2047, 2048, 2064),
                                                ("f32", 1, 4, 16), ("f32", 7, 8, 16), ("f32", 63, 72, 64), ("f32", 257, 260, 288),
                                                ("f32", 1000, 1000, 1008), ("f32", 1023, 1024, 1040)])
def test_quantiser_of_difficult_rows_in_both_vector_forms(gpu, dtype, cols, ldw, ldq, rows):
    """Ties, subnormal, huge, zero and non-finite rows with one wave a row (1032 rows) and four (24)."""
    w = np.concatenate([_special_rows(cols, dtype, 100 * cols + i) for i in range(rows // 24)])
    src = torch.full((rows, ldw), 1e30, dtype=BF if dtype == "bf16" else F32, device=gpu)
    src[:, :cols] = torch.from_numpy(w).to(gpu).to(src.dtype)
    q = torch.full((rows, ldq), SENTINEL, dtype=torch.int8, device=gpu)
    s = torch.full((rows + 1,), -1.0, device=gpu)
    (name,) = kernels(lambda: moe.i8_quantize_rows(src[:, :cols], q[:, :cols], s))
    assert re.search(r"i8_quant_rows_kernelI[tf]Li(\d)ELi(\d+)ELb(\d)E", name).groups() == \
        (("1", "4", "1") if rows >= 1024 else ("4", "3", "1"))
    moe.i8_quantize_rows(src[:, :cols], q[:, :cols], s)
    codes, scale = oracle.i8_quantize_rows(w)
    np.testing.assert_array_equal(s[:rows].cpu().numpy(), scale)
    np.testing.assert_array_equal(q[:, :cols].cpu().numpy(), codes)
    assert (q[:, cols:] == SENTINEL).all() and s[rows] == -1

"""Every form of the INT8 kernels, each at a size for which it is the one launched.

The name of the launched kernel is part of each test, so a moved limit between
the forms cannot leave one of them without its test.  Outputs that the header
gives as a sequence of float32 operations are compared bit for bit:
  linear     fl(fl(fl(fl(S) xs) ws) + b), then one rounding to the output type,
with S the whole-number sum, taken here in float64, where it is exact.
"""
import re

import pytest
import torch

import mixture_experts_layer_02_amd as moe
from launched import kernels
from test_gpu_i8 import SENTINEL

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

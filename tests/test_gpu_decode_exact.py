"""The decode step on layers with one right answer, bit for bit, and on random ones by 64 columns of each token.

Every form of the kernel that a call can reach runs: bf16 and 4 bits with each group, one token, two, up to 16
(in 4 bits with 16 and with 8 channels of f an item) and more, 8 and 24 channels of d an item.  The form is pinned by
the name of the launched kernel.
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_02_amd as moe
from exact_layer import BLOCK_TOL, FORMS, Layer, pack, worst_block
from gpu_util import to_host
from launched import kernels

pytestmark = pytest.mark.gpu

CASES = [(shape, i4 if group else bf16, group) for shape, bf16, i4 in FORMS for group in (0, 32, 64, 128)]


def _id(v):
    return "-".join(map(str, v)) if isinstance(v, tuple) else str(v)


def _decode(b, x, wr, weights, group, **kw):
    if group:
        return moe.decode_i4(b, x, wr, moe.Int4Experts.from_codes(*[t for w in weights for t in w], group=group), **kw)
    return moe.decode(b, x, wr, *weights, **kw)


def _pinned(call, form, group):
    """call() launches the form that it is meant to."""
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        return
    name = "decode_kernelI" + "".join(f"Li{v}E" for v in (group, *form[:4]))
    assert any(name in k for k in kernels(call)), (name, kernels(call))


@pytest.mark.parametrize("shape,form,group", CASES, ids=_id)
def test_whole_numbers_are_exact(gpu, shape, form, group):
    a = Layer(*shape, group, seed=4)
    want = a.y()
    assert (want != 0).mean() > 0.4 or a.e0
    weights = [a.weights(n, gpu) for n in ("w1", "w3", "w2")]
    b = moe.DecodeBuffers(moe.make_desc(*shape[:5], a.e0, a.NL, "bf16"))
    b.ws.fill_(0xFF)
    b.y.fill_(float("nan"))
    x = torch.from_numpy(a.x).to(gpu).bfloat16()
    routing = (torch.from_numpy(a.idx).to(gpu), torch.from_numpy(a.w).to(gpu))
    _decode(b, x, None, weights, group, routing=routing)
    got = to_host(b.y)
    bad = np.argwhere(got != want)
    assert len(bad) == 0, (len(bad), [(*p, got[tuple(p)], want[tuple(p)]) for p in bad[:4].tolist()])
    _pinned(lambda: _decode(b, x, None, weights, group, routing=routing), form, group)


WIDTHS = [((1, 6144, 1792, 16, 4, 0, 16), (2, 2, 16, 24), (2, 2, 32, 24)), ((5, 6144, 1792, 16, 4, 0, 16), (16, 16, 16, 24), (16, 4, 32, 24)),
          ((64, 6144, 1792, 16, 4, 0, 16), (64, 12, 16, 24), (64, 8, 32, 24))]


@pytest.mark.parametrize("shape,form,group", CASES + [(s, i if g else h, g) for s, h, i in WIDTHS for g in (0, 128)], ids=_id)
def test_random_layers_by_blocks(gpu, shape, form, group):
    """y against 64-bit arithmetic on the selection that the step itself made."""
    T, d, f, E, k, e0, NL = shape
    g = torch.Generator(device="cuda").manual_seed(T + d)
    x = (torch.randn(T, d, generator=g, device=gpu) * torch.exp(0.3 * torch.randn(T, 1, generator=g, device=gpu))).bfloat16()
    wr = (torch.randn(E, d, generator=g, device=gpu) * d ** -0.5).bfloat16()
    weights, value = [], {}
    for name, rows, cols in (("w1", f, d), ("w3", f, d), ("w2", d, f)):
        if group:
            codes = torch.randint(-8, 8, (NL, rows, cols), dtype=torch.int8, generator=g, device=gpu)
            scale = torch.rand(NL, rows, -(-cols // group), generator=g, device=gpu) * 6e-3 + 2e-3
            weights.append((torch.cat([pack(c)[None] for c in codes]), scale))
            value[name] = lambda e, c=codes, s=scale, n=cols: c[e].double() * s[e].double().repeat_interleave(group, dim=1)[:, :n]
        else:
            w = torch.empty(NL, rows, cols, dtype=torch.bfloat16, device=gpu).normal_(0, 0.02, generator=g)
            weights.append(w)
            value[name] = lambda e, w=w: w[e].double()
    b = moe.DecodeBuffers(moe.make_desc(*shape[:5], e0, NL, "bf16"))
    _decode(b, x, wr, weights, group)
    want = torch.zeros(T, d, dtype=torch.float64, device=gpu)
    for e in range(NL):
        t, j = torch.nonzero(b.topk_idx - e0 == e, as_tuple=True)
        if len(t):
            G, U = (x[t].double() @ value[n](e).t().contiguous() for n in ("w1", "w3"))
            want.index_add_(0, t, b.topk_w[t, j][:, None].double() * ((G / (1 + torch.exp(-G)) * U) @ value["w2"](e).t().contiguous()))
    got, want = to_host(b.y), want.cpu().numpy()
    here = (want != 0).any(axis=1)  # (a token may have no local slot)
    assert (got[~here] == 0).all() and 2 * here.sum() >= T
    assert worst_block(got[here], want[here]) <= BLOCK_TOL
    assert worst_block(0.9 * got[here], want[here]) > BLOCK_TOL
    _pinned(lambda: _decode(b, x, wr, weights, group), form, group)

"""The whole-number layers of exact_layer.py against the layer's definition, and that mistakes show in them (CPU)."""
import numpy as np
import pytest
import torch

import oracle
from exact_layer import BLOCK_TOL, FORMS, Layer, bf, pack, worst_block

SMALL = [s for s, _, _ in FORMS if s[1] * s[2] * s[6] < 1 << 22]


def test_packed_codes_are_the_oracles():
    c = np.random.default_rng(1).integers(-8, 8, (5, 72)).astype(np.int8)
    np.testing.assert_array_equal(pack(torch.from_numpy(c)).numpy(), oracle.i4_pack(c))


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("shape", SMALL, ids=lambda s: "-".join(map(str, s)))
def test_the_sparse_sums_are_the_layer(shape, group):
    """y against oracle.layer_forward on the dense weights: silu(G) = G to 2^-28, h and y rounded to bf16 (2^-8 each; a term of
    y is at most 8 * 2 * 792 * 2^-8 off, six of them a slot), and the dense weights from the bytes that the kernels get."""
    a = Layer(*shape, group, seed=1)
    dense = {}
    for n in ("w1", "w3", "w2"):
        w = a.weights(n, "cpu")
        if group:
            q, s = w
            codes = oracle.i4_unpack(q.reshape(-1, q.shape[2]).numpy())
            dense[n] = oracle.i4_dequantize(codes, s.reshape(codes.shape[0], -1).numpy(), group).reshape(a.NL, q.shape[1], -1)
        else:
            dense[n] = w.double().numpy()
    ref = sum(oracle.layer_forward(a.x, np.zeros((a.E, a.d)), dense["w1"], dense["w3"], dense["w2"], 1, a.e0, a.NL,
                                   routing=(a.idx[:, j:j + 1], a.w[:, j:j + 1]))["y"] for j in range(a.k))  # (an expert may be named twice)
    room = np.zeros(a.T)
    np.add.at(room, np.nonzero((a.idx >= a.e0) & (a.idx < a.e0 + a.NL))[0], 1)
    assert (np.abs(a.y() - ref) <= 2.0 ** -8 * (np.abs(ref) + 2 * 6 * 8 * 2 * 792 * room[:, None] + 1)).all()
    assert (a.y() != 0).mean() > 0.5


@pytest.mark.parametrize("shape,form", [(s, f) for s, f, _ in FORMS] + [(s, f) for s, _, f in FORMS],
                         ids=lambda s: "-".join(map(str, s)))
def test_mistakes_show(shape, form):
    """A stage of k left out of one matrix, an expert left out, a group's scale twice over, zeros and nine tenths: y differs."""
    group = 0 if form[2] == 16 and form[1] in (2, 12, 16) else 64
    a = Layer(*shape, group, seed=2)
    want = a.y()
    T, d, f = shape[:3]
    step = 256 if group else 64
    rng = np.random.default_rng(3)
    for n, cols in (("w1", d), ("w3", d), ("w2", f)):
        for lo in {0, int(rng.integers(0, -(-cols // step))) * step, (cols - 1) // step * step}:
            assert (a.y(skip=(n, lo, lo + step)) != want).any(), (n, lo)
        assert (a.y(scales=(n, int(rng.integers(0, -(-cols // 64))))) != want).any()
    for e in set((a.idx - a.e0).ravel().tolist()):
        if 0 <= e < a.NL:
            assert (a.y(without=e) != want).any()
            break
    assert (want != 0).any() and (0.9 * want != want).any()


def test_blocks_tell_roundings_from_mistakes():
    """A down product with h and y rounded passes; zeros, nine tenths, one column, one of 24 shares of k and one of 64 groups with
    its scale half as large again do not."""
    rng = np.random.default_rng(5)
    h, w = rng.normal(0, 1, (3, 1536)), rng.normal(0, 0.02, (1536, 640))
    want = h @ w
    got = bf(bf(h).astype(np.float64) @ w).astype(np.float64)
    assert worst_block(got, want) <= BLOCK_TOL
    one, share, scale = got.copy(), w.copy(), w.copy()
    one[1, 100] *= -1
    share[64:128] = 0
    scale[24:48] *= 1.5
    for bad in (0 * got, 0.9 * got, one, h @ share, h @ scale, np.where(np.arange(640) == 9, np.nan, got)):
        assert worst_block(bad, want) > BLOCK_TOL

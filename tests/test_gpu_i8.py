"""The INT8 row quantiser and products on the GPU against the oracle's
whole-number arithmetic in float64.

Codes and scales must match bit for bit.  The products' integer sums are
exact, so their outputs are off by float32 roundings and one rounding to the
output type; with u = 2^-24 (float32) and U = 2^-8 (bf16; 0 for float32):
  linear  y = fl(fl(fl(S) xs) ws) + b: at most 3 u |p| for the product p, u for
          the bias' sum and U for the output: 4 u (|p| + |b|) + U |y|;
  G, U    3 u of the value, then U;
  h       silu(G) U in float32: G's 3 u weighs up to 1 + |G| in silu, exp(-G)
          costs |G| u for its argument and 2 u for itself, the sum, reciprocal
          and two products 5 u, U's 3 u: (13 + 4 |G|) u, then U; below 2^-100
          (exp(-G) past float32) anything goes to 0.
Bounds are on each value, doubled in their float32 part for second-order terms.
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_02_amd as moe
import oracle
import synth
from gpu_util import to_dev, to_host
from layer_checks import TOL, random_routing
from metrics import max_row_rel_err

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8
SENTINEL = 77


def _dev_rows(a, ld, dtype, fill):
    """Rows of a on the GPU, ld elements apart, `fill` in between."""
    t = torch.full((a.shape[0], ld), fill, dtype=dtype, device="cuda")
    t[:, :a.shape[1]] = torch.from_numpy(a).to("cuda").to(dtype)
    return t


def _special_rows(cols, dtype, seed=0):
    rng = np.random.default_rng(seed)
    w = rng.normal(0, 1, (24, cols)).astype(np.float32)
    w[1] = 0.0
    w[2] = -0.0
    w[3] = 0.0
    w[3, cols // 2] = -0.25
    w[4] *= 1e-38                                     # 127 / max overflows; subnormal bf16 and fp32 among them
    w[5] *= 1e-41
    w[6] *= 1e38 / 5
    w[7, cols - 1] = np.inf
    w[8, 0] = np.nan
    w[9, cols // 3] = -np.inf
    for r, m in ((10, 254.0), (11, 127 * 2.0 ** -30), (12, 1.7), (13, 3e-39), (14, 3e38), (15, 255.0)):
        n = rng.integers(-126, 126, cols)
        v = ((n + 0.5) / 127.0 * m).astype(np.float32)          # ties and their neighbours
        v = np.where(np.arange(cols) % 3 == 1, np.nextafter(v, np.float32(-3.4e38)), v)
        v = np.where(np.arange(cols) % 3 == 2, np.nextafter(v, np.float32(3.4e38)), v)
        w[r] = np.clip(v, -m, m)
        w[r, 0] = m
    return synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(w)) if dtype == "bf16" else w


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols,ldw,ldq", [(1, 1, 16), (7, 7, 16), (16, 16, 16), (63, 70, 64), (257, 264, 288), (1000, 1000, 1008),
                                          (1792, 1792, 1792), (2049, 2056, 2064), (6144, 6144, 6144), (6145, 6152, 6160),
                                          (20000, 20000, 20000), (20003, 20003, 20016)])
def test_quantize_rows_matches_the_oracle(gpu, dtype, cols, ldw, ldq):
    w = _special_rows(cols, dtype, cols)
    wd = _dev_rows(w, ldw, torch.bfloat16 if dtype == "bf16" else torch.float32, 1e30)
    q = torch.full((24, ldq), SENTINEL, dtype=torch.int8, device=gpu)
    s = torch.full((24,), -1.0, device=gpu)
    moe.i8_quantize_rows(wd[:, :cols], q[:, :cols], s)
    codes, scale = oracle.i8_quantize_rows(w)
    np.testing.assert_array_equal(s.cpu().numpy(), scale)
    np.testing.assert_array_equal(q[:, :cols].cpu().numpy(), codes)
    assert (q[:, cols:] == SENTINEL).all()


@pytest.mark.parametrize("rows,nrows", [(1, 1), (5, 0), (1000, 999), (40000, 1), (40000, 50000), (3, -2)])
def test_quantize_rows_leaves_rows_past_nrows(gpu, rows, nrows):
    w = np.random.default_rng(rows).normal(0, 1, (rows, 64)).astype(np.float32)
    q = torch.full((rows, 64), SENTINEL, dtype=torch.int8, device=gpu)
    s = torch.full((rows,), -1.0, device=gpu)
    moe.i8_quantize_rows(torch.from_numpy(w).cuda(), q, s, nrows=torch.tensor([nrows], dtype=torch.int32, device=gpu))
    n = max(0, min(rows, nrows))
    codes, scale = oracle.i8_quantize_rows(w)
    np.testing.assert_array_equal(q[:n].cpu().numpy(), codes[:n])
    np.testing.assert_array_equal(s[:n].cpu().numpy(), scale[:n])
    assert (q[n:] == SENTINEL).all() and (s[n:] == -1).all()


def _codes(rng, *shape):
    return rng.integers(-127, 128, shape, dtype=np.int8)


def _scales(rng, *shape):
    return (rng.random(shape) * 1e-3 + 1e-4).astype(np.float32)


def _within(got, ref, slack, bf16):
    """|got - ref| within slack (float32 part) and the output's own rounding."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    tol = 2 * slack + (UBF if bf16 else 0.0) * (np.abs(ref) + 2 * slack) + 2.0 ** -100
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4])


def _linear(gpu, M, N, K, dtype, bias, pad=0, seed=0, codes=None):
    rng = np.random.default_rng([M, N, K, seed])
    xq, wq = (_codes(rng, M, K), _codes(rng, N, K)) if codes is None else codes
    xs, ws = _scales(rng, M), _scales(rng, N)
    b = rng.normal(0, 1, N).astype(np.float32) if bias else None
    ld = (K + 15) // 16 * 16
    X = _dev_rows(xq, ld + 16 * pad, torch.int8, 127)          # what follows a row is not zero
    W = _dev_rows(wq, ld + 32 * pad, torch.int8, -127)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    Y = torch.full((M, N + pad), float(SENTINEL), dtype=dt, device=gpu)
    moe.i8_linear(X[:, :K], to_dev(xs), W[:, :K], to_dev(ws), Y[:, :N], bias=None if b is None else to_dev(b))
    p = oracle.i8_linear(xq, xs, wq, ws)
    ref = p if b is None else p + b
    _within(to_host(Y[:, :N].contiguous()), ref, 4 * U32 * (np.abs(p) + (0 if b is None else np.abs(b))), dtype == "bf16")
    assert (Y[:, N:] == SENTINEL).all()


@pytest.mark.parametrize("dtype,bias", [("bf16", False), ("f32", True)])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 16, 16), (1, 3, 17), (2, 64, 128), (15, 63, 127), (16, 65, 129), (17, 1003, 1990),
                                   (31, 32, 33), (33, 48, 512), (63, 128, 640), (64, 64, 64), (65, 100, 1000), (1, 3584, 6144),
                                   (130, 260, 1024), (257, 257, 1024), (300, 520, 2048), (1000, 777, 1537), (513, 1024, 6144),
                                   (500, 2500, 100), (1500, 3150, 100), (2600, 2601, 130), (8200, 6144, 512), (2040, 6136, 2048),
                                   (1100, 23000, 100)])
def test_linear_matches_the_oracle(gpu, M, N, K, dtype, bias):
    _linear(gpu, M, N, K, dtype, bias)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,pad", [(5, 40, 100, 1), (40, 72, 256, 3), (300, 512, 1024, 8), (700, 264, 1000, 5), (1100, 2050, 1536, 7)])
def test_linear_with_rows_apart(gpu, M, N, K, pad, dtype):
    _linear(gpu, M, N, K, dtype, True, pad)


@pytest.mark.parametrize("M", [1, 20, 70, 520])
def test_linear_sums_of_the_largest_codes_do_not_overflow(gpu, M):
    K = 131072
    _linear(gpu, M, 520, K, "f32", False, codes=(np.full((M, K), 127, np.int8), np.full((520, K), -127, np.int8)))


@pytest.mark.parametrize("dtype,bias", [("bf16", True), ("f32", False)])
@pytest.mark.parametrize("M,N,K", [(1, 6144, 4096), (1, 5, 4097), (16, 1003, 4223), (17, 100, 8191), (40, 33, 6000), (130, 31, 131072)])
def test_linear_of_few_channels_and_a_long_k(gpu, M, N, K, dtype, bias):
    _linear(gpu, M, N, K, dtype, bias)


def test_linear_of_no_rows(gpu):
    w = torch.zeros(8, 16, dtype=torch.int8, device=gpu)
    s = torch.zeros(8, device=gpu)
    moe.i8_linear(w[:0], s, w, s, torch.empty(0, 8, device=gpu))
    moe.i8_quantize_rows(torch.empty(0, 16, device=gpu), w[:0], s)
    torch.cuda.synchronize()


def test_linear_beyond_32_bit_offsets(gpu):
    """Weights of 2.1 GiB and an output of 2.2 G values: sampled entries against the oracle."""
    rng = np.random.default_rng(3)
    for M, N, K in ((2, 17000, 131072), (40000, 56000, 32)):
        xq = torch.randint(-127, 128, (M, K), dtype=torch.int8, device=gpu)
        wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=gpu)
        xs, ws = torch.rand(M, device=gpu), torch.rand(N, device=gpu)
        y = torch.empty(M, N, dtype=torch.bfloat16, device=gpu)
        moe.i8_linear(xq, xs, wq, ws, y)
        m = np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, 40)]))
        n = np.unique(np.concatenate([[0, N - 1], rng.integers(0, N, 40)]))
        ref = oracle.i8_linear(xq[m].cpu().numpy(), xs[m].cpu().numpy(), wq[n].cpu().numpy(), ws[n].cpu().numpy())
        _within(to_host(y[m][:, n].contiguous()), ref, 4 * U32 * np.abs(ref), True)
        del y, wq


@pytest.mark.parametrize("M,N,K,ldx,ldw,ldy", [(40, 1100, 300, 1 << 22, 1 << 22, 1 << 26), (1100, 2050, 1536, 1 << 22, 1 << 22, 1 << 21),
                                               (8200, 6144, 512, 1 << 20, 1 << 20, 1 << 19), (2400001, 1024, 512, 512, 512, 1024)])
def test_linear_of_rows_far_apart(gpu, M, N, K, ldx, ldw, ldy):
    """Every operand past 32-bit offsets, through each kind of kernel: sampled rows in whole, every value written."""
    rng = np.random.default_rng(M)
    X = torch.empty(M, ldx, dtype=torch.int8, device=gpu)[:, :K]
    W = torch.empty(N, ldw, dtype=torch.int8, device=gpu)[:, :K]
    Y = torch.empty(M, ldy, dtype=torch.bfloat16, device=gpu)[:, :N]
    X.random_(-127, 128)
    W.random_(-127, 128)
    Y.fill_(float("nan"))
    xs, ws = torch.rand(M, device=gpu), torch.rand(N, device=gpu)
    moe.i8_linear(X, xs, W, ws, Y)
    assert not torch.isnan(Y).any()
    m = np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, 30)]))
    ref = oracle.i8_linear(X[m].cpu().numpy(), xs[m].cpu().numpy(), W.cpu().numpy(), ws.cpu().numpy())
    _within(to_host(Y[m].contiguous()), ref, 4 * U32 * np.abs(ref), True)


def test_quantize_rows_far_apart(gpu):
    w = torch.empty(70000, 1 << 16, dtype=torch.bfloat16, device=gpu)[:, :300]
    q = torch.empty(70000, 1 << 16, dtype=torch.int8, device=gpu)[:, :300]
    w.normal_()
    s = torch.empty(70000, device=gpu)
    moe.i8_quantize_rows(w, q, s)
    for m in (slice(0, 50), slice(32750, 32800), slice(65500, 65560), slice(69950, 70000)):
        codes, scale = oracle.i8_quantize_rows(w[m].float().cpu().numpy())
        np.testing.assert_array_equal(q[m].cpu().numpy(), codes)
        np.testing.assert_array_equal(s[m].cpu().numpy(), scale)


# ---- the expert products ----------------------------------------------------

SHAPES = {  # T, d, f, E, k, e0, NL, skew
    "one token": (1, 128, 64, 8, 2, 0, 8, 0.0),
    "one token, none local": (1, 128, 64, 64, 1, 63, 1, 0.0),
    "odd sizes": (37, 192, 448, 24, 3, 5, 13, 0.0),
    "many experts, few rows": (50, 256, 128, 1024, 4, 100, 700, 0.0),
    "about 16 rows": (180, 512, 192, 32, 3, 0, 32, 0.0),
    "about 60 rows": (500, 640, 320, 40, 5, 8, 32, 0.3),
    "one busy expert": (1500, 576, 256, 16, 2, 0, 16, 3.0),
    "tails of 256": (2300, 1024, 512, 8, 2, 1, 6, 0.0),
    "long": (5000, 768, 640, 16, 4, 0, 16, 0.5),
    "1T sizes": (300, 6144, 1792, 16, 2, 0, 4, 0.0),
    # enough tiles for the larger tiles of the few-rows kernel and the shared-operand kernel; K in half chunks
    "6 rows, many tiles": (48, 832, 448, 64, 8, 0, 64, 0.0),
    "20 rows, many tiles": (160, 832, 448, 64, 8, 0, 64, 0.0),
    "5 rows, very many tiles": (120, 832, 448, 192, 8, 0, 192, 0.5),
    "40 rows, many tiles": (480, 832, 448, 96, 8, 0, 96, 0.0),
    "75 rows, many tiles": (600, 832, 448, 64, 8, 0, 64, 0.0),
    "125 rows, many tiles": (1000, 832, 448, 64, 8, 0, 64, 0.0),
    "125 rows, skewed": (1000, 832, 448, 64, 8, 0, 64, 1.0),
    "180 rows, many tiles": (1440, 832, 448, 64, 8, 0, 64, 0.0),
    "180 rows, skewed": (1440, 832, 448, 64, 8, 0, 64, 0.6),
    "about 330 rows, many tiles": (1300, 1792, 1024, 32, 8, 0, 32, 0.3),
    "500 rows, K no multiple of 128": (2000, 832, 448, 32, 8, 0, 32, 0.3),
}


def _layer(name, gpu, dyn=False, scale=1.0):
    T, d, f, E, k, e0, NL, skew = SHAPES[name]
    rng = np.random.default_rng(T + d)
    D = moe.make_desc(T, d, f, E, k, e0, NL, "bf16", tile_counters=moe.new_tile_counters() if dyn else None)
    idx = random_routing(rng, T, E, k, skew)
    b = moe.Buffers(D, gather=True)
    moe.permute(D, to_dev(idx), None, b.counts, b.offsets, b.row_token, b.slot_row, None, b.ws_permute)
    off = b.offsets.cpu().numpy()
    tok = b.row_token.cpu().numpy()[:off[-1]]
    c = dict(rng=rng, D=D, b=b, off=off, tok=tok, idx=idx)
    c["xq"], c["xs"] = _codes(rng, T, d), _scales(rng, T) * scale
    for n, (r, m) in (("w1", (f, d)), ("w3", (f, d)), ("w2", (d, f))):
        c[n + "q"], c[n + "s"] = _codes(rng, NL, r, m), _scales(rng, NL, r)
    return c


def _products(c, rows, rs, wq, ws):
    """Exact products of rows [R][K] with their experts' weights, scaled in float64."""
    out = np.zeros((rows.shape[0], wq.shape[1]))
    for n in range(len(c["off"]) - 1):
        a, z = c["off"][n], c["off"][n + 1]
        if z > a:
            out[a:z] = oracle.i8_linear(rows[a:z], rs[a:z], wq[n], ws[n])
    return out


@pytest.mark.parametrize("gu,dyn", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("name", list(SHAPES))
def test_gate_up_matches_the_oracle(gpu, name, gu, dyn):
    c = _layer(name, gpu, dyn)
    D, R = c["D"], c["off"][-1]
    f = D.f
    h = torch.full((D.R_cap, f), float(SENTINEL), dtype=torch.bfloat16, device=gpu)
    g = torch.full((D.R_cap, 2 * f), float(SENTINEL), dtype=torch.bfloat16, device=gpu) if gu else None
    for _ in range(2):                                         # (the dynamic order's counters are left zero)
        moe.expert_gate_up_i8(D, c["b"].offsets, c["b"].row_token, to_dev(c["xq"]), to_dev(c["xs"]), to_dev(c["w1q"]),
                              to_dev(c["w1s"]), to_dev(c["w3q"]), to_dev(c["w3s"]), g, h)
    rows, rs = c["xq"][c["tok"]], c["xs"][c["tok"]]
    G, U = _products(c, rows, rs, c["w1q"], c["w1s"]), _products(c, rows, rs, c["w3q"], c["w3s"])
    H = G / (1 + np.exp(-G)) * U
    _within(to_host(h[:R]), H, U32 * (13 + 4 * np.abs(G)) * np.abs(H), True)
    assert (h[R:] == SENTINEL).all()
    if gu:
        _within(to_host(g[:R]), np.concatenate([G, U], 1), 3 * U32 * np.abs(np.concatenate([G, U], 1)), True)
        assert (g[R:] == SENTINEL).all()


def test_gate_up_of_large_and_of_not_finite_rows(gpu):
    """|G| past the range of exp, and a token whose scale is NaN: its rows alone are NaN."""
    c = _layer("about 60 rows", gpu, scale=4000.0)
    c["xs"][3] = np.nan
    D, R = c["D"], c["off"][-1]
    h = torch.empty(D.R_cap, D.f, dtype=torch.bfloat16, device=gpu)
    moe.expert_gate_up_i8(D, c["b"].offsets, c["b"].row_token, to_dev(c["xq"]), to_dev(c["xs"]), to_dev(c["w1q"]),
                          to_dev(c["w1s"]), to_dev(c["w3q"]), to_dev(c["w3s"]), None, h)
    got = to_host(h[:R])
    nan = c["tok"] == 3
    assert nan.any() and np.isnan(got[nan]).all()
    rows, rs = c["xq"][c["tok"]], np.where(nan, 0, c["xs"][c["tok"]])
    G, U = _products(c, rows, rs, c["w1q"], c["w1s"]), _products(c, rows, rs, c["w3q"], c["w3s"])
    assert np.abs(G).max() > 100
    with np.errstate(over="ignore"):
        H = G / (1 + np.exp(-G)) * U
    _within(got[~nan], H[~nan], (U32 * (13 + 4 * np.abs(G)) * np.abs(H))[~nan], True)


@pytest.mark.parametrize("dyn", [False, True])
@pytest.mark.parametrize("name", list(SHAPES))
def test_down_matches_the_oracle(gpu, name, dyn):
    c = _layer(name, gpu, dyn)
    D, R, rng = c["D"], c["off"][-1], c["rng"]
    hq, hs = _codes(rng, D.R_cap, D.f), _scales(rng, D.R_cap)
    hs[R:] = np.nan                                            # rows past the last segment are not read
    y = torch.full((D.R_cap, D.d), float(SENTINEL), dtype=torch.bfloat16, device=gpu)
    for _ in range(2):
        moe.expert_down_i8(D, c["b"].offsets, to_dev(hq), to_dev(hs), to_dev(c["w2q"]), to_dev(c["w2s"]), y)
    Y = _products(c, hq[:R], hs[:R], c["w2q"], c["w2s"])
    _within(to_host(y[:R]), Y, 3 * U32 * np.abs(Y), True)
    assert (y[R:] == SENTINEL).all()


@pytest.mark.parametrize("T,groups", [(1, 1), (70, 2), (2500, 1)])
def test_forward_i8_matches_the_oracle(gpu, T, groups):
    """The layer end to end: the codes of x and of the layer's own h bit for bit, y against the products of those
    codes, and the whole against the oracle's layer on the weights the codes stand for."""
    cfg = synth.Config("t", 7, T, 512, 16, 4, 256, 0, 16, "bf16", 1.0, "router", False)
    inp = synth.make_inputs(cfg)
    D = moe.make_desc(T, cfg.d, cfg.f, cfg.E, cfg.k, 0, 16, "bf16")
    dev = {n: to_dev(inp[n]) for n in ("x", "wr", "w1", "w3", "w2")}
    b, i8, ex = moe.Buffers(D, gather=True), moe.Int8Buffers(D), moe.Int8Experts(dev["w1"], dev["w3"], dev["w2"])
    y = to_host(moe.forward_i8(b, i8, dev["x"], dev["wr"], ex, n_groups=groups))
    wide = {n: synth.as_f32(inp[n], "bf16") for n in ("x", "w1", "w3", "w2")}
    deq = {}
    for n in ("w1", "w3", "w2"):
        codes, scale = oracle.i8_quantize_rows(wide[n].reshape(-1, wide[n].shape[-1]))
        np.testing.assert_array_equal(getattr(ex, n + "q").cpu().numpy().reshape(codes.shape), codes)
        np.testing.assert_array_equal(getattr(ex, n + "s").cpu().numpy().reshape(-1), scale)
        deq[n] = oracle.i8_dequantize_rows(codes, scale).reshape(wide[n].shape)
    xc, xs = oracle.i8_quantize_rows(wide["x"])
    np.testing.assert_array_equal(i8.xq.cpu().numpy(), xc)
    R = int(b.offsets[-1])
    hc, hs = oracle.i8_quantize_rows(to_host(b.h[:R]))
    np.testing.assert_array_equal(i8.hq[:R].cpu().numpy(), hc)
    off, tok, slot, w = (t.cpu().numpy() for t in (b.offsets, b.row_token, b.slot_row, b.topk_w))
    xd = oracle.i8_dequantize_rows(xc, xs)
    _, _, H, _ = oracle.expert_ffn(xd[tok[:R]], off, deq["w1"], deq["w3"], deq["w2"])
    assert max_row_rel_err(to_host(b.h[:R]), H) <= TOL["bf16"]
    Y = oracle.expert_down(oracle.i8_dequantize_rows(hc, hs), off, deq["w2"])
    assert max_row_rel_err(y, oracle.combine(Y, slot, w)) <= TOL["bf16"]


def test_captured_forward_and_two_streams(gpu):
    """A captured forward replayed on new inputs between eager work, and two layers running at once on two streams,
    give bitwise what one eager call gives."""
    cfg = synth.Config("t", 9, 300, 512, 16, 4, 256, 0, 16, "bf16", 1.0, "router", False)
    inp = [synth.make_inputs(synth.scaled(cfg, seed=s)) for s in (1, 2, 3)]
    D = moe.make_desc(cfg.T, cfg.d, cfg.f, cfg.E, cfg.k, 0, 16, "bf16")
    w = {n: to_dev(inp[0][n]) for n in ("wr", "w1", "w3", "w2")}
    ex = moe.Int8Experts(w["w1"], w["w3"], w["w2"])
    xs = [to_dev(i["x"]) for i in inp]
    b, i8 = moe.Buffers(D, gather=True), moe.Int8Buffers(D)
    want = [moe.forward_i8(b, i8, x, w["wr"], ex).clone() for x in xs]
    x = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        moe.forward_i8(b, i8, x, w["wr"], ex)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.y, want[i])
        assert torch.isfinite(x.float().sum())
    sets = [(moe.Buffers(D, gather=True), moe.Int8Buffers(D)) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                moe.forward_i8(*sets[j], xs[j], w["wr"], ex)
    torch.cuda.synchronize()
    for j in range(2):
        assert torch.equal(sets[j][0].y, want[j])


def test_python_checks_of_the_expert_calls(gpu):
    c = _layer("odd sizes", gpu)
    D, b = c["D"], c["b"]
    a = dict(offsets=b.offsets, row_token=b.row_token, xq=to_dev(c["xq"]), xs=to_dev(c["xs"]), w1q=to_dev(c["w1q"]),
             w1s=to_dev(c["w1s"]), w3q=to_dev(c["w3q"]), w3s=to_dev(c["w3s"]), gu=None, h=b.h)
    for n, bad in (("xq", a["xq"][:-1]), ("xq", a["xq"].float()), ("w1q", a["w1q"].transpose(1, 2)), ("h", b.h[:-1]),
                   ("xs", a["xs"].double()), ("offsets", b.offsets[:-1]), ("xq", a["xq"].cpu())):
        with pytest.raises(ValueError):
            moe.expert_gate_up_i8(D, **{**a, n: bad})
    with pytest.raises(ValueError):
        moe.expert_down_i8(D, b.offsets, torch.empty(D.R_cap, D.f, device=gpu), a["xs"], a["w1q"], a["w1s"], b.y_perm)
    with pytest.raises(ValueError):
        moe.i8_linear(a["xq"].t(), a["xs"], a["xq"], a["xs"], b.h)


@pytest.mark.parametrize("per", [2, 60, 200])
def test_experts_whose_weights_pass_32_bit_offsets(gpu, per):
    """96 experts of 25 M weights each, 2.4 GiB a matrix; the last one among those that have rows."""
    E, d, f = 96, 4096, 6272
    T = per * E
    D = moe.make_desc(T, d, f, E, 1, 0, E, "bf16")
    idx = torch.full((T, 1), E - 1, dtype=torch.int32, device=gpu)
    idx[: T // 3] = 0
    b = moe.Buffers(D, gather=True)
    moe.permute(D, idx, None, b.counts, b.offsets, b.row_token, b.slot_row, None, b.ws_permute)
    w = [torch.empty(E, r, c, dtype=torch.int8, device=gpu) for r, c in ((f, d), (f, d), (d, f))]
    s = [torch.rand(E, r, device=gpu) * 1e-3 + 1e-4 for r in (f, f, d)]
    for v in w:
        for e in (0, E - 1):
            v[e].random_(-127, 128)
    xq = torch.empty(T, d, dtype=torch.int8, device=gpu).random_(-127, 128)
    hq = torch.empty(T, f, dtype=torch.int8, device=gpu).random_(-127, 128)
    xs, hs = torch.rand(T, device=gpu) * 1e-3 + 1e-4, torch.rand(T, device=gpu) * 1e-3 + 1e-4
    moe.expert_gate_up_i8(D, b.offsets, b.row_token, xq, xs, w[0], s[0], w[1], s[1], None, b.h)
    moe.expert_down_i8(D, b.offsets, hq, hs, w[2], s[2], b.y_perm)
    tok = b.row_token.cpu().numpy()
    cut = T // 3
    for e, rows in ((0, [0, cut - 1]), (E - 1, [cut, (cut + T) // 2, T - 1])):
        a, z = xq.cpu().numpy()[tok[rows]], xs.cpu().numpy()[tok[rows]]
        G, U = (oracle.i8_linear(a, z, w[j][e].cpu().numpy(), s[j][e].cpu().numpy()) for j in (0, 1))
        H = G / (1 + np.exp(-G)) * U
        _within(to_host(b.h[rows]), H, U32 * (13 + 4 * np.abs(G)) * np.abs(H), True)
        Y = oracle.i8_linear(hq.cpu().numpy()[rows], hs.cpu().numpy()[rows], w[2][e].cpu().numpy(), s[2][e].cpu().numpy())
        _within(to_host(b.y_perm[rows]), Y, 3 * U32 * np.abs(Y), True)

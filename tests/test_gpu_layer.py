"""The operators that run a calibrated layer, on the GPU, against the oracle and plain FP64: tokens sorted by expert,
rows gathered and combined with the gradient, NVFP4 tokens, NVFP4 products, and all of them in a run."""
import numpy as np
import pytest
import torch

import oracle
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step, relative


def _lh():
    import scale_calibration_b200 as lh
    return lh


def pitch(c, t):
    per = 8 if t == "bf16" else 4
    return -(-max(c, 1) // per) * per


def rows_of(rng, n, c, t, fill=None):
    """(device buffer with padded rows, its [n, c] values in f64)."""
    b = torch.full((n, pitch(c, t)), -7.0, dtype=DT[t], device="cuda")
    v = torch.from_numpy(rng.standard_normal((n, c)).astype(np.float32)).to(DT[t])
    b[:, :c] = v.cuda()
    return b, v.double().numpy()


# ---------------------------------------------------------------- route

@pytest.mark.parametrize("n,k,e,kind", [
    (0, 2, 5, "any"), (1, 1, 1, "any"), (1, 8, 64, "any"), (48, 4, 64, "any"), (33, 3, 7, "masked"),
    (1000, 2, 16, "all masked"), (513, 1, 1024, "any"), (4096, 1, 8, "one"), (4097, 1, 8, "any"),
    (9000, 8, 96, "masked"), (70000, 3, 1000, "any"), (40001, 1, 3, "one"), (2048, 6, 64, "same twice"),
])
def test_route_is_the_stable_sort(cuda_ok, n, k, e, kind):
    lh = _lh()
    rng = np.random.default_rng(n * 31 + k + e)
    ids = rng.integers(0, e, (n, k)).astype(np.int32)
    if kind == "masked":
        ids[rng.random((n, k)) < 0.3] = -1
        ids[rng.random((n, k)) < 0.05] = e
        ids[rng.random((n, k)) < 0.02] = np.iinfo(np.int32).min
    elif kind == "all masked":
        ids[:] = -1
    elif kind == "one":
        ids[:] = e - 1
    elif kind == "same twice":
        ids[:, 1] = ids[:, 0]
    d = torch.from_numpy(ids).cuda()
    off = torch.full((e + 1,), -5, dtype=torch.int64, device="cuda")
    order = torch.full((n * k + 3,), 12345, dtype=torch.int32, device="cuda")
    pos = torch.full((n * k + 3,), 12345, dtype=torch.int32, device="cuda")
    lh.lh_route_tokens(d, n, k, e, off, order, pos)
    ro, rr, rp = ref.route(ids, e)
    assert np.array_equal(off.cpu().numpy(), ro)
    assert np.array_equal(order.cpu().numpy()[:n * k], rr) and (order[n * k:] == 12345).all()
    assert np.array_equal(pos.cpu().numpy()[:n * k], rp) and (pos[n * k:] == 12345).all()


# ---------------------------------------------------------------- gather, combine, gradient

CASES = [(1, 1, 3, 1), (5, 2, 4, 7), (48, 4, 64, 1536), (37, 3, 5, 129), (300, 8, 16, 264), (1, 8, 64, 2048), (64, 2, 3, 3)]


def routed(rng, n, k, e, masked=True):
    ids = rng.integers(0, e, (n, k)).astype(np.int32)
    if masked and n > 2:
        ids[rng.random((n, k)) < 0.2] = -1
        ids[0] = -1  # a token without any expert
    return ref.route(ids, e)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,e,c", CASES)
def test_gather_copies_the_rows(cuda_ok, n, k, e, c, t):
    lh = _lh()
    rng = np.random.default_rng(c)
    _, order, _ = routed(rng, n, k, e)
    x, _ = rows_of(rng, n, c, t)
    xs = torch.full((n * k, pitch(c, t)), 3.0, dtype=DT[t], device="cuda")
    want = xs.clone()
    for p, f in enumerate(order):
        if f >= 0:
            want[p, :c] = x[f // k, :c]
    lh.lh_gather_tokens(x, x, n, c, x.stride(0), torch.from_numpy(order).cuda(), k, n * k, xs, xs.stride(0))
    assert torch.equal(xs, want)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("n,k,e,c", CASES)
def test_combine_is_the_weighted_sum(cuda_ok, n, k, e, c, weighted, t):
    lh = _lh()
    rng = np.random.default_rng(c + k)
    _, _, pos = routed(rng, n, k, e)
    ys, yv = rows_of(rng, n * k, c, t)
    used = np.zeros(n * k, bool)
    used[pos[pos >= 0]] = True
    ys[torch.from_numpy(~used).cuda()] = float("nan")  # rows that nothing names are not read
    w = rng.standard_normal((n, k)).astype(np.float32)
    y = torch.full((n, pitch(c, t)), 5.0, dtype=DT[t], device="cuda")
    lh.lh_combine_tokens(ys, ys, n * k, c, ys.stride(0), torch.from_numpy(pos).cuda(),
                         torch.from_numpy(w).cuda() if weighted else None, n, k, y, y.stride(0))
    wm = (w if weighted else np.ones_like(w)).astype(np.float64) * (pos.reshape(n, k) >= 0)
    terms = wm[:, :, None] * np.where(used[:, None], yv, 0)[np.maximum(pos, 0)].reshape(n, k, c)
    want, mag = terms.sum(1), np.abs(terms).sum(1)
    got = y.double().cpu().numpy()
    tol = k * 2.0 ** -24 * mag  # k fused multiply-adds, each rounded once
    tol = tol + (np.abs(want) + tol) * HALF[t]
    assert (np.abs(got[:, :c] - want) <= tol).all()
    assert (got[:, c:] == 5.0).all()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("n,k,e,c", CASES)
def test_combine_gradient_is_the_formula(cuda_ok, n, k, e, c, weighted, t):
    lh = _lh()
    rng = np.random.default_rng(c + 3 * k)
    _, _, pos = routed(rng, n, k, e)
    ys, yv = rows_of(rng, n * k, c, t)
    dy, dv = rows_of(rng, n, c, t)
    w = rng.standard_normal((n, k)).astype(np.float32)
    wd = torch.from_numpy(w).cuda() if weighted else None
    pd = torch.from_numpy(pos).cuda()
    dys = torch.full((n * k, pitch(c, t)), 9.0, dtype=DT[t], device="cuda")
    dw = torch.full((n, k), 9.0, device="cuda")
    lh.lh_combine_tokens_grad(dy, dy, n, k, c, dy.stride(0), ys, ys.stride(0), n * k, pd, wd, dys, dys.stride(0), dw)
    got, gw = dys.double().cpu().numpy(), dw.double().cpu().numpy()
    wm = (w if weighted else np.ones_like(w)).astype(np.float64)
    want = np.full((n * k, c), 9.0)
    ww, wt = np.zeros((n, k)), np.zeros((n, k))
    for f, p in enumerate(pos):
        if p >= 0:
            t0, s = f // k, f % k
            want[p] = wm[t0, s] * dv[t0]
            ww[t0, s] = dv[t0] @ yv[p]
            wt[t0, s] = np.abs(dv[t0]) @ np.abs(yv[p])
    # one product rounded to FP32, then to the type
    assert (np.abs(got[:, :c] - want) <= np.abs(want) * (2.0 ** -24 + HALF[t] * (1 + 2.0 ** -24))).all()
    assert (got[:, c:] == 9.0).all()
    # c products and sums in FP32
    assert (np.abs(gw - ww) <= (c + 5) * 2.0 ** -24 * wt).all()
    # each output alone
    d2, w2 = torch.full_like(dys, 9.0), torch.full_like(dw, 9.0)
    lh.lh_combine_tokens_grad(dy, dy, n, k, c, dy.stride(0), None, 0, n * k, pd, wd, d2, d2.stride(0), None)
    lh.lh_combine_tokens_grad(dy, dy, n, k, c, dy.stride(0), ys, ys.stride(0), n * k, pd, wd, None, 0, w2)
    assert torch.equal(d2, dys) and torch.equal(w2, dw)


def test_combine_gradient_is_that_of_differences(cuda_ok):
    # the combination is linear in Ys and in the weights: its difference quotient is the gradient up to rounding
    lh = _lh()
    rng = np.random.default_rng(0)
    n, k, e, c = 9, 3, 4, 40
    _, _, pos = routed(rng, n, k, e)
    pd = torch.from_numpy(pos).cuda()
    ys, _ = rows_of(rng, n * k, c, "f32")
    dy, dv = rows_of(rng, n, c, "f32")
    w = torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32)).cuda()
    dys, dw = torch.zeros_like(ys), torch.zeros_like(w)
    lh.lh_combine_tokens_grad(dy, dy, n, k, c, c, ys, c, n * k, pd, w, dys, c, dw)

    def loss(ys_, w_):
        y = torch.empty(n, c, device="cuda")
        lh.lh_combine_tokens(ys_, ys_, n * k, c, c, pd, w_, n, k, y, c)
        return float((y.double().cpu().numpy() * dv).sum())

    base = loss(ys, w)
    for _ in range(5):
        p, i = int(rng.choice(pos[pos >= 0])), int(rng.integers(c))
        y2 = ys.clone()
        y2[p, i] += 1.0
        assert abs(loss(y2, w) - base - float(dys[p, i])) <= 1e-4
        t, s = int(rng.integers(n)), int(rng.integers(k))
        w2 = w.clone()
        w2[t, s] += 1.0
        assert abs(loss(ys, w2) - base - float(dw[t, s])) <= 1e-4


def test_gather_and_unweighted_combine_are_adjoint(cuda_ok):
    # <gather(X), G> = <X, combine(G)>: small whole numbers, so both sides are exact
    lh = _lh()
    rng = np.random.default_rng(4)
    n, k, e, c = 50, 4, 6, 72
    _, order, pos = routed(rng, n, k, e)
    x = torch.from_numpy(rng.integers(-4, 5, (n, c)).astype(np.float32)).cuda()
    g = torch.from_numpy(rng.integers(-4, 5, (n * k, c)).astype(np.float32)).cuda()
    xs, dx = torch.zeros_like(g), torch.zeros_like(x)
    lh.lh_gather_tokens(x, x, n, c, c, torch.from_numpy(order).cuda(), k, n * k, xs, c)
    lh.lh_combine_tokens(g, g, n * k, c, c, torch.from_numpy(pos).cuda(), None, n, k, dx, c)
    assert float((xs.double() * g.double()).sum()) == float((x.double() * dx.double()).sum())


# ---------------------------------------------------------------- NVFP4 tokens

def quantize(x, n_src, c, rows=None, row_div=1, n_rows=None, offsets=None, amax=None, out=None):
    lh = _lh()
    n_rows = n_src if n_rows is None else n_rows
    G = 1 if offsets is None else offsets.numel() - 1
    packed = torch.full((n_rows, c // 2), 0xEE, dtype=torch.uint8, device="cuda")
    tiles = torch.full((max(lh.lh_nvfp4_token_scale_bytes(n_rows, c, G), 1),), 0xEE, dtype=torch.uint8, device="cuda")
    g = torch.full((n_rows,), -3.0, device="cuda")
    values = torch.full((n_rows, c), -3.0, dtype=out, device="cuda") if out is not None else None
    lh.lh_quantize_tokens(x, x, n_src, c, x.stride(0), rows, row_div, n_rows, offsets, G, amax, packed, tiles, g,
                          values, values if out is not None else x)
    return packed, tiles, g, values


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["token", "tensor", "small amax"])
@pytest.mark.parametrize("n,c", [(1, 16), (3, 48), (130, 64), (1, 4096), (129, 272), (33, 4112), (260, 80), (5, 17408)])
def test_tokens_match_the_oracle(cuda_ok, n, c, mode, t):
    rng = np.random.default_rng(n + c)
    v = rng.standard_normal((n, c)).astype(np.float32) * np.exp(rng.standard_normal(c)).astype(np.float32)
    v[rng.random((n, c)) < 0.1] = 0
    v[rng.random((n, c)) < 0.05] *= -0.0
    if n > 2:
        v[1] = 0           # a token of zeros
        v[2] *= 2.0 ** -120  # and a tiny one
    x = torch.from_numpy(v).to(DT[t])
    v = x.float().numpy()
    amax = None if mode == "token" else np.float32(np.abs(v).max() * (1 if mode == "tensor" else 0.1))
    da = None if amax is None else torch.tensor([amax], device="cuda")
    buf = torch.full((n, c + 16), 1e9, dtype=DT[t], device="cuda")  # a leading dimension beyond c
    buf[:, :c] = x.cuda()
    packed, tiles, g, values = quantize(buf, n, c, amax=da, out=torch.float32)
    rp, rc, rg, rv = ref.quantize_tokens(v, amax)
    assert np.array_equal(g.cpu().numpy().view(np.uint32), rg.view(np.uint32))
    got = ref.untile(tiles.cpu().numpy(), n, c // 16)
    assert np.array_equal(got[:, :c // 16], rc) and (got[:, c // 16:] == 0).all()
    assert np.array_equal(packed.cpu().numpy(), rp)
    assert np.array_equal(values.cpu().numpy().view(np.uint32), rv.view(np.uint32))
    _, _, _, vb = quantize(buf, n, c, amax=da, out=torch.bfloat16)
    assert torch.equal(vb.cpu().view(torch.int16), torch.from_numpy(rv).to(torch.bfloat16).view(torch.int16))


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("amax", [0.0, 1e-42, 1e-37, 1e-30, 1e-20, 1.0, 1e20, 3e33, 3e38])
def test_tokens_far_from_the_given_amax(cuda_ok, amax, t):
    # every order of magnitude against scales at both ends of the range: they saturate, or vanish, with their signs
    rng = np.random.default_rng(3)
    v = np.ldexp(rng.choice([-1.0, 1.0], (60, 64)) * (1 + rng.random((60, 64))), np.arange(-126, 114, 4)[:, None])
    x = torch.from_numpy(v.astype(np.float32)).to(DT[t])
    a = np.float32(amax)
    packed, tiles, g, values = quantize(x.cuda(), 60, 64, amax=torch.tensor([a], device="cuda"), out=torch.float32)
    rp, rc, rg, rv = ref.quantize_tokens(x.float().numpy(), a)
    assert np.array_equal(packed.cpu().numpy(), rp)
    assert np.array_equal(ref.untile(tiles.cpu().numpy(), 60, 4), rc)
    assert np.array_equal(g.cpu().numpy(), rg) and np.array_equal(values.cpu().numpy(), rv)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_tokens_of_every_magnitude(cuda_ok, t):
    # each token's own scale, from the smallest numbers to the largest
    rng = np.random.default_rng(4)
    v = np.ldexp(rng.standard_normal((270, 48)), np.arange(-148, 122)[:, None])
    x = torch.from_numpy(v.astype(np.float32)).to(DT[t])
    packed, tiles, g, values = quantize(x.cuda(), 270, 48, out=torch.float32)
    rp, rc, rg, rv = ref.quantize_tokens(x.float().numpy())
    assert np.array_equal(packed.cpu().numpy(), rp)
    assert np.array_equal(ref.untile(tiles.cpu().numpy(), 270, 3)[:, :3], rc)
    assert np.array_equal(g.cpu().numpy(), rg) and np.array_equal(values.cpu().numpy(), rv)


@pytest.mark.parametrize("div", [1, 2, 3, 5, 6, 7, 8, 31, 1000])
def test_rows_over_their_divisor(cuda_ok, div):
    rng = np.random.default_rng(div)
    n_src, c = 37, 32
    x = torch.from_numpy(rng.standard_normal((n_src, c)).astype(np.float32)).cuda()
    src = rng.integers(0, n_src * div, 500).astype(np.int32)
    packed, _, _, _ = quantize(x, n_src, c, torch.from_numpy(src).cuda(), div, 500)
    rp, _, _, _ = ref.quantize_tokens(x.cpu().numpy()[src // div])
    assert np.array_equal(packed.cpu().numpy(), rp)


@pytest.mark.parametrize("counts,before,after", [([5, 0, 130, 1, 0], 0, 0), ([128, 128], 3, 9), ([0, 0, 1], 0, 200),
                                                 ([127, 129, 257], 1, 0)])
def test_grouped_and_gathered_tokens(cuda_ok, counts, before, after):
    rng = np.random.default_rng(sum(counts))
    n_src, k, c = 90, 3, 112
    off = np.concatenate([[0], np.cumsum(counts)]) + before
    n_rows = int(off[-1]) + after
    v = rng.standard_normal((n_src, c)).astype(np.float32)
    src = rng.integers(0, n_src * k, n_rows).astype(np.int32)
    src[rng.random(n_rows) < 0.1] = -1
    src[rng.random(n_rows) < 0.1] = n_src * k + 5
    x = torch.from_numpy(v).cuda()
    packed, tiles, g, values = quantize(x, n_src, c, torch.from_numpy(src).cuda(), k, n_rows,
                                        torch.from_numpy(off).cuda(), out=torch.float32)
    packed, tiles, g, values = (a.cpu().numpy() for a in (packed, tiles, g, values))
    tok = src // k
    inside = (np.arange(n_rows) >= off[0]) & (np.arange(n_rows) < off[-1]) & (src >= 0) & (tok < n_src)
    rp, rc, rg, rv = ref.quantize_tokens(v[np.where(inside, tok, 0)])
    assert np.array_equal(packed[inside], rp[inside]) and (packed[~inside] == 0xEE).all()
    assert np.array_equal(g[inside], rg[inside]) and (g[~inside] == -3.0).all()
    assert np.array_equal(values[inside], rv[inside]) and (values[~inside] == -3.0).all()
    for i, m in enumerate(counts):
        lo = off[i]
        got = ref.untile(tiles, m, c // 16, lo, i)
        ok = inside[lo:lo + m]
        assert np.array_equal(got[ok][:, :c // 16], rc[lo:lo + m][ok])


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("tensor", [False, True])
def test_tokens_that_are_not_finite(cuda_ok, bad, tensor, t):
    rng = np.random.default_rng(1)
    n, c = 6, 96
    x = torch.from_numpy(rng.standard_normal((n, c)).astype(np.float32)).to(DT[t])
    x[2, 37] = bad
    x[4, 0] = bad
    amax = torch.tensor([3.0], device="cuda") if tensor else None
    packed, tiles, g, values = quantize(x.cuda(), n, c, amax=amax, out=torch.float32)
    codes = ref.untile(tiles.cpu().numpy(), n, c // 16)[:, :c // 16]
    hit = np.zeros((n, c // 16), bool)
    hit[2, 2] = hit[4, 0] = True
    if not tensor:
        hit[[2, 4]] = True
    good = np.array([0, 1, 3, 5])
    rp, rc, rg, rv = ref.quantize_tokens(x[good].float().numpy(), 3.0 if tensor else None)
    assert np.array_equal(packed.cpu().numpy()[good], rp) and np.array_equal(codes[good], rc)
    assert np.array_equal(values.cpu().numpy()[good], rv) and np.array_equal(g.cpu().numpy()[good], rg)
    assert np.isnan(g.cpu().numpy()[[2, 4]]).all()
    assert ((codes == 0x7F) == hit).all()
    v = values.cpu().numpy().reshape(n, c // 16, 16)
    assert (np.isnan(v).all(-1) == hit).all()


# ---------------------------------------------------------------- products

def tiles_of(codes):
    """Weight scale bytes [mats, m, J] tiled by the library, checked against the definition."""
    lh = _lh()
    mats, m, J = codes.shape
    out = torch.full((lh.lh_nvfp4_weight_scale_bytes(mats, m, 16 * J),), 0xEE, dtype=torch.uint8, device="cuda")
    lh.lh_nvfp4_tile_scales(torch.from_numpy(codes).cuda(), mats, m, 16 * J, out)
    per = -(-m // 128) * -(-J // 4) * 512
    want = np.zeros((mats, per), np.uint8)
    for i in range(mats):
        ref.tile(codes[i], out=want[i])
    assert np.array_equal(out.cpu().numpy(), want.reshape(-1))
    return out


def whole_operand(rng, shape):
    """Codes of every E2M1 value and block scales of 1/2, 1 and 2: sums of their products are whole multiples of
    1/16, exact in FP32 in any order while they stay below 2^20 (c up to 4096: 4096 * 36 * 4 < 2^20)."""
    *lead, c = shape
    packed = rng.integers(0, 256, (*lead, c // 2)).astype(np.uint8)
    codes = rng.choice(np.array([0x30, 0x38, 0x40], np.uint8), (*lead, c // 16))  # E4M3 0.5, 1, 2
    return packed, codes


def matmul(xp, xt, xg, wp, wt, wg, off, y, c_out, c):
    lh = _lh()
    G = 1 if off is None else off.numel() - 1
    lh.lh_nvfp4_matmul(xp, xt, xg, wp, wt, wg, off, G, xp.shape[0], c_out, c, y, y, y.stride(0))
    assert lh.lh_nvfp4_status() == 0


def token_tiles(codes, off):
    """Token scale bytes [n, J] in tiles with the groups' places; what lies between them is NaN (0x7F)."""
    lh = _lh()
    n, J = codes.shape
    off = np.array([0, n]) if off is None else off
    out = np.full(lh.lh_nvfp4_token_scale_bytes(n, 16 * J, len(off) - 1), 0x7F, np.uint8)
    for i in range(len(off) - 1):
        m = off[i + 1] - off[i]
        if m > 0:  # blocks past c are 0 in a row's step
            padded = np.zeros((m, -(-J // 4) * 4), np.uint8)
            padded[:, :J] = codes[off[i]:off[i + 1]]
            ref.tile(padded, int(off[i]), i, out)
    return torch.from_numpy(out).cuda()


SIZES = [(1, 1, 32), (1, 128, 256), (2, 130, 64), (7, 33, 96), (16, 128, 512), (31, 200, 224), (33, 129, 288),
         (100, 5, 1024), (128, 256, 4096), (129, 127, 320), (200, 640, 800), (257, 300, 1056), (513, 384, 2048),
         (1, 4096, 4096), (3, 1536, 2080), (1000, 1100, 512), (20, 12300, 96),
         (60, 9700, 64), (1, 100, 17408), (32, 384, 8192), (33, 384, 8192), (90, 130, 17408 // 4)]


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("n,m,c", SIZES)
def test_product_of_whole_numbers_is_exact(cuda_ok, n, m, c, t):
    rng = np.random.default_rng(n + m + c)
    xp, xc = whole_operand(rng, (n, c))
    wp, wc = whole_operand(rng, (1, m, c))
    xg = np.exp2(rng.integers(-3, 4, n)).astype(np.float32)
    y = torch.full((n + 2, pitch(m, t)), 11.0, dtype=DT[t], device="cuda")
    matmul(torch.from_numpy(xp).cuda(), token_tiles(xc, None), torch.from_numpy(xg).cuda(),
           torch.from_numpy(wp).cuda(), tiles_of(wc), torch.tensor([0.5], device="cuda"), None, y, m, c)
    want, _ = ref.product(ref.decode(xp, xc), ref.decode(wp[0], wc[0]), xg, 0.5)
    want = torch.from_numpy(want).float().to(DT[t])
    assert torch.equal(y[:n, :m].cpu(), want)
    assert (y[n:] == 11.0).all() and (y[:, m:] == 11.0).all()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("counts,before,after,m,c", [
    ([1], 0, 0, 128, 256), ([0, 1, 0, 0, 3], 0, 0, 96, 64), ([5, 17, 130, 0, 1, 300], 0, 0, 200, 544),
    ([128, 256, 129], 2, 7, 257, 96), ([0] * 70 + [2, 1] + [0] * 30 + [33], 0, 5, 64, 128), ([0, 0], 4, 0, 32, 32),
    ([1] * 100, 0, 0, 130, 1024), ([300, 700, 0, 513, 16], 5, 3, 300, 352), ([1024, 1], 0, 0, 520, 128),
    ([40, 0, 33, 2, 65], 0, 0, 70, 4352),
    ([257, 20, 300, 500, 33, 1, 2000, 129, 160], 1, 4, 400, 288), ([3000, 32, 31, 33, 97], 0, 0, 1152, 64), ([64, 31, 97, 255, 2], 1, 1, 384, 2048),
])
def test_grouped_product_of_whole_numbers_is_exact(cuda_ok, counts, before, after, m, c, t):
    rng = np.random.default_rng(len(counts) + m)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64) + before
    n, G = int(off[-1]) + after, len(counts)
    xp, xc = whole_operand(rng, (n, c))
    wp, wc = whole_operand(rng, (G, m, c))
    xg = np.exp2(rng.integers(-3, 4, n)).astype(np.float32)
    wg = np.exp2(rng.integers(-3, 4, G)).astype(np.float32)
    y = torch.full((n, pitch(m, t)), 11.0, dtype=DT[t], device="cuda")
    matmul(torch.from_numpy(xp).cuda(), token_tiles(xc, off), torch.from_numpy(xg).cuda(), torch.from_numpy(wp).cuda(),
           tiles_of(wc), torch.from_numpy(wg).cuda(), torch.from_numpy(off).cuda(), y, m, c)
    want = torch.full((n, m), 11.0, dtype=DT[t])
    for g in range(G):
        a, b = off[g], off[g + 1]
        if b > a:
            yg, _ = ref.product(ref.decode(xp[a:b], xc[a:b]), ref.decode(wp[g], wc[g]), xg[a:b], wg[g])
            want[a:b] = torch.from_numpy(yg).float().to(DT[t])
    assert torch.equal(y[:, :m].cpu(), want)
    assert (y[:, m:] == 11.0).all()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("counts,m,c", [
    ([1500], 5000, 2080), ([2000], 4999, 96), ([1100], 5121, 1280),   # several rounds of 256-token tiles
    ([100] * 40, 1100, 1312), ([1, 120, 0, 64, 33] * 12, 1000, 1824),  # and of 128-token tiles, one and two a group
    ([400] * 12, 1300, 1600), ([290, 0, 161, 32, 384] * 8, 520, 2336),
])
def test_many_tiles_for_every_pair(cuda_ok, counts, m, c, t):
    # the ring, the scales' places and the halves of the way to Y go on from tile to tile
    rng = np.random.default_rng(len(counts) + m)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    n, G = int(off[-1]), len(counts)
    xp, xc = whole_operand(rng, (n, c))
    wp, wc = whole_operand(rng, (G, m, c))
    xg = np.exp2(rng.integers(-3, 4, n)).astype(np.float32)
    wg = np.exp2(rng.integers(-3, 4, G)).astype(np.float32)
    y = torch.full((n + 1, pitch(m, t)), 11.0, dtype=DT[t], device="cuda")
    given = off if G > 1 else None
    matmul(torch.from_numpy(xp).cuda(), token_tiles(xc, given), torch.from_numpy(xg).cuda(), torch.from_numpy(wp).cuda(),
           tiles_of(wc), torch.from_numpy(wg).cuda(), None if G == 1 else torch.from_numpy(off).cuda(), y, m, c)
    for g in range(G):
        a, b = off[g], off[g + 1]
        if b > a:
            x = torch.from_numpy(ref.decode(xp[a:b], xc[a:b])).double()
            w = torch.from_numpy(ref.decode(wp[g], wc[g])).double()
            want = (x @ w.T) * torch.from_numpy(xg[a:b]).double()[:, None] * float(wg[g])
            assert torch.equal(y[a:b, :m].cpu(), want.float().to(DT[t]))
    assert (y[n:] == 11.0).all() and (y[:, m:] == 11.0).all()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("n,m,c", [(1, 256, 4096), (60, 384, 1024), (300, 130, 17408)])
def test_product_of_quantised_tokens(cuda_ok, n, m, c, t):
    # every scale code and value that quantisation makes, against FP64 with the bound of FP32 sums
    rng = np.random.default_rng(c)
    x = (rng.standard_normal((n, c)) * np.exp(rng.standard_normal(c))).astype(np.float32)
    w = (rng.standard_normal((m, c)) * 0.02).astype(np.float32)
    xp, xc, xg, _ = ref.quantize_tokens(x)
    wp, wc, wg, _ = ref.quantize_tokens(w, np.abs(w).max())
    y = torch.empty(n, pitch(m, t), dtype=DT[t], device="cuda")
    matmul(torch.from_numpy(xp).cuda(), token_tiles(xc, None), torch.from_numpy(xg).cuda(),
           torch.from_numpy(wp[None]).cuda(), tiles_of(wc[None]), torch.from_numpy(wg[:1]).cuda(), None, y, m, c)
    want, s = ref.product(ref.decode(xp, xc), ref.decode(wp, wc), xg, wg[0])
    err = np.abs(y[:, :m].double().cpu().numpy() - want)
    assert (err <= ref.product_tolerance(want, s, c, t == "bf16")).all()


def test_decreasing_offsets_stay_in_bounds(cuda_ok):
    # results are unspecified, but nothing outside the rows that some group names is touched
    lh = _lh()
    rng = np.random.default_rng(0)
    n, m, c = 500, 130, 96
    w, _, _ = bank(rng, 4, m, c)
    x = torch.from_numpy(rng.standard_normal((n, c)).astype(np.float32)).cuda()
    for off in ([10, 300, 20, 260, 100], [-50, 40, 10 ** 12, 3, 200], [400, 300, 200, 100, 50]):
        y = torch.full((n + 8, pitch(m, "f32")), 6.0, device="cuda")
        linear(x, n, c, w, m, y[:n], off=torch.tensor(off, dtype=torch.int64, device="cuda"))
        assert lh.lh_nvfp4_status() == 0
        named = np.zeros(n + 8, bool)
        for a, b in zip(off, off[1:]):
            named[max(min(a, n), 0):max(min(b, n), 0)] = True
        assert (y[torch.from_numpy(~named).cuda()] == 6.0).all() and (y[:, m:] == 6.0).all()


def test_outputs_beyond_32_bits(cuda_ok):
    # offsets in Y, in the quantised values and in gathered rows past 2^32 bytes: the far rows equal the near ones
    lh = _lh()
    rng = np.random.default_rng(5)
    w, _, _ = bank(rng, 1, 66000, 32)
    n = 34000
    near = torch.from_numpy(rng.standard_normal((200, 32)).astype(np.float32)).cuda()
    x = near.repeat(n // 200, 1).contiguous()
    y = torch.zeros(n, 66000, dtype=torch.bfloat16, device="cuda")
    linear(x, n, 32, w, 66000, y)
    assert torch.equal(y[-200:], y[:200]) and torch.equal(y[n // 2 // 200 * 200:][:200], y[:200])
    assert float(y[:200].float().abs().sum()) > 0
    del y, w
    n, c = 40000, 32768
    x = torch.from_numpy(rng.standard_normal((8, c)).astype(np.float32)).cuda()
    src = (torch.arange(n, device="cuda") % 8).to(torch.int32)
    packed, _, g, values = quantize(x, 8, c, src, 1, n, out=torch.float32)
    assert torch.equal(values[-8:], values[:8]) and torch.equal(packed[-8:], packed[:8]) and torch.equal(g[-8:], g[:8])
    rows = torch.zeros_like(values)
    lh.lh_gather_tokens(x, x, 8, c, c, src, 1, n, rows, c)
    assert torch.equal(rows[-8:], x) and torch.equal(rows[:8], x)
    back = torch.zeros(2, c, device="cuda")
    pos = torch.tensor([n - 8, n - 7, n - 6, -1], dtype=torch.int32, device="cuda")
    lh.lh_combine_tokens(rows, rows, n, c, c, pos, None, 2, 2, back, c)
    assert torch.equal(back[1], x[2]) and torch.equal(back[0], x[0] + x[1])
    dw = torch.zeros(2, 2, device="cuda")
    lh.lh_combine_tokens_grad(back, back, 2, 2, c, c, rows, c, n, pos, None, None, 0, dw)
    want = (back[1].double() * x[2].double()).sum()
    assert abs(float(dw[1, 0]) - float(want)) <= (c + 5) * 2.0 ** -24 * float((back[1].double() * x[2].double()).abs().sum())


def test_every_scale_code_multiplies_by_its_value(cuda_ok):
    # token r has block scale code r + 1 and values 1; the weights are 1 with scale 1: each output is 32 v(r + 1), exact
    c, m = 32, 8
    codes = np.arange(1, 127, dtype=np.uint8)
    n = len(codes)
    xc = np.repeat(codes[:, None], 2, 1)
    ones = np.full((n, c // 2), 0x22, np.uint8)
    wc = np.full((1, m, 2), 0x38, np.uint8)
    y = torch.empty(n, m, device="cuda")
    one = torch.ones(n, device="cuda")
    matmul(torch.from_numpy(ones).cuda(), token_tiles(xc, None), one, torch.from_numpy(ones[None, :m].copy()).cuda(),
           tiles_of(wc), one[:1], None, y, m, c)
    want = 32 * ref.e4m3_table()[codes]
    assert np.array_equal(y.double().cpu().numpy(), np.repeat(want[:, None], m, 1))


# ---------------------------------------------------------------- one call, and all of them in a run

def linear(x, n_src, c, w, m, y, rows=None, row_div=1, n_rows=None, off=None, amax=None, ws=None, stream=None):
    lh = _lh()
    n_rows = n_src if n_rows is None else n_rows
    G = 1 if off is None else off.numel() - 1
    need = lh.lh_nvfp4_linear_workspace_bytes(n_rows, c, G)
    if ws is None:
        ws = torch.full((max(need, 1),), 0x7F, dtype=torch.uint8, device="cuda")
    lh.lh_nvfp4_linear(x, x, n_src, c, x.stride(0), rows, row_div, n_rows, off, G, amax, *w, m, y, y, y.stride(0), ws,
                       need, stream)
    return ws


def bank(rng, mats, m, c):
    """(device operands, FP64 values without the global scale, global scales) of a bank calibrated by max scaling."""
    lh = _lh()
    w = torch.from_numpy((rng.standard_normal((mats, m, c)) * 0.02).astype(np.float32)).cuda()
    J = c // 16
    amax = torch.empty(mats, device="cuda")
    lh.lh_absmax(w, w, mats, m, c, c, amax)
    ba, codes = torch.empty(mats, m, J, device="cuda"), torch.empty(mats, m, J, dtype=torch.uint8, device="cuda")
    lh.lh_baseline_scales(w, w, mats, m, c, c, amax, lh.LH_SCALE_MAX, ba, codes)
    packed = torch.empty(mats, m, c // 2, dtype=torch.uint8, device="cuda")
    scales, g = torch.empty_like(codes), torch.empty(mats, device="cuda")
    lh.lh_quantize_nvfp4(w, w, mats, m, c, c, amax, codes, packed, scales, g)
    tiles = torch.empty(lh.lh_nvfp4_weight_scale_bytes(mats, m, c), dtype=torch.uint8, device="cuda")
    lh.lh_nvfp4_tile_scales(scales, mats, m, c, tiles)
    return (packed, tiles, g), ref.decode(packed.cpu().numpy(), scales.cpu().numpy()), g.cpu().numpy()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("tensor", [False, True])
@pytest.mark.parametrize("n,m,c", [(1, 128, 64), (1, 4096, 4096), (2, 1000, 1056), (17, 384, 512), (140, 257, 2048)])
def test_linear_from_the_tokens(cuda_ok, n, m, c, tensor, t):
    rng = np.random.default_rng(n + m)
    w, wv, wg = bank(rng, 1, m, c)
    x = torch.from_numpy((rng.standard_normal((n, c)) * np.exp(rng.standard_normal(c))).astype(np.float32)).to(DT[t])
    v = x.float().numpy()
    amax = np.abs(v).max() if tensor else None
    y = torch.full((n, pitch(m, t)), 4.0, dtype=DT[t], device="cuda")
    linear(x.cuda(), n, c, w, m, y, amax=None if amax is None else torch.tensor([amax], device="cuda"))
    assert _lh().lh_nvfp4_status() == 0
    xp, xc, xg, _ = ref.quantize_tokens(v, amax)
    want, s = ref.product(ref.decode(xp, xc), wv[0], xg, wg[0])
    err = np.abs(y[:, :m].double().cpu().numpy() - want)
    assert (err <= ref.product_tolerance(want, s, c, t == "bf16")).all()
    assert (y[:, m:] == 4.0).all()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("given", [None, 3.0, 1e-30, 0.0])
@pytest.mark.parametrize("n,m,c", [(1, 100, 32), (1, 4096, 4096), (2, 700, 1056), (3, 130, 9248), (5, 64, 480),
                                   (8, 19000, 64), (8, 1536, 512), (8, 9000, 480), (7, 128, 4384),
                                   (4, 300, 1024), (1, 12288, 4096), (1, 257, 17408)])
def test_linear_of_few_tokens_equals_its_two_calls(cuda_ok, n, m, c, given, t):
    lh = _lh()
    rng = np.random.default_rng(n + m + c)
    w, _, _ = bank(rng, 1, m, c)
    buf = torch.full((n, c + 8), 9.0, dtype=DT[t], device="cuda")
    x = buf[:, :c]
    x.copy_(torch.from_numpy((rng.standard_normal((n, c)) * np.exp(rng.standard_normal(c))).astype(np.float32)))
    if n > 2:
        x[0] = 0
        x[1, c // 3] = float("nan")
        x[2, c - 1] = -float("inf")
    amax = None if given is None else torch.tensor([given], device="cuda")
    y = torch.full((n, pitch(m, t)), 4.0, dtype=DT[t], device="cuda")
    linear(x, n, c, w, m, y, amax=amax)
    packed, tiles, g, _ = quantize(x, n, c, amax=amax)
    y2 = torch.full_like(y, 4.0)
    matmul(packed, tiles, g, *w, None, y2, m, c)
    a, b = y.float().cpu().numpy(), y2.float().cpu().numpy()
    assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.nan_to_num(a), np.nan_to_num(b))
    assert lh.lh_nvfp4_status() == 0


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("given", [None, 3.0])
@pytest.mark.parametrize("n,m,c", [(1, 4096, 8192), (1, 130, 8224), (2, 200, 4096), (3, 257, 2720), (4, 1536, 2048),
                                   (4, 9000, 480), (5, 300, 1024)])
def test_the_most_tokens_of_one_launch(cuda_ok, n, m, c, given, t):
    test_linear_of_few_tokens_equals_its_two_calls(cuda_ok, n, m, c, given, t)


def test_linear_of_tokens_that_are_not_finite(cuda_ok):
    rng = np.random.default_rng(2)
    w, wv, wg = bank(rng, 1, 200, 128)
    for n in (1, 5, 130):
        x = torch.from_numpy(rng.standard_normal((n, 128)).astype(np.float32)).cuda()
        x[n // 2, 100] = float("inf")
        for amax in (None, torch.tensor([4.0], device="cuda")):
            y = torch.empty(n, 200, device="cuda")
            linear(x, n, 128, w, 200, y, amax=amax)
            nan = torch.isnan(y).all(1)
            assert nan[n // 2] and int(nan.sum()) == 1 and torch.isfinite(y[~nan]).all()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,e,m,c", [(1, 4, 16, 130, 160), (48, 4, 64, 256, 512), (600, 2, 5, 384, 320)])
def test_a_layer_of_experts(cuda_ok, n, k, e, m, c, t):
    # route, products of the gathered tokens, and the weighted sum back, as a serving step runs them
    lh = _lh()
    rng = np.random.default_rng(n)
    w, wv, wg = bank(rng, e, m, c)
    x = torch.from_numpy(rng.standard_normal((n, c)).astype(np.float32)).to(DT[t])
    ids = np.stack([rng.choice(e, k, replace=False) for _ in range(n)]).astype(np.int32)
    if n > 1:
        ids[n // 2] = -1  # a padded token
    cw = rng.random((n, k)).astype(np.float32)
    xd, idd, cwd = x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(cw).cuda()
    off = torch.empty(e + 1, dtype=torch.int64, device="cuda")
    order, pos = (torch.empty(n * k, dtype=torch.int32, device="cuda") for _ in range(2))
    ys = torch.full((n * k, pitch(m, t)), float("nan"), dtype=DT[t], device="cuda")
    y = torch.empty(n, pitch(m, t), dtype=DT[t], device="cuda")
    ws = torch.empty(lh.lh_nvfp4_linear_workspace_bytes(n * k, c, e), dtype=torch.uint8, device="cuda")

    def step():
        lh.lh_route_tokens(idd, n, k, e, off, order, pos)
        linear(xd, n, c, w, m, ys, rows=order, row_div=k, n_rows=n * k, off=off, ws=ws)
        lh.lh_combine_tokens(ys, ys, n * k, m, ys.stride(0), pos, cwd, n, k, y, y.stride(0))

    step()
    xp, xc, xg, _ = ref.quantize_tokens(x.float().numpy())
    xv = ref.decode(xp, xc)
    want, tol = np.zeros((n, m)), np.zeros((n, m))
    mag = np.zeros((n, m))
    for i in range(n):
        for s in range(k):
            if ids[i, s] >= 0:
                yy, ss = ref.product(xv[i:i + 1], wv[ids[i, s]], xg[i:i + 1], wg[ids[i, s]])
                want[i] += cw[i, s] * yy[0]
                tol[i] += cw[i, s] * ref.product_tolerance(yy, ss, c, t == "bf16")[0]
                mag[i] += cw[i, s] * (np.abs(yy[0]) + tol[i])
    tol = tol + k * 2.0 ** -24 * mag
    tol = tol + (np.abs(want) + tol) * HALF[t]
    assert (np.abs(y[:, :m].double().cpu().numpy() - want) <= tol).all()

    # captured and replayed with other inputs in the same buffers
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ids2 = np.roll(ids, 1, 1)
    idd.copy_(torch.from_numpy(ids2).cuda())
    xd.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    once = y.clone()
    step()
    assert torch.equal(once, y)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(once, y)
    assert lh.lh_nvfp4_status() == 0


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("tensor", [False, True])
@pytest.mark.parametrize("n,k,c,kind", [(1100, 4, 96, "route"), (1100, 4, 4128, "route"), (2100, 2, 544, "twice"),
                                        (520, 8, 2080, "holes"), (140, 32, 64, "route"), (1400, 3, 9248, "twice")])
def test_linear_of_tokens_with_several_rows(cuda_ok, n, k, c, kind, tensor, t):
    # one call equals the two calls it stands for, row by row, whatever rows name the tokens' slots
    lh = _lh()
    rng = np.random.default_rng(n + k)
    e, m = 7, 72
    R = n * k
    x = torch.from_numpy(rng.standard_normal((n, c)).astype(np.float32)).to(DT[t]).cuda()
    x[3, c // 2] = float("nan")
    w, _, _ = bank(rng, e, m, c)
    ids = rng.integers(0, e, (n, k)).astype(np.int32)
    if kind == "holes":
        ids[rng.random((n, k)) < 0.3] = -1
    off, order, _ = ref.route(ids, e)
    src = order.copy()
    if kind == "twice":  # several rows name one slot, some slots have none, some rows name nothing
        src[:R] = rng.integers(-1, R + 9, R)
        src[10:20] = 5
        off[0], off[-1] = 3, R - 17
    amax = torch.tensor([3.0], device="cuda") if tensor else None
    sd, od = torch.from_numpy(src).cuda(), torch.from_numpy(off).cuda()
    y = torch.full((R, pitch(m, t)), 4.0, dtype=DT[t], device="cuda")
    linear(x, n, c, w, m, y, rows=sd, row_div=k, n_rows=R, off=od, amax=amax)
    packed, tiles, g, _ = quantize(x, n, c, sd, k, R, od, amax)
    y2 = torch.full_like(y, 4.0)
    matmul(packed, tiles, g, *w, od, y2, m, c)
    rows = np.arange(R)
    inside = (rows >= off[0]) & (rows < off[-1])
    named = inside & (src >= 0) & (src < R)
    a, b = y.float().cpu().numpy()[named], y2.float().cpu().numpy()[named]
    assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.nan_to_num(a), np.nan_to_num(b))
    assert (y[torch.from_numpy(~inside).cuda()] == 4.0).all()
    assert lh.lh_nvfp4_status() == 0


def test_calibration_of_routed_tokens(cuda_ok):
    # the sorted rows and offsets are what the Hessian takes: each expert's H is that of its own tokens
    lh = _lh()
    rng = np.random.default_rng(8)
    n, k, e, c = 700, 2, 9, 128
    x = torch.from_numpy(rng.standard_normal((n, c)).astype(np.float32)).to(torch.bfloat16)
    ids = rng.integers(0, e - 1, (n, k)).astype(np.int32)
    ids[rng.random((n, k)) < 0.1] = -1
    xd = x.cuda()
    off = torch.empty(e + 1, dtype=torch.int64, device="cuda")
    order, pos = (torch.empty(n * k, dtype=torch.int32, device="cuda") for _ in range(2))
    xs = torch.full((n * k, c), float("nan"), dtype=torch.bfloat16, device="cuda")
    lh.lh_route_tokens(torch.from_numpy(ids).cuda(), n, k, e, off, order, pos)
    lh.lh_gather_tokens(xd, xd, n, c, c, order, k, n * k, xs, c)
    H = torch.zeros(e, c // 16, 16, 16, device="cuda")
    need = lh.lh_hessian_workspace_bytes(n * k, c, e)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    lh.lh_accumulate_hessian(xs, lh.LH_BF16, n * k, c, c, off, e, H, ws, need)
    assert lh.lh_workspace_status(ws) == 0
    bits = x.view(torch.int16).numpy().view(np.uint16)
    got = H.double().cpu().numpy()
    for i in range(e):
        mine = np.repeat(bits, (ids == i).sum(1), 0)
        want = oracle.hessian(mine)[0] if len(mine) else np.zeros((c // 16, 16, 16))
        assert np.linalg.norm(got[i] - want) <= 1e-5 * np.linalg.norm(want)

"""The operators that run a calibrated layer at the ends of what they accept, on the GPU."""
import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from tests import test_gpu_layer as layer

pytestmark = pytest.mark.gpu


def _lh():
    import scale_calibration_b200 as lh
    return lh


@pytest.fixture
def big(cuda_ok):
    """Room for tens of GB, given back afterwards."""
    torch.cuda.empty_cache()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


PIECE = 1 << 27  # rows looked at together


def test_the_most_rows_of_tokens(big):
    # 2^31 - 513 rows of one block each: a counter of rows that steps past the last one must not come round again
    lh = _lh()
    n, c, n_src = (1 << 31) - 513, 16, 37
    v = np.random.default_rng(0).standard_normal((n_src, c)).astype(np.float32)
    x = torch.from_numpy(v).cuda()
    rows = torch.empty(n, dtype=torch.int32, device="cuda")
    for a in range(0, n, PIECE):
        b = min(a + PIECE, n)
        rows[a:b] = (torch.arange(a, b, device="cuda") % n_src).to(torch.int32)
    packed = torch.zeros(n, c // 2, dtype=torch.uint8, device="cuda")
    tiles = torch.zeros(lh.lh_nvfp4_token_scale_bytes(n, c, 1), dtype=torch.uint8, device="cuda")
    g = torch.zeros(n, device="cuda")
    lh.lh_quantize_tokens(x, x, n_src, c, c, rows, 1, n, None, 1, None, packed, tiles, g)
    rp, rc, rg, _ = ref.quantize_tokens(v)
    rp, rg, rc = (torch.from_numpy(a.copy()).cuda() for a in (rp, rg, rc))
    rp = rp.view(torch.int64).view(-1)
    packed = packed.view(torch.int64).view(-1)
    for a in range(0, n, PIECE):
        b = min(a + PIECE, n)
        i = rows[a:b].long()
        assert torch.equal(g[a:b], rg[i])
        assert torch.equal(packed[a:b], rp[i])
    # row r's code: byte 0 of (r % 32, r % 128 / 32) of tile r / 128
    words = tiles.view(torch.int32).view(-1, 32, 4)
    for t0 in range(0, words.shape[0], PIECE // 128):
        w = words[t0:t0 + PIECE // 128].permute(0, 2, 1).reshape(-1)
        a, b = 128 * t0, min(128 * t0 + w.numel(), n)
        assert torch.equal(w[:b - a], rc.view(-1)[rows[a:b].long()].to(torch.int32))


def test_the_most_rows_of_a_product(big):
    # 2^31 - 513 rows of 32 values by 8 channels: every row equals that of the same token in a small call
    lh = _lh()
    n, m, c, n_src = (1 << 31) - 513, 8, 32, 37
    rng = np.random.default_rng(1)
    w, _, _ = layer.bank(rng, 1, m, c)
    x = torch.from_numpy(rng.standard_normal((n_src, c)).astype(np.float32)).cuda()
    small = torch.zeros(n_src, m, dtype=torch.bfloat16, device="cuda")
    layer.linear(x, n_src, c, w, m, small)
    rows = torch.empty(n, dtype=torch.int32, device="cuda")
    for a in range(0, n, PIECE):
        b = min(a + PIECE, n)
        rows[a:b] = (torch.arange(a, b, device="cuda") % n_src).to(torch.int32)
    y = torch.zeros(n, m, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(lh.lh_nvfp4_linear_workspace_bytes(n, c, 1), dtype=torch.uint8, device="cuda")
    layer.linear(x, n_src, c, w, m, y, rows=rows, n_rows=n, ws=ws)
    assert lh.lh_nvfp4_status() == 0
    assert float(small.float().abs().sum()) > 0
    for a in range(0, n, PIECE):
        b = min(a + PIECE, n)
        assert torch.equal(y[a:b], small[rows[a:b].long()])


def test_the_most_ids(big):
    # 2^31 - 513 ids, every third of them without an expert
    lh = _lh()
    n, e = (1 << 31) - 513, 2
    ids = torch.empty(n, dtype=torch.int32, device="cuda")
    for a in range(0, n, PIECE):
        b = min(a + PIECE, n)
        ids[a:b] = (torch.arange(a, b, device="cuda") % 3).to(torch.int32)
    off = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    order, pos = (torch.full((n,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    lh.lh_route_tokens(ids, n, 1, e, off, order, pos)
    n0, n1 = -(-n // 3), -(-(n - 1) // 3)
    assert off.tolist() == [0, n0, n0 + n1]
    for a in range(0, n, PIECE):
        p = torch.arange(a, min(a + PIECE, n), device="cuda")
        want = torch.where(p < n0, 3 * p, torch.where(p < n0 + n1, 3 * (p - n0) + 1, -1))
        assert torch.equal(order[a:a + len(p)], want.to(torch.int32))
        want = torch.where(p % 3 == 0, p // 3, torch.where(p % 3 == 1, p // 3 + n0, -1))
        assert torch.equal(pos[a:a + len(p)], want.to(torch.int32))


@pytest.mark.parametrize("n,m,grouped", [(3, 200, False), (16, 130, False), (200, 300, False), (700, 520, False), (90, 300, True)])
def test_rows_of_every_number_of_stages_one_after_another(cuda_ok, n, m, grouped):
    # a kernel waits for the last arrivals on its ring, whatever is left over of it: split and paired products of one
    # stage to three rings, launched back to back, all right and none of their waits run out
    rng = np.random.default_rng(n)
    calls = []
    for stages in range(1, 22):
        c = 256 * stages - 32 * int(rng.integers(8))
        xp, xc = layer.whole_operand(rng, (n, c))
        wp, wc = layer.whole_operand(rng, (1, m, c))
        xg = np.exp2(rng.integers(-3, 4, n)).astype(np.float32)
        off = np.array([0, n], np.int64) if grouped else None
        a = (torch.from_numpy(xp).cuda(), layer.token_tiles(xc, off), torch.from_numpy(xg).cuda(), torch.from_numpy(wp).cuda(),
             layer.tiles_of(wc), torch.tensor([0.5], device="cuda"), torch.from_numpy(off).cuda() if grouped else None)
        x, w = (torch.from_numpy(v).double() for v in (ref.decode(xp, xc), ref.decode(wp[0], wc[0])))
        want = ((x @ w.T) * torch.from_numpy(xg).double()[:, None] * 0.5).float()
        calls.append((a, c, want, torch.empty(n, layer.pitch(m, "f32"), device="cuda")))
    for _ in range(20):
        for a, c, _, y in calls:
            _lh().lh_nvfp4_matmul(*a, 1, n, m, c, y, y, y.stride(0))
    for a, c, want, y in calls:
        assert torch.equal(y[:, :m].cpu(), want), c
    assert _lh().lh_nvfp4_status() == 0


def test_a_bank_calibrated_without_tokens(cuda_ok):
    lh = _lh()
    W = torch.randn(3, 8, 64, device="cuda")
    X = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    cal = lh.calibrate_routed(W, X, torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert (cal["codes"] == 1).all() and (cal["H"] == 0).all()  # H = 0: every code is as good, the lowest is taken
    q = lh.QuantizedLayer(W, cal["global_amax"], cal["codes"])
    r = lh.Routing(0, 2, 3).route(torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert r.offsets.tolist() == [0, 0, 0, 0] and q.forward_routed(X, r).shape == (0, 8)
    one = lh.calibrate(W[0], X)
    assert torch.equal(one["codes"][0], cal["codes"][0])


def test_a_combination_without_rows_is_zero(cuda_ok):
    lh = _lh()
    pos = torch.full((6,), 3, dtype=torch.int32, device="cuda")  # past the end of no rows
    rows, dy = torch.empty(0, 8, device="cuda"), torch.randn(3, 8, device="cuda")
    y, dw = torch.full((3, 8), 5.0, device="cuda"), torch.full((3, 2), 5.0, device="cuda")
    lh.lh_combine_tokens(rows, rows, 0, 8, 8, pos, None, 3, 2, y, 8)
    lh.lh_combine_tokens_grad(dy, dy, 3, 2, 8, 8, rows, 8, 0, pos, None, rows, 8, dw)
    assert (y == 0).all() and (dw == 0).all()


def test_a_layer_runs_on_detached_tokens(cuda_ok):
    lh = _lh()
    W = torch.randn(3, 8, 64, device="cuda")
    cal = lh.calibrate_routed(W, torch.randn(9, 64, device="cuda").bfloat16(), torch.zeros(9, 2, dtype=torch.int32, device="cuda"))
    q = lh.QuantizedLayer(W, cal["global_amax"], cal["codes"])
    x = torch.randn(9, 64, device="cuda", requires_grad=True)
    w = torch.rand(9, 2, device="cuda", requires_grad=True)
    r = lh.Routing(9, 2, 3).route(torch.arange(18, dtype=torch.int32, device="cuda").view(9, 2) % 3)
    with pytest.raises(ValueError):
        q.forward_routed(x, r, w)
    with torch.no_grad():
        y = q.forward_routed(x, r, w)
    assert torch.equal(y, q.forward_routed(x.detach(), r, w.detach())) and not y.requires_grad


def test_a_layer_reports_an_expired_wait(cuda_ok):
    lh = _lh()
    W = torch.randn(8, 64, device="cuda")
    cal = lh.calibrate(W, torch.randn(40, 64, device="cuda").bfloat16())
    q = lh.QuantizedLayer(W, cal["global_amax"], cal["codes"])
    x = torch.randn(300, 64, device="cuda")
    y = q(x)
    q.check()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    lh.lh_debug_nvfp4_wait_timeout(50000, 0)  # 50 ms, nothing arrives
    end.record()
    with pytest.raises(lh.LHError, match="LH_ERR_TIMEOUT") as e:
        q.check()
    assert e.value.status == 6 and 45 <= start.elapsed_time(end) <= 500
    q.check()  # told once
    lh.lh_debug_nvfp4_wait_timeout(50000, 1)  # completed: nothing to tell
    q.check()
    s = torch.cuda.Stream()
    lh.lh_debug_nvfp4_wait_timeout(1000, 0, s)
    with pytest.raises(lh.LHError):
        q.check(s)
    assert torch.equal(q(x), y)
    q.check()


def test_calibration_of_tensors_that_lie_otherwise(cuda_ok):
    # every other expert of a bank, transposed weights, transposed and unaligned tokens: the same as their copies
    lh = _lh()
    W = torch.randn(6, 16, 64, device="cuda")
    X = torch.randn(40, 64, device="cuda").bfloat16()
    ids = (torch.arange(80, device="cuda").view(40, 2) % 3).to(torch.int32)
    wide = torch.zeros(40, 69, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:67] = X
    turned = W[::2].transpose(1, 2).contiguous().transpose(1, 2)
    want = lh.calibrate_routed(W[::2].contiguous(), X, ids)
    for w in (W[::2], turned, W[1::2].clone().copy_(W[::2])):
        for x in (X, X.t().contiguous().t(), wide[:, 3:67]):
            got = lh.calibrate_routed(w, x, ids)
            assert all(torch.equal(got[key], want[key]) for key in want)
    want = lh.calibrate(W[1].contiguous(), X)
    for x in (X.t().contiguous().t(), wide[:, 3:67]):
        got = lh.calibrate(W.transpose(1, 2).contiguous().transpose(1, 2)[1], x)
        assert all(torch.equal(got[key], want[key]) for key in want)
    bank = lh.calibrate_routed(W[::2], X, ids)
    a, b = (lh.QuantizedLayer(w, bank["global_amax"], bank["codes"]) for w in (W[::2], turned))
    assert torch.equal(a.packed, b.packed) and torch.equal(a.scale_tiles, b.scale_tiles)


@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_streams_handle_is_the_default_stream(cuda_ok, handle):
    # work that waits on the default stream comes before a call with its handle
    lh = _lh()
    W = torch.randn(3, 8, 64, device="cuda")
    X = torch.randn(9, 64, device="cuda").bfloat16()
    ids = (torch.arange(18, device="cuda").view(9, 2) % 3).to(torch.int32)
    want = lh.calibrate_routed(W, X, ids)
    q = lh.QuantizedLayer(W, want["global_amax"], want["codes"])
    r = lh.Routing(9, 2, 3).route(ids)
    y = q.forward_routed(X, r)
    x, i, w = torch.zeros_like(X), torch.zeros_like(ids), torch.zeros_like(W)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # a tenth of a second
    x.copy_(X), i.copy_(ids), w.copy_(W)
    got = lh.calibrate_routed(w, x, i, stream=handle)
    q2 = lh.QuantizedLayer(w, got["global_amax"], got["codes"], stream=handle)
    y2 = q2.forward_routed(x, lh.Routing(9, 2, 3).route(i, stream=handle), stream=handle)
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and all(torch.equal(got[key], want[key]) for key in want)


def test_calibration_on_a_stream_does_all_of_it_there(cuda_ok):
    # the current stream is busy for a while: what calibration needs set to zero must not wait for it
    lh = _lh()
    W, X = torch.randn(16, 64, device="cuda"), torch.randn(400, 64, device="cuda").bfloat16()
    want = lh.calibrate(W, X)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert all(torch.equal(v, want[key]) for key, v in lh.calibrate(W, X, stream=0).items())  # the default stream
    for stream in (s, s.cuda_stream):
        torch.cuda._sleep(200_000_000)  # a tenth of a second
        got = lh.calibrate(W, X, stream=stream)
        s.synchronize()
        host = {key: got[key].cpu() for key in got}  # behind the sleep
        assert all(torch.equal(host[key], want[key].cpu()) for key in want)


def far_rows(rng, n, k, e):
    """(ids with masked slots, order, pos) of n tokens on the device."""
    ids = rng.integers(0, e, (n, k)).astype(np.int32)
    ids[rng.random((n, k)) < 0.2] = -1
    ids[::7] = -1
    _, order, pos = ref.route(ids, e)
    return torch.from_numpy(order).cuda(), torch.from_numpy(pos).cuda()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,c", [(5000, 5, 521), (5000, 3, 1536), (40001, 2, 72), (2500, 9, 1030)])
def test_rows_of_many_rounds(cuda_ok, n, k, c, t):
    # more vectors, rows and tokens than the grids take at once, every one of them looked at
    lh = _lh()
    rng = np.random.default_rng(n + k)
    dt, e = layer.DT[t], 64
    order, pos = far_rows(rng, n, k, e)
    R = n * k
    gen = torch.Generator(device="cuda")
    gen.manual_seed(c)

    def rows(m, fill):
        b = torch.full((m, layer.pitch(c, t)), fill, dtype=dt, device="cuda")
        b[:, :c] = torch.randn(m, c, generator=gen, device="cuda")
        return b

    x, ys, dy = rows(n, -7.0), rows(R, -7.0), rows(n, -7.0)
    w = torch.randn(n, k, generator=gen, device="cuda")
    named = order >= 0
    xs = torch.full_like(ys, 3.0)
    lh.lh_gather_tokens(x, x, n, c, x.stride(0), order, k, R, xs, xs.stride(0))
    want = torch.full_like(xs, 3.0)
    want[named, :c] = x[order[named].long() // k, :c]
    assert torch.equal(xs, want)

    ys[~named] = float("nan")  # read by nothing
    y = torch.full_like(x, 5.0)
    lh.lh_combine_tokens(ys, ys, R, c, ys.stride(0), pos, w, n, k, y, y.stride(0))
    there = (pos >= 0).view(n, k)
    taken = torch.where(there[..., None], ys[pos.clamp(min=0).long(), :c].view(n, k, c).double(), 0.0)
    terms = w.double()[..., None] * taken
    sums, mag = terms.sum(1), terms.abs().sum(1)
    tol = k * 2.0 ** -24 * mag  # k fused multiply-adds, each rounded once
    tol = tol + (sums.abs() + tol) * layer.HALF[t]
    assert ((y[:, :c].double() - sums).abs() <= tol).all() and (y[:, c:] == 5.0).all()

    dys, dw = torch.full_like(ys, 9.0), torch.full_like(w, 9.0)
    lh.lh_combine_tokens_grad(dy, dy, n, k, c, dy.stride(0), ys, ys.stride(0), R, pos, w, dys, dys.stride(0), dw)
    d = dy[:, :c].double()
    want = torch.full((R, c), 9.0, dtype=torch.float64, device="cuda")
    want[pos[there.view(-1)].long()] = (w.double()[..., None] * d[:, None])[there]
    # one product rounded to FP32, then to the type
    assert ((dys[:, :c].double() - want).abs() <= want.abs() * (2.0 ** -24 + layer.HALF[t] * (1 + 2.0 ** -24))).all()
    assert (dys[:, c:] == 9.0).all()
    dots, size = (d[:, None] * taken).sum(2), (d[:, None] * taken).abs().sum(2)
    assert ((dw.double() - dots).abs() <= (c + 5) * 2.0 ** -24 * size).all()  # c products and sums in FP32


def test_matrices_of_one_row(cuda_ok):
    # their row's stride is arbitrary, and a copy's was taken for the way from matrix to matrix
    lh = _lh()
    W = torch.randn(1, 3, 64, device="cuda").transpose(0, 1)
    X = torch.randn(40, 64, device="cuda").bfloat16()
    ids = (torch.arange(80, device="cuda").view(40, 2) % 3).to(torch.int32)
    same = torch.empty(3, 1, 64, device="cuda").copy_(W)
    assert W.stride(1) == 192 and same.stride(1) == 64
    want, got = lh.calibrate_routed(same, X, ids), lh.calibrate_routed(W, X, ids)
    assert all(torch.equal(got[key], want[key]) for key in want)
    a, b = (lh.QuantizedLayer(w, want["global_amax"], want["codes"]) for w in (same, W))
    assert torch.equal(a.packed, b.packed) and torch.equal(a.block_scales, b.block_scales)

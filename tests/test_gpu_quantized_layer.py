"""QuantizedLayer, Routing and calibrate_routed: what a user of the package runs after (and for) a calibration."""
import numpy as np
import pytest
import torch

import synth
from tests import gpu_util as gu
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _lh():
    import scale_calibration_b200 as lh
    return lh


def expected(layer, W, X, m=0):
    """FP64 product of the layer's codes with the tokens' own, and the bound of its rounding."""
    J = layer.c_in // 16
    wv = ref.decode(layer.packed[m].cpu().numpy(), layer.block_scales[m].cpu().numpy().reshape(layer.c_out, J))
    xp, xc, xg, _ = ref.quantize_tokens(X.float().cpu().numpy(), None if layer.x_amax is None else float(layer.x_amax))
    y, s = ref.product(ref.decode(xp, xc), wv, xg, float(layer.global_scale[m]))
    return y, ref.product_tolerance(y, s, layer.c_in, X.dtype == torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("given", [False, True])
def test_a_calibrated_layer_runs(cuda_ok, dtype, given):
    lh = _lh()
    layer = synth.make_layer(70, 160, 300, seed=5)
    W, X, _ = gu.to_device(layer)
    cal = lh.calibrate(W, X)
    x = X[:33].to(dtype)
    q = lh.QuantizedLayer(W, cal["global_amax"], cal["codes"], X.float().abs().max().view(1) if given else None)
    assert torch.equal(q.block_scales.view(-1), cal["codes"].view(-1))
    y = q(x)
    want, tol = expected(q, W, x)
    assert y.shape == (33, 70) and y.dtype == dtype
    assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()
    # rows that are not aligned, and columns of a wider matrix, are the same tokens
    wide = torch.zeros(33, 163, dtype=dtype, device="cuda")
    wide[:, 1:161] = x
    assert torch.equal(q(wide[:, 1:161]), y)
    assert q(x[:0]).shape == (0, 70)
    # on a stream of its own
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2 = q(x)
    y3, y4 = q(x, stream=s), q(x, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(y2, y) and torch.equal(y3, y) and torch.equal(y4, y)


def test_a_routed_bank_is_calibrated_and_runs(cuda_ok):
    lh = _lh()
    rng = np.random.default_rng(1)
    e, m, c, n, k = 6, 72, 96, 150, 2
    W = torch.from_numpy((rng.standard_normal((e, m, c)) * 0.02).astype(np.float32)).cuda()
    X = torch.from_numpy(rng.standard_normal((n, c)).astype(np.float32)).cuda().to(torch.bfloat16)
    ids = rng.integers(0, e - 1, (n, k)).astype(np.int32)  # one expert without tokens
    ids[7] = -1
    cal = lh.calibrate_routed(W, X, torch.from_numpy(ids).cuda())
    # the same as calibrating the rows sorted by hand
    off, order, _ = ref.route(ids, e)
    rows = X[torch.from_numpy(order[order >= 0] // k).cuda().long()]
    by_hand = lh.calibrate(W, rows, torch.from_numpy(off).cuda())
    assert torch.equal(cal["codes"], by_hand["codes"])
    assert (cal["codes"][e - 1] == 1).all()
    q = lh.QuantizedLayer(W, cal["global_amax"], cal["codes"])
    r = lh.Routing(n, k, e).route(torch.from_numpy(ids).cuda())
    w = torch.from_numpy(rng.random((n, k)).astype(np.float32)).cuda()
    y = q.forward_routed(X, r, w).double().cpu().numpy()
    want, tol = np.zeros((n, m)), np.zeros((n, m))
    per = [expected(q, W, X, i) for i in range(e)]
    for t in range(n):
        for s in range(k):
            if ids[t, s] >= 0:
                want[t] += float(w[t, s]) * per[ids[t, s]][0][t]
                tol[t] += float(w[t, s]) * per[ids[t, s]][1][t] * (1 + 2.0 ** -20)
    tol += (np.abs(want) + tol) * (2.0 ** -8 + k * 2.0 ** -24) + 1e-30
    assert (np.abs(y - want) <= tol).all()
    assert (y[7] == 0).all()
    # the layer in two graphs that run at the same time, against the layer alone
    x2 = (X * 2).contiguous()
    q.forward_routed(X, r, w), q.forward_routed(x2, r, w)
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        ya = q.forward_routed(X, r, w)
    with torch.cuda.graph(gb):
        yb = q.forward_routed(x2, r, w)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(sa):
            ga.replay()
        with torch.cuda.stream(sb):
            gb.replay()
    torch.cuda.synchronize()
    assert np.array_equal(ya.double().cpu().numpy(), y)
    assert torch.equal(yb, lh.QuantizedLayer(W, cal["global_amax"], cal["codes"]).forward_routed(x2, r, w))


def test_refusals(cuda_ok):
    lh = _lh()
    W = torch.randn(64, 64, device="cuda")
    cal = lh.calibrate(W, torch.randn(40, 64, device="cuda").bfloat16())
    q = lh.QuantizedLayer(W, cal["global_amax"], cal["codes"])
    with pytest.raises(ValueError):
        q(torch.randn(3, 48, device="cuda"))
    with pytest.raises(ValueError):
        q(torch.randn(3, 64))
    with pytest.raises(ValueError):
        q(torch.randn(3, 64, device="cuda").half())
    with pytest.raises(ValueError):
        q(torch.randn(3, 64, device="cuda"), offsets=torch.zeros(2, dtype=torch.int64, device="cuda"))
    r = lh.Routing(5, 2, 1)
    with pytest.raises(ValueError):
        r.route(torch.zeros(5, 2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        r.route(torch.zeros(4, 2, dtype=torch.int32, device="cuda"))
    r.route(torch.zeros(5, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        q.forward_routed(torch.randn(4, 64, device="cuda"), r)
    with pytest.raises(ValueError):
        q.forward_routed(torch.randn(5, 64, device="cuda"), r, torch.ones(5, 2, device="cuda").double())
    with pytest.raises(ValueError):
        lh.QuantizedLayer(W[:, :48], cal["global_amax"], cal["codes"][..., :3])

"""Arguments that the package's classes refuse before anything reaches the library (no GPU: the tensors' types and
shapes are looked at before their device)."""
import pytest
import torch


def _lh():
    import scale_calibration_b200 as lh
    return lh


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.int16])
def test_calibration_takes_bf16_tokens_only(dtype):
    # other types' bits would be read as bf16
    lh = _lh()
    W, X = torch.zeros(2, 8, 64), torch.zeros(10, 64).to(dtype)
    with pytest.raises(ValueError, match="X must be bf16"):
        lh.calibrate_routed(W, X, torch.zeros(10, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="X must be bf16"):
        lh.calibrate(W[0], X)
    cal = lh.Calibrator(1, 8, 64, 10, False, device="cpu")
    with pytest.raises(ValueError, match="X must be bf16"):
        cal.run(W[:1], X)


def parts(n_mats=3, c_out=8, c_in=64):
    return dict(W=torch.zeros(n_mats, c_out, c_in), global_amax=torch.ones(n_mats),
                codes=torch.ones(n_mats, c_out, c_in // 16, dtype=torch.uint8), x_amax=None)


@pytest.mark.parametrize("over,what", [
    (dict(codes=torch.ones(3, 8, 4, dtype=torch.int32)), "codes"), (dict(codes=torch.ones(3, 8, 3, dtype=torch.uint8)), "codes"),
    (dict(codes=torch.ones(3, 8, 4)), "codes"), (dict(global_amax=torch.ones(3).double()), "global_amax"),
    (dict(global_amax=torch.ones(3).bfloat16()), "global_amax"), (dict(global_amax=torch.ones(2)), "global_amax"),
    (dict(global_amax=torch.ones(6)[::2]), "global_amax"), (dict(x_amax=torch.ones(1).bfloat16()), "x_amax"),
    (dict(x_amax=torch.ones(1).double()), "x_amax"), (dict(x_amax=torch.ones(0)), "x_amax"),
])
def test_a_layer_refuses_other_types_and_sizes(over, what):
    with pytest.raises(ValueError, match=what):
        _lh().QuantizedLayer(**dict(parts(), **over))


@pytest.mark.parametrize("offsets", [torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int64), torch.zeros(4),
                                     torch.zeros(8, dtype=torch.int64)[::2]])
def test_offsets_of_other_types_and_sizes_are_refused(offsets):
    # they would be read past their end
    lh = _lh()
    layer = object.__new__(lh.QuantizedLayer)
    layer.n_mats, layer.c_out, layer.c_in, layer.x_amax, layer.packed = 3, 8, 64, None, torch.zeros(1)
    with pytest.raises(ValueError, match="offsets must be 4"):
        layer(torch.zeros(5, 64), offsets)
    with pytest.raises(ValueError, match="offsets must be 4"):
        lh.Calibrator(3, 8, 64, 5, True, device="cpu").run(torch.zeros(3, 8, 64), torch.zeros(5, 64).bfloat16(), offsets)


def test_a_layer_refuses_to_lose_a_gradient():
    lh = _lh()
    one, bank = (object.__new__(lh.QuantizedLayer) for _ in range(2))
    for layer, n_mats in ((one, 1), (bank, 3)):
        layer.n_mats, layer.c_out, layer.c_in, layer.x_amax, layer.packed = n_mats, 8, 64, None, torch.zeros(1)
    x = torch.zeros(5, 64, requires_grad=True)
    off = torch.zeros(4, dtype=torch.int64)
    w = torch.ones(5, 2, requires_grad=True)
    routing = lh.Routing(5, 2, 3, device="cpu")
    for call in (lambda: one(x), lambda: bank(x, off), lambda: bank.forward_routed(x, routing),
                 lambda: bank.forward_routed(x.detach(), routing, w)):
        with pytest.raises(ValueError, match="requires a gradient"):
            call()


class OnGPU0(torch.Tensor):
    """Says that it is on the first GPU."""
    is_cuda = True
    device = torch.device("cuda:0")


def test_tensors_have_to_be_on_the_streams_device(monkeypatch):
    # a stream makes its device the current one: tensors of the device that was current before are not there
    import contextlib
    lh = _lh()
    current = [0]

    @contextlib.contextmanager
    def on(stream):
        current[0] = 1
        yield
        current[0] = 0

    monkeypatch.setattr(lh, "_on", on)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    gpu0 = lambda t: t.as_subclass(OnGPU0)  # noqa: E731
    ids = gpu0(torch.zeros(10, 2, dtype=torch.int32))
    routing = lh.Routing(10, 2, 3, device="cpu")
    routing.pos = gpu0(routing.pos)
    layer = object.__new__(lh.QuantizedLayer)
    layer.n_mats = 3
    w = gpu0(torch.ones(10, 2))
    for call in (lambda: lh.QuantizedLayer(**{k: v if v is None else gpu0(v) for k, v in parts().items()}),
                 lambda: routing.route(ids), lambda: layer.forward_routed(gpu0(torch.zeros(10, 64)), routing, w),
                 lambda: lh.calibrate_routed(gpu0(torch.zeros(3, 8, 64)), gpu0(torch.zeros(10, 64).bfloat16()), ids)):
        with pytest.raises(ValueError, match="is on cuda:0, the current device is cuda:1"):
            call()


def test_calibration_refuses_other_shapes():
    # rows and matrices past the tensors' ends would be read
    lh = _lh()
    cal = lh.Calibrator(2, 8, 64, 5, True, device="cpu")
    off, x, w = torch.zeros(3, dtype=torch.int64), torch.zeros(5, 64).bfloat16(), torch.zeros(2, 8, 64)
    for bad in (torch.zeros(5, 80)[:, :48], torch.zeros(5, 80), torch.zeros(5, 1, 64)):
        with pytest.raises(ValueError, match="X must be"):
            cal.run(w, bad.bfloat16(), off)
    for bad in (w[:1], w[0], torch.zeros(2, 8, 48), torch.zeros(2, 4, 64), torch.zeros(2, 2, 8, 64)):
        with pytest.raises(ValueError, match="W must be"):
            cal.run(bad, x, off)


@pytest.mark.parametrize("w", [
    torch.arange(192.0).view(1, 3, 64).transpose(0, 1),  # [3, 1, 64] with a stride of 192 for its one row: "contiguous"
    torch.arange(64.0).view(64, 1).t(), torch.arange(64.0).view(1, 64, 1).transpose(1, 2), torch.arange(64.0).expand(2, 3, 64),
    torch.arange(384.0).view(2, 3, 64), torch.arange(768.0).view(4, 3, 64)[::2], torch.arange(480.0).view(2, 3, 80)[..., :64],
    torch.arange(384.0).view(2, 64, 3).transpose(1, 2),
])
def test_matrices_lie_as_the_library_reads_them(w):
    lh = _lh()
    m = lh._matrices(w)
    assert torch.equal(m, w) and m.stride(-1) == 1 and m.stride(-2) >= m.shape[-1]
    if m.dim() == 3 and m.shape[0] > 1:
        assert m.stride(0) == m.shape[1] * m.stride(1)

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

"""backward refuses what another layer's forward saved."""
import pytest

torch = pytest.importorskip("torch")

from weight_communication_gb300 import build, fp8  # noqa: E402


def test_saved_of_another_layer():
    if not build.LIB.exists() or not build.CALLS.exists():
        build.build()
    lin = fp8.Fp8Linear.__new__(fp8.Fp8Linear)    # (its weights are on a GPU in earnest)
    lin.N, lin.K = 24, 40
    lin.w, lin.wt = fp8.Fp8Tensor.empty(24, 40, 128, "cpu"), fp8.Fp8Tensor.empty(40, 24, 128, "cpu")
    dy = torch.zeros(7, 24)
    with pytest.raises(ValueError, match="another layer"):
        lin.backward(dy, fp8.Fp8Tensor.empty(48, 7, device="cpu"))
    with pytest.raises(ValueError, match="dy has shape"):
        lin.backward(dy, fp8.Fp8Tensor.empty(40, 8, device="cpu"))
    with pytest.raises(ValueError, match="CUDA tensor"):    # its own: goes on to the quantization
        lin.backward(dy, fp8.Fp8Tensor.empty(40, 7, device="cpu"))

"""Refusals of the operators between the layers and of the loss, on the CPU: every
documented rule broken one at a time gives its status code and a message that
names the entry point, before anything is launched.  The pointers are placeholders
that nothing dereferences, so the file runs only where no GPU is visible."""
import ctypes
import math

import pytest

from weight_communication_gb300 import binding

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="placeholder pointers: run where no GPU is reachable")

from test_abi import FAKE, MIS, lib  # noqa: E402,F401  (the library fixture)
from test_ops_abi import BIG, EALIGN, EINVAL, ERANGE, OK, refused  # noqa: E402

ODD = FAKE + 1
ROWS = 8388481          # one more than the limit
FAR = 1 << 38


def kept(codes=FAKE, ld_codes=208, scales=FAKE, ld_scales=100):
    return ctypes.pointer(binding.WcKept(codes, ld_codes, scales, ld_scales))


BAD_KEPT = [(kept(codes=None), EINVAL), (kept(scales=None), EINVAL), (kept(codes=MIS), EALIGN),
            (kept(scales=MIS), EALIGN), (kept(ld_codes=200), EINVAL), (kept(ld_codes=192), EINVAL),
            (kept(ld_scales=99), EINVAL), (kept(ld_codes=FAR), ERANGE), (kept(ld_scales=FAR), ERANGE)]


def test_struct():
    assert ctypes.sizeof(binding.WcKept) == 32


def test_dequant(lib):
    names = ["q", "ldq", "s", "lds", "per", "rows", "cols", "out", "ot", "ldo", "st"]
    ok = (FAKE, 208, FAKE, 100, 1, 100, 200, FAKE, 1, 200, None)
    refused(lib, "wc_fp8_dequant", ok, names, [
        ({"q": None}, EINVAL), ({"q": MIS}, EALIGN), ({"s": None}, EINVAL), ({"s": MIS}, EALIGN),
        ({"out": None}, EINVAL), ({"out": ODD}, EALIGN), ({"out": FAKE + 2, "ot": 0}, EALIGN), ({"ot": 2}, EINVAL),
        ({"per": 64}, EINVAL), ({"per": 0}, EINVAL), ({"ldq": 192}, EINVAL), ({"ldq": 200}, EINVAL),
        ({"lds": 99}, EINVAL), ({"per": 128, "lds": 0}, EINVAL), ({"ldo": 199}, EINVAL), ({"rows": -1}, EINVAL),
        ({"cols": -1}, EINVAL), ({"rows": ROWS, "lds": BIG}, ERANGE), ({"cols": ROWS, "ldq": BIG, "ldo": BIG}, ERANGE),
        ({"rows": 1 << 20, "cols": 1 << 20, "lds": BIG, "ldq": BIG, "ldo": BIG}, ERANGE),
        ({"ldo": FAR}, ERANGE), ({"ldq": FAR}, ERANGE), ({"lds": FAR}, ERANGE),
        ({"rows": 0, "q": None, "s": None, "out": None}, OK), ({"cols": 0, "out": None}, OK)])


def test_activation(lib):
    names = ["gate", "ldg", "up", "ldu", "dtype", "kind", "rows", "cols", "h", "ldh", "kg", "ku", "st"]
    ok = (FAKE, 200, FAKE, 200, 1, 1, 100, 200, FAKE, 200, kept(), kept(), None)
    refused(lib, "wc_activation", ok, names, [
        ({"gate": None}, EINVAL), ({"gate": ODD}, EALIGN), ({"up": ODD}, EALIGN), ({"h": None}, EINVAL),
        ({"h": ODD}, EALIGN), ({"gate": FAKE + 2, "dtype": 0}, EALIGN), ({"dtype": 2}, EINVAL), ({"kind": 3}, EINVAL),
        ({"kind": -1}, EINVAL), ({"rows": -1}, EINVAL), ({"cols": -1}, EINVAL), ({"ldg": 199}, EINVAL),
        ({"ldu": 199}, EINVAL), ({"ldh": 199}, EINVAL), ({"ldh": FAR}, ERANGE), ({"rows": ROWS}, ERANGE),
        ({"cols": ROWS, "ldg": BIG, "ldu": BIG, "ldh": BIG}, ERANGE),
        # a kept gate without the kept up, or the other way round
        ({"ku": None}, EINVAL), ({"up": None}, EINVAL), ({"kg": None}, EINVAL),
        *[({"kg": k}, want) for k, want in BAD_KEPT], *[({"ku": k}, want) for k, want in BAD_KEPT],
        ({"rows": 0, "gate": None, "up": None, "h": None}, OK), ({"cols": 0, "gate": None, "h": None}, OK)])


def test_activation_grad(lib):
    names = ["dh", "ldd", "dtype", "kind", "rows", "cols", "kg", "ku", "dg", "ldg", "du", "ldu", "st"]
    ok = (FAKE, 200, 1, 2, 100, 200, kept(), kept(), FAKE, 200, FAKE, 200, None)
    refused(lib, "wc_activation_grad", ok, names, [
        ({"dh": None}, EINVAL), ({"dh": ODD}, EALIGN), ({"dg": None}, EINVAL), ({"dg": ODD}, EALIGN),
        ({"du": None}, EINVAL), ({"du": ODD}, EALIGN), ({"ku": None}, EINVAL), ({"kg": None}, EINVAL),
        ({"dtype": -1}, EINVAL), ({"kind": 7}, EINVAL), ({"rows": -1}, EINVAL), ({"cols": -1}, EINVAL),
        ({"ldd": 199}, EINVAL), ({"ldg": 199}, EINVAL), ({"ldu": 199}, EINVAL), ({"ldd": FAR}, ERANGE),
        ({"rows": ROWS}, ERANGE), *[({"kg": k}, want) for k, want in BAD_KEPT],
        *[({"ku": k}, want) for k, want in BAD_KEPT], ({"rows": 0, "dh": None, "dg": None, "du": None}, OK)])


def test_rms_norm(lib):
    names = ["x", "ldx", "add", "lda", "dtype", "rows", "cols", "w", "wt", "eps", "y", "ldy", "total", "ldt",
             "rstd", "kept", "st"]
    ok = (FAKE, 200, FAKE, 200, 1, 100, 200, FAKE, 1, 1e-6, FAKE, 200, FAKE, 200, FAKE, kept(), None)
    refused(lib, "wc_rms_norm", ok, names, [
        ({"x": None}, EINVAL), ({"x": ODD}, EALIGN), ({"add": ODD}, EALIGN), ({"w": None}, EINVAL), ({"w": ODD}, EALIGN),
        ({"w": FAKE + 2, "wt": 0}, EALIGN), ({"y": None}, EINVAL), ({"y": ODD}, EALIGN), ({"total": None}, EINVAL),
        ({"total": ODD}, EALIGN), ({"add": None}, EINVAL), ({"rstd": None}, EINVAL), ({"rstd": FAKE + 2}, EALIGN),
        ({"kept": None}, EINVAL), ({"dtype": 3}, EINVAL), ({"wt": 3}, EINVAL), ({"eps": -1e-9}, EINVAL),
        ({"eps": math.inf}, EINVAL), ({"eps": math.nan}, EINVAL), ({"rows": -1}, EINVAL), ({"cols": 0}, EINVAL),
        ({"ldx": 199}, EINVAL), ({"lda": 199}, EINVAL), ({"ldy": 199}, EINVAL), ({"ldt": 199}, EINVAL),
        ({"ldx": FAR}, ERANGE), ({"rows": ROWS}, ERANGE),
        ({"cols": 16385, "ldx": 20000, "lda": 20000, "ldy": 20000, "ldt": 20000}, ERANGE),
        *[({"kept": k}, want) for k, want in BAD_KEPT], ({"rows": 0, "x": None, "y": None}, OK)])


def test_rms_norm_grad(lib):
    names = ["dy", "ldy", "add", "lda", "dtype", "rows", "cols", "w", "wt", "rstd", "kept", "dx", "ldx", "dw", "dwt",
             "acc", "ws", "bytes", "st"]
    ok = (FAKE, 200, FAKE, 200, 1, 100, 200, FAKE, 1, FAKE, kept(), FAKE, 200, FAKE, 0, 0, FAKE, BIG, None)
    need = lib.wc_rms_norm_grad_workspace(100, 200)
    assert need >= 4 * 200
    refused(lib, "wc_rms_norm_grad", ok, names, [
        ({"dy": None}, EINVAL), ({"dy": ODD}, EALIGN), ({"add": ODD}, EALIGN), ({"w": None}, EINVAL), ({"w": ODD}, EALIGN),
        ({"rstd": None}, EINVAL), ({"rstd": FAKE + 2}, EALIGN), ({"kept": None}, EINVAL), ({"dx": None}, EINVAL),
        ({"dx": ODD}, EALIGN), ({"dw": None}, EINVAL), ({"dw": FAKE + 2}, EALIGN), ({"ws": None}, EINVAL),
        ({"ws": MIS}, EALIGN), ({"bytes": need - 1}, EINVAL), ({"dtype": 3}, EINVAL), ({"wt": -1}, EINVAL),
        ({"dwt": 2}, EINVAL), ({"rows": -1}, EINVAL), ({"cols": 0}, EINVAL), ({"ldy": 199}, EINVAL), ({"lda": 199}, EINVAL),
        ({"ldx": 199}, EINVAL), ({"ldx": FAR}, ERANGE), ({"rows": ROWS}, ERANGE),
        ({"cols": 16385, "ldy": 20000, "lda": 20000, "ldx": 20000}, ERANGE), *[({"kept": k}, want) for k, want in BAD_KEPT],
        ({"rows": 0, "acc": 1, "dy": None, "dx": None, "ws": None}, OK)])
    assert lib.wc_rms_norm_grad_workspace(-1, 10) == EINVAL
    assert lib.wc_rms_norm_grad_workspace(5, 20000) == ERANGE
    assert lib.wc_rms_norm_grad_workspace(0, 10) == 0


SIZES = [({"T": -1}, EINVAL), ({"V": 0}, EINVAL), ({"D": 0}, EINVAL), ({"ldx": 63}, EINVAL), ({"ldw": 63}, EINVAL),
         ({"T": (1 << 31) - 1}, ERANGE), ({"V": (1 << 31) - 1}, ERANGE), ({"T": 1 << 30, "V": 1 << 14}, ERANGE),
         ({"D": (1 << 22) + 1, "ldx": 1 << 23, "ldw": 1 << 23}, ERANGE),
         ({"T": 1 << 20, "D": 1 << 20, "ldx": 1 << 20, "ldw": 1 << 20}, ERANGE),
         ({"V": 1 << 20, "D": 1 << 20, "ldx": 1 << 20, "ldw": 1 << 20}, ERANGE), ({"ldx": FAR}, ERANGE), ({"ldw": FAR}, ERANGE)]


def test_cross_entropy(lib):
    names = ["x", "ldx", "w", "ldw", "y", "it", "T", "V", "D", "losses", "lse", "ws", "bytes", "st"]
    ok = (FAKE, 64, FAKE, 64, FAKE, 1, 10, 100, 64, FAKE, FAKE, FAKE, BIG, None)
    need = lib.wc_cross_entropy_workspace(FAKE, 64, FAKE, 64, 10, 100, 64)
    assert need > 0
    # rows that do not start on 16 bytes are copied
    assert lib.wc_cross_entropy_workspace(FAKE, 65, FAKE, 64, 10, 100, 64) >= need + 10 * 64 * 2
    assert lib.wc_cross_entropy_workspace(FAKE, 64, FAKE + 2, 64, 10, 100, 64) >= need + 100 * 64 * 2
    refused(lib, "wc_cross_entropy", ok, names, SIZES + [
        ({"x": None}, EINVAL), ({"x": ODD}, EALIGN), ({"w": None}, EINVAL), ({"w": ODD}, EALIGN), ({"y": None}, EINVAL),
        ({"y": MIS}, EALIGN), ({"y": FAKE + 2, "it": 0}, EALIGN), ({"it": 2}, EINVAL), ({"losses": FAKE + 2}, EALIGN),
        ({"lse": FAKE + 2}, EALIGN), ({"losses": None, "lse": None}, EINVAL), ({"ws": None}, EINVAL), ({"ws": MIS}, EALIGN),
        ({"bytes": need - 1}, EINVAL), ({"T": 0, "x": None, "y": None, "losses": None, "ws": None}, OK)])
    assert lib.wc_cross_entropy_workspace(FAKE, 64, FAKE, 64, 10, 0, 64) == EINVAL
    assert lib.wc_cross_entropy_workspace(None, 64, None, 64, 0, 10, 64) == 0


def test_cross_entropy_grad(lib):
    names = ["x", "ldx", "w", "ldw", "y", "it", "T", "V", "D", "lse", "dl", "dloss", "dx", "dxt", "lddx", "dw", "dwt",
             "lddw", "acc", "ws", "bytes", "st"]
    ok = (FAKE, 64, FAKE, 64, FAKE, 1, 10, 100, 64, FAKE, None, 0.1, FAKE, 1, 64, FAKE, 1, 64, 0, FAKE, BIG, None)
    need = lib.wc_cross_entropy_grad_workspace(FAKE, 64, FAKE, 64, 10, 100, 64)
    refused(lib, "wc_cross_entropy_grad", ok, names, SIZES + [
        ({"x": None}, EINVAL), ({"x": ODD}, EALIGN), ({"w": None}, EINVAL), ({"w": ODD}, EALIGN), ({"y": None}, EINVAL),
        ({"y": MIS}, EALIGN), ({"it": 2}, EINVAL), ({"lse": None}, EINVAL), ({"lse": FAKE + 2}, EALIGN),
        ({"dl": FAKE + 2}, EALIGN), ({"dx": None, "dw": None}, EINVAL), ({"dx": ODD}, EALIGN), ({"dw": ODD}, EALIGN),
        ({"dxt": 2}, EINVAL), ({"dwt": 2}, EINVAL), ({"dw": FAKE + 2, "dwt": 0}, EALIGN), ({"lddx": 63}, EINVAL),
        ({"lddw": 63}, EINVAL), ({"lddx": FAR}, ERANGE), ({"lddw": FAR}, ERANGE), ({"ws": None}, EINVAL),
        ({"ws": MIS}, EALIGN), ({"bytes": need - 1}, EINVAL), ({"T": 0, "acc": 1, "x": None, "ws": None}, OK),
        ({"T": 0, "dw": None, "x": None, "ws": None}, OK)])
    assert lib.wc_cross_entropy_grad_workspace(FAKE, 64, FAKE, 64, -1, 100, 64) == EINVAL
    # the logits' gradients of a piece of the vocabulary, not of all of it
    big = lib.wc_cross_entropy_grad_workspace(FAKE, 2048, FAKE, 2048, 8192, 256000, 2048)
    assert big < (1 << 28) + 3 * 8192 * 2048 * 4 + (1 << 20)


def test_python_refusals():
    """What the composed calls refuse before they reach the library."""
    from weight_communication_gb300 import activation, fp8, loss, norm
    cpu = torch.zeros(4, 32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        activation.forward(cpu)
    with pytest.raises(ValueError, match="kind"):
        activation.forward(cpu, kind="tanh")
    q = fp8.Fp8Tensor.empty(4, 32, device="cpu")
    with pytest.raises(ValueError, match="kind"):
        activation.backward(cpu, activation.Kept("tanh", q, None))
    with pytest.raises(ValueError, match="CUDA tensor"):
        activation.backward(cpu, activation.Kept("silu", q, None))
    with pytest.raises(ValueError, match="CUDA tensor"):
        norm.rms(cpu, cpu[0])
    with pytest.raises(ValueError, match="CUDA tensor"):
        norm.rms_grad(cpu, cpu[0], norm.Kept(q, cpu[:, 0]))
    with pytest.raises(ValueError, match="GPU"):
        fp8.dequantize(q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        loss.cross_entropy(cpu, cpu, torch.zeros(4, dtype=torch.int64))


def test_calls_refuse_wrong_arguments():
    calls = binding.calls()
    for name in ("fp8_dequantize", "activation", "activation_grad", "rms_norm", "rms_norm_grad", "cross_entropy",
                 "cross_entropy_grad"):
        with pytest.raises(TypeError, match=name):
            getattr(calls, name)(1)
    with pytest.raises(TypeError, match="gate must be a tensor"):
        calls.activation(1, None, 0, False, None)
    with pytest.raises(TypeError, match="8-bit matrix"):
        calls.fp8_dequantize((1, 2), None, torch.float32)

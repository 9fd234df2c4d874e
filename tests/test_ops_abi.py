"""Refusals of the training-step operators, on the CPU: every documented rule
broken one at a time gives its status code and a message that names the entry
point, before anything is launched.  The pointers are placeholders that
nothing dereferences, so the file runs only where no GPU is visible."""
import ctypes
import math

import pytest

from weight_communication_gb300 import binding

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="placeholder pointers: run where no GPU is reachable")

from test_abi import FAKE, MIS, lib  # noqa: E402,F401  (the library fixture)

OK, EINVAL, EALIGN, ERANGE = (binding.WC_OK, binding.WC_EINVAL, binding.WC_EALIGN,
                              binding.WC_ERANGE)
BIG = 1 << 60


def spans(*items):
    a = (binding.WcSpan * max(1, len(items)))()
    for i, (p, n, t) in enumerate(items):
        a[i] = binding.WcSpan(p, n, t, 0)
    return a


def refused(lib, name, ok, names, changes):
    f = getattr(lib, name)
    for what, want in changes:
        a = dict(zip(names, ok))
        a.update(what)
        rc = f(*a.values())
        assert rc == want, (name, what, rc, lib.wc_last_error())
        if want != OK:
            assert name in lib.wc_last_error().decode()


def test_grad_clip_refusals(lib):
    names = ["spans", "dst", "count", "max_norm", "eps", "stats", "ws", "bytes", "st"]
    two = spans((FAKE, 100, 0), (FAKE + 1024, 100, 1))
    ok = (two, None, 2, 1.0, 1e-6, FAKE, FAKE, BIG, None)
    refused(lib, "wc_grad_clip", ok, names, [
        ({"count": -1}, EINVAL), ({"spans": None}, EINVAL), ({"max_norm": -1.0}, EINVAL),
        ({"max_norm": math.nan}, EINVAL), ({"eps": -1e-9}, EINVAL), ({"eps": math.inf}, EINVAL),
        ({"eps": math.nan}, EINVAL), ({"stats": None}, EINVAL), ({"stats": MIS}, EALIGN),
        ({"ws": None}, EINVAL), ({"ws": MIS}, EALIGN), ({"bytes": 100}, EINVAL),
        ({"spans": spans((FAKE, 100, 0), (FAKE, 100, 7))}, EINVAL),
        ({"spans": spans((FAKE, -1, 0), (FAKE, 1, 0))}, EINVAL),
        ({"spans": spans((None, 5, 0), (FAKE, 1, 0))}, EINVAL),
        ({"spans": spans((FAKE + 2, 5, 0), (FAKE + 64, 1, 0))}, EALIGN),
        ({"spans": spans((FAKE + 1, 5, 1), (FAKE + 64, 1, 0))}, EALIGN),
        ({"spans": spans((FAKE, 1 << 40, 0), (FAKE, 1, 0))}, ERANGE),
        ({"spans": spans((FAKE, 1 << 39, 1), (FAKE + (1 << 41), 1 << 39, 1))}, ERANGE),
        # in place: the second tensor starts inside the first
        ({"spans": spans((FAKE, 100, 0), (FAKE + 396, 100, 0))}, EINVAL),
        ({"spans": spans((FAKE + 396, 100, 0), (FAKE, 100, 0))}, EINVAL),
        ({"spans": spans((FAKE, 100, 0), (FAKE, 100, 0))}, EINVAL),
        # into other buffers: lengths, and overlaps with a source or each other
        ({"dst": spans((FAKE + 8192, 100, 0), (FAKE + 16384, 99, 0))}, EINVAL),
        ({"dst": spans((FAKE + 8192, 100, 0), (FAKE + 8192, 100, 0))}, EINVAL),
        ({"dst": spans((FAKE + 8192, 100, 0), (FAKE + 200, 100, 0))}, EINVAL),
        ({"dst": spans((FAKE + 8192, 100, 5), (FAKE + 16384, 100, 0))}, EINVAL),
    ])


def test_grad_norm_refusals(lib):
    names = ["spans", "count", "stats", "ws", "bytes", "st"]
    ok = (spans((FAKE, 100, 0), (FAKE + 64, 100, 1)), 2, FAKE, FAKE, BIG, None)
    refused(lib, "wc_grad_norm", ok, names, [
        ({"count": -1}, EINVAL), ({"spans": None}, EINVAL), ({"stats": None}, EINVAL),
        ({"stats": MIS}, EALIGN), ({"ws": None}, EINVAL), ({"bytes": 0}, EINVAL),
        ({"spans": spans((FAKE, 100, 2), (FAKE, 1, 0))}, EINVAL)])
    assert lib.wc_grad_norm_workspace(0) > 0
    assert lib.wc_grad_norm_workspace(1025) == 2 * lib.wc_grad_norm_workspace(1024)


def test_embedding_refusals(lib):
    names = ["table", "dtype", "ldt", "ids", "it", "n", "first", "V", "D", "scale", "out", "ldo", "st"]
    ok = (FAKE, 1, 64, FAKE, 1, 10, 0, 100, 64, 1.0, FAKE, 64, None)
    refused(lib, "wc_embedding", ok, names, [
        ({"table": None}, EINVAL), ({"table": MIS}, EALIGN), ({"ids": None}, EINVAL),
        ({"ids": MIS}, EALIGN), ({"out": None}, EINVAL), ({"out": MIS}, EALIGN),
        ({"dtype": 2}, EINVAL), ({"it": 2}, EINVAL), ({"n": -1}, EINVAL), ({"V": -1}, EINVAL),
        ({"D": -1}, EINVAL), ({"first": -1}, EINVAL), ({"first": 1 << 62}, EINVAL),
        ({"ldt": 63}, EINVAL), ({"ldo": 63}, EINVAL), ({"n": 1 << 31}, ERANGE),
        ({"V": (1 << 31) - 1}, ERANGE), ({"D": 1 << 31, "ldt": 1 << 31, "ldo": 1 << 31}, ERANGE),
        ({"n": (1 << 31) - 1, "D": 1024, "ldt": 1024, "ldo": 1024}, ERANGE),
        ({"n": 0, "table": None, "ids": None, "out": None}, OK),
        ({"D": 0, "table": None, "ids": None, "out": None}, OK)])


def test_embedding_grad_refusals(lib):
    names = ["dy", "dt", "ldy", "ids", "it", "n", "first", "V", "D", "scale", "acc", "out", "ot",
             "ldo", "ws", "bytes", "st"]
    ok = (FAKE, 1, 64, FAKE, 1, 10, 0, 100, 64, 1.0, 0, FAKE, 0, 64, FAKE, BIG, None)
    need = lib.wc_embedding_grad_workspace(10, 100, 64)
    assert need > 0
    refused(lib, "wc_embedding_grad", ok, names, [
        ({"dy": None}, EINVAL), ({"dy": MIS}, EALIGN), ({"ids": None}, EINVAL), ({"ids": MIS}, EALIGN),
        ({"out": None}, EINVAL), ({"out": MIS}, EALIGN), ({"ws": None}, EINVAL), ({"ws": MIS}, EALIGN),
        ({"bytes": need - 1}, EINVAL), ({"dt": 3}, EINVAL), ({"ot": -1}, EINVAL), ({"it": 5}, EINVAL),
        ({"n": -1}, EINVAL), ({"first": -5}, EINVAL), ({"ldy": 60}, EINVAL), ({"ldo": 60}, EINVAL),
        ({"n": 1 << 31}, ERANGE), ({"V": 1 << 31}, ERANGE),
        ({"V": 0, "out": None, "ws": None}, OK), ({"D": 0, "out": None}, OK),
        ({"n": 0, "acc": 1, "dy": None, "ids": None, "out": None, "ws": None}, OK)])
    assert lib.wc_embedding_grad_workspace(-1, 10, 10) == EINVAL
    assert lib.wc_embedding_grad_workspace(1 << 31, 10, 10) == ERANGE


def test_fp8_quant_refusals(lib):
    names = ["x", "dtype", "rows", "cols", "ld", "square", "q", "ldq", "s", "lds", "qt", "ldqt",
             "st_", "ldst", "stream"]
    ok = (FAKE, 1, 100, 200, 200, 0, FAKE, 208, FAKE, 100, FAKE, 112, FAKE, 200, None)
    refused(lib, "wc_fp8_quant", ok, names, [
        ({"x": None}, EINVAL), ({"x": MIS}, EALIGN), ({"dtype": 4}, EINVAL), ({"rows": -1}, EINVAL),
        ({"cols": -1}, EINVAL), ({"ld": 199}, EINVAL), ({"s": None}, EINVAL), ({"q": None}, EINVAL),
        ({"st_": None}, EINVAL), ({"qt": None}, EINVAL), ({"q": MIS}, EALIGN), ({"s": MIS}, EALIGN),
        ({"qt": MIS}, EALIGN), ({"st_": MIS}, EALIGN), ({"ldq": 192}, EINVAL), ({"ldq": 200}, EINVAL),
        ({"ldqt": 96}, EINVAL), ({"ldqt": 100}, EINVAL), ({"lds": 99}, EINVAL), ({"ldst": 199}, EINVAL),
        ({"rows": 8388481, "lds": BIG, "ldqt": 1 << 40}, ERANGE),
        ({"cols": 8388481, "ld": BIG, "ldq": 1 << 40, "ldst": BIG}, ERANGE),
        ({"q": None, "s": None, "qt": None, "st_": None}, EINVAL),
        ({"square": 1, "lds": 0}, EINVAL), ({"square": 1, "ldst": 1}, EINVAL),
        ({"rows": 0, "x": None, "q": None, "s": None, "qt": None, "st_": None}, OK),
        ({"cols": 0, "x": None}, OK)])


def test_fp8_matmul_refusals(lib):
    names = ["a", "lda", "sa", "ldsa", "ga", "b", "ldb", "sb", "ldsb", "gb", "M", "N", "K", "out",
             "ot", "ldo", "acc", "st"]
    ok = (FAKE, 256, FAKE, 100, 1, FAKE, 256, FAKE, 2, 128, 100, 200, 250, FAKE, 1, 200, 0, None)
    refused(lib, "wc_fp8_matmul", ok, names, [
        ({"a": None}, EINVAL), ({"a": MIS}, EALIGN), ({"sa": None}, EINVAL), ({"sa": MIS}, EALIGN),
        ({"b": None}, EINVAL), ({"b": MIS}, EALIGN), ({"sb": None}, EINVAL), ({"sb": MIS}, EALIGN),
        ({"out": None}, EINVAL), ({"out": MIS}, EALIGN), ({"ga": 64}, EINVAL), ({"gb": 0}, EINVAL),
        ({"lda": 250}, EINVAL), ({"lda": 240}, EINVAL), ({"ldb": 264}, EINVAL), ({"ldsa": 99}, EINVAL),
        ({"ldsb": 1}, EINVAL), ({"ot": 2}, EINVAL), ({"ldo": 199}, EINVAL), ({"M": -1}, EINVAL),
        ({"N": -1}, EINVAL), ({"K": -1}, EINVAL), ({"M": 1 << 31, "ldsa": BIG}, ERANGE),
        ({"M": 1 << 30, "N": 1 << 14, "ldsa": BIG, "ldsb": BIG, "ldo": BIG}, ERANGE),
        ({"M": 0, "a": None, "out": None}, OK), ({"N": 0, "b": None, "out": None}, OK)])


def test_python_refusals():
    """What the composed calls refuse before they reach the library."""
    from weight_communication_gb300 import embedding, fp8, gradnorm
    cpu = torch.zeros(4, 32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gradnorm.TensorList([cpu])
    with pytest.raises(ValueError, match="empty list"):
        gradnorm.norm([])
    with pytest.raises(ValueError, match="matrix"):
        embedding.lookup(torch.zeros(5), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="contiguous"):
        embedding.lookup(cpu, torch.zeros(4, 6, dtype=torch.int64)[:, ::2])
    with pytest.raises(ValueError, match="matrix"):
        fp8.quantize(torch.zeros(3))
    with pytest.raises(ValueError, match="neither"):
        fp8.quantize(cpu, rows=False)
    with pytest.raises(ValueError, match="block_rows"):
        fp8.Fp8Tensor(cpu, cpu, 4, 32, 64)
    a = fp8.Fp8Tensor.empty(4, 32, device="cpu")
    with pytest.raises(ValueError, match="columns"):
        fp8.matmul(a, fp8.Fp8Tensor.empty(4, 48, device="cpu"))
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.fp8_quant(cpu, a.codes, a.scales)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.embedding_grad(cpu, torch.zeros(4, dtype=torch.int64), torch.zeros(9, 32),
                               torch.zeros(16, dtype=torch.uint8))
    assert ctypes.sizeof(binding.WcSpan) == 24

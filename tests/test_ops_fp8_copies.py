"""Copies of 8-bit matrices and layers (copy, pickle, torch.save) stand for
themselves: their own memory, and nothing of the original's."""
import copy
import io
import pickle

import pytest

torch = pytest.importorskip("torch")

from weight_communication_gb300 import binding, build, fp8  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    if not build.LIB.exists() or not build.CALLS.exists():
        build.build()


def saved(t):
    f = io.BytesIO()
    torch.save(t, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


COPIES = {"deepcopy": copy.deepcopy, "pickle": lambda t: pickle.loads(pickle.dumps(t)), "save": saved}


def made(rows, cols, block_rows):
    t = fp8.Fp8Tensor.empty(rows, cols, block_rows, device="cpu")
    t.codes.view(torch.uint8).copy_(torch.arange(t.codes.numel()).view(t.codes.shape) % 251)
    t.scales.copy_(torch.arange(1.0, 1.0 + t.scales.numel()).view(t.scales.shape))
    return t


def viewed(rows, cols, block_rows):
    """The same matrix in rows further apart, past the start of their storage."""
    m = made(rows, cols, block_rows)
    codes = torch.zeros(rows + 2, m.codes.shape[1] + 32, dtype=torch.uint8)
    scales = torch.zeros(m.scales.shape[0], m.scales.shape[1] + 4)
    codes[2:, :m.codes.shape[1]] = m.codes.view(torch.uint8)
    scales[:, :m.scales.shape[1]] = m.scales
    return fp8.Fp8Tensor(codes.view(torch.float8_e4m3fn)[2:], scales, rows, cols, block_rows)


def bytes_of(t):
    return t.codes.view(torch.uint8)[:, :t.cols].clone(), t.scales.clone()


def addresses(t):
    return {t.codes.data_ptr(), t.scales.data_ptr()}


@pytest.mark.parametrize("how", COPIES)
@pytest.mark.parametrize("make", [made, viewed])
@pytest.mark.parametrize("rows,cols,block_rows", [(5, 300, 1), (300, 257, 128), (1, 16, 1)])
def test_copy_has_its_own_memory(how, make, rows, cols, block_rows):
    t = make(rows, cols, block_rows)
    codes, scales = bytes_of(t)
    c = COPIES[how](t)
    assert (c.rows, c.cols, c.block_rows, c.device) == (rows, cols, block_rows, t.device)
    assert not addresses(c) & addresses(t)
    # what the calls are given names none of the original's memory, and is the
    # memory that the copy shows
    assert not addresses(t) & {p for p in c._parts if isinstance(p, int)}
    first = c._parts[0]
    assert first.untyped_storage().data_ptr() == c.codes.untyped_storage().data_ptr()
    assert all(torch.equal(x, y) for x, y in zip(bytes_of(c), (codes, scales)))
    t.codes.view(torch.uint8).fill_(1)
    t.scales.fill_(-1.0)
    assert all(torch.equal(x, y) for x, y in zip(bytes_of(c), (codes, scales)))
    del t
    assert all(torch.equal(x, y) for x, y in zip(bytes_of(c), (codes, scales)))


def test_shallow_copy_is_the_same_matrix():
    t = made(5, 300, 1)
    c = copy.copy(t)
    assert addresses(c) == addresses(t)


def test_parts_that_do_not_fit_are_refused():
    """Sizes are checked against the tensors at each call, not once."""
    calls = binding.calls()
    buffer = made(4, 130, 1)._parts[0]
    good = (buffer, None, 4, 130, 1)
    for parts in ((buffer, None, 5, 130, 1), (buffer[:-16], None, 4, 130, 1),
                  (buffer.view(torch.int32), None, 4, 130, 1)):
        with pytest.raises(ValueError, match="buffer"):
            calls.fp8_matmul(parts, good, None, torch.bfloat16, False)
    t = viewed(4, 130, 1)
    t.scales.resize_(1, 4)
    with pytest.raises(ValueError, match="scales has shape"):
        fp8.matmul(t, t)


@pytest.mark.gpu
@pytest.mark.parametrize("how", COPIES)
def test_copied_layer(how):
    """A copy keeps the weights it was made with, whatever becomes of the
    original, and its own loads and passes leave the original alone."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(91)
    w, w2 = (torch.randn(200, 300, generator=g, device=dev).bfloat16() for _ in range(2))
    x = torch.randn(70, 300, generator=g, device=dev).bfloat16()
    dy = torch.randn(70, 200, generator=g, device=dev).bfloat16()
    lin = fp8.Fp8Linear(w)
    y, saved_x = lin.forward(x, save=True)
    dx, dw = lin.backward(dy, saved_x)
    y2 = fp8.Fp8Linear(w2).forward(x)
    c, cx = COPIES[how](lin), COPIES[how](saved_x)
    lin.load(w2)
    assert torch.equal(lin.forward(x), y2)
    assert torch.equal(c.forward(x), y)
    c_dx, c_dw = c.backward(dy, cx)
    assert torch.equal(c_dx, dx) and torch.equal(c_dw, dw)
    c.load(w2)
    lin.load(w)
    assert torch.equal(c.forward(x), y2) and torch.equal(lin.forward(x), y)

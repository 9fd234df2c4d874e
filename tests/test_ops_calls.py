"""What the Python calls of the training-step operators accept and refuse:
types, shapes, strides, devices and streams, with the exception's class and a
message that names the argument."""
import pytest

torch = pytest.importorskip("torch")

from weight_communication_gb300 import binding, build, embedding, fp8, gradnorm  # noqa: E402


@pytest.fixture(scope="module")
def calls():
    if not build.LIB.exists() or not build.CALLS.exists():
        build.build()
    return binding.calls()


def test_calls_refuse_wrong_arguments(calls):
    for name in ("embedding", "embedding_grad", "grad_norm", "fp8_empty", "fp8_view", "fp8_quantize",
                 "fp8_quantize_into", "fp8_matmul", "setup"):
        with pytest.raises(TypeError, match=name):
            getattr(calls, name)(1)
    with pytest.raises(TypeError, match="table must be a tensor"):
        calls.embedding([1.0], torch.zeros(2, dtype=torch.int64), 1.0, 0, None)
    with pytest.raises(TypeError, match="8-bit matrix"):
        calls.fp8_matmul((1, 2), (1, 2), None, torch.bfloat16, False)
    with pytest.raises(ValueError, match="address of"):
        calls.setup({}, RuntimeError)
    with pytest.raises(ValueError, match="negative"):
        calls.fp8_empty(-1, 4, 1, torch.device("cpu"))


def test_matrix_in_one_buffer(calls):
    for rows, cols, block in ((1, 1, 1), (3, 130, 1), (300, 257, 128), (0, 5, 1), (5, 0, 128)):
        t = fp8.Fp8Tensor.empty(rows, cols, block, device="cpu")
        assert t.codes.shape == (rows, -(-cols // 16) * 16) and t.codes.dtype == torch.float8_e4m3fn
        assert t.scales.shape == (-(-cols // 128), -(-rows // block)) and t.scales.dtype == torch.float32
        assert (t.rows, t.cols, t.block_rows, t.device) == (rows, cols, block, torch.device("cpu"))
        if rows and cols:  # the two views do not overlap, and end inside the buffer
            t.codes.view(torch.uint8).fill_(0x7F)
            t.scales.fill_(1.0)
            assert bool((t.codes.view(torch.uint8) == 0x7F).all()) and bool((t.scales == 1.0).all())


def test_view_refusals(calls):
    codes = torch.zeros(4, 144, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.ones(2, 4)
    fp8.Fp8Tensor(codes, scales, 4, 130)
    with pytest.raises(TypeError, match="codes"):
        fp8.Fp8Tensor(codes.view(torch.uint8), scales, 4, 130)
    with pytest.raises(TypeError, match="scales"):
        fp8.Fp8Tensor(codes, scales.double(), 4, 130)
    with pytest.raises(ValueError, match="codes has shape"):
        fp8.Fp8Tensor(codes, scales, 5, 130)
    with pytest.raises(ValueError, match="codes has shape"):
        fp8.Fp8Tensor(codes, scales, 4, 145)
    with pytest.raises(ValueError, match="scales has shape"):
        fp8.Fp8Tensor(codes, scales[:1], 4, 130)
    with pytest.raises(ValueError, match="consecutive"):
        fp8.Fp8Tensor(codes, torch.ones(4, 2).t(), 4, 130)
    with pytest.raises(ValueError, match="overlapping"):
        fp8.Fp8Tensor(codes[:1].expand(4, 144), scales, 4, 130)


@pytest.mark.gpu
def test_refusals_on_the_gpu(calls):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d = torch.device("cuda:0")
    table = torch.randn(10, 24, device=d)
    ids = torch.tensor([1, 2, 3], device=d)
    with pytest.raises(ValueError, match="ids is on cpu"):
        embedding.lookup(table, ids.cpu())
    with pytest.raises(TypeError, match="ids must be"):
        embedding.lookup(table, ids.float())
    with pytest.raises(TypeError, match="table must be"):
        embedding.lookup(table.half(), ids)
    with pytest.raises(TypeError, match="out must be"):
        embedding.lookup(table, ids, out=torch.empty(3, 24, device=d, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="out has shape"):
        embedding.lookup(table, ids, out=torch.empty(2, 24, device=d))
    with pytest.raises(ValueError, match="out has shape"):
        embedding.lookup(table, ids, out=torch.empty(3, 25, device=d))
    with pytest.raises(ValueError, match="consecutive"):
        embedding.lookup(torch.randn(24, 10, device=d).t(), ids)
    with pytest.raises(binding.WcError, match="first"):
        embedding.lookup(table, ids, first_row=-1)
    with pytest.raises(binding.WcError, match="aligned") as e:
        embedding.lookup(table.view(-1)[1:1 + 9 * 24].view(9, 24), ids)
    assert e.value.code == binding.WC_EALIGN

    dy = torch.randn(3, 24, device=d)
    with pytest.raises(ValueError, match="accumulate needs"):
        embedding.grad(dy, ids, 10, accumulate=True)
    with pytest.raises(ValueError, match="dy has shape"):
        embedding.grad(dy[:2], ids, 10)
    with pytest.raises(ValueError, match="dy has shape"):
        embedding.grad(torch.randn(3, 2, 24, device=d), ids, 10)
    with pytest.raises(ValueError, match="out has shape"):
        embedding.grad(dy, ids, 10, out=torch.empty(9, 24, device=d))
    with pytest.raises(TypeError, match="out must be"):
        embedding.grad(dy, ids, 10, out=torch.empty(10, 24, device=d), out_dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="out_dtype"):
        embedding.grad(dy, ids, 10, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="negative"):
        embedding.grad(dy, ids, -1)

    with pytest.raises(TypeError, match="x must be"):
        fp8.quantize(table.half())
    with pytest.raises(ValueError, match="consecutive"):
        fp8.quantize(table.t())
    with pytest.raises(ValueError, match="overlapping"):
        fp8.quantize(table[:1].expand(5, 24))
    a, b = fp8.quantize(table)[0], fp8.quantize(torch.randn(7, 24, device=d))[0]
    with pytest.raises(ValueError, match="out has shape"):
        fp8.matmul(a, b, out=torch.empty(10, 8, device=d))
    with pytest.raises(TypeError, match="out_dtype"):
        fp8.matmul(a, b, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="accumulate needs"):
        fp8.matmul(a, b, accumulate=True)
    with pytest.raises(ValueError, match="b is on"):
        fp8.matmul(a, fp8.Fp8Tensor.empty(7, 24, device="cpu"))
    lin = fp8.Fp8Linear(torch.randn(16, 24, device=d), training=False)
    with pytest.raises(ValueError, match="x has shape"):
        lin.load(torch.randn(24, 16, device=d))
    with pytest.raises(ValueError, match="training"):
        lin.backward(torch.randn(10, 16, device=d), a)

    with pytest.raises(ValueError, match="stats has"):
        gradnorm.norm([table], stats=torch.empty(2, device=d))
    with pytest.raises(TypeError, match="stats must be"):
        gradnorm.clip([table], 1.0, stats=torch.empty(2, device=d, dtype=torch.float64))
    with pytest.raises(binding.WcError, match="max_norm"):
        gradnorm.clip([table], -1.0)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_new_tensors_belong_to_the_given_stream(calls):
    """A result made on a side stream is usable there while the default stream
    reuses memory that was freed on it: nothing of the call is allocated from
    another stream's pool."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d = torch.device("cuda:0")
    table = torch.randn(1000, 64, device=d)
    ids = torch.randint(0, 1000, (5000,), device=d)
    want = embedding.lookup(table, ids, scale=2.0)
    grad = embedding.grad(want, ids, 1000)
    s = torch.cuda.Stream(d)
    s.wait_stream(torch.cuda.current_stream(d))
    for _ in range(5):
        out = embedding.lookup(table, ids, scale=2.0, stream=s)
        got = embedding.grad(out, ids, 1000, stream=s)
        junk = torch.full((5000, 64), 7.0, device=d)  # on the default stream
        del junk
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(got, grad)

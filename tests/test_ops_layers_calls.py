"""What the Python calls of activations, norms and 8-bit values refuse on a GPU, and
how they and the loss stand to autograd and to copies of what they keep."""
import copy
import pickle
import warnings

import pytest
import torch

from gpu_util import dev  # noqa: F401

pytestmark = pytest.mark.gpu


def test_refusals(dev):
    from weight_communication_gb300 import activation, binding, fp8, norm
    x = torch.randn(10, 40, device=dev)
    h, kept = activation.forward(x, x, save=True)
    for call, kind, match in ((lambda: activation.forward(x.half()), TypeError, "gate must be"),
                              (lambda: activation.forward(x, x[:9]), ValueError, "up has shape"),
                              (lambda: activation.forward(x, x.bfloat16()), TypeError, "up must be"),
                              (lambda: activation.forward(x, x.cpu()), ValueError, "up is on"),
                              (lambda: activation.forward(x.t()), ValueError, "consecutive"),
                              (lambda: activation.forward(x[:1].expand(5, 40)), ValueError, "overlapping"),
                              (lambda: activation.forward(x.view(2, 5, 40).transpose(0, 1)), ValueError, "contiguous"),
                              (lambda: activation.forward(x, out=x.bfloat16()), TypeError, "out must be"),
                              (lambda: activation.forward(x, out=x[:9]), ValueError, "out has shape"),
                              (lambda: activation.forward(torch.zeros((), device=dev)), ValueError, "columns"),
                              (lambda: activation.backward(x[:9], kept), ValueError, "the kept gate is"),
                              (lambda: activation.backward(x[:, :39], kept), ValueError, "the kept gate is"),
                              (lambda: activation.backward(x.half(), kept), TypeError, "dh must be"),
                              (lambda: activation.backward(x, activation.Kept("silu", kept.gate, fp8.quantize_weight(x)[0])),
                               ValueError, "rows per scale"),
                              (lambda: fp8.dequantize(kept.gate, torch.float16), TypeError, "out_dtype"),
                              (lambda: fp8.dequantize(kept.gate, out=x[:9]), ValueError, "out has shape"),
                              (lambda: fp8.dequantize(kept.gate, out=x.cpu()), ValueError, "out is on"),
                              (lambda: norm.rms(x, x[0, :39]), ValueError, "weight has shape"),
                              (lambda: norm.rms(x, x[0].half()), TypeError, "weight must be"),
                              (lambda: norm.rms(x, x[0].cpu()), ValueError, "weight is on"),
                              (lambda: norm.rms(x, x[0], add=x[:9]), ValueError, "add has shape"),
                              (lambda: norm.rms(x, x[0], eps=-1.0), binding.WcError, "eps"),
                              (lambda: norm.rms(torch.zeros(2, 16385, device=dev), torch.zeros(16385, device=dev)),
                               binding.WcError, "16384")):
        with pytest.raises(kind, match=match):
            call()
    y, _, k = norm.rms(x, x[0], save=True)
    for call, kind, match in ((lambda: norm.rms_grad(x[:9], x[0], k), ValueError, "rstd has shape|kept input"),
                              (lambda: norm.rms_grad(x, x[0], norm.Kept(k.input, k.rstd[:9])), ValueError, "rstd has shape"),
                              (lambda: norm.rms_grad(x, x[0], norm.Kept(k.input, k.rstd.double())), TypeError, "rstd must be"),
                              (lambda: norm.rms_grad(x, x[0], k, add=x.bfloat16()), TypeError, "add must be"),
                              (lambda: norm.rms_grad(x, x[0], k, dweight=x), ValueError, "dweight has shape"),
                              (lambda: norm.rms_grad(x, x[0], k, dweight=x[0].half()), TypeError, "dweight must be"),
                              (lambda: norm.rms_grad(x, x[0], k, accumulate=True), ValueError, "accumulate needs")):
        with pytest.raises(kind, match=match):
            call()
    torch.cuda.synchronize()


def test_copies_have_their_own_memory(dev):
    from weight_communication_gb300 import activation, norm
    x = torch.randn(30, 300, device=dev)
    w = torch.ones(300, device=dev)
    _, kept = activation.forward(x, x, save=True)
    _, _, kn = norm.rms(x, w, save=True)
    want, want_n = activation.backward(x, kept), norm.rms_grad(x, w, kn)
    for c, n in ((copy.deepcopy(kept), copy.deepcopy(kn)), (pickle.loads(pickle.dumps(kept)), pickle.loads(pickle.dumps(kn)))):
        kept.gate.codes.view(torch.uint8).fill_(0x7F)
        kn.rstd.fill_(3.0)
        got, got_n = activation.backward(x, c), norm.rms_grad(x, w, n)
        assert all(torch.equal(a, b) for a, b in zip(want + want_n, got + got_n))
        kept, kn = c, n


def writes(dev):
    from weight_communication_gb300 import activation, fp8, loss, norm
    x = torch.randn(12, 16, device=dev)
    b = x.bfloat16()
    y = torch.arange(12, device=dev)
    _, lse = loss.cross_entropy(b, b, y, save=True)
    _, _, k = norm.rms(x, x[0], save=True)
    q, _ = fp8.quantize(x)
    return {
        "activation": lambda t: activation.forward(x, out=t),
        "dequantize": lambda t: fp8.dequantize(q, out=t),
        "dweight": lambda t: norm.rms_grad(x, x[0], k, dweight=t.view(-1)[:16]),
        "dw": lambda t: loss.cross_entropy_grad(b, b, y, lse, 1.0, dw=t),
        "dw_added": lambda t: loss.cross_entropy_grad(b, b, y, lse, 1.0, dw=t, accumulate=True),
    }


@pytest.mark.parametrize("name", ["activation", "dequantize", "dweight", "dw", "dw_added"])
def test_written_tensors_have_a_new_version(dev, name):
    x = torch.ones(12, 16, device=dev, requires_grad=True)
    y = 2 * x
    value = (y * y).sum()    # saves y
    before = y._version
    writes(dev)[name](y.detach())
    assert y._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        value.backward()
    with torch.inference_mode():
        t = torch.full((12, 16), 5.0, device=dev)
        writes(dev)[name](t)
        assert bool((t != 5.0).any())


def test_a_gradient_that_ends_is_told_of(dev):
    from weight_communication_gb300 import activation, loss, norm
    x = torch.randn(12, 16, device=dev)
    b, y = x.bfloat16(), torch.arange(12, device=dev)
    _, kept = activation.forward(x, save=True)
    _, _, k = norm.rms(x, x[0], save=True)
    _, lse = loss.cross_entropy(b, b, y, save=True)
    leaf = lambda t: t.clone().requires_grad_()  # noqa: E731
    for call, name in ((lambda: activation.forward(leaf(x)), "activation.forward"),
                       (lambda: activation.forward(x, leaf(x)), "activation.forward"),
                       (lambda: activation.backward(leaf(x), kept), "activation.backward"),
                       (lambda: norm.rms(leaf(x), x[0]), "norm.rms"), (lambda: norm.rms(x, leaf(x[0])), "norm.rms"),
                       (lambda: norm.rms(x, x[0], add=leaf(x)), "norm.rms"),
                       (lambda: norm.rms_grad(leaf(x), x[0], k), "norm.rms_grad"),
                       (lambda: loss.cross_entropy(leaf(b), b, y), "loss.cross_entropy"),
                       (lambda: loss.cross_entropy(b, leaf(b), y), "loss.cross_entropy"),
                       (lambda: loss.cross_entropy_grad(b, b, y, lse, leaf(lse)), "loss.cross_entropy_grad")):
        with pytest.warns(UserWarning, match=f"{name} stands outside autograd"):
            call()
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with torch.no_grad():
                call()


def test_new_tensors_belong_to_the_given_stream(dev):
    """Results, workspaces and kept matrices of a side stream come from its pool."""
    from weight_communication_gb300 import activation, loss, norm
    g = torch.Generator(device=dev)
    g.manual_seed(0)
    x = torch.randn(3000, 512, generator=g, device=dev).bfloat16()
    w = torch.randn(1000, 512, generator=g, device=dev).bfloat16()
    y = torch.randint(0, 1000, (3000,), generator=g, device=dev)

    def run(stream):
        n, t, kn = norm.rms(x, x[0], add=x, save=True, stream=stream)
        h, ka = activation.forward(n, t, save=True, stream=stream)
        losses, lse = loss.cross_entropy(h, w, y, save=True, stream=stream)
        dh, dw = loss.cross_entropy_grad(h, w, y, lse, 0.01, stream=stream)
        dn, dt = activation.backward(dh, ka, stream=stream)
        dx, dweight = norm.rms_grad(dn, x[0], kn, add=dt, stream=stream)
        return losses, dw, dx, dweight

    want = run(None)
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    for _ in range(4):
        got = run(s)
        junk = [torch.full((3000, 512), 7.0, device=dev) for _ in range(4)]  # on the default stream
        del junk
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

"""The largest sizes of the training-step operators: the first value past each
is refused on the CPU, before anything is launched (placeholder pointers, so
the file runs only where no GPU is visible); the largest rows run on the GPU."""
import pytest
import torch

from test_abi import FAKE, lib  # noqa: F401
from weight_communication_gb300 import binding, embedding

N_MAX = (1 << 31) - 4096
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers")


@no_gpu
def test_first_sizes_past_the_limits(lib):  # noqa: F811
    E = binding.WC_ERANGE
    assert lib.wc_embedding_grad_workspace(N_MAX, 10, 8) > 0
    assert lib.wc_embedding_grad_workspace(10, N_MAX, 8) > 0
    assert lib.wc_embedding_grad_workspace(10, 10, 1 << 22) > 0
    assert lib.wc_embedding_grad_workspace(N_MAX + 1, 10, 8) == E
    assert lib.wc_embedding_grad_workspace(10, N_MAX + 1, 8) == E
    assert lib.wc_embedding_grad_workspace(10, 10, (1 << 22) + 1) == E
    for n, V in ((N_MAX + 1, 10), (10, N_MAX + 1)):
        assert lib.wc_embedding(FAKE, 1, 8, FAKE, 1, n, 0, V, 8, 1.0, FAKE, 8, None) == E
        assert lib.wc_embedding_grad(FAKE, 1, 8, FAKE, 1, n, 0, V, 8, 1.0, 0, FAKE, 1, 8, FAKE, 1 << 60,
                                     None) == E
    top = (1 << 31) - 255
    for M, N, K in ((top, 1, 16), (1, top, 16), (1, 1, top)):
        assert lib.wc_fp8_matmul(FAKE, 1 << 32, FAKE, 1 << 32, 1, FAKE, 1 << 32, FAKE, 1 << 32, 1, M, N, K,
                                 FAKE, 1, 1 << 32, 0, None) == E


@pytest.mark.gpu
@pytest.mark.parametrize("D,pad", [(1 << 22, 1), ((1 << 22) - 1, 0), (1 << 22, 0)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_longest_rows(D, pad, accumulate):
    """Rows of 2^22 values that start anywhere: one column per thread, more
    slices than a grid's second axis takes."""
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(D + pad)
    dy = torch.randint(-8, 9, (6, D + pad), generator=g, device=dev).float()[:, :D]  # sums are exact
    ids = torch.tensor([1, 0, 1, 1, -1, 1], device=dev)
    out = torch.randint(-8, 9, (3, D + pad), generator=g, device=dev).float()[:, :D]
    want = torch.stack([dy[1], dy[0] + dy[2] + dy[3] + dy[5], torch.zeros(D, device=dev)]) * 0.5
    if accumulate:
        want = want + out
    assert torch.equal(embedding.grad(dy, ids, 3, scale=0.5, out=out, accumulate=accumulate), want)

"""Token ids that start on any id of a longer row: the next-token slice, and the
rows of a batch of an odd number of tokens."""
import pytest
import torch

from test_abi import FAKE, lib  # noqa: F401
from weight_communication_gb300 import binding

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers")
TYPES = [torch.int32, torch.int64]


@no_gpu
def test_alignment_of_ids(lib):  # noqa: F811
    """Ids on a boundary of their own pass this check (the call then stops at
    the output's address); others are refused."""
    OK_IDS, MIS = b"out", FAKE + 2
    for id_type, steps in ((0, (4, 8, 12)), (1, (8,))):
        for step in steps:
            assert lib.wc_embedding(FAKE, 1, 64, FAKE + step, id_type, 10, 0, 100, 64, 1.0, None, 64,
                                    None) == binding.WC_EINVAL
            assert OK_IDS in lib.wc_last_error()
            assert lib.wc_embedding_grad(FAKE, 1, 64, FAKE + step, id_type, 10, 0, 100, 64, 1.0, 0, None, 0,
                                         64, FAKE, 1 << 60, None) == binding.WC_EINVAL
            assert b"dtable" in lib.wc_last_error()
        for bad in (MIS, FAKE + 1) + ((FAKE + 4,) if id_type else ()):
            assert lib.wc_embedding(FAKE, 1, 64, bad, id_type, 10, 0, 100, 64, 1.0, FAKE, 64,
                                    None) == binding.WC_EALIGN
            assert b"ids" in lib.wc_last_error()
            assert lib.wc_embedding_grad(FAKE, 1, 64, bad, id_type, 10, 0, 100, 64, 1.0, 0, FAKE, 0, 64,
                                         FAKE, 1 << 60, None) == binding.WC_EALIGN
            assert b"ids" in lib.wc_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("id_type", TYPES)
@pytest.mark.parametrize("start", [1, 2, 3])
@pytest.mark.parametrize("n", [1, 37, 12_001])
def test_ids_from_any_place(id_type, start, n):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_communication_gb300 import embedding
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(start + n)
    table = torch.randint(-8, 9, (500, 24), generator=g, device=dev).float()
    ids = torch.randint(0, 500, (n + start,), generator=g, device=dev).to(id_type)[start:]
    assert ids.data_ptr() % 16 or start * ids.element_size() % 16 == 0
    out = embedding.lookup(table, ids)
    assert torch.equal(out, table[ids.long()])
    want = torch.zeros(500, 24, device=dev).index_add_(0, ids.long(), out)    # small whole numbers
    assert torch.equal(embedding.grad(out, ids, 500), want)


@pytest.mark.gpu
def test_training_step_with_an_odd_number_of_tokens():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_communication_gb300.train_step import TrainStep, batch
    model = TrainStep(vocab=203, width=96, hidden=200, ranks=2, lr=1.0)
    losses = [float(model.step(*batch(203, 2, 301, i))[0]) for i in range(3)]
    assert losses[2] < losses[0]

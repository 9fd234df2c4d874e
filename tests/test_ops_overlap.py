"""Calls whose results would be written over what they read, or over one another, are
refused, on the CPU; matrices between one another's rows are not.  The pointers are
placeholders that nothing dereferences, so the file runs only where no GPU is visible:
calls that are not refused end at their launch."""
import random

import pytest

from weight_communication_gb300 import binding

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="placeholder pointers: run where no GPU is reachable")

from test_abi import lib  # noqa: E402,F401  (the library fixture)
from test_ops_abi import BIG, EINVAL  # noqa: E402

ECUDA = binding.WC_ECUDA
MB = 1 << 20
X, W, Y, LSE, DL, DX, DW, WS = (k * MB for k in (16, 32, 48, 64, 80, 96, 112, 512))
T, V, D = 10, 100, 64


def forward(lib, **k):
    a = dict(x=X, ldx=D, w=W, ldw=D, y=Y, it=1, T=T, V=V, D=D, losses=DX, lse=LSE, ws=WS, bytes=BIG, st=None)
    a.update(k)
    return lib.wc_cross_entropy(*a.values()), lib.wc_last_error().decode()


def backward(lib, **k):
    a = dict(x=X, ldx=D, w=W, ldw=D, y=Y, it=1, T=T, V=V, D=D, lse=LSE, dl=DL, dloss=0.0, dx=DX, dxt=1, lddx=D, dw=DW, dwt=1,
             lddw=D, acc=0, ws=WS, bytes=BIG, st=None)
    a.update(k)
    return lib.wc_cross_entropy_grad(*a.values()), lib.wc_last_error().decode()


@pytest.mark.parametrize("tokens", [1, 4, 10])
def test_cross_entropy(lib, tokens):
    assert forward(lib, T=tokens)[0] == ECUDA        # nothing overlaps: no GPU to launch on
    for k, words in ((dict(losses=LSE), "losses overlaps lse"), (dict(losses=X), "losses overlaps x"),
                     (dict(lse=W + 2 * V * D - 4), "lse overlaps w"), (dict(losses=Y + 8 * tokens - 4), "losses overlaps targets"),
                     (dict(ws=W + 16), "workspace overlaps w"), (dict(ws=X), "workspace overlaps x"),
                     (dict(losses=WS), "losses overlaps workspace")):
        rc, message = forward(lib, T=tokens, **k)
        assert rc == EINVAL and words in message, (k, rc, message)
    for k in (dict(losses=None, lse=X + 2 * tokens * D), dict(lse=None, losses=W + 2 * V * D)):
        assert forward(lib, T=tokens, **k)[0] == ECUDA, k


@pytest.mark.parametrize("tokens", [1, 4, 10])
def test_cross_entropy_grad(lib, tokens):
    assert backward(lib, T=tokens)[0] == ECUDA
    end_w = W + 2 * V * D
    for k, words in ((dict(dw=W), "dw overlaps w"), (dict(dw=W, acc=1), "dw overlaps w"), (dict(dw=W + 2 * D * (V - 1)), "dw overlaps w"),
                     (dict(dw=W - 4 * V * D + 4, dwt=0), "dw overlaps w"), (dict(dx=W + 2 * D), "dx overlaps w"),
                     (dict(dx=X), "dx overlaps x"), (dict(dw=X), "dw overlaps x"), (dict(dx=DW), "dx overlaps dw"),
                     (dict(dw=LSE), "dw overlaps lse"), (dict(dx=DL), "dx overlaps dlosses"), (dict(dw=Y), "dw overlaps targets"),
                     (dict(ws=X), "workspace overlaps x"), (dict(dx=WS), "dx overlaps workspace"), (dict(ws=W), "workspace overlaps w"),
                     # rows between the weight's, but longer than the room there
                     (dict(ldw=2 * D, dw=W + 2 * D - 2, lddw=2 * D), "dw overlaps w"),
                     (dict(ldw=2 * D, dw=W + 2 * D + 2, lddw=2 * D), "dw overlaps w"),
                     (dict(ldw=2 * D, dw=W + 2 * D, lddw=2 * D, dwt=0), "dw overlaps w"),
                     # another distance of rows, only some of which meet
                     (dict(ldw=2 * D, dw=W + 2 * D, lddw=3 * D), "dw overlaps w")):
        rc, message = backward(lib, T=tokens, **k)
        assert rc == EINVAL and words in message, (k, rc, message)
    for k in (dict(dw=end_w), dict(dw=W - 2 * V * D), dict(dx=None, dl=DX), dict(dw=None, dl=DW), dict(dl=None, dw=DL),
              dict(ldw=2 * D, dw=W + 2 * D, lddw=2 * D), dict(ldw=3 * D, dw=W + 2 * D, lddw=3 * D, dwt=0),
              dict(ldw=4 * D, dw=W + 2 * D, lddw=2 * D, V=1), dict(ldw=2 * D, dw=W + 2 * D, lddw=4 * D),
              # dx in the room beside x
              dict(ldx=2 * D, dx=X + 2 * D, lddx=2 * D)):
        assert backward(lib, T=tokens, **k)[0] == ECUDA, (k, lib.wc_last_error())


def test_every_way_that_rows_meet(lib):
    """Against sets of bytes."""
    rng = random.Random(1)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        v, d = rng.randint(1, 6), rng.randint(1, 5)
        ldw, lddw, dwt = d + rng.randint(0, 12), d + rng.randint(0, 12), rng.randint(0, 1)
        if rng.random() < 0.5:
            lddw = max(d, ldw // (1 if dwt else 2))
        size = 2 if dwt else 4
        at = W + size * rng.randint(-30, 30)
        w = {W + 2 * (r * ldw + c) + b for r in range(v) for c in range(d) for b in range(2)}
        dw = {at + size * (r * lddw + c) + b for r in range(v) for c in range(d) for b in range(size)}
        rc, message = backward(lib, T=1, V=v, D=d, ldx=d, lddx=d, ldw=ldw, dw=at, lddw=lddw, dwt=dwt)
        assert rc == (EINVAL if w & dw else ECUDA), (v, d, ldw, lddw, dwt, at - W, message)
        seen[bool(w & dw)] += 1
    assert min(seen.values()) > 300

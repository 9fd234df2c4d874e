"""Calls whose results would be written over what they read, or over one another, are
refused, on the CPU; matrices between one another's rows are not.  The pointers are
placeholders that nothing dereferences, so the file runs only where no GPU is visible:
calls that are not refused end at their launch."""
import ctypes
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


R, C = 100, 200
SLOTS = [k * MB for k in range(16, 64)]


def kept(at, ld=208):
    return ctypes.pointer(binding.WcKept(at, ld, at + MB, R))


def calls(lib, name, ok, cases):
    """Changes of `ok` that nothing overlaps in, and those that are refused, with their words."""
    f = getattr(lib, name)
    for change, words in [({}, None)] + cases:
        a = dict(ok)
        a.update(change)
        rc, message = f(*a.values()), lib.wc_last_error().decode()
        if words is None:
            assert rc == ECUDA, (name, change, rc, message)
        else:
            assert rc == EINVAL and words in message, (name, change, rc, message)


def test_activation(lib):
    g, u, h, kg, ku = SLOTS[0], SLOTS[4], SLOTS[8], SLOTS[12], SLOTS[16]
    ok = dict(gate=g, ldg=C, up=u, ldu=C, dtype=1, kind=1, rows=R, cols=C, h=h, ldh=C, kg=kept(kg), ku=kept(ku), st=None)
    calls(lib, "wc_activation", ok, [
        (dict(h=g), None), (dict(h=u), None), (dict(h=g, up=g), None),   # the same rows
        (dict(h=g + 2), "h overlaps gate"), (dict(h=g + 2 * C), "h overlaps gate"), (dict(h=g, ldh=C + 1), "h overlaps gate"),
        (dict(h=u + 2 * R * C - 2), "h overlaps up"), (dict(h=g + 2 * C, ldh=2 * C, ldg=2 * C), None),
        (dict(kg=kept(g)), "codes of kept_gate overlaps gate"), (dict(kg=kept(h - MB)), "scales of kept_gate overlaps h"),
        (dict(ku=kept(kg)), "codes of kept_gate overlaps codes of kept_up"), (dict(up=None, kg=None, ku=None, h=g), None)])
    ok = dict(dh=g, ldd=C, dtype=1, kind=2, rows=R, cols=C, kg=kept(kg), ku=kept(ku), dg=u, ldg=C, du=h, ldu=C, st=None)
    calls(lib, "wc_activation_grad", ok, [
        (dict(dg=g), None), (dict(du=g), None), (dict(dg=h), "dgate overlaps dup"), (dict(dg=g + 2), "dgate overlaps dh"),
        (dict(du=g - 2), "dup overlaps dh"), (dict(dg=kg), "dgate overlaps codes of kept_gate"),
        (dict(du=ku + MB), "dup overlaps scales of kept_up")])


def test_norm(lib):
    x, add, w, y, t, r, k = (SLOTS[4 * i] for i in range(7))
    ok = dict(x=x, ldx=C, add=add, lda=C, dtype=1, rows=R, cols=C, w=w, wt=1, eps=1e-6, y=y, ldy=C, total=t, ldt=C, rstd=r,
              kept=kept(k), st=None)
    calls(lib, "wc_rms_norm", ok, [
        (dict(y=x), None), (dict(total=x), None), (dict(y=x, total=add), None), (dict(y=t), "y overlaps total"),
        (dict(y=x + 2), "y overlaps x"), (dict(total=add + 2 * C), "total overlaps add"), (dict(y=w - 2), "y overlaps weight"),
        (dict(rstd=x), "rstd overlaps x"), (dict(kept=kept(add)), "codes of kept overlaps add"), (dict(rstd=k), "rstd overlaps codes of kept"),
        (dict(add=None, total=None, y=x, rstd=None, kept=None), None)])
    ws = SLOTS[28]
    ok = dict(dy=x, ldy=C, add=add, lda=C, dtype=1, rows=R, cols=C, w=w, wt=1, rstd=r, kept=kept(k), dx=y, ldx=C, dw=t, dwt=0, acc=0,
              ws=ws, bytes=BIG, st=None)
    calls(lib, "wc_rms_norm_grad", ok, [
        (dict(dx=x), None), (dict(dx=add), None), (dict(dw=w, dwt=1), None), (dict(dw=w, dwt=0), "dweight overlaps weight"),
        (dict(dx=x + 2), "dx overlaps dy"), (dict(dx=add - 2), "dx overlaps add"), (dict(dw=x), "dweight overlaps dy"),
        (dict(dw=y), "dx overlaps dweight"), (dict(dx=k), "dx overlaps codes of kept"), (dict(dw=r), "dweight overlaps rstd"),
        (dict(ws=w), "workspace overlaps weight"), (dict(ws=k + MB), "workspace overlaps scales of kept"), (dict(dx=w), "dx overlaps weight")])


def test_dequant(lib):
    q, s, out = SLOTS[0], SLOTS[4], SLOTS[8]
    ok = dict(q=q, ldq=208, s=s, lds=R, per=1, rows=R, cols=C, out=out, ot=1, ldo=C, st=None)
    calls(lib, "wc_fp8_dequant", ok, [(dict(out=q), "out overlaps q"), (dict(out=s + 8 * R - 4), "out overlaps s"),
                                      (dict(out=s + 8 * R), None), (dict(per=128, lds=1, out=s + 8), None),
                                      (dict(per=128, lds=1, out=s + 4), "out overlaps s")])


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

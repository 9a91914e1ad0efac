"""Refusals of the vocabulary operators, decided on the host before anything
is launched, and the workspace convention.  No GPU is needed."""
import ctypes
import types

import pytest


@pytest.fixture(scope="module")
def rlt():
    import stateful_decoder_b200 as rlt
    return rlt


P = ctypes.c_void_p(4096)  # pointers that no refused call follows
Q, R = ctypes.c_void_p(8192), ctypes.c_void_p(12288)


def operands(rlt, **kw):
    a = dict(h=4096, ld_h=64, w=4096, ld_w=64, N=3, V=100, d=64, dtype=1)
    a.update(kw)
    return rlt.Vocab(**a)


def sized(n):
    return ctypes.byref(ctypes.c_size_t(n))


BIG = 1 << 40


def test_operands_are_checked(rlt):
    lib = rlt._lib
    for bad in (dict(N=-1), dict(V=0), dict(d=0), dict(ld_h=63), dict(ld_w=63), dict(dtype=2), dict(h=None), dict(w=None),
                dict(N=(1 << 28) + 1), dict(V=(1 << 28) + 1), dict(d=(1 << 28) + 1, ld_h=1 << 29, ld_w=1 << 29)):
        a = ctypes.byref(operands(rlt, **bad))
        assert lib.rlt_op_cross_entropy(a, P, P, P, P, sized(BIG), None) == rlt.RLT_E_INVAL, bad
        assert lib.rlt_op_distill(a, P, P, 4, 1.0, P, P, P, sized(BIG), None) == rlt.RLT_E_INVAL, bad
        assert lib.rlt_op_cross_entropy_backward(a, P, P, P, P, 64, P, 64, 0, P, sized(BIG), None) == rlt.RLT_E_INVAL, bad
        assert lib.rlt_op_distill_backward(a, P, P, 4, 1.0, P, P, P, 64, P, 64, 0, P, sized(BIG), None) == rlt.RLT_E_INVAL, bad
    a = ctypes.byref(operands(rlt))
    assert lib.rlt_op_cross_entropy(None, P, P, P, P, sized(BIG), None) == rlt.RLT_E_INVAL
    assert lib.rlt_op_cross_entropy(a, None, P, P, P, sized(BIG), None) == rlt.RLT_E_INVAL
    assert lib.rlt_op_cross_entropy(a, P, None, P, P, sized(BIG), None) == rlt.RLT_E_INVAL
    assert lib.rlt_op_cross_entropy(a, P, P, None, P, sized(BIG), None) == rlt.RLT_E_INVAL
    assert lib.rlt_op_cross_entropy(a, P, P, P, P, None, None) == rlt.RLT_E_INVAL
    for K, T in ((0, 1.0), (257, 1.0), (4, 0.0), (4, -1.0), (4, float("nan")), (4, float("inf")), (4, 1e-45)):
        assert lib.rlt_op_distill(a, P, P, K, T, P, P, P, sized(BIG), None) == rlt.RLT_E_INVAL, (K, T)
    assert lib.rlt_op_distill(a, P, None, 4, 1.0, P, P, P, sized(BIG), None) == rlt.RLT_E_INVAL
    back = lib.rlt_op_cross_entropy_backward
    assert back(a, P, None, P, P, 64, P, 64, 0, P, sized(BIG), None) == rlt.RLT_E_INVAL
    assert back(a, P, P, None, P, 64, P, 64, 0, P, sized(BIG), None) == rlt.RLT_E_INVAL
    assert back(a, P, P, P, None, 0, None, 0, 0, P, sized(BIG), None) == rlt.RLT_E_INVAL
    assert back(a, P, P, P, P, 63, P, 64, 0, P, sized(BIG), None) == rlt.RLT_E_INVAL
    assert back(a, P, P, P, P, 64, P, 63, 0, P, sized(BIG), None) == rlt.RLT_E_INVAL


def test_outputs_in_an_operands_place_are_refused(rlt):
    """By their addresses: an output that is an operand, or the other output."""
    lib = rlt._lib
    a = ctypes.byref(operands(rlt, h=4096, w=8192))
    assert lib.rlt_op_cross_entropy(a, P, R, R, P, sized(BIG), None) == rlt.RLT_E_INVAL
    assert lib.rlt_op_distill(a, P, P, 4, 1.0, R, R, P, sized(BIG), None) == rlt.RLT_E_INVAL
    other = ctypes.c_void_p(1 << 20)
    for dh, dw in ((P, R), (Q, R), (R, P), (R, Q), (R, R), (P, None), (None, Q)):
        assert lib.rlt_op_cross_entropy_backward(a, other, other, other, dh, 64, dw, 64, 0, other, sized(BIG), None) == rlt.RLT_E_INVAL
        assert lib.rlt_op_distill_backward(a, other, other, 4, 1.0, other, other, dh, 64, dw, 64, 0, other, sized(BIG), None) == rlt.RLT_E_INVAL
    assert lib.rlt_op_embed(P, 64, 1, 100, 64, Q, 3, 1.0, P, 64, 1, None) == rlt.RLT_E_INVAL
    assert lib.rlt_op_embed_backward(P, 64, 1, Q, 3, 100, 64, 1.0, P, 64, 1, 0, R, sized(BIG), None) == rlt.RLT_E_INVAL


def test_embedding_arguments_are_checked(rlt):
    lib = rlt._lib
    good = [P, 64, 1, 100, 64, P, 3, 1.0, Q, 64, 0, None]
    for at, bad in ((0, None), (1, 63), (2, 2), (3, 0), (4, 0), (5, None), (6, -1), (8, None), (9, 63), (10, -1)):
        args = list(good)
        args[at] = bad
        assert lib.rlt_op_embed(*args) == rlt.RLT_E_INVAL, at
    good = [P, 64, 1, P, 3, 100, 64, 1.0, Q, 64, 0, 0, R, sized(BIG), None]
    for at, bad in ((0, None), (1, 63), (2, 7), (3, None), (4, -1), (5, 0), (6, 0), (8, None), (9, 63), (10, 2), (13, None)):
        args = list(good)
        args[at] = bad
        assert lib.rlt_op_embed_backward(*args) == rlt.RLT_E_INVAL, at
    size, wide = ctypes.c_size_t(), 1 << 23
    for d, code in ((wide, rlt.RLT_OK), (wide + 1, rlt.RLT_E_INVAL)):
        assert lib.rlt_op_embed_backward(P, d, 1, P, 3, 100, d, 1.0, Q, d, 0, 0, None, ctypes.byref(size), None) == code


def test_workspace_convention(rlt):
    """A null workspace reports the size; a short or misaligned one is refused."""
    lib = rlt._lib
    a = ctypes.byref(operands(rlt, N=300, V=5000))
    n = ctypes.c_size_t()
    calls = (
        lambda ws, s: lib.rlt_op_cross_entropy(a, P, P, Q, ws, s, None),
        lambda ws, s: lib.rlt_op_cross_entropy_backward(a, P, P, P, Q, 64, R, 64, 0, ws, s, None),
        lambda ws, s: lib.rlt_op_distill(a, P, P, 50, 0.8, P, Q, ws, s, None),
        lambda ws, s: lib.rlt_op_distill_backward(a, P, P, 50, 0.8, P, P, Q, 64, R, 64, 0, ws, s, None),
    )
    for call in calls:
        assert call(None, ctypes.byref(n)) == rlt.RLT_OK
        assert 0 < n.value < 1 << 32
        assert call(P, sized(n.value - 1)) == rlt.RLT_E_CAPACITY
        assert call(ctypes.c_void_p(4096 + 128), sized(n.value)) == rlt.RLT_E_INVAL
    code, text = rlt.rlt_last_error()
    assert code == rlt.RLT_E_INVAL and "256" in text


def test_workspace_does_not_hold_the_logits(rlt):
    """The loss over 65,536 rows and 256,000 ids: its logits would take 67 GB in
    fp32; forward and backward need a few GB at most."""
    lib = rlt._lib
    n = ctypes.c_size_t()
    a = ctypes.byref(operands(rlt, N=65536, V=256000, d=2048, ld_h=2048, ld_w=2048))
    assert lib.rlt_op_cross_entropy(a, P, P, Q, None, ctypes.byref(n), None) == rlt.RLT_OK
    assert n.value < 2 << 30
    assert lib.rlt_op_cross_entropy_backward(a, P, P, P, Q, 2048, R, 2048, 0, None, ctypes.byref(n), None) == rlt.RLT_OK
    assert n.value < 4 << 30


def test_outputs_that_reach_into_an_operand_are_refused(rlt):
    """By their whole extents, not their first addresses: an output that begins
    inside an operand or ends in it, in the workspace, or in the other output.
    (Every call here is refused: the addresses are not memory.)"""
    lib = rlt._lib
    MB = 1 << 20

    def at(n, off=0):
        return ctypes.c_void_p(n * MB + off)

    H, W, IDS, TE, O1, O2, WS = 16, 32, 48, 49, 50, 51, 64
    N, V, d = 3, 100, 64  # bf16: rows of 128 bytes, h 384 bytes, w 12,800
    a = ctypes.byref(operands(rlt, h=H * MB, w=W * MB, N=N, V=V, d=d))
    for o in (at(H, 4), at(H, -4), at(H, 380), at(W, 12796), at(IDS, -8), at(IDS, 8), at(O2, 8), at(O2, -8), at(WS, 4)):
        assert lib.rlt_op_cross_entropy(a, at(IDS), o, at(O2), at(WS), sized(BIG), None) == rlt.RLT_E_INVAL, o
        assert lib.rlt_op_cross_entropy(a, at(IDS), at(O2), o, at(WS), sized(BIG), None) == rlt.RLT_E_INVAL, o
    for o in (at(H, 4), at(W, 12796), at(IDS, 44), at(TE, -8), at(TE, 44), at(O2, 8), at(WS, 4)):
        assert lib.rlt_op_distill(a, at(IDS), at(TE), 4, 1.0, o, at(O2), at(WS), sized(BIG), None) == rlt.RLT_E_INVAL, o

    def back(dh, ld_dh, dw, ld_dw, a=a):
        return (lib.rlt_op_cross_entropy_backward(a, at(IDS), at(O1), at(O2), dh, ld_dh, dw, ld_dw, 0, at(WS), sized(BIG), None),
                lib.rlt_op_distill_backward(a, at(IDS), at(TE), 4, 1.0, at(O1), at(O2), dh, ld_dh, dw, ld_dw, 0, at(WS), sized(BIG), None))

    refused = (rlt.RLT_E_INVAL, rlt.RLT_E_INVAL)
    for g in (at(H, 64), at(H, -64), at(W, 12672), at(W, -256), at(IDS, 8), at(O1, -380), at(O2, 8), at(WS, 128)):
        assert back(g, d, None, 0) == refused, g
    for g in (at(H, 64), at(W, 64), at(W, -12672), at(H, -12672), at(IDS, 0), at(O1, 0), at(O2, -12672), at(WS, 0)):
        assert back(None, 0, g, d) == refused, g
    assert back(at(80), d, at(80, 256), d) == refused
    # rows that stand apart: a gradient whose rows reach into the operand's, at
    # the operand's own row distance and at another
    a2 = ctypes.byref(operands(rlt, h=H * MB, ld_h=200, w=W * MB, ld_w=200, N=N, V=V, d=d))
    for off in (126, -126, 400 + 126, -800 - 126, 99 * 400 - 126):
        assert back(None, 0, at(W, off), 200, a2) == refused, off
    assert back(None, 0, at(W, 126), 1000, a2) == refused
    assert back(None, 0, at(W, 3 * 400 + 200), 201, a2) == refused  # meets w's rows further on
    assert back(at(W, 126), 1000, None, 0, a2) == refused
    assert back(at(W, 99 * 400 + 126), 1000, None, 0, a2) == refused
    # no rows: dw is still written whole
    none = ctypes.byref(operands(rlt, h=None, w=W * MB, N=0, V=V, d=d))
    assert lib.rlt_op_cross_entropy_backward(none, None, None, None, None, 0, at(W), d, 0, at(WS), sized(BIG), None) == rlt.RLT_E_INVAL

    E, T, G = 16, 32, 48
    for o in (at(E, 4), at(E, -4), at(T, 8), at(T, -4)):
        assert lib.rlt_op_embed(at(E), d, 0, V, d, at(T), N, 1.0, o, d, 1, None) == rlt.RLT_E_INVAL, o
    for o in (at(E, 4), at(E, -4), at(T, 8), at(T, -4), at(WS, 0)):
        assert lib.rlt_op_embed_backward(at(E), d, 1, at(T), N, V, d, 1.0, o, d, 0, 0, at(WS), sized(BIG), None) == rlt.RLT_E_INVAL, o


@pytest.mark.parametrize("N", [0, 1])
def test_a_reported_size_is_never_zero(rlt, N):
    """With no rows too: an allocation of 0 bytes may be the null pointer, which
    asks for the size again and launches nothing, so a gradient that is to be
    written whole (zeros) would keep what it held."""
    lib = rlt._lib
    a = ctypes.byref(operands(rlt, N=N))
    n = ctypes.c_size_t(0)
    for call in (
        lambda ws, s: lib.rlt_op_cross_entropy(a, P, P, Q, ws, s, None),
        lambda ws, s: lib.rlt_op_cross_entropy_backward(a, P, P, P, Q, 64, R, 64, 0, ws, s, None),
        lambda ws, s: lib.rlt_op_distill(a, P, P, 4, 0.8, P, Q, ws, s, None),
        lambda ws, s: lib.rlt_op_distill_backward(a, P, P, 4, 0.8, P, P, Q, 64, R, 64, 0, ws, s, None),
        lambda ws, s: lib.rlt_op_embed_backward(P, 64, 1, P, N, 100, 64, 1.0, Q, 64, 0, 0, ws, s, None),
    ):
        n.value = 0
        assert call(None, ctypes.byref(n)) == rlt.RLT_OK
        assert n.value >= 256
        assert call(R, sized(0)) == rlt.RLT_E_CAPACITY


class _Fake:
    """A CPU tensor that passes for a CUDA one: what the binding refuses, it
    refuses by shape, type and stride, before the library sees a pointer."""

    def __init__(self, t):
        self.t, self.is_cuda, self.shape, self.dtype = t, True, t.shape, t.dtype
        self.device = types.SimpleNamespace(index=0)

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_refuses_wrong_tensors(rlt, monkeypatch):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def f(*shape, dtype=torch.float32):
        return _Fake(torch.zeros(*shape, dtype=dtype))

    i32, bf = torch.int32, torch.bfloat16
    h, w, t, o, e = f(4, 8), f(9, 8), f(4, dtype=i32), f(4), f(4)
    ids, te = f(4, 3, dtype=i32), f(4, 3)
    calls = [
        lambda: rlt.rlt_op_cross_entropy(f(4, 7), w, t, o, e),
        lambda: rlt.rlt_op_cross_entropy(f(4, 8, dtype=bf), w, t, o, e),
        lambda: rlt.rlt_op_cross_entropy(f(4, 8, dtype=torch.float16), f(9, 8, dtype=torch.float16), t, o, e),
        lambda: rlt.rlt_op_cross_entropy(_Fake(torch.zeros(8, 4).t()), w, t, o, e),
        lambda: rlt.rlt_op_cross_entropy(_Fake(torch.zeros(1, 8).expand(4, 8)), w, t, o, e),
        lambda: rlt.rlt_op_cross_entropy(h, w, f(5, dtype=i32), o, e),
        lambda: rlt.rlt_op_cross_entropy(h, w, f(4, dtype=torch.int64), o, e),
        lambda: rlt.rlt_op_cross_entropy(h, w, t, f(3), e),
        lambda: rlt.rlt_op_cross_entropy(h, w, t, f(4, dtype=bf), e),
        lambda: rlt.rlt_op_cross_entropy_backward(h, w, t, e, f(3), dh=f(4, 8)),
        lambda: rlt.rlt_op_cross_entropy_backward(h, w, t, e, o, dh=f(4, 9)),
        lambda: rlt.rlt_op_cross_entropy_backward(h, w, t, e, o, dh=f(4, 8, dtype=bf)),
        lambda: rlt.rlt_op_cross_entropy_backward(h, w, t, e, o, dw=f(8, 8)),
        lambda: rlt.rlt_op_distill(h, w, f(4, 3), te, 1.0, o, e),
        lambda: rlt.rlt_op_distill(h, w, ids, f(4, 2), 1.0, o, e),
        lambda: rlt.rlt_op_distill(h, w, f(12, dtype=i32), te, 1.0, o, e),
        lambda: rlt.rlt_op_embed(w, f(4, dtype=torch.int64), f(4, 8)),
        lambda: rlt.rlt_op_embed(w, t, f(4, 7)),
        lambda: rlt.rlt_op_embed_backward(f(5, 8), t, w),
        lambda: rlt.rlt_op_embed_backward(f(4, 8), t, f(9, 8, dtype=torch.float16)),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    far = f(9, 8)
    far.device = types.SimpleNamespace(index=1)
    with pytest.raises(ValueError, match="current device"):
        rlt.rlt_op_cross_entropy(h, far, t, o, e)


def test_binding_refuses_an_empty_workspace(rlt, monkeypatch):
    """A tensor without elements has a null pointer, which asks the library for
    the size: the call would return with nothing launched."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def f(*shape, dtype=torch.float32):
        return _Fake(torch.zeros(*shape, dtype=dtype))

    i32 = torch.int32
    h, w, t, o, e = f(4, 8), f(9, 8), f(4, dtype=i32), f(4), f(4)
    ids, te, none = f(4, 3, dtype=i32), f(4, 3), f(0, dtype=torch.uint8)
    for call in (
        lambda: rlt.rlt_op_cross_entropy(h, w, t, o, e, workspace=none, stream=0),
        lambda: rlt.rlt_op_cross_entropy_backward(h, w, t, e, o, dh=f(4, 8), workspace=none, stream=0),
        lambda: rlt.rlt_op_distill(h, w, ids, te, 1.0, o, e, workspace=none, stream=0),
        lambda: rlt.rlt_op_distill_backward(h, w, ids, te, 1.0, e, o, dw=f(9, 8), workspace=none, stream=0),
        lambda: rlt.rlt_op_embed_backward(f(4, 8), t, w, workspace=none, stream=0),
    ):
        with pytest.raises(ValueError, match="workspace"):
            call()

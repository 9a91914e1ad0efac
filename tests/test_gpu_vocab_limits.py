"""The vocabulary operators at the ends of what their calls allow: outputs in
slices beside their operands, lists and rows of extreme values, few rows that
take part among many, long sorts.  Formulas and bounds are those of
test_gpu_vocab."""
import ctypes
import math

import pytest

from test_gpu_vocab import U, ce, embed_reference, env, half_step, kl, make, make_list, reference, types, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_beside_their_operands(env, dtype):
    """Gradients in slices of the operands' own buffers, between their rows,
    are no overlap: same bits as in buffers of their own, operands untouched."""
    rlt, torch = env
    N, V, d = 140, 300, 40
    h0, w0, target, weight = make(torch, N, V, d, dtype, seed=12)
    want = ce(env, h0, w0, target, weight)
    hb, wb = (torch.full((x.shape[0], 2 * d + 16), 5.0, dtype=x.dtype, device="cuda") for x in (h0, w0))
    h, dh, w, dw = hb[:, :d], hb[:, d + 8:2 * d + 8], wb[:, 8:d + 8], wb[:, d + 8:2 * d + 8]
    h.copy_(h0)
    w.copy_(w0)
    rlt.rlt_op_cross_entropy_backward(h, w, target, want["lse"], weight, dh=dh, dw=dw)
    assert torch.equal(dh, want["dh"]) and torch.equal(dw, want["dw"])
    assert torch.equal(h, h0) and torch.equal(w, w0)
    assert (hb[:, d:d + 8] == 5).all() and (hb[:, 2 * d + 8:] == 5).all() and (wb[:, :8] == 5).all()
    tok = target.clamp(min=0)
    both = torch.full((V + N, d), 5.0, device="cuda")
    both[:V] = w0.float()
    rlt.rlt_op_embed(both[:V], tok, both[V:])
    assert torch.equal(both[V:], w0.float()[tok.long()])
    with pytest.raises(rlt.RltError):
        rlt.rlt_op_embed(both[:V], tok, both[V - 1:V - 1 + N])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [6, 150])
@pytest.mark.parametrize("T", [0.25, 0.8, 2.0])
def test_teacher_logits_of_extreme_values(env, T, N, dtype):
    """Masks of the type's lowest value are a softmax's ordinary members: a row
    that holds nothing else is uniform, at any temperature; largest values do
    not overflow; -inf alone empties a row."""
    rlt, torch = env
    V, d, K = 300, 32, 8
    h, w, _, weight = make(torch, N, V, d, dtype, seed=N)
    ids, teacher = make_list(torch, N, V, K, seed=3, empty=0.0)
    low, high = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    teacher[0] = low
    teacher[1, ::2] = low
    teacher[2] = -math.inf
    teacher[3], teacher[3, 2:5] = low, high
    teacher[4], ids[4, 3:] = low, -1
    teacher[5], teacher[5, 1], teacher[5, 2] = -math.inf, low, low
    got = kl(env, h, w, ids, teacher, T, weight)
    ref = reference(torch, h, w, T=T, ids=ids, teacher=teacher, weight=weight)
    for k in ("loss", "lse", "dh", "dw"):
        within(torch, got[k], ref[k], k)
    assert got["loss"][2] == 0 and got["lse"][2] == 0 and got["lse"][0] != 0

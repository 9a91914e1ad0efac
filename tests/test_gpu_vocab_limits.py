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

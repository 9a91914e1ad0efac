"""The vocabulary operators at the ends of what their calls allow: outputs in
slices beside their operands, lists and rows of extreme values, few rows that
take part among many, long sorts.  Formulas and bounds are those of
test_gpu_vocab."""
import ctypes
import math

import pytest

from test_gpu_vocab import U, ce, dense_targets, embed_reference, env, half_step, kl, make, make_list, reference, types, within  # noqa: F401

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


# ------------------------------------------------------------------ single rows
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [40, 6504])
def test_the_distance_of_a_single_row_does_not_matter(env, d, dtype):
    """With one row there is no other to stand apart from: any ld >= d."""
    rlt, torch = env
    h, w, target, weight = make(torch, 1, 1, d, dtype, seed=d, ignored=0.0)
    h2, w2, _, _ = make(torch, 5, 7, d, dtype, seed=d, ignored=0.0)
    t5 = torch.zeros(5, dtype=torch.int32, device="cuda")
    wt5 = torch.ones(5, device="cuda")
    far = 1 << 59
    for hh, ww, t, wt in ((h, w, target * 0, weight), (h, w2, target * 0, weight), (h2, w, t5, wt5)):
        N, V = hh.shape[0], ww.shape[0]
        want = ce(env, hh, ww, t, wt)
        a = rlt.Vocab(hh.data_ptr(), far if N == 1 else d, ww.data_ptr(), far if V == 1 else d, N, V, d, int(dtype == "bf16"))
        out = {"loss": torch.empty(N, device="cuda"), "lse": torch.empty(N, device="cuda"), "dh": torch.empty_like(hh), "dw": torch.empty_like(ww)}
        ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        size = ctypes.c_size_t(ws.numel())
        p = {k: ctypes.c_void_p(x.data_ptr()) for k, x in {**out, "t": t, "wt": wt, "ws": ws}.items()}
        st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert rlt._lib.rlt_op_cross_entropy(ctypes.byref(a), p["t"], p["loss"], p["lse"], p["ws"], ctypes.byref(size), st) == 0
        size.value = ws.numel()
        assert rlt._lib.rlt_op_cross_entropy_backward(ctypes.byref(a), p["t"], p["lse"], p["wt"], p["dh"], far if N == 1 else d, p["dw"],
                                                      far if V == 1 else d, 0, p["ws"], ctypes.byref(size), st) == 0
        for k in want:
            assert torch.equal(out[k], want[k]), k
        if V > 1:
            continue
        # the embedding of a table of one row, and its gradient, without ids too
        tok = torch.tensor([0, -1, 0], dtype=torch.int32, device="cuda")[:1 if N == 1 else 3]
        e = torch.empty(tok.numel(), d, device="cuda")
        one = tok.numel() == 1
        assert rlt._lib.rlt_op_embed(ww.data_ptr(), far, int(dtype == "bf16"), 1, d, tok.data_ptr(), tok.numel(), 2.0, e.data_ptr(),
                                     far if one else d, 0, st) == 0
        assert torch.equal(e, torch.where((tok == 0)[:, None], 2 * ww.float(), torch.zeros((), device="cuda")))
        for n in (tok.numel(), 0):
            demb = torch.full((1, d), 7.0, device="cuda")
            size.value = ws.numel()
            assert rlt._lib.rlt_op_embed_backward(e.data_ptr(), far if n < 2 else d, 0, tok.data_ptr(), n, 1, d, 1.0, demb.data_ptr(), far, 0, 0,
                                                  p["ws"], ctypes.byref(size), st) == 0
            want_e = e[tok[:n] == 0] if n else e[:0]
            assert torch.equal(demb[0], want_e.sum(0))


# ------------------------------------------------------------------ fp32 rows of wide range
def check_all(env, h, w, target, weight, T=1.0):
    rlt, torch = env
    got = ce(env, h, w, target, weight)
    ref = reference(torch, h, w, target=target, weight=weight)
    for k in ("loss", "lse", "dh", "dw"):
        within(torch, got[k], ref[k], k)
    rlt.rlt_check_device()
    return got


@pytest.mark.parametrize("N", [12, 200])
def test_fp32_rows_of_every_scale(env, N):
    """Whole rows near the ends of the type, rows of zeros, and products of
    large rows that have nothing in common (0, not 0 * inf)."""
    rlt, torch = env
    V, d = 150, 64
    h, w, target, weight = make(torch, N, V, d, "f32", seed=N, ignored=0.0)
    check_all(env, h * 2.0 ** 100, w * 2.0 ** -100, target, weight)
    check_all(env, h * 2.0 ** -118, w * 2.0 ** 118, target, weight)
    hz, wz = h.clone(), w.clone()
    hz[::3], wz[::4] = 0.0, 0.0
    check_all(env, hz, wz, target, weight)
    # the columns' halves: rows of h at 2^90 in the first; rows of w at 2^90 in
    # the second, or at 2^-90 in the first
    hs, ws = h.clone(), w.clone()
    hs[:, :32] *= 2.0 ** 90
    hs[:, 32:] = 0.0
    ws[::2, 32:] *= 2.0 ** 90
    ws[::2, :32] = 0.0
    ws[1::2, :32] *= 2.0 ** -90
    ws[1::2, 32:] = 0.0
    got = check_all(env, hs, ws, target, weight)
    assert not torch.isnan(got["lse"]).any()
    ids, teacher = make_list(torch, N, V, 9, seed=2)
    got = kl(env, hs, ws, ids, teacher, 2.0, weight)
    ref = reference(torch, hs, ws, T=2.0, ids=ids, teacher=teacher, weight=weight)
    for k in ("loss", "lse", "dh", "dw"):
        within(torch, got[k], ref[k], k)


@pytest.mark.parametrize("N", [5, 9, 130, 300])
@pytest.mark.parametrize("power", [20, 27, 33, 60, 100])
@pytest.mark.parametrize("side,d", [("h", 64), ("w", 64), ("both", 64), ("both", 1040)])
def test_fp32_outlier_columns(env, side, d, power, N):
    """A column that is large in one operand where the other has none: the
    logits come from the elements far below the row's largest, to the accuracy
    of an fp32 sum of products all the same; with both, from products of two
    such elements."""
    rlt, torch = env
    h, w, target, weight = make(torch, N, 333, d, "f32", seed=N + power, ignored=0.0)
    if side != "w":
        h[:, 5], w[:, 5] = 2.0 ** power, 0.0
        h[0, 17], w[:, 17] = 2.0 ** power, 0.0
    if side != "h":
        w[:, 9], h[:, 9] = 2.0 ** power, 0.0
        w[0, 30], h[:, 30] = -2.0 ** power, 0.0
    check_all(env, h, w, target, weight)


def test_fp32_rows_with_elements_of_every_size(env):
    """Elements from 2^-60 to 2^60 of the row's typical one, met by their
    inverses; and the pair whose small elements carry the product."""
    rlt, torch = env
    N, V, d = 40, 200, 96
    h, w, target, weight = make(torch, N, V, d, "f32", seed=5, ignored=0.0)
    s = torch.exp2(torch.linspace(-60, 60, d, device="cuda").round())
    check_all(env, h * s, w / s, target, weight)
    h, w = torch.zeros(9, 2, device="cuda"), torch.zeros(3, 2, device="cuda")
    h[:, 0], h[:, 1] = 1.0, 3.1e-10
    w[:, 0], w[:, 1] = 2.7e-10, torch.tensor([1.234, -0.5, 0.25], device="cuda")
    target = torch.tensor([0, 1, 2] * 3, dtype=torch.int32, device="cuda")
    got = check_all(env, h, w, target, torch.ones(9, device="cuda"))
    assert not torch.isnan(got["lse"]).any()


def test_fp32_wide_rows_over_several_pieces(env):
    """The backward walks the vocabulary in pieces; one wide row of w, in the
    last of them."""
    rlt, torch = env
    N, V, d = 44000, 4999, 16
    h, w, target, weight = make(torch, N, V, d, "f32", seed=6)
    weight /= N
    h[:, 3], w[:, 3] = 0.0, 0.0
    w[V - 2, 3] = 2.0 ** 70
    w[V - 2, 7] = 1.0
    h[:, 7] = 2.0 ** -3
    got = ce(env, h, w, target, weight)
    dw = [0.0, 0.0]
    for i in range(0, N, 11000):
        s = slice(i, i + 11000)
        ref = reference(torch, h[s], w, target=target[s], weight=weight[s])
        for k in ("loss", "lse", "dh"):
            within(torch, got[k][s], ref[k], k)
        dw[0] = dw[0] + ref["dw"][0]
        dw[1] = dw[1] + ref["dw"][1] * 4  # (2 n + 8) u counts all N terms
    within(torch, got["dw"], dw, "dw")


def test_fp32_wide_rows_in_a_replayed_graph(env):
    """The kernels choose by the values they are given: captured on ordinary
    rows, replayed on wide ones and back, with an eager call's bits."""
    rlt, torch = env
    h, w, target, weight = make(torch, 150, 400, 48, "f32", seed=16, ignored=0.0)
    h2, w2 = h.clone(), w.clone()
    h2[:, 5], w2[:, 5] = 2.0 ** 80, 0.0
    a, b = h.clone(), w.clone()
    ce(env, a, b, target, weight)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ce(env, a, b, target, weight)
    for x, y in ((h2, w2), (h, w), (h2, w2)):
        a.copy_(x)
        b.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        eager = check_all(env, a, b, target, weight)
        for k in out:
            assert torch.equal(out[k], eager[k]), k


# ------------------------------------------------------------------ accuracy where the bounds of sums are wide
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d", [(1100, 5000, 2048), (300, 9000, 1600), (100, 3001, 2112)])
def test_logits_of_long_rows(env, N, V, d, dtype):
    """Pairs of CTAs, several rounds of tiles and several tensor-memory sums.
    The bound on a logit's error here is of root mean square, (2/3) d^1.5 u s
    with s that of the products h w: every one of d additions off, all one
    way, by u times a partial sum of sqrt(k) s.  It is below the 2^-12 sqrt(d)
    s that an fp32 operand's lost lower half would leave.  The logit is logp +
    lse, each of them a rounding of its own and the sum's 2^-21 of lse."""
    rlt, torch = env
    h, w, target, weight = make(torch, N, V, d, dtype, seed=d, ignored=0.3)
    got = ce(env, h, w, target, weight)
    ref = reference(torch, h, w, target=target, weight=weight)
    for k in ("loss", "lse", "dh", "dw"):
        within(torch, got[k], ref[k], k)
    on = target >= 0
    z = (h[on].double() * w[target[on].long()].double()).sum(1)
    s = (h[on].double().square() * w[target[on].long()].double().square()).mean().sqrt()
    off = (got["loss"][on].double() + got["lse"][on].double() - z).square().mean().sqrt()
    stored = 2.0 ** -21 * got["lse"][on].double().abs().max()
    assert off <= 2 / 3 * d ** 1.5 * U * s + stored, (off.item(), s.item())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 2, 8])
def test_few_rows_past_the_streaming_kernel(env, N, dtype):
    """d over 6,400: the rows of h no longer fit the streaming kernel."""
    rlt, torch = env
    h, w, target, weight = make(torch, N, 301, 6504, dtype, seed=N, ignored=0.0)
    got = ce(env, h, w, target, weight)
    ref = reference(torch, h, w, target=target, weight=weight)
    for k in ("loss", "lse", "dh", "dw"):
        within(torch, got[k], ref[k], k)


@pytest.mark.parametrize("N,part", [(4096, 100), (257, 256), (3000, 256), (300, 1)])
def test_gradient_of_few_rows_among_many(env, N, part):
    """bf16 gradients over few rows that take part carry one rounding, the
    output's, whatever N is: the root mean square of the error is that of the
    exact gradient rounded once.  (Another rounding of dz would make it 1.4 of
    that; 16 bits of dz and fp32 sums add less than a hundredth.)"""
    rlt, torch = env
    V, d = 2000, 128
    h, w, _, weight = make(torch, N, V, d, "bf16", seed=part)
    g = torch.Generator().manual_seed(part)
    target = torch.full((N,), -1, dtype=torch.int32)
    rows = torch.randperm(N, generator=g)[:part]
    target[rows] = torch.randint(0, V, (part,), generator=g, dtype=torch.int32)
    target = target.cuda()
    ids = torch.full((N, 3), -1, dtype=torch.int32)
    ids[rows] = torch.randint(0, V, (part, 3), generator=g, dtype=torch.int32)
    teacher = torch.randn(N, 3, generator=g).cuda()
    for got, lists, T in ((ce(env, h, w, target, weight), {"target": target}, 1.0),
                          (kl(env, h, w, ids.cuda(), teacher, 0.8, weight), {"ids": ids.cuda(), "teacher": teacher}, 0.8)):
        ref = reference(torch, h, w, T=T, weight=weight, **lists)
        for k in ("dh", "dw"):
            within(torch, got[k], ref[k], k)
            exact = ref[k][0]
            once = (exact.to(torch.bfloat16).double() - exact).square().mean().sqrt()
            off = (got[k].double() - exact).square().mean().sqrt()
            assert off <= 1.05 * once, (k, (off / once).item())


@pytest.mark.parametrize("N,V,d,K,lean", [(300, 2000, 24, 1, 6.0), (1200, 700, 40, 5, 3.0), (2000, 300, 333, 200, 1.0), (700, 5000, 1032, 1, 4.0),
                                          (41000, 8003, 20, 1, 5.0), (41000, 8003, 25, 3, 5.0)])
def test_dh_keeps_its_listed_entries_whole(env, N, V, d, K, lean):
    """Many bf16 rows: dz is rounded once, but dh gets the residuals of its
    listed entries back (of a long list all but an eighth of the largest).  So
    the error's mean square is that of the output's rounding, once, and that of
    the other entries, each off by a relative 2^-8.9 (a bf16 rounding's root mean
    square is 2^-7 / sqrt 12 of the step below, at most 2^-8.7 of the value)
    where they are independent; a list's left-outs are within the 1.1.  At
    41,000 rows the vocabulary is walked in pieces."""
    rlt, torch = env
    h, w, target, weight = make(torch, N, V, d, "bf16", seed=N + d)
    on = target >= 0
    if K == 1:  # rows that lean to their target: p of it is not small, and the sum is near zero
        t = w[target[on].long()].float()
        h[on] = (h[on].float() + lean * t / (t.square().sum(1, keepdim=True) + 1e-3)).to(h.dtype)
        got, lists, T = ce(env, h, w, target, weight), {"target": target}, 1.0
    else:
        ids, teacher = make_list(torch, N, V, K, seed=d)
        ids[:, 1] = ids[:, 0]  # an id in two slots
        got, lists, T = kl(env, h, w, ids, teacher, 0.8, weight), {"ids": ids, "teacher": teacher}, 0.8
    err = once = rest = 0.0
    W = w.double()
    for i in range(0, N, 10000):
        s = slice(i, i + 10000)
        part = {k: v[s] for k, v in lists.items()}
        ref = reference(torch, h[s], w, T=T, weight=weight[s], **part)["dh"]
        within(torch, got["dh"][s], ref, "dh")
        want, has, _ = dense_targets(torch, V, T=T, **part)
        p = torch.softmax(torch.where(has[:, None], h[s].double(), torch.zeros((), device="cuda", dtype=torch.float64)) @ W.T / T, 1)
        c = torch.where(has, weight[s].double() / T, torch.zeros((), device="cuda", dtype=torch.float64))[:, None]
        g = torch.where(want > 0, torch.zeros_like(p), c * p)
        rest = rest + (2.0 ** -17.4 * (g.square() @ W.square())).sum()
        once = once + (ref[0].to(torch.bfloat16).double() - ref[0]).square().sum()
        err = err + (got["dh"][s].double() - ref[0]).square().sum()
    assert err.sqrt() <= 1.1 * (once + rest).sqrt(), ((err / (once + rest)).sqrt().item(), (err / once).sqrt().item())


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 8, 9, 64])
def test_fp32_probabilities_of_the_backward_sum_to_one(env, N):
    """The backward's logits have the errors of those the lse was made of, so
    sum_v p - 1 is lse's own rounding, half a step of it, and the roundings of
    the exponentials, planes and sums (4 + 1 + 24 u for the terms up to 1, and
    4 additions towards zero of 2 u in tensor memory: 40 u).  A w whose first
    column is 1 (and none of h) shows it as dh's first: weight (sum p - 1).
    Logits of about 80: half a step of lse is 64 u."""
    rlt, torch = env
    V, d = 1500, 1001
    for seed in range(4):
        h, w, target, _ = make(torch, N, V, d, "f32", seed=seed, ignored=0.0)
        h, weight = 25 * h, torch.ones(N, device="cuda")
        h[:, 0], w[:, 0] = 0.0, 1.0
        got = ce(env, h, w, target, weight)
        half = torch.exp2(torch.floor(torch.log2(got["lse"].double()))) * U
        off = got["dh"][:, 0].double().abs()
        assert (off <= half + 40 * U).all(), (off / U, half / U)
        ids, teacher = make_list(torch, N, V, 30, seed=seed, empty=0.0)
        got = kl(env, h, w, ids, teacher, 1.0, weight)  # sum q is 1 to 2 u a term
        assert (got["dh"][:, 0].double().abs() <= half + (40 + 60) * U).all()


@pytest.mark.parametrize("N", [1, 3, 8])
def test_few_fp32_rows_some_left_out(env, N):
    """Odd widths, rows apart and off the grid, rows left out among the few, a
    vocabulary in pieces, gradients added to and one at a time."""
    rlt, torch = env
    for V, d in ((17, 5), (333, 75), (1000, 264), (400_003, 4)):
        h0, w0, target, weight = make(torch, N, V, d, "f32", seed=V, ignored=0.0)
        hb, wb = (torch.full((x.shape[0], d + 3), math.nan, device="cuda") for x in (h0, w0))
        h, w = hb[:, 1:1 + d], wb[:, 2:2 + d]
        h.copy_(h0)
        w.copy_(w0)
        if N > 2:
            target[0], weight[2] = -1, 0.0
            h[0], h[2] = math.nan, math.inf
            h0[0] = h0[2] = 0.0
        want = reference(torch, h0, w0, target=target, weight=weight)
        lse, loss = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
        rlt.rlt_op_cross_entropy(h0, w0, target, loss, lse)
        dh, dw = torch.full((N, d), 7.0, device="cuda"), torch.full((V, d), 7.0, device="cuda")
        rlt.rlt_op_cross_entropy_backward(h, w, target, lse, weight, dh=dh, dw=dw)
        within(torch, dh, want["dh"], "dh")
        within(torch, dw, want["dw"], "dw")
        again = torch.full((V, d), 2.0, device="cuda")
        rlt.rlt_op_cross_entropy_backward(h, w, target, lse, weight, dw=again, accumulate=True)
        value, bound = want["dw"]
        within(torch, again, (value + 2, bound + U * (value + 2).abs()), "dw added")
        one = torch.empty_like(dh)
        rlt.rlt_op_cross_entropy_backward(h, w, target, lse, weight, dh=one)
        assert torch.equal(one, dh)
        none = torch.full((V, d), 7.0, device="cuda")
        rlt.rlt_op_cross_entropy_backward(h, w, torch.full_like(target, -1), lse, weight, dh=dh, dw=none)
        assert (dh == 0).all() and (none == 0).all()


# ------------------------------------------------------------------ long sorts
@pytest.mark.parametrize("V", [200, 255, 256, 32000, 65535, 65536, 70000])
@pytest.mark.parametrize("N,dist", [(16384, "uniform"), (16385, "zipf"), (20001, "uniform"), (65536, "zipf")])
def test_embedding_gradient_of_many_ids(env, N, dist, V):
    """One block's sort at its largest and several blocks', in one to three
    passes (keys go to V, the ids that do not count), a tenth of the ids
    outside, into a table of its own, a slice of rows off the 16-byte grid, and
    one that is added to."""
    rlt, torch = env
    d = 24 if N < 60000 else 8
    g = torch.Generator().manual_seed(N + V)
    tok = torch.randint(0, V, (N,), generator=g) if dist == "uniform" else (V * torch.rand(N, generator=g) ** 6).long().clamp(max=V - 1)
    out = torch.rand(N, generator=g) < 0.1
    tok[out] = torch.tensor([-1, V, V + 1, 2 ** 31 - 1, -2 ** 31])[torch.randint(0, 5, (int(out.sum()),), generator=g)]
    tok = tok.to(torch.int32).cuda()
    dout = torch.randn(N, d, generator=g).cuda()
    dout[out.cuda()] = math.nan
    value, bound = embed_reference(torch, dout, tok, V, 1.5, torch.float32)
    table = torch.full((V, d), 7.0, device="cuda")
    rlt.rlt_op_embed_backward(dout, tok, table, scale=1.5)
    within(torch, table, (value, bound), "whole")
    absent = torch.bincount(tok[~out.cuda()].long(), minlength=V) == 0
    assert (table[absent] == 0).all()
    wide = torch.full((V, d + 5), 9.0, device="cuda")
    rlt.rlt_op_embed_backward(dout, tok, wide[:, 3:3 + d], scale=1.5)
    assert torch.equal(wide[:, 3:3 + d], table)
    assert (wide[:, :3] == 9).all() and (wide[:, 3 + d:] == 9).all()
    half = torch.full((V, d), 2.0, dtype=torch.bfloat16, device="cuda")
    rlt.rlt_op_embed_backward(dout, tok, half, scale=1.5, accumulate=True)
    within(torch, half, (value + 2, bound + half_step(half.dtype) * (value + 2).abs() + U * (value + 2).abs()), "added")

"""The vocabulary operators against their formulas in 64 bits: cross entropy and
distillation over h w^T without kept logits, the embedding lookup and its
gradient, each with its masks, strides, odd sizes, streams and graphs.

Tolerances.  Every bound is elementwise and follows from the arithmetic, with
u = 2^-24 (fp32) and half a bf16 step 2^-8:
  logits     a sum of d fp32 products in any order, and as much again for fp32
             operands taken as 16-bit parts, whose own error and left-out
             products are below (d + 8) u |h||w|: |dz| <= (2 d + 8) u sum|h||w|
  lse        2 |dz| plus the exponentials' and sums' own (1024 + 4 |z|) u
  p          relative: |dz| + |dlse| + (8 + 2 |z - lse|) u
  dz         c p dp, plus one rounding to bf16 (bf16 operands) or to three
             bf16 parts (fp32: 2^-23)
  gradients  the error of dz through |w| or |h|, a sum of V or N terms
             (2 n + 8) u, and the output's own rounding
"""
import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    import stateful_decoder_b200 as rlt
    return rlt, torch


def half_step(t):
    return {"torch.bfloat16": 2.0 ** -8, "torch.float32": U}[str(t)]


def types(torch, name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


# ------------------------------------------------------------------ formulas in 64 bits
def dense_targets(torch, V, target=None, ids=None, teacher=None, T=1.0):
    """(want [N, V], has [N], sum q log q [N])."""
    if target is not None:
        N = target.numel()
        want = torch.zeros(N, V, dtype=torch.float64, device="cuda")
        has = (target >= 0) & (target < V)
        want[has.nonzero()[:, 0], target[has].long()] = 1.0
        return want, has, torch.zeros(N, dtype=torch.float64, device="cuda")
    N, K = ids.shape
    ok = (ids >= 0) & (ids < V)
    t = (teacher.double() / T).masked_fill(~ok, -math.inf)
    has = (t > -math.inf).any(1)
    q = torch.where(has[:, None], torch.softmax(t.masked_fill(~has[:, None], 0.0), 1), torch.zeros_like(t))
    want = torch.zeros(N, V, dtype=torch.float64, device="cuda")
    rows = torch.arange(N, device="cuda")[:, None].expand(N, K)
    want.index_put_((rows[ok], ids[ok].long()), q[ok], accumulate=True)
    return want, has, torch.special.xlogy(q, q).sum(1)


def reference(torch, h, w, T=1.0, weight=None, **lists):
    """Values and elementwise error bounds of loss, lse, dh and dw."""
    H, W = h.double(), w.double()
    V, d = W.shape
    N = H.shape[0]
    want, has, ent = dense_targets(torch, V, T=T, **lists)
    H = torch.where(has[:, None], H, torch.zeros_like(H))
    z = H @ W.T / T
    dz = ((2 * d + 8) * U * (H.abs() @ W.abs().T) / T).amax(1) + U * z.abs().amax(1)
    lse = torch.logsumexp(z, 1)
    big = z.abs().amax(1)
    dlse = 2 * dz + (1024 + 4 * big) * U + U * lse.abs()
    ce = "target" in lists
    lp = z - lse[:, None]
    loss = (want * lp).sum(1) if ce else ent - (want * lp).sum(1)
    zero = torch.zeros_like(lse)
    # a list of K terms q (log q - z + lse), q to a few ulp of its exponent
    dloss = dz + dlse + (16 + 4 * big + (0 if ce else 600)) * U * (1 + ent.abs() + loss.abs())
    r = {"loss": (torch.where(has, loss, zero), torch.where(has, dloss, zero)),
         "lse": (torch.where(has, lse, zero), torch.where(has, dlse, zero))}
    if weight is None:
        return r
    c = torch.where(has, weight.double() / T, zero)[:, None]
    p = lp.exp()
    g = c * (p - want)
    r_g = half_step(torch.bfloat16) if str(h.dtype) == "torch.bfloat16" else 2 * U
    e_g = c.abs() * p * (dz + dlse)[:, None] + c.abs() * p * (16 + 2 * lp.abs()) * U + c.abs() * want * 600 * U
    e_g = e_g + r_g * g.abs()
    step = half_step(h.dtype)
    for name, a, b, n in (("dh", lambda x: x @ W, lambda x: x @ W.abs(), V),
                          ("dw", lambda x: x.T @ H, lambda x: x.T @ H.abs(), N)):
        value = a(g)
        r[name] = (value, b(e_g) * (1 + 2.0 ** -7) + (2 * n + 8) * U * b(g.abs()) + step * value.abs() + 1e-38)
    return r


def within(torch, got, ref, what=""):
    value, bound = ref
    off = (got.double() - value).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), (off - bound).max().item(), off.max().item())


def make(torch, N, V, d, dtype, seed, spread=1.0, ignored=0.25):
    g = torch.Generator().manual_seed(seed)
    w = (spread / math.sqrt(d) * torch.randn(V, d, generator=g)).to(types(torch, dtype)).cuda()
    h = torch.randn(N, d, generator=g).to(types(torch, dtype)).cuda()
    target = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    target[torch.rand(N, generator=g) < ignored] = -1
    weight = torch.randn(N, generator=g)
    return h, w, target.cuda(), weight.cuda()


def make_list(torch, N, V, K, seed, empty=0.2):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, V, (N, K), generator=g, dtype=torch.int32)
    ids[torch.rand(N, K, generator=g) < empty] = -1
    teacher = 3 * torch.randn(N, K, generator=g)
    return ids.cuda(), teacher.cuda()


def ce(env, h, w, target, weight=None, **kw):
    rlt, torch = env
    N = h.shape[0]
    loss, lse = (torch.full((N,), 7.0, device="cuda") for _ in range(2))
    rlt.rlt_op_cross_entropy(h, w, target, loss, lse, **kw)
    out = {"loss": loss, "lse": lse}
    if weight is not None:
        out["dh"] = torch.full(h.shape, 7.0, dtype=h.dtype, device="cuda")
        out["dw"] = torch.full(w.shape, 7.0, dtype=w.dtype, device="cuda")
        rlt.rlt_op_cross_entropy_backward(h, w, target, lse, weight, dh=out["dh"], dw=out["dw"], **kw)
    return out


def kl(env, h, w, ids, teacher, T, weight=None, **kw):
    rlt, torch = env
    N = h.shape[0]
    loss, lse = (torch.full((N,), 7.0, device="cuda") for _ in range(2))
    rlt.rlt_op_distill(h, w, ids, teacher, T, loss, lse, **kw)
    out = {"loss": loss, "lse": lse}
    if weight is not None:
        out["dh"] = torch.full(h.shape, 7.0, dtype=h.dtype, device="cuda")
        out["dw"] = torch.full(w.shape, 7.0, dtype=w.dtype, device="cuda")
        rlt.rlt_op_distill_backward(h, w, ids, teacher, T, lse, weight, dh=out["dh"], dw=out["dw"], **kw)
    return out


SIZES = [  # N, V, d
    (1, 1, 1), (1, 200, 17), (2, 257, 64), (127, 255, 63), (128, 256, 64), (129, 513, 65), (300, 1000, 136),
    (64, 5000, 512), (1, 32000, 256), (257, 771, 1000), (1000, 130, 24), (520, 4099, 200),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d", SIZES)
def test_cross_entropy_matches_formula(env, N, V, d, dtype):
    rlt, torch = env
    h, w, target, weight = make(torch, N, V, d, dtype, seed=N + V + d, ignored=0.25 if N > 1 else 0.0)
    got = ce(env, h, w, target, weight)
    ref = reference(torch, h, w, target=target, weight=weight)
    for k in ("loss", "lse", "dh", "dw"):
        within(torch, got[k], ref[k], k)
    rlt.rlt_check_device()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d,K,T", [(1, 1, 1, 1, 1.0), (3, 300, 64, 50, 0.8), (129, 513, 65, 256, 2.0),
                                       (200, 2000, 128, 33, 0.5), (64, 40, 32, 200, 1.0), (400, 4099, 72, 7, 0.8)])
def test_distill_matches_formula(env, N, V, d, K, T, dtype):
    """Among them lists longer than the vocabulary, so every id repeats."""
    rlt, torch = env
    h, w, _, weight = make(torch, N, V, d, dtype, seed=N * K)
    ids, teacher = make_list(torch, N, V, K, seed=V, empty=0.2 if K > 1 else 0.0)
    if N > 2:
        ids[1] = -1            # an empty row
        ids[2] = V             # ids past the vocabulary are empty slots too
        teacher[0, 0] = -math.inf
    got = kl(env, h, w, ids, teacher, T, weight)
    ref = reference(torch, h, w, T=T, ids=ids, teacher=teacher, weight=weight)
    for k in ("loss", "lse", "dh", "dw"):
        within(torch, got[k], ref[k], k)
    rlt.rlt_check_device()


@pytest.mark.parametrize("N,dtype", [(90001, "bf16"), (90001, "f32"), (60000, "f32")])
def test_several_pieces_of_the_vocabulary(env, N, dtype):
    """Many rows: the backward walks the vocabulary in more than one piece,
    the last one short and odd; at 60,000 fp32 rows the last round of row
    tiles is split over k as well."""
    rlt, torch = env
    V, d = 5121, 16
    h, w, target, weight = make(torch, N, V, d, dtype, seed=5)
    weight /= N
    got = ce(env, h, w, target, weight)
    value, bound = [], []
    dw = [0.0, 0.0]
    for i in range(0, N, 15000):
        s = slice(i, i + 15000)
        ref = reference(torch, h[s], w, target=target[s], weight=weight[s])
        for k in ("loss", "lse", "dh"):
            within(torch, got[k][s], ref[k], k)
        dw[0] = dw[0] + ref["dw"][0]
        dw[1] = dw[1] + ref["dw"][1] * 7  # (2 n + 8) u counts all N terms (at most 6.01 times 15,000)
    within(torch, got["dw"], dw, "dw")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d", [(2, 1000, 300), (3, 900, 61), (4, 5000, 520), (5, 70, 2100), (8, 3001, 130), (9, 640, 256),
                                   (256, 900, 64), (257, 900, 64), (40, 20000, 192), (12, 251, 2432), (3000, 700, 74),
                                   (300, 4000, 264)])
def test_each_way_of_cutting_the_work(env, N, V, d, dtype):
    """Few rows (streamed, and just past that), one and two planes of the logit
    gradient, long sums split over the SMs with few and many tiles, narrow
    tiles; with a list that has the target in it, at half temperature."""
    rlt, torch = env
    h, w, target, weight = make(torch, N, V, d, dtype, seed=N + d, ignored=0.1 if N > 8 else 0.0)
    ids, teacher = make_list(torch, N, V, 6, seed=N)
    got = ce(env, h, w, target, weight)
    ref = reference(torch, h, w, target=target, weight=weight)
    for k in ("loss", "lse", "dh", "dw"):
        within(torch, got[k], ref[k], k)
    got = kl(env, h, w, ids, teacher, 0.5, weight)
    ref = reference(torch, h, w, T=0.5, ids=ids, teacher=teacher, weight=weight)
    for k in ("loss", "lse", "dh", "dw"):
        within(torch, got[k], ref[k], k)
    rlt.rlt_check_device()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_few_of_many_rows_take_part(env, dtype):
    """The work is cut by the rows that have a target, a count only the device
    knows: one in a hundred, in runs and alone, first and last among them."""
    rlt, torch = env
    N, V, d = 5000, 3000, 136
    h, w, target, weight = make(torch, N, V, d, dtype, seed=8, ignored=0.99)
    target[0], target[N - 1], target[1200:1210] = 5, 2999, 7
    got = ce(env, h, w, target, weight)
    ref = reference(torch, h, w, target=target, weight=weight)
    for k in ("loss", "lse", "dh", "dw"):
        within(torch, got[k], ref[k], k)


def test_few_rows_off_the_grid(env):
    """Up to eight rows whose operands are not 16-byte aligned."""
    rlt, torch = env
    for dtype in ("bf16", "f32"):
        for N in (1, 2, 7):
            h, w, target, _ = make(torch, N, 333, 75, dtype, seed=N, ignored=0.0)
            hb, wb = (torch.full((x.shape[0], 78), math.nan, dtype=x.dtype, device="cuda") for x in (h, w))
            hb[:, 1:76], wb[:, 3:] = h, w
            loss, lse = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
            rlt.rlt_op_cross_entropy(hb[:, 1:76], wb[:, 3:], target, loss, lse)
            ref = reference(torch, h, w, target=target)
            within(torch, loss, ref["loss"])
            within(torch, lse, ref["lse"])


def test_strided_and_misaligned_operands(env):
    """Rows that stand apart by odd distances, bases off the 16-byte grid, and
    gradients written into slices whose surroundings stay as they were."""
    rlt, torch = env
    for dtype in ("bf16", "f32"):
        N, V, d = 140, 600, 72
        h0, w0, target, weight = make(torch, N, V, d, dtype, seed=9)
        hb = torch.full((N, d + 9), math.nan, dtype=h0.dtype, device="cuda")
        wb = torch.full((V, d + 5), math.nan, dtype=h0.dtype, device="cuda")
        h, w = hb[:, 3:3 + d], wb[:, 1:1 + d]
        h.copy_(h0)
        w.copy_(w0)
        gh, gw = (torch.full_like(x, 5.0) for x in (hb, wb))
        loss, lse = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
        rlt.rlt_op_cross_entropy(h, w, target, loss, lse)
        rlt.rlt_op_cross_entropy_backward(h, w, target, lse, weight, dh=gh[:, 2:2 + d], dw=gw[:, 4:4 + d])
        ref = reference(torch, h0, w0, target=target, weight=weight)
        for got, k in ((loss, "loss"), (lse, "lse"), (gh[:, 2:2 + d], "dh"), (gw[:, 4:4 + d], "dw")):
            within(torch, got, ref[k], k)
        assert (gh[:, :2] == 5).all() and (gh[:, 2 + d:] == 5).all()
        assert (gw[:, :4] == 5).all() and (gw[:, 4 + d:] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [5, 300])
def test_rows_without_a_target_do_not_matter(env, dtype, N):
    """Rows without a target, or of weight 0, may hold anything."""
    rlt, torch = env
    h, w, target, weight = make(torch, N, 700, 64, dtype, seed=3)
    target[0], target[1], target[3] = -1, 700, 2 ** 31 - 1
    weight[4], target[4] = 0.0, 3
    clean = ce(env, h, w, target, weight)
    h2, wt2 = h.clone(), weight.clone()
    h2[0], h2[1], h2[3] = math.nan, math.inf, -math.inf
    wt2[0] = math.nan
    dirty = ce(env, h2, w, target, wt2)
    for k in clean:
        assert torch.equal(clean[k], dirty[k]), k
    for k in ("loss", "lse"):
        assert (clean[k][[0, 1, 3]] == 0).all()
    assert (clean["dh"][[0, 1, 3, 4]] == 0).all()
    # a zero-weight row with a target: its h stays out of the gradient too
    h3 = h.clone()
    h3[4] = math.nan
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    rlt.rlt_op_cross_entropy_backward(h3, w, target, clean["lse"], weight, dh=dh, dw=dw)
    assert torch.equal(dh, clean["dh"]) and torch.equal(dw, clean["dw"])
    # nothing left at all
    none = ce(env, h, w, torch.full_like(target, -1), weight)
    assert all((none[k] == 0).all() for k in none)


def test_no_rows(env):
    rlt, torch = env
    for t in ("bf16", "f32"):
        h, w, target, weight = make(torch, 0, 300, 40, t, seed=1)
        got = ce(env, h, w, target, weight)
        assert (got["dw"] == 0).all()
        dw = torch.full_like(w, 3.0)
        rlt.rlt_op_cross_entropy_backward(h, w, target, got["lse"], weight, dw=dw, accumulate=True)
        assert (dw == 3).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_accumulate_and_single_gradients(env, dtype):
    rlt, torch = env
    h, w, target, weight = make(torch, 150, 400, 64, dtype, seed=11)
    full = ce(env, h, w, target, weight)
    dh, dw = torch.full_like(h, 2.0), torch.full_like(w, 2.0)
    rlt.rlt_op_cross_entropy_backward(h, w, target, full["lse"], weight, dh=dh)
    assert torch.equal(dh, full["dh"])
    rlt.rlt_op_cross_entropy_backward(h, w, target, full["lse"], weight, dw=dw, accumulate=True)
    value, bound = reference(torch, h, w, target=target, weight=weight)["dw"]
    within(torch, dw, (value + 2, bound + half_step(w.dtype) * (value + 2).abs()), "dw")


def test_extreme_logits(env):
    """Logits of hundreds, where exponentials without the maximum overflow, and
    rows whose whole mass is one id."""
    rlt, torch = env
    for dtype in ("bf16", "f32"):
        h, w, target, weight = make(torch, 130, 500, 64, dtype, seed=21, spread=150.0, ignored=0.0)
        got = ce(env, h, w, target, weight)
        ref = reference(torch, h, w, target=target, weight=weight)
        for k in ("loss", "lse"):
            within(torch, got[k], ref[k], k)
        for k in ("dh", "dw"):
            within(torch, got[k], ref[k], k)
        h[7] = math.nan  # a row that has a target and holds NaN poisons itself alone in the forward
        bad = ce(env, h, w, target)
        assert torch.isnan(bad["loss"][7]) and torch.isnan(bad["lse"][7])
        keep = torch.arange(130, device="cuda") != 7
        assert torch.equal(bad["lse"][keep], got["lse"][keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_twice_and_any_workspace(env, dtype):
    """Results do not depend on timing, nor on what the workspace held."""
    rlt, torch = env
    h, w, target, weight = make(torch, 333, 3001, 96, dtype, seed=2)
    ids, teacher = make_list(torch, 333, 3001, 40, seed=8)
    ws = torch.full((512 << 20,), 255, dtype=torch.uint8, device="cuda")
    for f in (lambda **kw: ce(env, h, w, target, weight, **kw), lambda **kw: kl(env, h, w, ids, teacher, 0.8, weight, **kw)):
        a, b, c = f(), f(), f(workspace=ws)
        for k in a:
            assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]), k


def test_gradient_against_differences(env):
    """Central differences of the loss in 64 bits along random directions."""
    rlt, torch = env
    h, w, target, weight = make(torch, 20, 300, 48, "f32", seed=4)
    ids, teacher = make_list(torch, 20, 300, 12, seed=4)
    for T, lists, got, sign in ((1.0, {"target": target}, ce(env, h, w, target, weight), -1.0),
                                (0.8, {"ids": ids, "teacher": teacher}, kl(env, h, w, ids, teacher, 0.8, weight), 1.0)):
        g = torch.Generator().manual_seed(0)
        for name in ("dh", "dw"):
            x = h if name == "dh" else w
            u = torch.randn(x.shape, generator=g).double().cuda()
            u /= u.norm()
            eps = 1e-4

            def loss(s):
                hh, ww = (h.double() + s * u, w) if name == "dh" else (h, w.double() + s * u)
                return sign * (reference(torch, hh, ww, T=T, **lists)["loss"][0] * weight.double()).sum()

            diff = ((loss(eps) - loss(-eps)) / (2 * eps)).item()
            value, bound = reference(torch, h, w, T=T, weight=weight, **lists)[name]
            # the gradient's own bound along u, and eps^2 of a third derivative of order |weight| |h|^3
            tol = (bound * u.abs()).sum().item() + 1e-8 * 1e2
            assert abs((got[name].double() * u).sum().item() - diff) <= tol


def test_side_stream_and_graph_replay(env):
    """On a stream of the caller's, and captured once and replayed on new
    inputs, with the same bits as an eager call."""
    rlt, torch = env
    h, w, target, weight = make(torch, 200, 1500, 128, "bf16", seed=6)
    ids, teacher = make_list(torch, 200, 1500, 20, seed=6)
    want = ce(env, h, w, target, weight)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    loss, lse = torch.empty(200, device="cuda"), torch.empty(200, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    rlt.rlt_op_cross_entropy(h, w, target, loss, lse, stream=s)
    s.synchronize()
    assert torch.equal(lse, want["lse"]) and torch.equal(loss, want["loss"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = ce(env, h, w, target, weight)
        b = kl(env, h, w, ids, teacher, 0.8, weight)
    for seed in (31, 32):
        h2, w2, t2, wt2 = make(torch, 200, 1500, 128, "bf16", seed=seed, ignored=0.1 * (seed - 30))
        for x, y in ((h, h2), (w, w2), (target, t2), (weight, wt2)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        for got, eager in ((a, ce(env, h, w, target, weight)), (b, kl(env, h, w, ids, teacher, 0.8, weight))):
            for k in got:
                assert torch.equal(got[k], eager[k]), k


def test_streams_of_every_kind_and_two_calls_at_once(env):
    """The legacy default stream by number and by object, and two calls at once
    on two streams, each with the workspace that its call takes."""
    rlt, torch = env
    a = make(torch, 700, 3000, 128, "bf16", seed=1)
    b = make(torch, 650, 2500, 192, "bf16", seed=2)
    want = [ce(env, *x) for x in (a, b)]
    torch.cuda.synchronize()
    for stream in (0, torch.cuda.default_stream()):
        got = ce(env, *a, stream=stream)
        torch.cuda.synchronize()
        for k in got:
            assert torch.equal(got[k], want[0][k]), k
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [ce(env, *x, stream=s) for x, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        for g, e in zip(got, want):
            for k in g:
                assert torch.equal(g[k], e[k]), k
    tok = torch.randint(0, 3000, (700,), dtype=torch.int32).cuda()
    grad = [torch.empty(3000, 128, device="cuda") for _ in range(2)]
    rlt.rlt_op_embed_backward(a[0].float(), tok, grad[0])
    torch.cuda.synchronize()
    rlt.rlt_op_embed_backward(a[0].float(), tok, grad[1], stream=0)
    torch.cuda.synchronize()
    assert torch.equal(*grad)


# ------------------------------------------------------------------ embedding
def embed_reference(torch, dout, tok, V, scale, dt):
    """Gradient and bound: a sum of n fp32 terms, a product, the output's rounding."""
    ok = (tok >= 0) & (tok < V)
    g = torch.zeros(V, dout.shape[1], dtype=torch.float64, device="cuda")
    m = torch.zeros_like(g)
    g.index_add_(0, tok[ok].long(), dout[ok].double())
    m.index_add_(0, tok[ok].long(), dout[ok].double().abs())
    n = torch.bincount(tok[ok].long(), minlength=V).double()[:, None]
    return g * scale, abs(scale) * m * (n + 4) * U + half_step(dt) * (g * scale).abs()


@pytest.mark.parametrize("et,ot", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("N,V,d,dist", [(1, 1, 1, "uniform"), (7, 5, 3, "uniform"), (300, 1000, 64, "uniform"),
                                        (1025, 17, 130, "uniform"), (5000, 3000, 33, "zipf"), (2049, 70000, 8, "zipf"),
                                        (40000, 300, 96, "one")])
def test_embedding_and_its_gradient(env, N, V, d, dist, et, ot):
    rlt, torch = env
    g = torch.Generator().manual_seed(N + d)
    emb = torch.randn(V, d, generator=g).to(types(torch, et)).cuda()
    if dist == "uniform":
        tok = torch.randint(0, V, (N,), generator=g)
    elif dist == "zipf":
        tok = (V * torch.rand(N, generator=g) ** 6).long().clamp(max=V - 1)
    else:
        tok = torch.full((N,), V - 1)
    tok = tok.to(torch.int32)
    if N > 5:
        tok[1], tok[3], tok[5] = -1, V, -2 ** 31
    tok = tok.cuda()
    scale = 1.75
    out = torch.full((N, d), 7.0, dtype=types(torch, ot), device="cuda")
    rlt.rlt_op_embed(emb, tok, out, scale=scale)
    ok = (tok >= 0) & (tok < V)
    want = torch.where(ok[:, None], emb.double()[tok.long().clamp(0, V - 1)] * scale, torch.zeros((), dtype=torch.float64, device="cuda"))
    within(torch, out, (want, half_step(out.dtype) * want.abs() + U * want.abs()), "out")
    dout = torch.randn(N, d, generator=g).to(out.dtype).cuda()
    dout[~ok] = math.nan  # never read
    demb = torch.full((V, d), 7.0, dtype=emb.dtype, device="cuda")
    rlt.rlt_op_embed_backward(dout, tok, demb, scale=scale)
    value, bound = embed_reference(torch, dout, tok, V, scale, emb.dtype)
    within(torch, demb, (value, bound), "demb")
    again = torch.full((V, d), -3.0, dtype=emb.dtype, device="cuda")
    rlt.rlt_op_embed_backward(dout, tok, again, scale=scale)
    assert torch.equal(again, demb)
    acc = torch.full((V, d), 0.5, dtype=emb.dtype, device="cuda")
    rlt.rlt_op_embed_backward(dout, tok, acc, scale=scale, accumulate=True)
    within(torch, acc, (value + 0.5, bound + half_step(emb.dtype) * (value + 0.5).abs() + U), "accumulate")


def test_embedding_of_slices_and_nothing(env):
    rlt, torch = env
    V, d, N = 50, 24, 70
    g = torch.Generator().manual_seed(1)
    table = torch.randn(V, d + 7, generator=g).to(torch.bfloat16).cuda()
    emb = table[:, 3:3 + d]
    tok = torch.randint(0, V, (N,), generator=g, dtype=torch.int32).cuda()
    buf = torch.full((N, d + 3), 9.0, device="cuda")
    rlt.rlt_op_embed(emb, tok, buf[:, 1:1 + d])
    assert torch.equal(buf[:, 1:1 + d], emb.float()[tok.long()])
    assert (buf[:, 0] == 9).all() and (buf[:, 1 + d:] == 9).all()
    grad = torch.full((V, d + 5), 9.0, device="cuda")
    dout = torch.randn(N, d + 3, generator=g).cuda()[:, 2:2 + d]
    rlt.rlt_op_embed_backward(dout, tok, grad[:, 5:])
    within(torch, grad[:, 5:], embed_reference(torch, dout, tok, V, 1.0, grad.dtype), "demb")
    assert (grad[:, :5] == 9).all()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    rlt.rlt_op_embed(emb, none, torch.empty(0, d, device="cuda"))
    rlt.rlt_op_embed_backward(torch.empty(0, d, device="cuda"), none, grad[:, 5:])
    assert (grad[:, 5:] == 0).all()


# ------------------------------------------------------------------ together
def test_a_training_step_of_a_tied_vocabulary(env):
    """Embedding -> a residual map -> cross entropy and distillation on the same
    table, and all gradients back into it (the readout's written, the
    embedding's added), in fp32 against autograd of the formulas in 64 bits."""
    rlt, torch = env
    N, V, d, K = 190, 777, 80, 9
    g = torch.Generator().manual_seed(77)
    emb = (torch.randn(V, d, generator=g) / math.sqrt(d)).cuda()
    tok = torch.randint(0, V, (N,), generator=g, dtype=torch.int32).cuda()
    target = torch.cat([tok[1:], tok.new_tensor([-1])])
    ids, teacher = make_list(torch, N, V, K, seed=3)
    a, b = (torch.rand(N, generator=g).cuda() / N for _ in range(2))
    scale = math.sqrt(d)

    x = torch.empty(N, d, device="cuda")
    rlt.rlt_op_embed(emb, tok, x, scale=scale)
    h = torch.tanh(x)
    logp, lse, div, lse_t = (torch.empty(N, device="cuda") for _ in range(4))
    rlt.rlt_op_cross_entropy(h, emb, target, logp, lse)
    rlt.rlt_op_distill(h, emb, ids, teacher, 0.8, div, lse_t)
    dh, dh2, grad = torch.empty_like(h), torch.empty_like(h), torch.empty_like(emb)
    rlt.rlt_op_cross_entropy_backward(h, emb, target, lse, a, dh=dh, dw=grad)
    rlt.rlt_op_distill_backward(h, emb, ids, teacher, 0.8, lse_t, b, dh=dh2, dw=grad, accumulate=True)
    dx = (dh + dh2) * (1 - h * h)
    rlt.rlt_op_embed_backward(dx, tok, grad, scale=scale, accumulate=True)
    loss = -(a * logp).sum() + (b * div).sum()

    e = emb.double().requires_grad_()
    hh = torch.tanh(e[tok.long()] * scale)
    lp = torch.log_softmax(hh @ e.T, 1)
    lpt = torch.log_softmax(hh @ e.T / 0.8, 1)
    has = target >= 0
    t = (teacher.double() / 0.8).masked_fill(ids < 0, -math.inf)
    some = (ids >= 0).any(1)
    q = torch.softmax(t.masked_fill(~some[:, None], 0.0), 1) * some[:, None]
    kl64 = torch.special.xlogy(q, q).sum(1) - (q * lpt.gather(1, ids.long().clamp(min=0))).sum(1)
    want = -(a.double() * has * lp.gather(1, target.long().clamp(min=0)[:, None])[:, 0]).sum() + (b.double() * kl64).sum()
    want.backward()
    # fp32 throughout: logits to (2 d + 8) u sum|h||w|, about 170 u * 80 * 0.8 / sqrt(80) < 1e-4 at worst over
    # every term, and each gradient row a sum of at most N + V such terms of weight ~ 1/N
    assert abs(loss.item() - want.item()) <= 1e-4 * abs(want.item()) + 1e-4
    assert (grad.double() - e.grad).abs().max().item() <= 1e-4 * (1 + scale) * e.grad.abs().max().item()

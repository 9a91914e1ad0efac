"""Cases that measure the vocabulary operators: the softmax cross entropy over
a large vocabulary without kept logits (rlt_op_cross_entropy), the
distillation from a teacher's top logits (rlt_op_distill) and the embedding
lookup with its gradient by sorted tokens (rlt_op_embed).

Sizes are those of the workloads in synth (d = 64, 512, 2048; V = 256, 32000;
batches of 16, 128, 256 sequences of up to 1,024 tokens; top-k 50 at
temperature 0.8) and generic odd ones.  `own` selects the library's kernels;
otherwise the plain form runs in elementary fp32 torch operations.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # log-probability of one token under the current weights: a single sequence being scored
        {"name": "ce score one token", "op": "ce", "N": 1, "V": 32000, "d": 2048, "dtype": "bf16", "backward": False, "ignored": 0.0},
        # one decode batch of the reference-depth workload scored at once
        {"name": "ce score decode batch", "op": "ce", "N": 128, "V": 32000, "d": 2048, "dtype": "bf16", "backward": False, "ignored": 0.0},
        # a training step of the tiny fp32 workload: 2 sequences of 32 tokens
        {"name": "ce train tiny fp32", "op": "ce", "N": 62, "V": 256, "d": 64, "dtype": "f32", "backward": True, "ignored": 0.0},
        # a micro-batch of replay training: 16 sequences of 1,024 tokens, prompts without a target
        {"name": "ce train replay", "op": "ce", "N": 16368, "V": 32000, "d": 2048, "dtype": "bf16", "backward": True, "ignored": 0.3},
        # full-precision training at the small width
        {"name": "ce train small fp32", "op": "ce", "N": 4088, "V": 32000, "d": 512, "dtype": "f32", "backward": True, "ignored": 0.0},
        # a ragged batch of spans, odd vocabulary, most rows user or tool tokens
        {"name": "ce train ragged", "op": "ce", "N": 1333, "V": 32003, "d": 1000, "dtype": "bf16", "backward": True, "ignored": 0.6},
        # KL of one decode batch to the behaviour sampler's candidates
        {"name": "kl decode batch", "op": "kl", "N": 128, "V": 32000, "d": 2048, "dtype": "bf16", "backward": False, "K": 50, "T": 0.8, "ignored": 0.0},
        # policy distillation over 8 sequences of 1,024 tokens from recorded top-50 logits
        {"name": "kl train replay", "op": "kl", "N": 8184, "V": 32000, "d": 2048, "dtype": "bf16", "backward": True, "K": 50, "T": 0.8, "ignored": 0.1},
        # full precision, the widest teacher list, a softened temperature
        {"name": "kl train wide list fp32", "op": "kl", "N": 501, "V": 32000, "d": 512, "dtype": "f32", "backward": True, "K": 256, "T": 2.0, "ignored": 0.1},
        # the embedding rows of one decode step
        {"name": "embed decode batch", "op": "embed", "N": 128, "V": 32000, "d": 2048, "dtype": "bf16", "out": "f32", "grad": "f32", "backward": False, "ignored": 0.0},
        # 64 sequences of 1,024 Zipf tokens, the bf16 residual stream
        {"name": "embed train replay", "op": "embed", "N": 65536, "V": 32000, "d": 2048, "dtype": "bf16", "out": "bf16", "grad": "bf16", "backward": True, "ignored": 0.0},
        # fp32 stream and gradient, spans of odd lengths, padded rows
        {"name": "embed train small fp32", "op": "embed", "N": 8191, "V": 32000, "d": 512, "dtype": "f32", "out": "f32", "grad": "f32", "backward": True, "ignored": 0.1},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ce", "ce", "kl", "embed"])
    backward = rng.random() < 0.7
    dtype = rng.choice(["bf16", "bf16", "f32"])
    V = _log_int(rng, 200, 64000)
    if rng.random() < 0.5:  # widths that tiles like, and any others
        d = 64 * _log_int(rng, 1, 40)
    else:
        d = _log_int(rng, 17, 2560)
    ignored = rng.choice([0.0, 0.1, 0.6])
    if op == "embed":
        N = _log_int(rng, 1, 65536)
        out = rng.choice(["f32", "bf16"])
        N = max(1, min(N, int(65536 * 2048 / d)))
        return {"op": op, "N": N, "V": min(V, int(32000 * 2048 / d)), "d": d, "dtype": dtype, "out": out,
                "grad": rng.choice(["f32", "bf16"]), "backward": backward, "ignored": ignored}
    N = _log_int(rng, 1, 16384)
    top = 16368 * 32000 * 2048 * (1.0 if dtype == "bf16" else 0.25)
    N = max(1, min(N, int(top / (V * d))))
    case = {"op": op, "N": N, "V": V, "d": d, "dtype": dtype, "backward": backward, "ignored": ignored}
    if op == "kl":
        case["K"] = _log_int(rng, 1, 256)
        case["T"] = rng.choice([0.8, 1.0, 2.0])
    return case


def _tokens(g, N, V):
    """Zipf(1.1) ids, as the synthetic workloads draw them."""
    r = torch.arange(1, V + 1, dtype=torch.float64, device="cuda")
    cdf = torch.cumsum(r ** -1.1, 0)
    u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64) * cdf[-1]
    return torch.searchsorted(cdf, u).clamp_(max=V - 1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    N, V, d, t = case["N"], case["V"], case["d"], TYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    tok = _tokens(g, N, V)
    skip = torch.rand(N, generator=g, device="cuda") < case["ignored"]
    s = {"case": case, "backward": case["backward"]}
    if case["op"] == "embed":
        s["emb"] = (0.02 * randn(V, d)).to(t)
        s["tokens"] = torch.where(skip, torch.full_like(tok, -1), tok)
        s["scale"] = math.sqrt(d)
        s["out"], s["grad"] = TYPES[case["out"]], TYPES[case["grad"]]
        if case["backward"]:
            s["dout"] = randn(N, d).to(s["out"])
        return s
    # a readout after its norm: unit rows, logits of spread 1 to 3, and a lean
    # towards the target that differs from row to row
    w = 0.9 / math.sqrt(d) * randn(V, d)
    h = randn(N, d) * (1 + 2 * torch.rand(N, 1, generator=g, device="cuda"))
    lean = 10 * torch.rand(N, 1, generator=g, device="cuda")
    wt = w[tok.long()]
    h = h + lean * wt / (wt.square().sum(1, keepdim=True) + 1e-3)
    s["h"], s["w"] = h.to(t), w.to(t)
    a = torch.rand(N, generator=g, device="cuda") + 0.5
    s["weight"] = torch.where(skip, torch.zeros_like(a), a / N)
    if case["op"] == "ce":
        s["target"] = torch.where(skip, torch.full_like(tok, -1), tok)
        return s
    K = case["K"]
    # a teacher's list: the token, then distinct-ish others, logits falling; a
    # skipped row is empty and some lists are shorter than K
    ids = torch.randint(0, V, (N, K), generator=g, device="cuda", dtype=torch.int32)
    ids[:, 0] = tok
    t_logits = 4 - 3 * torch.log1p(torch.arange(K, device="cuda", dtype=torch.float32)) + 0.5 * randn(N, K)
    kept = torch.randint((K + 1) // 2, K + 1, (N, 1), generator=g, device="cuda")
    empty = (torch.arange(K, device="cuda")[None, :] >= kept) | skip[:, None]
    s["ids"] = torch.where(empty, torch.full_like(ids, -1), ids)
    s["teacher"], s["T"] = t_logits.contiguous(), case["T"]
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        import stateful_decoder_b200 as rlt
        if op == "ce":
            h, w = s["h"], s["w"]
            N = h.shape[0]
            logp = torch.empty(N, device="cuda")
            lse = torch.empty(N, device="cuda")
            rlt.rlt_op_cross_entropy(h, w, s["target"], logp, lse)
            if not s["backward"]:
                return {"logp": logp, "lse": lse}
            dh, dw = torch.empty_like(h), torch.empty_like(w)
            rlt.rlt_op_cross_entropy_backward(h, w, s["target"], lse, s["weight"], dh=dh, dw=dw)
            return {"logp": logp, "lse": lse, "dh": dh, "dw": dw}
        if op == "kl":
            h, w = s["h"], s["w"]
            N = h.shape[0]
            kl = torch.empty(N, device="cuda")
            lse = torch.empty(N, device="cuda")
            rlt.rlt_op_distill(h, w, s["ids"], s["teacher"], s["T"], kl, lse)
            if not s["backward"]:
                return {"kl": kl, "lse": lse}
            dh, dw = torch.empty_like(h), torch.empty_like(w)
            rlt.rlt_op_distill_backward(h, w, s["ids"], s["teacher"], s["T"], lse, s["weight"], dh=dh, dw=dw)
            return {"kl": kl, "lse": lse, "dh": dh, "dw": dw}
        emb, tok = s["emb"], s["tokens"]
        out = torch.empty(tok.shape[0], emb.shape[1], dtype=s["out"], device="cuda")
        rlt.rlt_op_embed(emb, tok, out, scale=s["scale"])
        if not s["backward"]:
            return {"out": out}
        demb = torch.empty(emb.shape, dtype=s["grad"], device="cuda")
        rlt.rlt_op_embed_backward(s["dout"], tok, demb, scale=s["scale"])
        return {"out": out, "demb": demb}
    if op == "ce":
        return _plain_ce(s)
    if op == "kl":
        return _plain_kl(s)
    return _plain_embed(s)


def _plain_ce(s):
    h, w, target = s["h"].float(), s["w"].float(), s["target"].long()
    valid = target >= 0
    y = target.clamp(min=0)[:, None]
    z = h @ w.t()
    m = z.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
    none = torch.zeros_like(lse[:, 0])
    out = {"logp": torch.where(valid, (z.gather(1, y) - lse)[:, 0], none), "lse": torch.where(valid, lse[:, 0], none)}
    if not s["backward"]:
        return out
    a = torch.where(valid, s["weight"], none)[:, None]
    gz = torch.exp(z - lse) * a
    gz.scatter_add_(1, y, -a)
    return {**out, "dh": (gz @ w).to(s["h"].dtype), "dw": (gz.t() @ h).to(s["w"].dtype)}


def _plain_kl(s):
    h, w, T = s["h"].float(), s["w"].float(), s["T"]
    full = s["ids"] >= 0
    ids = s["ids"].long().clamp(min=0)
    t = torch.where(full, s["teacher"] / T, torch.full_like(s["teacher"], -math.inf))
    some = full.any(1, keepdim=True)
    mt = torch.where(some, t.amax(1, keepdim=True), torch.zeros_like(t[:, :1]))
    e = torch.exp(t - mt)
    se = torch.where(some, e.sum(1, keepdim=True), torch.ones_like(mt))
    q = e / se
    logq = torch.where(full, t - mt - torch.log(se), torch.zeros_like(t))
    z = (h @ w.t()) / T
    m = z.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
    none = torch.zeros_like(lse[:, 0])
    out = {"kl": (q * (logq - (z.gather(1, ids) - lse))).sum(1), "lse": torch.where(some[:, 0], lse[:, 0], none)}
    if not s["backward"]:
        return out
    a = torch.where(some[:, 0], s["weight"], none)[:, None] / T
    gz = torch.exp(z - lse) * a
    gz.scatter_add_(1, ids, -a * q)
    return {**out, "dh": (gz @ w).to(s["h"].dtype), "dw": (gz.t() @ h).to(s["w"].dtype)}


def _plain_embed(s):
    emb, tok = s["emb"], s["tokens"].long()
    ok = (tok >= 0)[:, None]
    at = tok.clamp(min=0)
    out = torch.where(ok, emb[at].float() * s["scale"], torch.zeros((), device="cuda")).to(s["out"])
    if not s["backward"]:
        return {"out": out}
    g = torch.where(ok, s["dout"].float() * s["scale"], torch.zeros((), device="cuda"))
    demb = torch.zeros(emb.shape, device="cuda").index_add_(0, at, g)
    return {"out": out, "demb": demb.to(s["grad"])}


def work(case):
    N, V, d = case["N"], case["V"], case["d"]
    size = {"bf16": 2, "f32": 4}
    e = size[case["dtype"]]
    if case["op"] == "embed":
        o, gr = size[case["out"]], size[case["grad"]]
        b = N * d * (e + o) + 4 * N
        if case["backward"]:
            b += N * d * o + V * d * gr
        return {"bytes": b, "flops": N * d * (2 if case["backward"] else 1)}
    M = max(1, int(N * (1 - case["ignored"])))  # rows with a target: the others need no logits
    b = (M + V) * d * e + 12 * N
    f = 2 * M * V * d
    if case["op"] == "kl":
        b += 8 * N * case["K"]
    if case["backward"]:
        b += (N + V) * d * e + 4 * N  # dh and dw whole
        f *= 3
    return {"bytes": b, "flops": f}


def exact(case, seed):
    """The operators' definitions in 64 bits, over blocks of token rows."""
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "embed":
        ok = s["tokens"] >= 0
        rows = s["tokens"][ok].long()
        out = torch.zeros(case["N"], case["d"], dtype=f64, device="cuda")
        out[ok] = s["emb"].to(f64)[rows] * s["scale"]
        if not case["backward"]:
            return {"out": out}
        order = torch.argsort(rows, stable=True)
        uniq, counts = torch.unique_consecutive(rows[order], return_counts=True)
        sums = torch.segment_reduce(s["dout"][ok][order].to(f64), "sum", lengths=counts, axis=0)
        demb = torch.zeros(case["V"], case["d"], dtype=f64, device="cuda")
        demb[uniq] = sums * s["scale"]
        return {"out": out, "demb": demb}
    W = s["w"].to(f64)
    loss, lses, dhs = [], [], []
    dw = torch.zeros_like(W)
    for i in range(0, case["N"], 2048):
        h = s["h"][i:i + 2048].to(f64)
        z = torch.mm(h, W.T)
        n = torch.arange(h.shape[0], device="cuda")
        # the distribution the loss compares with, dense over the vocabulary
        want = torch.zeros_like(z)
        if case["op"] == "ce":
            y = s["target"][i:i + 2048].long()
            has = y >= 0
            want[n[has], y[has]] = 1.0
        else:
            z = z / case["T"]
            ids = s["ids"][i:i + 2048].long()
            t = s["teacher"][i:i + 2048].to(f64) / case["T"]
            has = (ids >= 0).any(1)
            q = torch.softmax(t.masked_fill(ids < 0, -math.inf), 1)
            q = torch.where(has[:, None], q, torch.zeros_like(q))
            want.index_put_((n[:, None].expand_as(ids)[ids >= 0], ids[ids >= 0]), q[ids >= 0], accumulate=True)
        lse = torch.logsumexp(z, 1)
        lp = z - lse[:, None]
        lses.append(torch.where(has, lse, torch.zeros_like(lse)))  # a row without a target has none
        if case["op"] == "ce":
            loss.append((want * lp).sum(1))
        else:
            loss.append(torch.special.xlogy(q, q).sum(1) - (want * lp).sum(1))
        if case["backward"]:
            c = s["weight"][i:i + 2048].to(f64) * has
            if case["op"] == "kl":
                c = c / case["T"]
            dz = (lp.exp() - want) * c[:, None]
            dhs.append(dz @ W)
            dw += dz.T @ h
    first = "logp" if case["op"] == "ce" else "kl"
    r = {first: torch.cat(loss), "lse": torch.cat(lses)}
    if case["backward"]:
        r["dh"], r["dw"] = torch.cat(dhs), dw
    return r

"""Routing with its gradient, 8-bit integer products and the weighted sum of a
token's routes, as measurable cases.

* ``route``, ``route_bwd`` -- experts by sigmoid or softmax scores, a balance
  bias, groups, top-k and (optionally) renormalised weights; the gradient of
  the weights by the logits.
* ``linear``, ``gmm`` -- products of 8-bit integers with one scale per row and
  output channel from 16-bit activations: quantised row by row, then
  multiplied, dense or grouped by expert over a routing plan, with the
  epilogue (bias, activation, residual).
* ``combine``, ``combine_bwd`` -- the routes' rows weighted and added up per
  token, and its gradient by the rows and by the weights.

``run`` computes them in plain torch operations where ``own`` is false and by
the library's entry points where it is true; ``exact`` computes them from the
definition in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("none", "silu", "gelu", "swiglu")


# ------------------------------------------------------------------ cases --

def _route(name, op, dtype, M, E, top_k, score, renorm, bias=False, n_group=1, topk_group=1, group_top=2,
           scale=1.0, shared=0, masked=0.0):
    return {"name": name, "op": op, "dtype": dtype, "M": M, "E": E, "top_k": top_k, "score": score,
            "renorm": renorm, "bias": bias, "n_group": n_group, "topk_group": topk_group,
            "group_top": group_top, "scale": scale, "shared": shared, "masked": masked}


def _lin(name, dtype, M, K, N, act, bias, residual):
    return {"name": name, "op": "linear", "dtype": dtype, "M": M, "K": K, "N": N, "act": act, "bias": bias,
            "residual": residual}


def _gmm(name, dtype, M, E, K, N, top_k, block_m, act, per_route=False, shards=1):
    return {"name": name, "op": "gmm", "dtype": dtype, "M": M, "E": E, "K": K, "N": N, "top_k": top_k,
            "block_m": block_m, "act": act, "per_route": per_route, "shards": shards}


def _comb(name, op, dtype, M, K, top_k, residual=True, masked=0.0):
    return {"name": name, "op": op, "dtype": dtype, "M": M, "K": K, "top_k": top_k, "residual": residual,
            "masked": masked}


def listed():
    return [
        # a decode batch of 16 behind 256 routed experts and a shared one: pure latency
        _route("route_decode", "route", "f32", 16, 256, 8, "sigmoid", True, bias=True, n_group=8,
               topk_group=4, scale=2.5, shared=1),
        # a long prefill behind the page-1 geometry's experts
        _route("route_prefill", "route", "bf16", 8192, 288, 8, "softmax", True, bias=True),
        # a training step's gradient: softmax scores as they are, every logit has one
        _route("route_bwd_dense", "route_bwd", "bf16", 2048, 512, 10, "softmax", False),
        # a training step over long sequences with grouped, renormalised sigmoid scores
        _route("route_bwd_long", "route_bwd", "f32", 16384, 256, 8, "sigmoid", True, bias=True, n_group=8,
               topk_group=4, scale=2.5, shared=1),
        # a shared expert's gate/up for a decode batch
        _lin("linear_batch", "f16", 48, 4096, 2048, "swiglu", False, False),
        # odd rows and columns
        _lin("linear_odd", "bf16", 1000, 2048, 1001, "gelu", True, True),
        # a dense projection over a long prefill
        _lin("linear_large", "bf16", 8192, 7168, 4096, "silu", True, True),
        # four decoded tokens: the touched experts' gate/up weights streamed once
        _gmm("gmm_decode", "bf16", 4, 257, 7168, 512, 9, 16, "swiglu"),
        # the page-1 geometry's gate/up over a long prefill (largest)
        _gmm("gmm_page1", "bf16", 8192, 288, 4096, 2048, 8, 128, "swiglu"),
        # the page-1 geometry's routes, after the down product
        _comb("combine_page1", "combine", "bf16", 4096, 4096, 8),
        # the tiny workload: the smallest gradient
        _comb("combine_bwd_tiny", "combine_bwd", "f16", 4, 256, 2),
        # a training step over the skewed batch, with masked routes
        _comb("combine_bwd_skew", "combine_bwd", "bf16", 2048, 2048, 10, masked=0.01),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "route_bwd", "linear", "linear", "gmm", "gmm", "combine", "combine_bwd"))
    dtype = rng.choice(("bf16", "f16"))
    if op in ("route", "route_bwd"):
        n_group = rng.choice((1, 1, 2, 4, 8))
        per = _log_int(rng, 8, 512 // n_group)
        topk_group = rng.randint(1, n_group)
        score = rng.choice(("sigmoid", "softmax"))
        c = _route("", op, rng.choice(("f32", dtype)), _log_int(rng, 1, 16384), per * n_group,
                   rng.randint(1, min(16, per * topk_group)), score, rng.random() < 0.6,
                   rng.random() < 0.6, n_group, topk_group, rng.choice((1, 2)), rng.choice((1.0, 2.5)),
                   rng.choice((0, 1)), rng.choice((0.0, 0.0, 0.1)))
    elif op == "linear":
        while True:
            act = rng.choice(ACTS)
            K, N, M = 16 * _log_int(rng, 16, 448), _log_int(rng, 64, 8192), _log_int(rng, 1, 8192)
            N += N % 2 if act == "swiglu" else 0
            if M * K * N <= 8192 * 7168 * 4096:
                break
        c = _lin("", dtype, M, K, N, act, rng.random() < 0.5, rng.random() < 0.5)
    elif op == "gmm":
        while True:
            E = _log_int(rng, 1, 512)
            top_k = min(E, rng.randint(1, 10))
            K, N, M = 16 * _log_int(rng, 16, 448), 8 * _log_int(rng, 16, 512), _log_int(rng, 1, 8192)
            if M * top_k * K * N <= 8192 * 8 * 4096 * 2048 and E * K * N <= 288 * 4096 * 2048 // 2:
                break
        c = _gmm("", dtype, M, E, K, N, top_k, rng.choice((8, 16, 32, 64, 128)), rng.choice(ACTS),
                 rng.random() < 0.4, rng.choice((1, 1, 2, 4)))
    else:
        c = _comb("", op, dtype, _log_int(rng, 1, 4096), 8 * _log_int(rng, 16, 896), rng.randint(1, 10),
                  rng.random() < 0.5, rng.choice((0.0, 0.01, 0.5)))
        c["M"] = min(c["M"], 4096 * 4096 * 8 // (c["K"] * c["top_k"]))
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs --

def _gen(seed, kind):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1_000_003 + kind)
    return g


def _route_inputs(case, seed):
    g = _gen(seed, 1)
    M, E, k = case["M"], case["E"], case["top_k"]
    l = torch.randn((M, E), generator=g, device=DEV) * 1.5
    if case["masked"] > 0:                       # experts that are out of service
        l[:, torch.rand(E, generator=g, device=DEV) < case["masked"]] = -math.inf
    s = {"logits": l.to(DTYPES[case["dtype"]])}
    s["bias"] = torch.randn(E, generator=g, device=DEV) * 0.02 if case["bias"] else None
    if case["op"] == "route_bwd":
        ids, _ = _plain_route(case, s["logits"], s["bias"])
        s["ids"] = ids
        s["d_weights"] = torch.randn(ids.shape, generator=g, device=DEV)
    return s


def _lin_inputs(case, seed):
    M, K, N = case["M"], case["K"], case["N"]
    dt = DTYPES[case["dtype"]]
    g = _gen(seed, 2)
    s = {"x": torch.randn((M, K), generator=g, device=DEV).to(dt)}
    s["w"] = (torch.randn((N, K), generator=g, device=DEV) * 32).round_().clamp_(-127, 127).to(torch.int8)
    s["ws"] = torch.exp(torch.randn(N, generator=g, device=DEV) * 0.2) * 6e-4
    s["bias"] = torch.randn(N, generator=g, device=DEV) * 0.5 if case["bias"] else None
    n_out = N // 2 if case["act"] == "swiglu" else N
    s["residual"] = torch.randn((M, n_out), generator=g, device=DEV).to(dt) if case["residual"] else None
    return s


def _gmm_inputs(case, seed):
    M, E, K, N, k = case["M"], case["E"], case["K"], case["N"], case["top_k"]
    g = _gen(seed, 3)
    # ids of other ranks' experts lie outside [0, E): masked here
    ids = torch.topk(torch.randn((M, E * case["shards"]), generator=g, device=DEV), k, dim=1).indices
    rows = M * k if case["per_route"] else M
    s = {"ids": ids, "x": torch.randn((rows, K), generator=g, device=DEV).to(DTYPES[case["dtype"]])}
    w = torch.empty((E, N, K), dtype=torch.int8, device=DEV)
    for e in range(E):
        w[e] = (torch.randn((N, K), generator=g, device=DEV) * 32).round_().clamp_(-127, 127).to(torch.int8)
    s["w"] = w
    s["ws"] = torch.exp(torch.randn((E, N), generator=g, device=DEV) * 0.2) * 6e-4
    return s


def _comb_inputs(case, seed):
    M, K, k = case["M"], case["K"], case["top_k"]
    dt = DTYPES[case["dtype"]]
    g = _gen(seed, 4)
    s = {"y": torch.randn((M * k, K), generator=g, device=DEV).to(dt)}
    s["weights"] = torch.softmax(torch.randn((M, k), generator=g, device=DEV), dim=1)
    ids = torch.randint(0, 64, (M, k), generator=g, device=DEV, dtype=torch.int32)
    s["ids"] = torch.where(torch.rand((M, k), generator=g, device=DEV) < case["masked"], -1, ids).to(torch.int32)
    x = torch.randn((M, K), generator=g, device=DEV).to(dt)
    if case["op"] == "combine_bwd":
        s["dout"] = x
    else:
        s["residual"] = x if case["residual"] else None
    return s


def _plan(ids, E, block_m):
    """The routing plan of these ids: routes grouped by expert, each expert's
    segment padded with the sentinel R to a multiple of block_m."""
    flat = ids.reshape(-1)
    R = flat.numel()
    cap = (R + min(E, R) * (block_m - 1) + block_m - 1) // block_m * block_m
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    padded = (counts + block_m - 1) // block_m * block_m
    start = torch.cumsum(padded, 0) - padded
    first = torch.cumsum(counts, 0) - counts
    nv = int(counts.sum())
    routes = order[:nv]
    e = key[routes]
    srt = torch.full((cap,), R, dtype=torch.int32, device=DEV)
    srt[start[e] + torch.arange(nv, device=DEV) - first[e]] = routes.to(torch.int32)
    blocks = torch.repeat_interleave(torch.arange(E, device=DEV), padded // block_m)
    eids = torch.zeros(cap // block_m, dtype=torch.int32, device=DEV)
    eids[:blocks.numel()] = blocks.to(torch.int32)
    segments = [(i, s, n) for i, (s, n) in enumerate(zip(start.tolist(), counts.tolist())) if n > 0]
    return srt, eids, padded.sum().to(torch.int32).reshape(1), segments


def prepare(case, seed):
    op, st = case["op"], {"case": dict(case)}
    M, k = case["M"], case.get("top_k", 1)
    dt = DTYPES[case["dtype"]]
    if op in ("route", "route_bwd"):
        st.update(_route_inputs(case, seed))
        kk = k + case["shared"]
        if op == "route":
            st["topk_ids"] = torch.zeros((M, kk), dtype=torch.int32, device=DEV)
            st["topk_weights"] = torch.zeros((M, kk), dtype=torch.float32, device=DEV)
        else:
            st["d_logits"] = torch.zeros((M, case["E"]), dtype=dt, device=DEV)
        return st
    if op in ("combine", "combine_bwd"):
        st.update(_comb_inputs(case, seed))
        if op == "combine":
            st["out"] = torch.zeros((M, case["K"]), dtype=dt, device=DEV)
        else:
            # rows of masked routes are left as they were: zero from here on
            st["dy"] = torch.zeros((M * k, case["K"]), dtype=dt, device=DEV)
            st["d_weights"] = torch.zeros((M, k), dtype=torch.float32, device=DEV)
        return st
    n_out = case["N"] // 2 if case["act"] == "swiglu" else case["N"]
    if op == "linear":
        st.update(_lin_inputs(case, seed))
        st["out"] = torch.zeros((M, n_out), dtype=dt, device=DEV)
    else:
        st.update(_gmm_inputs(case, seed))
        st["srt"], st["eids"], st["ntp"], st["segments"] = _plan(st["ids"], case["E"], case["block_m"])
        st["out"] = torch.zeros((M * k, n_out), dtype=dt, device=DEV)
    st["x_q"] = torch.zeros(st["x"].shape, dtype=torch.int8, device=DEV)
    st["x_s"] = torch.zeros(st["x"].shape[0], dtype=torch.float32, device=DEV)
    if own:
        import fp8_block_scale_amd as moe
        act = _act(moe, case["act"])
        if op == "linear":
            n = moe.moe_i8_linear_workspace_size(M, case["N"], case["K"], act)
        else:
            n = moe.moe_i8_group_mm_workspace_size(M, case["K"], case["N"], case["E"], k, case["block_m"],
                                                   st["srt"].numel(), act, x_per_route=case["per_route"])
        st["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    return st


def _act(moe, act):
    return {"none": moe.MOE_ACT_NONE, "silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU,
            "swiglu": moe.MOE_ACT_SWIGLU}[act]


# -------------------------------------------------------------------- run --

def run(st):
    c = st["case"]
    if own:
        return _run_own(st, c)
    op = c["op"]
    if op == "route":
        return _plain_route(c, st["logits"], st["bias"])
    if op == "route_bwd":
        return _plain_route_bwd(c, st["logits"], st["ids"], st["d_weights"])
    if op == "combine":
        return _plain_combine(st, c)
    if op == "combine_bwd":
        return _plain_combine_bwd(st, c)
    return _plain_linear(st, c) if op == "linear" else _plain_gmm(st, c)


def _run_own(st, c):
    import fp8_block_scale_amd as moe
    op = c["op"]
    if op in ("route", "route_bwd"):
        score = moe.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX
        if op == "route_bwd":
            moe.moe_route_scored_bwd(st["logits"], st["ids"], st["d_weights"], st["d_logits"], score,
                                     renorm=c["renorm"], routed_scaling=c["scale"])
            return st["d_logits"]
        moe.moe_route_scored(st["logits"], c["top_k"], st["topk_ids"], st["topk_weights"], score,
                             bias=st["bias"], n_group=c["n_group"], topk_group=c["topk_group"],
                             group_top=c["group_top"], renorm=c["renorm"], routed_scaling=c["scale"],
                             n_shared=c["shared"])
        return st["topk_ids"], st["topk_weights"]
    if op == "combine":
        moe.moe_combine(st["y"], st["weights"], st["out"], topk_ids=st["ids"], E=64,
                        residual=st["residual"])
        return st["out"]
    if op == "combine_bwd":
        moe.moe_combine_bwd(st["dout"], st["y"], st["weights"], st["dy"], st["d_weights"],
                            topk_ids=st["ids"], E=64)
        return st["dy"], st["d_weights"]
    moe.moe_quant_i8(st["x"], st["x_q"], st["x_s"])
    if op == "linear":
        moe.moe_i8_linear(st["x_q"], st["x_s"], st["w"], st["ws"], st["out"], bias=st["bias"],
                          residual=st["residual"], act=_act(moe, c["act"]), workspace=st["workspace"])
    else:
        moe.moe_i8_group_mm(st["x_q"], st["x_s"], st["w"], st["ws"], st["srt"], st["eids"], st["ntp"],
                            c["top_k"], c["block_m"], st["out"], act=_act(moe, c["act"]),
                            workspace=st["workspace"], x_per_route=c["per_route"])
    return st["out"]


def _scores(l, score):
    """Scores of logits in 64 bits; 0 for those of -infinity."""
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(dim=1, keepdim=True).clamp_min(-1e300))
    return e / e.sum(dim=1, keepdim=True).clamp_min(1e-300)


def _plain_route(c, logits, bias):
    M, E, k, G = c["M"], c["E"], c["top_k"], c["n_group"]
    l = logits.double()                          # values next to each other decide who is chosen
    s = _scores(l, c["score"])
    choice = s if bias is None else s + bias.double()
    choice = torch.where(l == -math.inf, -math.inf, choice)
    if c["topk_group"] < G:
        best = torch.sort(choice.view(M, G, E // G), dim=2, descending=True).values[..., :c["group_top"]]
        there = best > -math.inf
        score = torch.where(there, best, 0.0).sum(dim=2)
        score = torch.where(there.any(dim=2), score, -math.inf)
        first = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros((M, G), dtype=torch.bool, device=DEV).scatter_(1, first, True)
        choice = torch.where(keep.repeat_interleave(E // G, dim=1), choice, -math.inf)
    top, ids = torch.sort(choice, dim=1, descending=True, stable=True)
    ids, there = ids[:, :k], top[:, :k] > -math.inf
    w = torch.where(there, torch.gather(s, 1, ids), 0.0)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp_min(1e-300)
    w = (w * c["scale"]).float()
    ids = torch.where(there, ids, -1).to(torch.int32)
    if c["shared"]:
        ids = torch.cat([ids, torch.full((M, 1), E, dtype=torch.int32, device=DEV)], dim=1)
        w = torch.cat([w, torch.ones((M, 1), device=DEV)], dim=1)
    return ids, w


def _plain_route_bwd(c, logits, ids, d_weights):
    l, E = logits.float(), c["E"]
    ok = (ids >= 0) & (ids < E)
    at = torch.where(ok, ids, 0).long()
    a = torch.where(ok, d_weights * c["scale"], 0.0)
    d = torch.zeros_like(l)
    if c["score"] == "softmax" and not c["renorm"]:
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
        d.scatter_add_(1, at, a)
        d = p * (d - (d * p).sum(dim=1, keepdim=True))
        return d.to(logits.dtype)
    z = torch.gather(l, 1, at)
    if c["score"] == "softmax":
        z = torch.where(ok, z, -math.inf)
        p = torch.where(ok, torch.exp(z - z.amax(dim=1, keepdim=True).clamp_min(-1e30)), 0.0)
        p = p / p.sum(dim=1, keepdim=True).clamp_min(1e-30)
        v = p * (a - (a * p).sum(dim=1, keepdim=True))
    else:
        s = torch.where(ok, 1.0 / (1.0 + torch.exp(-z)), 0.0)
        rest = 1.0 / (1.0 + torch.exp(z))
        if c["renorm"]:
            total = s.sum(dim=1, keepdim=True).clamp_min(1e-30)
            a = (a - (a * s).sum(dim=1, keepdim=True) / total) / total
        v = s * rest * a
    return d.scatter_add_(1, at, torch.where(ok, v, 0.0)).to(logits.dtype)


def _plain_quant(x):
    f = x.float()
    s = (f.abs().amax(dim=1) / 127.0).clamp_min(2.0 ** -126)
    return torch.round(f * (1.0 / s)[:, None]), s


def _plain_act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "swiglu":
        g, u = z[:, :z.shape[1] // 2], z[:, z.shape[1] // 2:]
        return g / (1.0 + torch.exp(-g)) * u
    return z


def _plain_linear(st, c):
    q, s = _plain_quant(st["x"])
    z = (q @ st["w"].float().t()) * s[:, None] * st["ws"]
    if st["bias"] is not None:
        z = z + st["bias"]
    z = _plain_act(z, c["act"])
    if st["residual"] is not None:
        z = z + st["residual"].float()
    st["out"].copy_(z)
    return st["out"]


def _plain_gmm(st, c):
    q, s = _plain_quant(st["x"])
    out = st["out"]
    for e, start, n in st["segments"]:
        rows = st["srt"][start:start + n].long()
        src = rows if c["per_route"] else rows // c["top_k"]
        z = (q[src] @ st["w"][e].float().t()) * s[src][:, None] * st["ws"][e]
        out[rows] = _plain_act(z, c["act"]).to(out.dtype)
    return out


def _plain_combine(st, c):
    M, K, k = c["M"], c["K"], c["top_k"]
    w = torch.where(st["ids"] >= 0, st["weights"], 0.0)
    z = (st["y"].view(M, k, K).float() * w[..., None]).sum(dim=1)
    if st["residual"] is not None:
        z = z + st["residual"].float()
    st["out"].copy_(z)
    return st["out"]


def _plain_combine_bwd(st, c):
    M, K, k = c["M"], c["K"], c["top_k"]
    ok = st["ids"] >= 0
    g = st["dout"].float()[:, None, :]
    dy = (st["weights"][..., None] * g).to(st["dy"].dtype)
    st["dy"].copy_(torch.where(ok[..., None], dy, st["dy"].view(M, k, K)).view(M * k, K))
    dw = (st["y"].view(M, k, K).float() * g).sum(dim=2)
    st["d_weights"].copy_(torch.where(ok, dw, 0.0))
    return st["dy"], st["d_weights"]


# ------------------------------------------------------------------- work --

def work(case):
    op, M, k = case["op"], case["M"], case.get("top_k", 1)
    size = 4 if case["dtype"] == "f32" else 2
    if op in ("route", "route_bwd"):
        E, kk = case["E"], k + case["shared"]
        dense = op == "route" or (case["score"] == "softmax" and not case["renorm"])
        read = M * E if dense else M * k          # logits that matter
        nbytes = read * size + 8 * M * kk + (4 * E if case["bias"] and op == "route" else 0)
        if op == "route_bwd":
            nbytes += M * E * size
        return {"bytes": nbytes, "flops": 4 * read}
    if op in ("combine", "combine_bwd"):
        R, K = M * k * (1.0 - case["masked"]), case["K"]
        if op == "combine":
            nbytes = 2 * K * (R + M * (2 if case["residual"] else 1)) + 8 * M * k
            return {"bytes": int(nbytes), "flops": int(2 * R * K)}
        return {"bytes": int(2 * K * (2 * R + M) + 12 * M * k), "flops": int(3 * R * K)}
    K, N = case["K"], case["N"]
    n_out = N // 2 if case["act"] == "swiglu" else N
    if op == "linear":
        nbytes = 2 * M * K + N * K + 4 * N * (2 if case["bias"] else 1)
        nbytes += 2 * M * n_out * (2 if case["residual"] else 1)
        return {"bytes": nbytes, "flops": 2 * M * K * N}
    E, shards = case["E"], case["shards"]
    R = M * k / shards
    p = min(1.0, k / (E * shards))
    hit = E * -math.expm1(M * math.log1p(-p)) if p < 1 else E
    rows = R if case["per_route"] else M * (1.0 - (1.0 - 1.0 / shards) ** k)
    nbytes = 2 * rows * K + hit * N * (K + 4) + 2 * R * n_out + 4 * R
    return {"bytes": int(nbytes), "flops": int(2 * R * K * N)}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    op = case["op"]
    if op == "route":
        return _exact_route(case, _route_inputs(case, seed))
    if op == "route_bwd":
        return _exact_route_bwd(case, _route_inputs(case, seed))
    if op in ("combine", "combine_bwd"):
        return _exact_combine(case, _comb_inputs(case, seed))
    if op == "linear":
        s = _lin_inputs(case, seed)
        x, xs = _exact_codes(s["x"])
        z = torch.mm(x, s["w"].double().t()) * xs * s["ws"].double()
        if s["bias"] is not None:
            z += s["bias"].double()
        z = _exact_act(z, case["act"])
        return z if s["residual"] is None else z + s["residual"].double()
    s = _gmm_inputs(case, seed)
    x, xs = _exact_codes(s["x"])
    n_out = case["N"] // 2 if case["act"] == "swiglu" else case["N"]
    res = torch.zeros((case["M"] * case["top_k"], n_out), dtype=torch.float64, device=DEV)
    flat = s["ids"].reshape(-1)
    for e in range(case["E"]):
        r = torch.nonzero(flat == e).flatten()
        if r.numel():
            t = r if case["per_route"] else torch.div(r, case["top_k"], rounding_mode="floor")
            z = torch.mm(x[t], s["w"][e].double().t()) * xs[t] * s["ws"][e].double()
            res[r] = _exact_act(z, case["act"])
    return res


def _exact_codes(x):
    """Codes and scales of rows as the quantisation rule defines them (its
    scale and reciprocal are 32-bit numbers)."""
    d = x.double()
    s = (d.abs().max(dim=1, keepdim=True).values / 127).clamp(min=2.0 ** -126).float().double()
    return torch.round(d * (1 / s).float().double()), s


def _exact_act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    if act == "swiglu":
        g, u = z.chunk(2, dim=1)
        return g * torch.sigmoid(g) * u
    return z


def _exact_route(case, s):
    """One rank at a time: the best remaining expert, until top_k are chosen."""
    l = s["logits"].double()
    M, E, G = case["M"], case["E"], case["n_group"]
    p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, dim=1).nan_to_num(0.0)
    c = p + (0 if s["bias"] is None else s["bias"].double())
    c = c.masked_fill(torch.isneginf(l), -math.inf)

    def take(v):                                 # (index of the largest, lowest first; whether there is one)
        best = v.amax(dim=1, keepdim=True)
        i = torch.where(v == best, torch.arange(v.shape[1], device=DEV), v.shape[1]).amin(dim=1, keepdim=True)
        return i, best > -math.inf

    per = E // G
    if case["topk_group"] < G:
        left, total, some = c.reshape(M * G, per).clone(), torch.zeros((M * G, 1), dtype=torch.float64, device=DEV), None
        for _ in range(min(case["group_top"], per)):
            i, there = take(left)
            total += torch.where(there, left.gather(1, i), 0.0)
            some = there if some is None else some
            left.scatter_(1, i, -math.inf)
        total = torch.where(some, total, -math.inf).view(M, G)
        open_ = torch.zeros((M, G), dtype=torch.bool, device=DEV)
        for _ in range(case["topk_group"]):
            i, there = take(total)
            open_ |= torch.zeros_like(open_).scatter_(1, i, there)
            total.scatter_(1, i, -math.inf)
        c = c.masked_fill(~open_[:, torch.arange(E, device=DEV) // per], -math.inf)
    ids, w = [], []
    for _ in range(case["top_k"]):
        i, there = take(c)
        ids.append(torch.where(there, i, -1))
        w.append(torch.where(there, p.gather(1, i), 0.0))
        c.scatter_(1, i, -math.inf)
    ids, w = torch.cat(ids, 1), torch.cat(w, 1)
    if case["renorm"]:
        w = (w / w.sum(dim=1, keepdim=True)).nan_to_num(0.0)
    w = w * case["scale"]
    if case["shared"]:
        ids = torch.cat([ids, torch.full_like(ids[:, :1], E)], 1)
        w = torch.cat([w, torch.ones_like(w[:, :1])], 1)
    return ids.to(torch.int32), w


def _exact_route_bwd(case, s):
    """By differentiating the weights' definition in 64 bits."""
    l = s["logits"].double().requires_grad_(True)
    ok = (s["ids"] >= 0) & (s["ids"] < case["E"])
    at = s["ids"].long().clamp(0, case["E"] - 1)
    if case["score"] == "sigmoid":
        w = torch.sigmoid(l).gather(1, at) * ok
        if case["renorm"]:
            w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    elif case["renorm"]:
        w = torch.softmax(l.gather(1, at).masked_fill(~ok, -1e300), dim=1) * ok
    else:
        w = torch.softmax(l, dim=1).gather(1, at) * ok
    return torch.autograd.grad((w * case["scale"] * s["d_weights"].double()).sum(), l)[0]


def _exact_combine(case, s):
    M, K, k = case["M"], case["K"], case["top_k"]
    there = s["ids"] >= 0
    w = s["weights"].double() * there
    if case["op"] == "combine":
        z = torch.zeros((M, K), dtype=torch.float64, device=DEV) if s["residual"] is None else s["residual"].double()
        for j in range(k):
            z = z + w[:, j:j + 1] * s["y"][j::k].double()
        return z
    g = s["dout"].double()
    dy = torch.zeros((M * k, K), dtype=torch.float64, device=DEV)
    dw = torch.zeros((M, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        dy[j::k] = w[:, j:j + 1] * g
        dw[:, j] = (s["y"][j::k].double() * g).sum(dim=1) * there[:, j]
    return dy, dw

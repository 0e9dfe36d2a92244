"""The matrix products beside the FP8 expert path, as measurable cases.

Two families, four operators:

* ``gmm``, ``gmm_dx``, ``gmm_dw`` -- matrix products grouped by expert, with
  ragged sizes, in BF16 or FP16 over a routing plan: the forward product
  ``y[r] = x[t(r)] w[e(r)]^T``, its gradient by the input and by the weights.
* ``linear`` -- the dense product of block-scaled FP8 codes with bias,
  activation and residual in its epilogue.

``run`` computes them in plain torch operations in 32 bits where ``own`` is
false and by the library's entry points where it is true; ``exact`` computes
them from the definition in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("none", "silu", "gelu", "swiglu")


# ------------------------------------------------------------------ cases --

def _gmm(name, op, dtype, M, E, K, N, top_k, block_m, routing, per_route=False, shards=1, out=None):
    return {"name": name, "op": op, "dtype": dtype, "M": M, "E": E, "K": K, "N": N, "top_k": top_k,
            "block_m": block_m, "routing": routing, "per_route": per_route, "shards": shards,
            "out": out or dtype}


def _lin(name, M, K, N, act, bias, residual):
    return {"name": name, "op": "linear", "dtype": "bf16", "M": M, "K": K, "N": N, "act": act,
            "bias": bias, "residual": residual}


def listed():
    return [
        # the tiny workload's gate/up product: pure latency
        _gmm("gmm_tiny", "gmm", "f16", 4, 8, 256, 512, 2, 16, "softmax"),
        # one decoded token: nine experts' gate/up weights streamed once
        _gmm("gmm_decode", "gmm", "bf16", 1, 257, 7168, 512, 9, 16, "softmax"),
        # a batch with four hot experts, long-tailed rest and 1% masked routes
        _gmm("gmm_skew", "gmm", "f16", 2048, 512, 2048, 1024, 10, 64, "skew"),
        # the page-1 geometry's gate/up product over a long prefill (largest)
        _gmm("gmm_page1", "gmm", "bf16", 8192, 288, 4096, 2048, 8, 128, "softmax"),
        # input gradient of a down product (one row per route), odd sizes
        _gmm("dx_odd", "gmm_dx", "f16", 333, 24, 712, 1288, 4, 32, "softmax", per_route=True),
        # input gradient of the gate/up product, summed over a token's routes
        _gmm("dx_page1", "gmm_dx", "bf16", 4096, 288, 4096, 2048, 8, 64, "softmax"),
        # weight gradient with few, long experts: the sum over rows is the long axis
        _gmm("dw_long", "gmm_dw", "f16", 8192, 8, 256, 512, 2, 16, "softmax", out="f32"),
        # one of eight ranks' share of the experts: most routes are masked here
        _gmm("dw_share", "gmm_dw", "bf16", 8192, 36, 4096, 2048, 8, 64, "softmax", shards=8),
        # a dense projection for one decoded token, added to the residual stream
        _lin("linear_one", 1, 7168, 4096, "none", False, True),
        # a shared expert's gate/up for a decode batch
        _lin("linear_batch", 48, 4096, 2048, "swiglu", False, False),
        # odd rows and columns
        _lin("linear_odd", 1000, 2048, 1001, "gelu", True, True),
        # a dense projection over a long prefill
        _lin("linear_large", 8192, 7168, 4096, "silu", True, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.35:
        while True:
            act = rng.choice(ACTS)
            K = 128 * _log_int(rng, 2, 56)
            N = _log_int(rng, 64, 8192)
            if act == "swiglu":
                N += N % 2
            M = _log_int(rng, 1, 8192)
            if M * K * N <= 8192 * 7168 * 4096:
                return _drop_name(_lin("", M, K, N, act, rng.random() < 0.5, rng.random() < 0.5))
    while True:
        op = rng.choice(("gmm", "gmm_dx", "gmm_dw"))
        E = _log_int(rng, 1, 512)
        top_k = min(E, rng.randint(1, 10))
        K = 8 * _log_int(rng, 16, 896)
        N = 8 * _log_int(rng, 16, 512)
        M = _log_int(rng, 1, 8192)
        dtype = rng.choice(("bf16", "f16"))
        out = "f32" if op == "gmm_dw" and rng.random() < 0.4 else dtype
        routing = "skew" if E > 8 and rng.random() < 0.3 else "softmax"
        shards = rng.choice((1, 1, 2, 4)) if routing == "softmax" else 1
        if M * top_k * K * N <= 8192 * 8 * 4096 * 2048 and E * K * N <= 288 * 4096 * 2048 // 2:
            return _drop_name(_gmm("", op, dtype, M, E, K, N, top_k, rng.choice((8, 16, 32, 64, 128)),
                                   routing, rng.random() < 0.4, shards, out))


def _drop_name(case):
    del case["name"]
    return case


# ----------------------------------------------------------------- inputs --

def _gen(seed, kind):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1_000_003 + kind)
    return g


def _routing(case, seed):
    """topk_ids [M, top_k]; ids of other ranks' experts and masked routes lie
    outside [0, E)."""
    g = _gen(seed, 1)
    M, E, k = case["M"], case["E"], case["top_k"]
    if case["routing"] == "skew":
        hot = torch.randint(0, E, (4,), generator=g, device=DEV)
        nh = k // 2
        a = hot[torch.randint(0, 4, (M, nh), generator=g, device=DEV)]
        b = torch.randint(0, E, (M, k - nh), generator=g, device=DEV)
        ids = torch.cat([a, b], dim=1)
        drop = torch.rand((M, k), generator=g, device=DEV) < 0.01
        return torch.where(drop, torch.full_like(ids, -1), ids)
    logits = torch.randn((M, E * case["shards"]), generator=g, device=DEV)
    return torch.topk(logits, k, dim=1).indices


def _plan(ids, E, block_m):
    """The routing plan of these ids: routes grouped by expert, each expert's
    segment padded with the sentinel R to a multiple of block_m."""
    flat = ids.reshape(-1)
    R = flat.numel()
    n = R + min(E, R) * (block_m - 1)
    cap = (n + block_m - 1) // block_m * block_m
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    padded = (counts + block_m - 1) // block_m * block_m
    start = torch.cumsum(padded, 0) - padded
    first = torch.cumsum(counts, 0) - counts
    nv = int(counts.sum())
    routes = order[:nv]
    e = key[routes]
    pos = start[e] + torch.arange(nv, device=DEV) - first[e]
    srt = torch.full((cap,), R, dtype=torch.int32, device=DEV)
    srt[pos] = routes.to(torch.int32)
    blocks = torch.repeat_interleave(torch.arange(E, device=DEV), padded // block_m)
    eids = torch.zeros(cap // block_m, dtype=torch.int32, device=DEV)
    eids[:blocks.numel()] = blocks.to(torch.int32)
    ntp = padded.sum().to(torch.int32).reshape(1)
    segments = list(zip(start.tolist(), counts.tolist()))
    return srt, eids, ntp, segments


def _gmm_inputs(case, seed):
    dt = DTYPES[case["dtype"]]
    M, E, K, N = case["M"], case["E"], case["K"], case["N"]
    R = M * case["top_k"]
    s = {"ids": _routing(case, seed)}
    g = _gen(seed, 2)
    rows = R if case["per_route"] else M
    if case["op"] != "gmm_dx":
        s["x"] = torch.randn((rows, K), generator=g, device=DEV).to(dt)
    if case["op"] != "gmm":
        s["dy"] = torch.randn((R, N), generator=g, device=DEV).to(dt)
    if case["op"] != "gmm_dw":
        w = torch.empty((E, N, K), dtype=dt, device=DEV)
        for e in range(E):
            w[e] = (torch.randn((N, K), generator=g, device=DEV) * 0.02).to(dt)
        s["w"] = w
    return s


def _lin_inputs(case, seed):
    M, K, N = case["M"], case["K"], case["N"]
    g = _gen(seed, 3)
    x = torch.randn((M, K // 128, 128), generator=g, device=DEV)
    xs = x.abs().amax(dim=2) / 448.0
    xq = (x / xs[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(M, K)
    nb = (N + 127) // 128
    w = torch.randn((nb, 128, K // 128, 128), generator=g, device=DEV) * 0.02
    ws = w.abs().amax(dim=(1, 3)) / 448.0
    wq = (w / ws[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s = {"xq": xq, "xs": xs, "w": wq.reshape(nb * 128, K)[:N].contiguous(), "ws": ws.contiguous()}
    n_out = N // 2 if case["act"] == "swiglu" else N
    s["bias"] = torch.randn((N,), generator=g, device=DEV) * 0.5 if case["bias"] else None
    s["residual"] = torch.randn((M, n_out), generator=g, device=DEV).to(torch.bfloat16) \
        if case["residual"] else None
    return s


def prepare(case, seed):
    st = {"case": dict(case)}
    if case["op"] == "linear":
        st.update(_lin_inputs(case, seed))
        n_out = case["N"] // 2 if case["act"] == "swiglu" else case["N"]
        st["out"] = torch.zeros((case["M"], n_out), dtype=torch.bfloat16, device=DEV)
        if own:
            import fp8_block_scale_amd as moe
            n = moe.moe_fp8_linear_workspace_size(case["M"], case["N"], case["K"], _act(moe, case["act"]))
            st["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
        return st
    st.update(_gmm_inputs(case, seed))
    M, E, K, N, k = case["M"], case["E"], case["K"], case["N"], case["top_k"]
    st["srt"], st["eids"], st["ntp"], st["segments"] = _plan(st["ids"], E, case["block_m"])
    rows = M * k if case["per_route"] else M
    shape = {"gmm": (M * k, N), "gmm_dx": (rows, K), "gmm_dw": (E, N, K)}[case["op"]]
    # rows of masked routes are left as they were: zero from here on
    st["out"] = torch.zeros(shape, dtype=DTYPES[case["out"]], device=DEV)
    if own:
        import fp8_block_scale_amd as moe
        op = {"gmm": moe.MOE_GMM_FWD, "gmm_dx": moe.MOE_GMM_DX, "gmm_dw": moe.MOE_GMM_DW}[case["op"]]
        n = moe.moe_group_mm_workspace_size(op, M, K, N, E, k, case["block_m"], st["srt"].numel(),
                                            x_per_route=case["per_route"])
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
    if c["op"] == "linear":
        return _plain_linear(st, c)
    return _plain_gmm(st, c)


def _run_own(st, c):
    import fp8_block_scale_amd as moe
    if c["op"] == "linear":
        moe.moe_fp8_linear(st["xq"], st["xs"], st["w"], st["ws"], st["out"], bias=st["bias"],
                           residual=st["residual"], act=_act(moe, c["act"]), workspace=st["workspace"])
        return st["out"]
    plan = (st["srt"], st["eids"], st["ntp"], c["top_k"], c["block_m"])
    if c["op"] == "gmm":
        moe.moe_group_mm(st["x"], st["w"], *plan, st["out"], st["workspace"],
                         x_per_route=c["per_route"])
    elif c["op"] == "gmm_dx":
        moe.moe_group_mm_dx(st["dy"], st["w"], *plan, st["out"], st["workspace"],
                            x_per_route=c["per_route"])
    else:
        moe.moe_group_mm_dw(st["dy"], st["x"], *plan, st["out"], st["workspace"],
                            x_per_route=c["per_route"])
    return st["out"]


def _plain_gmm(st, c):
    out, k = st["out"], c["top_k"]
    summed = c["op"] == "gmm_dx" and not c["per_route"]
    if summed:
        part = torch.zeros((c["M"] * k, c["K"]), dtype=torch.float32, device=DEV)
    for e, (start, n) in enumerate(st["segments"]):
        if n == 0:
            if c["op"] == "gmm_dw":
                out[e] = 0
            continue
        rows = st["srt"][start:start + n].long()
        src = rows if c["per_route"] else rows // k
        if c["op"] == "gmm":
            out[rows] = (st["x"][src].float() @ st["w"][e].float().t()).to(out.dtype)
        elif c["op"] == "gmm_dw":
            out[e] = (st["dy"][rows].float().t() @ st["x"][src].float()).to(out.dtype)
        elif summed:
            part[rows] = st["dy"][rows].float() @ st["w"][e].float()
        else:
            out[rows] = (st["dy"][rows].float() @ st["w"][e].float()).to(out.dtype)
    if summed:
        out.copy_(part.view(c["M"], k, c["K"]).sum(dim=1))
    return out


def _plain_linear(st, c):
    M, K, N = c["M"], c["K"], c["N"]
    x = st["xq"].view(torch.float8_e4m3fn).float().view(M, K // 128, 128) * st["xs"][..., None]
    scale = st["ws"].repeat_interleave(128, dim=0)[:N]
    w = st["w"].view(torch.float8_e4m3fn).float().view(N, K // 128, 128) * scale[..., None]
    z = x.view(M, K) @ w.view(N, K).t()
    if st["bias"] is not None:
        z = z + st["bias"]
    if c["act"] == "silu":
        z = z / (1.0 + torch.exp(-z))
    elif c["act"] == "gelu":
        z = 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    elif c["act"] == "swiglu":
        g, u = z[:, :N // 2], z[:, N // 2:]
        z = g / (1.0 + torch.exp(-g)) * u
    if st["residual"] is not None:
        z = z + st["residual"].float()
    st["out"].copy_(z)
    return st["out"]


# ------------------------------------------------------------------- work --

def _touched(case):
    """Expected (valid routes, experts with a route, tokens with a route)."""
    M, E, k = case["M"], case["E"], case["top_k"]
    if case["routing"] == "skew":
        R = M * k * 0.99
        cold = R * (k - k // 2) / k
        hit = E * -math.expm1(cold * math.log1p(-1.0 / E)) if E > 1 else 1.0
        return R, min(E, hit + (4 if k > 1 else 0)), M
    R = M * k / case["shards"]
    p = k / (E * case["shards"])
    hit = E * -math.expm1(M * math.log1p(-p)) if p < 1 else E
    tokens = M * (1.0 - (1.0 - 1.0 / case["shards"]) ** k)
    return R, hit, tokens


def work(case):
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        n_out = N // 2 if case["act"] == "swiglu" else N
        nbytes = M * K + M * K // 128 * 4 + N * K + (N + 127) // 128 * (K // 128) * 4
        nbytes += M * n_out * 2 * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0)
        return {"bytes": nbytes, "flops": 2 * M * K * N}
    K, N = case["K"], case["N"]
    R, hit, tokens = _touched(case)
    src = (R if case["per_route"] else tokens) * K
    wt = hit * K * N
    if case["op"] == "gmm":
        nbytes = 2 * (src + wt + R * N)
    elif case["op"] == "gmm_dx":
        nbytes = 2 * (R * N + wt + (R if case["per_route"] else case["M"]) * K)
    else:
        nbytes = 2 * (src + R * N) + case["E"] * K * N * (4 if case["out"] == "f32" else 2)
    return {"bytes": int(nbytes + 4 * R), "flops": int(2 * R * K * N)}


# ------------------------------------------------------------------ exact --

def _e4m3_values():
    """The 256 E4M3 values from the format's definition (bias 7, subnormals,
    0x7f NaN)."""
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        a = math.nan if (e == 15 and m == 7) else \
            (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-a if b & 128 else a)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def exact(case, seed):
    if case["op"] == "linear":
        return _exact_linear(case, _lin_inputs(case, seed))
    s = _gmm_inputs(case, seed)
    M, E, K, N, k = case["M"], case["E"], case["K"], case["N"], case["top_k"]
    flat = s["ids"].reshape(-1)
    op = case["op"]
    n_rows = M * k if (case["per_route"] or op == "gmm") else M
    if op == "gmm_dw":
        res = torch.zeros((E, N, K), dtype=torch.float64, device=DEV)
    else:
        res = torch.zeros((n_rows, N if op == "gmm" else K), dtype=torch.float64, device=DEV)
    for e in range(E):
        r = torch.nonzero(flat == e).flatten()
        if r.numel() == 0:
            continue
        t = r if case["per_route"] else torch.div(r, k, rounding_mode="floor")
        if op == "gmm":
            res[r] = torch.mm(s["x"][t].double(), s["w"][e].double().t())
        elif op == "gmm_dx":
            # a token may hold the same expert twice: add, do not assign
            res.index_add_(0, t, torch.mm(s["dy"][r].double(), s["w"][e].double()))
        else:
            res[e] = torch.mm(s["dy"][r].double().t(), s["x"][t].double())
    return res


def _exact_linear(case, s):
    N, K = case["N"], case["K"]
    vals = _e4m3_values()
    kg = torch.arange(K, device=DEV) // 128
    ng = torch.arange(N, device=DEV) // 128
    x = vals[s["xq"].long()] * s["xs"].double()[:, kg]
    res = torch.empty((case["M"], N), dtype=torch.float64, device=DEV)
    for lo in range(0, N, 1024):
        hi = min(N, lo + 1024)
        w = vals[s["w"][lo:hi].long()] * s["ws"].double()[ng[lo:hi]][:, kg]
        res[:, lo:hi] = torch.mm(x, w.t())
    if s["bias"] is not None:
        res = res + s["bias"].double()
    if case["act"] == "silu":
        res = res * torch.sigmoid(res)
    elif case["act"] == "gelu":
        inner = (2.0 / math.pi) ** 0.5 * (res + 0.044715 * res ** 3)
        res = res / (1.0 + torch.exp(-2.0 * inner))
    elif case["act"] == "swiglu":
        g, u = res.chunk(2, dim=1)
        res = g * torch.sigmoid(g) * u
    if s["residual"] is not None:
        res = res + s["residual"].double()
    return res

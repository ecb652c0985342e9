"""Cases, inputs, plain forms and 64-bit values of the MoE block's operators.

    norm      h = x + residual, RMS norm of h, as bf16/fp32 and/or block-FP8 rows
    norm_bw   its gradients
    route     group-limited expert routing with sigmoid or softmax scores and a balance bias
    route_bw  the gradient of its weights with respect to the logits
    permute   block-FP8 token rows into the expert-major buffer
    gemv      the experts' products with 4-bit weights, for few rows per expert

With ``own`` set, ``run`` calls the framework's entry points; otherwise it
computes the same from elementary torch operations.
"""
import math

import torch

own = False

EPS = 1e-6
MASK = -3.3e38                        # a logit or bias at or below this masks its expert
LOWEST = -1e300                       # where a NaN score ranks: below every number, above a masked expert
FP4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the norm in front of a decode step's experts (128 tokens): both the router's bf16 rows and the dispatch's FP8 rows
        {"name": "norm decode", "op": "norm", "T": 128, "H": 7168, "dt": "bf16", "out": "both", "res": True},
        # the same at a prefill chunk, where only the 8-bit rows leave
        {"name": "norm prefill fp8", "op": "norm", "T": 8192, "H": 7168, "dt": "bf16", "out": "fp8", "res": True},
        # training step of the bf16 layer (16384 tokens, H = 4096), with the residual stream's own gradient
        {"name": "norm backward bf16", "op": "norm_bw", "T": 16384, "H": 4096, "dt": "bf16", "res": True},
        # a short ragged fp32 batch: the dW reduction has few rows to split
        {"name": "norm backward f32 ragged", "op": "norm_bw", "T": 1001, "H": 1408, "dt": "f32", "res": False},
        # routing of one decode step: 256 experts in 8 groups of which 4 stay, top-8, sigmoid scores, balance bias
        {"name": "route decode", "op": "route", "T": 128, "E": 256, "K": 8, "score": "sigmoid", "groups": 8, "keep": 4,
         "top": 2, "renorm": True, "scale": 2.5, "bias": True, "pad": 3},
        # the same for a large prefill batch with padded tokens at its end
        {"name": "route prefill", "op": "route", "T": 65536, "E": 256, "K": 8, "score": "sigmoid", "groups": 8, "keep": 4,
         "top": 2, "renorm": True, "scale": 2.5, "bias": True, "pad": 517},
        # training step of the 64-expert top-6 layer with softmax scores: a dense gradient row
        {"name": "route backward softmax", "op": "route_bw", "T": 16384, "E": 64, "K": 6, "score": "softmax", "groups": 1,
         "keep": 1, "top": 1, "renorm": False, "scale": 1.0, "bias": False, "pad": 100},
        # training step with sigmoid scores at 256 experts: K values in a row of zeros
        {"name": "route backward sigmoid", "op": "route_bw", "T": 8192, "E": 256, "K": 8, "score": "sigmoid", "groups": 8,
         "keep": 4, "top": 2, "renorm": True, "scale": 2.5, "bias": True, "pad": 0},
        # FP8 rows of a decode step into the buffer of 32 of 256 experts
        {"name": "permute decode", "op": "permute", "T": 128, "K": 8, "E": 256, "L": 32, "R": 128, "H": 7168},
        # FP8 rows of a prefill chunk
        {"name": "permute prefill", "op": "permute", "T": 8192, "K": 8, "E": 256, "L": 32, "R": 512, "H": 7168},
        # gate/up products of a decode step: 32 experts with about 4 rows each, int4 weights with a scale per 128, block-FP8 rows
        {"name": "gemv gate/up int4", "op": "gemv", "T": 128, "K": 8, "E": 256, "L": 32, "R": 128, "D": 7168, "N": 4096,
         "fmt": "int4", "G": 128, "sdt": "f32", "act": "fp8", "epi": "silu", "odt": "bf16"},
        # down products of the same step, e2m1 weights with a bf16 scale per 32, bf16 rows
        {"name": "gemv down fp4", "op": "gemv", "T": 128, "K": 8, "E": 256, "L": 32, "R": 128, "D": 2048, "N": 7168,
         "fmt": "fp4", "G": 32, "sdt": "bf16", "act": "bf16", "epi": "store", "odt": "bf16"},
    ]


def draw(rng):
    def logint(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["norm", "norm_bw", "route", "route_bw", "permute", "gemv"])
    if op in ("norm", "norm_bw"):
        dt = rng.choice(["bf16", "bf16", "f32"])
        H = 128 * rng.randint(2, 56)
        T = logint(1, 8192 * 7168 // (H * (2 if dt == "f32" else 1)))
        c = {"op": op, "T": T, "H": H, "dt": dt, "res": rng.random() < 0.7}
        if op == "norm":
            c["out"] = rng.choice(["same", "fp8", "both"])
        return c
    if op in ("route", "route_bw"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(2, max(2, 384 // groups))
        keep = rng.randint(1, groups)
        K = rng.randint(1, min(16, keep * (E // groups)))
        T = logint(1, 65536 * 256 // max(256, E))
        if op == "route_bw":
            T = max(1, T // 4)
        return {"op": op, "T": T, "E": E, "K": K, "score": rng.choice(["sigmoid", "softmax"]), "groups": groups,
                "keep": keep, "top": rng.choice([1, 2]), "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5, 16.0]), "bias": rng.random() < 0.6, "pad": rng.randint(0, T // 16)}
    if op == "permute":
        E = rng.choice([8, 32, 64, 256])
        L = E // rng.choice([1, 2, 4, 8])
        K = rng.randint(1, min(8, E))
        T = logint(1, 8192)
        return {"op": op, "T": T, "K": K, "E": E, "L": L, "R": max(1, int(math.ceil(T * K / E * rng.uniform(0.8, 2.0)))),
                "H": 128 * rng.randint(1, 56)}
    E = rng.choice([32, 64, 128, 256])
    L = max(1, E // rng.choice([2, 4, 8, 16]))
    epi = rng.choice(["silu", "store"])
    D = 128 * rng.randint(2, 56)
    most = 32 * 4096 * 7168 // (L * D)
    N = 128 * rng.randint(1, max(1, min(56, most // 128)))
    return {"op": "gemv", "T": logint(1, 256), "K": rng.randint(1, 8), "E": E, "L": L, "R": rng.choice([16, 64, 128]),
            "D": D, "N": N, "fmt": rng.choice(["int4", "fp4"]), "G": rng.choice([32, 64, 128]),
            "sdt": rng.choice(["f32", "bf16"]), "act": rng.choice(["bf16", "fp8"]), "epi": epi,
            "odt": rng.choice(["bf16", "f32"])}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _quant(x):
    """Block-FP8 rows of x [.., H]: codes and a scale per 128 columns."""
    b = x.float().reshape(*x.shape[:-1], x.shape[-1] // 128, 128)
    amax = b.abs().amax(-1).clamp(min=1e-4)
    inv = torch.full_like(amax, 448.0) / amax
    q = (b * inv[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.reshape(x.shape), amax / 448.0


def _routes(g, T, K, E):
    """Expert ids of T tokens, as a skewed router gives them."""
    logits = _randn(g, T, E) + 0.6 * torch.arange(E, device="cuda") / E
    return logits.topk(K, dim=1).indices


def _slots(ids, L, R):
    """Rows of the routes to experts 0..L-1 in a buffer of R rows each (-1: elsewhere, or beyond R), and the experts' counts."""
    flat = ids.reshape(-1).clamp(max=L)
    order = flat.argsort(stable=True)
    total = torch.bincount(flat, minlength=L + 1)
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(flat.numel(), device="cuda") - (total.cumsum(0) - total)[flat[order]]
    slot = torch.where((flat < L) & (rank < R), flat * R + rank, torch.full_like(flat, -1))
    return slot.reshape(ids.shape).int(), total[:L].clamp(max=R).int()


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    s = {"case": dict(c)}
    if op in ("norm", "norm_bw"):
        T, H, dt = c["T"], c["H"], DT[c["dt"]]
        s["w"] = _randn(g, H).mul_(0.2).add_(1.0).to(dt)
        s["x"] = _randn(g, T, H, dtype=dt)
        if op == "norm":
            s["res"] = (_randn(g, T, H) * 4).to(dt) if c["res"] else None
            s["h"] = torch.empty(T, H, dtype=dt, device="cuda") if c["res"] else None
            s["y"] = torch.empty(T, H, dtype=dt, device="cuda") if c["out"] != "fp8" else None
            s["y8"] = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda") if c["out"] != "same" else None
            s["sc"] = torch.empty(T, H // 128, device="cuda") if c["out"] != "same" else None
        else:
            s["dy"] = _randn(g, T, H, dtype=dt)
            s["dh"] = _randn(g, T, H, dtype=dt) if c["res"] else None
            s["dx"] = torch.empty(T, H, dtype=dt, device="cuda")
            s["dw"] = torch.empty(H, device="cuda")
            if own:     # the scratch that a training program keeps
                import combine_top_expert_amd as ep
                s["ws"] = torch.empty(ep.moe_add_rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    elif op in ("route", "route_bw"):
        T, E, K = c["T"], c["E"], c["K"]
        s["logits"] = _randn(g, T, E) * 1.5
        if c["pad"]:
            s["logits"][T - c["pad"]:] = -math.inf          # tokens that only pad the batch
        s["bias"] = _randn(g, E) * 0.1 if c["bias"] else None
        s["ids"] = torch.empty(T, K, dtype=torch.int32, device="cuda")
        s["wts"] = torch.empty(T, K, device="cuda")
        if op == "route_bw":
            s["ids"] = _route(s)[0]
            s["dw"] = _randn(g, T, K)
            s["dl"] = torch.empty(T, E, device="cuda")
    elif op == "permute":
        s["x8"], s["xs"] = _quant(_randn(g, c["T"], c["H"]))
        s["slot"], _ = _slots(_routes(g, c["T"], c["K"], c["E"]), c["L"], c["R"])
        s["buf"] = torch.zeros(c["L"] * c["R"], c["H"], dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        s["bs"] = torch.zeros(c["L"] * c["R"], c["H"] // 128, device="cuda")
    else:
        L, R, D, N, G = c["L"], c["R"], c["D"], c["N"], c["G"]
        _, s["counts"] = _slots(_routes(g, c["T"], min(c["K"], c["E"]), c["E"]), L, R)
        s["offsets"] = torch.arange(L + 1, dtype=torch.int32, device="cuda") * R
        x = _randn(g, L * R, D, dtype=torch.bfloat16)
        s["a"], s["as"] = _quant(x) if c["act"] == "fp8" else (x, None)
        s["codes"] = torch.randint(0, 256, (L, N, D // 2), dtype=torch.uint8, generator=g, device="cuda")
        u = torch.rand(L, N, D // G, generator=g, device="cuda")
        s["ws"] = ((0.5 + u) / (4 * math.sqrt(D))).to(DT[c["sdt"]])
        cols = N // 2 if c["epi"] == "silu" else N
        s["out"] = torch.zeros(L * R, cols, dtype=DT[c["odt"]], device="cuda")
        if own:         # the weights as the products read them: laid out once, when they are loaded
            import combine_top_expert_amd as ep
            s["fmt"] = {"int4": ep.MOE_W4_INT4, "fp4": ep.MOE_W4_E2M1}[c["fmt"]]
            s["pw"], s["ps"] = torch.empty_like(s["codes"]), torch.empty_like(s["ws"])
            ep.moe_pack_w4(s["codes"], s["ws"], s["fmt"], s["pw"], s["ps"])
    return s


# ------------------------------------------------------------------ plain forms

def _norm(s):
    c = s["case"]
    h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["x"].dtype)
    f = h.float()
    y = f / (f.square().mean(-1, keepdim=True) + EPS).sqrt() * s["w"].float()
    out = {} if s["res"] is None else {"h": h}
    if c["out"] != "fp8":
        out["y"] = y.to(h.dtype)
    if c["out"] != "same":
        out["y8"], out["scales"] = _quant(y)
    return out


def _norm_bw(s):
    h, dy, w = s["x"].float(), s["dy"].float(), s["w"].float()
    r = 1.0 / (h.square().mean(-1, keepdim=True) + EPS).sqrt()
    n = h * r
    u = dy * w
    dx = r * (u - n * (u * n).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * n).sum(0)}


def _scores(logits, score):
    """fp64 scores: which expert comes first is decided next to ties."""
    l = logits.double()
    off = logits <= MASK
    if score == "sigmoid":
        return (1.0 / (1.0 + (-l).exp())).masked_fill(off, 0.0)
    l = l.masked_fill(off, -math.inf)
    m = l.amax(-1, keepdim=True)
    e = (l - m.masked_fill(m == -math.inf, 0.0)).exp()
    total = e.sum(-1, keepdim=True)
    return torch.where(total == 0, torch.zeros_like(e), e / total)


def _route(s):
    c, logits, bias = s["case"], s["logits"], s["bias"]
    T, E, K, n = c["T"], c["E"], c["K"], c["groups"]
    p = _scores(logits, c["score"])
    sel, off = p, logits <= MASK
    if bias is not None:
        sel, off = p + bias.double(), off | (bias <= MASK)
    sel = sel.nan_to_num(nan=LOWEST, posinf=math.inf).masked_fill(off, -math.inf)
    if n > 1:
        top = sel.reshape(T, n, E // n).sort(-1, descending=True).values[..., :c["top"]]
        gs = torch.where((top == -math.inf) & (top[..., :1] != -math.inf), torch.zeros_like(top), top).sum(-1)
        gs = torch.where((top == LOWEST).any(-1), torch.full_like(gs, LOWEST), gs)
        kept = gs.sort(dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        keep = torch.zeros(T, n, dtype=torch.bool, device=logits.device).scatter_(1, kept, True)
        sel = sel.masked_fill(~keep.repeat_interleave(E // n, 1), -math.inf)
    v, ids = sel.sort(dim=-1, descending=True, stable=True)
    v, ids = v[:, :K], ids[:, :K]
    none = v == -math.inf
    w = p.gather(1, ids).masked_fill(none, 0.0)
    if c["renorm"]:
        w = w / (w.sum(-1, keepdim=True) + 1e-20)
    return ids.masked_fill(none, -1).int(), (w * c["scale"]).float()


def _route_bw(s):
    c = s["case"]
    p = _scores(s["logits"], c["score"])
    none = s["ids"] < 0
    at = s["ids"].long().clamp(min=0)
    w, d = p.gather(1, at).masked_fill(none, 0.0), s["dw"].double().masked_fill(none, 0.0) * c["scale"]
    if c["renorm"]:
        total = w.sum(-1, keepdim=True) + 1e-20
        d = (d - (d * w).sum(-1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter_add_(1, at, d.masked_fill(none, 0.0))
    if c["score"] == "sigmoid":
        return (dp * p * (1.0 - p)).float()
    return (p * (dp - (dp * p).sum(-1, keepdim=True))).float()


def _permute(s):
    buf = torch.zeros(s["buf"].shape, dtype=torch.uint8, device="cuda")
    bs = torch.zeros_like(s["bs"])
    t, k = (s["slot"] >= 0).nonzero(as_tuple=True)
    rows = s["slot"][t, k].long()
    buf[rows] = s["x8"].view(torch.uint8)[t]
    bs[rows] = s["xs"][t]
    return {"buf": buf.view(torch.float8_e4m3fn), "scales": bs}


def _gemv(s):
    c = s["case"]
    L, R, D, N, G = c["L"], c["R"], c["D"], c["N"], c["G"]
    q = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).reshape(-1)
    if c["fmt"] == "int4":
        q = q.float() - 8.0
    else:
        q = torch.tensor(FP4 + [-v for v in FP4], device="cuda").index_select(0, q.int())
    w = (q.reshape(L, N, D // G, G) * s["ws"].float()[..., None]).reshape(L, N, D)
    a = s["a"].float()
    if c["act"] == "fp8":
        a = (a.reshape(L * R, D // 128, 128) * s["as"][..., None]).reshape(L * R, D)
    o = torch.bmm(a.reshape(L, R, D), w.transpose(1, 2))
    if c["epi"] == "silu":
        gate, up = o[..., :N // 2], o[..., N // 2:]
        o = gate / (1.0 + (-gate).exp()) * up
    valid = torch.arange(R, device="cuda")[None, :] < s["counts"][:, None]
    o = torch.where(valid[..., None], o, torch.zeros_like(o))
    return o.reshape(L * R, -1).to(s["out"].dtype)


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if not own:
        return {"norm": _norm, "norm_bw": _norm_bw, "route": _route, "route_bw": _route_bw, "permute": _permute,
                "gemv": _gemv}[op](s)
    import combine_top_expert_amd as ep
    if op == "norm":
        ep.moe_add_rms_norm(s["x"], s["res"], s["w"], EPS, s["h"], s["y"], s["y8"], s["sc"])
        out = {"h": s["h"], "y": s["y"], "y8": s["y8"], "scales": s["sc"]}
        return {k: v for k, v in out.items() if v is not None}
    if op == "norm_bw":
        ep.moe_add_rms_norm_backward(s["dy"], s["x"], s["w"], EPS, s["dx"], s["dw"], s["ws"], dh=s["dh"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op in ("route", "route_bw"):
        score = ep.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else ep.MOE_SCORE_SOFTMAX
        if op == "route_bw":
            ep.moe_router_group_topk_backward(s["logits"], s["ids"], s["dw"], s["dl"], score=score, renorm=c["renorm"],
                                              route_scale=c["scale"])
            return s["dl"]
        ep.moe_router_group_topk(s["logits"], c["K"], s["ids"], s["wts"], bias=s["bias"], score=score, n_group=c["groups"],
                                 topk_group=c["keep"], group_top=c["top"], renorm=c["renorm"], route_scale=c["scale"])
        return s["ids"], s["wts"]
    if op == "permute":
        ep.moe_permute_fp8(s["x8"], s["xs"], s["slot"], s["buf"], s["bs"])
        return {"buf": s["buf"], "scales": s["bs"]}
    epi = ep.MOE_EPI_SILU_MUL if c["epi"] == "silu" else ep.MOE_EPI_STORE_G
    ep.moe_grouped_gemv_w4(s["a"], s["as"], s["pw"], s["ps"], s["fmt"], s["counts"], s["offsets"], epi, s["out"])
    return s["out"]


# ------------------------------------------------------------------ work

def work(case):
    c, op = case, case["op"]
    if op in ("norm", "norm_bw"):
        e, n = (2 if c["dt"] == "bf16" else 4), c["T"] * c["H"]
        if op == "norm":
            per = e + (2 * e if c["res"] else 0) + (e if c["out"] != "fp8" else 0) + (1 + 4 / 128 if c["out"] != "same" else 0)
            return {"bytes": n * per + c["H"] * e, "flops": 6 * n}
        return {"bytes": n * e * (4 if c["res"] else 3) + c["H"] * (e + 4), "flops": 12 * n}
    if op == "route":
        return {"bytes": c["T"] * (4 * c["E"] + 8 * c["K"]) + (4 * c["E"] if c["bias"] else 0), "flops": 4 * c["T"] * c["E"]}
    if op == "route_bw":
        reads = c["E"] if c["score"] == "softmax" else c["K"]
        return {"bytes": c["T"] * (4 * c["E"] + 4 * reads + 8 * c["K"]), "flops": 4 * c["T"] * c["E"]}
    share = c["L"] / c["E"]
    rows = min(c["T"] * c["K"] * share, c["L"] * c["R"])
    if op == "permute":
        seen = c["T"] * (1 - (1 - share) ** c["K"])
        return {"bytes": (rows + seen) * (c["H"] + c["H"] / 32) + 4 * c["T"] * c["K"], "flops": 0}
    busy = c["L"] * (1 - (1 - min(c["K"], c["E"]) / c["E"]) ** c["T"])
    sb = 4 if c["sdt"] == "f32" else 2
    weights = busy * c["N"] * c["D"] * (0.5 + sb / c["G"])
    a = c["D"] * (2 if c["act"] == "bf16" else 1 + 4 / 128)
    o = (c["N"] // 2 if c["epi"] == "silu" else c["N"]) * (2 if c["odt"] == "bf16" else 4)
    return {"bytes": weights + rows * (a + o), "flops": 2 * rows * c["N"] * c["D"]}


# ------------------------------------------------------------------ 64-bit values

def _exact_norm(s):
    x = s["x"].double()
    h = x if s["res"] is None else (x + s["res"].double()).float().to(s["x"].dtype).double()
    y = torch.empty_like(h)
    for t in range(0, h.shape[0], 1024):
        b = h[t:t + 1024]
        y[t:t + 1024] = s["w"].double() * b * torch.rsqrt((b * b).sum(1) / b.shape[1] + EPS)[:, None]
    out = {} if s["res"] is None else {"h": h}
    if s["y"] is not None:
        out["y"] = y
    if s["y8"] is not None:
        top = y.unflatten(1, (-1, 128)).abs().max(2).values.clamp(min=float(torch.tensor(1e-4)))
        out["y8"] = (y.unflatten(1, (-1, 128)) / top[:, :, None] * 448).flatten(1)
        out["scales"] = top / 448
    return out


def _exact_norm_bw(s):
    h, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
    H = h.shape[1]
    ms = torch.linalg.vector_norm(h, dim=1) ** 2 / H + EPS
    dot = (h * (dy * w)).sum(1)
    dx = (dy * w) / ms.sqrt()[:, None] - h * (dot / (H * ms ** 1.5))[:, None]
    if s["dh"] is not None:
        dx += s["dh"].double()
    return {"dx": dx, "dw": (1 / ms.sqrt()) @ (dy * h)}


def _exact_score(row, score):
    live = row > MASK
    p = torch.zeros_like(row)
    if score == "sigmoid":
        p[live] = torch.sigmoid(row[live])
    elif bool(live.any()):
        p[live] = torch.softmax(row[live], 0)
    return p


def _exact_route(s):
    """Token by token, in plain Python."""
    c = s["case"]
    logits = s["logits"].double().cpu()
    bias = None if s["bias"] is None else s["bias"].double().cpu()
    E, n = c["E"], c["groups"]
    all_ids, all_w = [], []
    for row in logits:
        p = _exact_score(row, c["score"])
        v = (p if bias is None else p + bias).tolist()
        allowed = [e for e in range(E) if row[e] > MASK and (bias is None or bias[e] > MASK)]
        if n > 1:
            held = [sorted((v[e] for e in allowed if e // (E // n) == b), reverse=True)[:c["top"]] for b in range(n)]
            rank = sorted(range(n), key=lambda b: (-sum(held[b]) if held[b] else math.inf, b))[:c["keep"]]
            allowed = [e for e in allowed if e // (E // n) in rank]
        ids = sorted(allowed, key=lambda e: (-v[e], e))[:c["K"]]
        w = [float(p[e]) for e in ids]
        total = (math.fsum(w) + 1e-20) if c["renorm"] else 1.0
        all_ids.append(ids + [-1] * (c["K"] - len(ids)))
        all_w.append([x / total * c["scale"] for x in w] + [0.0] * (c["K"] - len(ids)))
    return torch.tensor(all_ids, dtype=torch.int32), torch.tensor(all_w, dtype=torch.float64)


def _exact_route_bw(s):
    """Through the weights' definition by automatic differentiation in 64 bits."""
    c = s["case"]
    l = s["logits"].double().requires_grad_(True)
    live = (s["logits"] > MASK)
    if c["score"] == "sigmoid":
        p = torch.where(live, torch.sigmoid(l), torch.zeros_like(l))
    else:
        some = live.any(1, keepdim=True)
        p = torch.softmax(torch.where(some, l, torch.zeros_like(l)), 1) * some
    w = torch.gather(p, 1, s["ids"].long().clamp(min=0)) * (s["ids"] >= 0)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    (w * c["scale"] * s["dw"].double()).sum().backward()
    return torch.nan_to_num(l.grad).masked_fill(~live, 0.0)


def _exact_permute(s):
    buf = torch.zeros(s["buf"].shape, dtype=torch.float32, device="cuda")
    bs = torch.zeros(s["bs"].shape, dtype=torch.float64, device="cuda")
    x, xs = s["x8"].float(), s["xs"].double()
    for k in range(s["slot"].shape[1]):
        at = s["slot"][:, k].long()
        buf[at[at >= 0]] = x[at >= 0]
        bs[at[at >= 0]] = xs[at >= 0]
    return {"buf": buf.double(), "scales": bs}


def _exact_gemv(s):
    c = s["case"]
    L, R, D, N = c["L"], c["R"], c["D"], c["N"]
    values = [v - 8.0 for v in range(16)] if c["fmt"] == "int4" else FP4 + [-v for v in FP4]
    table = torch.tensor(values, dtype=torch.float64, device="cuda")
    out = torch.zeros(L * R, s["out"].shape[1], dtype=torch.float64, device="cuda")
    for e, m in enumerate(s["counts"].tolist()):
        if m == 0:
            continue
        w = torch.empty(N, D, dtype=torch.float64, device="cuda")
        w[:, 0::2] = table[(s["codes"][e] % 16).long()]
        w[:, 1::2] = table[(s["codes"][e] // 16).long()]
        w *= s["ws"][e].double().repeat_interleave(c["G"], 1)
        a = s["a"][e * R:e * R + m].double()
        if s["as"] is not None:
            a = a * s["as"][e * R:e * R + m].double().repeat_interleave(128, 1)
        o = a @ w.T.contiguous()
        if c["epi"] == "silu":
            o = o[:, :N // 2] * torch.sigmoid(o[:, :N // 2]) * o[:, N // 2:]
        out[e * R:e * R + m] = o
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s) if case["T"] * case["E"] <= 1_500_000 else None
    return {"norm": _exact_norm, "norm_bw": _exact_norm_bw, "route_bw": _exact_route_bw, "permute": _exact_permute,
            "gemv": _exact_gemv}[op](s)

"""The operators of a decode step's sublayers, as they are measured: routing to
experts (mhc_moe_route), the experts' products (mhc_moe_experts) and the linear
product with bias, activation and residual in its epilogue (mhc_linear).

`listed` names the measured cases, `draw` gives further cases of the same ranges,
`prepare` makes a case's inputs on the GPU, `run` is one pass: the plain form in
elementary torch operations, or, where `own` is true, the library's calls.
`exact` is the operators' definition in 64 bits, `work` what a pass cannot do
without.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # Routing. One sequence being decoded: the call's latency is all there is.
        route_case("route, 1 row", rows=1, experts=64, top_k=8, scoring="softmax"),
        # The largest decode batch of the boundary, 15 of its rows padding (every logit -inf),
        # with a balance bias, 4 of 8 groups of experts and renormalised, scaled weights.
        route_case("route, decode batch", rows=128, padded=15, experts=256, top_k=8, scoring="sigmoid", bias=True,
                   groups=8, top_groups=4, group_top=2, scale=2.5),
        # A long prompt; an odd number of experts per group.
        route_case("route, long prompt", rows=8191, experts=200, top_k=6, scoring="sigmoid", bias=True, groups=8,
                   top_groups=3, group_top=2, scale=1.0),
        # Linear. The router's logits of a decode batch, kept in fp32.
        linear_case("linear, router logits", rows=32, k=7168, n=256, out="float32"),
        # The shared expert's gate and up products of a decode batch, one call.
        linear_case("linear, shared expert gate-up", rows=32, k=7168, n=2048, activation="swiglu"),
        # The product that reads a boundary's MXFP8 layer input.
        linear_case("linear, MXFP8 layer input", rows=64, k=7168, n=7168, mxfp8=True),
        # Sizes that no tile divides, with everything in the epilogue.
        linear_case("linear, odd sizes", rows=77, k=1000, n=333, activation="gelu", bias=True, residual=True),
        # A long prompt: bound by the tensor cores.
        linear_case("linear, long prompt", rows=4096, k=7168, n=7168, residual=True),
        # The experts' products. One sequence being decoded: eight experts' weights are read.
        experts_case("experts, 1 row", rows=1, top_k=8, experts=64, hidden=7168, inter=2048),
        # A decode batch: nearly every expert's weights are read for a few rows each.
        experts_case("experts, decode batch", rows=64, top_k=8, experts=64, hidden=7168, inter=2048),
        # Sizes that no tile divides, few rows, some experts without one.
        experts_case("experts, odd sizes", rows=37, top_k=3, experts=24, hidden=712, inter=328),
        # A long prompt: bound by the tensor cores.
        experts_case("experts, long prompt", rows=2048, top_k=8, experts=32, hidden=7168, inter=2048),
    ]


def route_case(name, *, rows, experts, top_k, scoring, padded=0, bias=False, groups=1, top_groups=1, group_top=1,
               renormalize=True, scale=1.0):
    return dict(name=name, op="route", rows=rows, padded=padded, experts=experts, top_k=top_k, scoring=scoring,
                bias=bias, groups=groups, top_groups=top_groups, group_top=group_top, renormalize=renormalize,
                scale=scale)


def linear_case(name, *, rows, k, n, activation="none", bias=False, residual=False, mxfp8=False, out="bfloat16"):
    return dict(name=name, op="linear", rows=rows, k=k, n=n, activation=activation, bias=bias, residual=residual,
                mxfp8=mxfp8, out=out)


def experts_case(name, *, rows, top_k, experts, hidden, inter):
    return dict(name=name, op="experts", rows=rows, top_k=top_k, experts=experts, hidden=hidden, inter=inter)


def _spread(rng, lo, hi):
    """A whole number in lo..hi, evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "linear", "linear", "experts", "experts"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * _spread(rng, 8, 256 // groups)
        rows = _spread(rng, 1, 8191)
        top_groups = rng.randint((groups + 1) // 2, groups)
        c = route_case("", rows=rows, padded=rng.choice((0, rows // 9)), experts=experts,
                       top_k=rng.randint(1, min(12, experts // groups * top_groups)),
                       scoring=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.6, groups=groups,
                       top_groups=top_groups, group_top=rng.choice((1, 2)), renormalize=rng.random() < 0.7,
                       scale=rng.choice((1.0, 2.5)))
    elif op == "linear":
        mxfp8 = rng.random() < 0.35
        activation = rng.choice(("none", "none", "relu", "silu", "gelu", "swiglu"))
        n = _spread(rng, 64, 7168 if activation != "swiglu" else 3584)
        if mxfp8 and activation == "swiglu":
            n = -(-n // 128) * 128
        k = _spread(rng, 8, 224) * 32 if mxfp8 else _spread(rng, 32, 896) * 8
        c = linear_case("", rows=_spread(rng, 1, 4096), k=k, n=n, activation=activation, bias=rng.random() < 0.5,
                        residual=rng.random() < 0.5, mxfp8=mxfp8, out=rng.choice(("bfloat16", "bfloat16", "float32")))
    else:
        experts = _spread(rng, 8, 64)
        c = experts_case("", rows=_spread(rng, 1, 1024), top_k=rng.randint(1, 8), experts=experts,
                         hidden=_spread(rng, 32, 896) * 8, inter=_spread(rng, 16, 256) * 8)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed, dev=DEV):
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    return g


def _routed(rows, experts, top_k, g, dev):
    """Expert ids [rows, top_k] of a router whose experts are unevenly popular."""
    popular = torch.randn(experts, generator=g, device=dev) * 0.5
    return (torch.randn(rows, experts, generator=g, device=dev) + popular).topk(top_k, dim=1).indices


def _quantized(v):
    """MXFP8 of the rows of v as the boundary writes it: E4M3 bytes, and E8M0 bytes in tiles of
    128 rows x 4 blocks, (r, c) of a tile at (r % 32) * 16 + (r // 32) * 4 + c."""
    rows, k = v.shape
    blocks = v.reshape(rows, k // 32, 32)
    m, e = torch.frexp(blocks.abs().amax(-1) / 448.0)
    e = torch.where(m == 0.5, e - 1, e).clamp(-127, 127)  # the smallest e with amax <= 448 * 2^e
    data = (blocks * torch.exp2(-e.float())[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(rows, k)
    sc = torch.zeros(-(-rows // 128) * 128, -(-k // 128) * 4, dtype=torch.uint8, device=v.device)
    sc[:rows, : k // 32] = (e + 127).to(torch.uint8)
    sc = sc.view(sc.shape[0] // 128, 4, 32, sc.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return data, sc


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    rows = case["rows"]
    if case["op"] == "route":
        s["logits"] = torch.randn(rows, case["experts"], generator=g, device=DEV) * 1.5
        if case["padded"]:
            s["logits"][rows - case["padded"]:] = -math.inf
        s["bias"] = torch.randn(case["experts"], generator=g, device=DEV) * 0.05 if case["bias"] else None
    elif case["op"] == "linear":
        k, n = case["k"], case["n"]
        wn = 2 * n if case["activation"] == "swiglu" else n
        x = torch.randn(rows, k, generator=g, device=DEV)
        w = torch.randn(wn, k, generator=g, device=DEV) * (1.5 / math.sqrt(k))
        s["x"] = _quantized(x) if case["mxfp8"] else x.to(torch.bfloat16)
        s["w"] = _quantized(w) if case["mxfp8"] else w.to(torch.bfloat16)
        s["bias"] = torch.randn(wn, generator=g, device=DEV) * 0.2 if case["bias"] else None
        s["residual"] = torch.randn(rows, n, generator=g, device=DEV).to(torch.bfloat16) if case["residual"] else None
    else:
        e, h, i, k = case["experts"], case["hidden"], case["inter"], case["top_k"]
        s["x"] = torch.randn(rows, h, generator=g, device=DEV).to(torch.bfloat16)
        s["w13"] = torch.empty(e, 2 * i, h, dtype=torch.bfloat16, device=DEV).normal_(0.0, 1.5 / math.sqrt(h), generator=g)
        s["w2"] = torch.empty(e, h, i, dtype=torch.bfloat16, device=DEV).normal_(0.0, 1.5 / math.sqrt(i), generator=g)
        ids = _routed(rows, e, k, g, DEV).reshape(-1)
        order = torch.sort(ids, stable=True).indices
        s["permuted_rows"] = (order // k).to(torch.int32)
        s["counts"] = torch.bincount(ids, minlength=e)
        s["offsets"] = torch.cat([s["counts"].new_zeros(1), s["counts"].cumsum(0)]).to(torch.int32)
        # the plain form's plan: which experts have rows, and the most rows of one
        s["active"] = torch.nonzero(s["counts"]).reshape(-1)
        s["most"] = int(s["counts"].max())
    return s


# ---------------------------------------------------------------- the plain forms

def _top(v, k):
    """Indices of the k largest of each row, the lowest index first among equals."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[..., :k]


def _plain_route(s):
    c = s["case"]
    rows, experts, k = c["rows"], c["experts"], c["top_k"]
    logits = s["logits"].double()  # in 64 bits: which of two near scores is larger decides
    if c["scoring"] == "softmax":
        score = torch.exp(logits - logits.amax(1, keepdim=True).clamp_min(-1e30))
        score = score / score.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    choice = logits if s["bias"] is None else score + s["bias"].double()
    choice = torch.where(torch.isneginf(logits), -math.inf, choice)
    if c["groups"] > 1:
        biased = score if s["bias"] is None else score + s["bias"].double()
        biased = torch.where(torch.isneginf(logits), -math.inf, biased).view(rows, c["groups"], -1)
        best = biased.sort(dim=-1, descending=True).values[..., : c["group_top"]]
        best = torch.where(torch.isneginf(best[..., :1]), -math.inf,
                           torch.where(torch.isneginf(best), 0.0, best).sum(-1, keepdim=True))[..., 0]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, _top(best, c["top_groups"]), True)
        choice = torch.where(kept[..., None], choice.view(rows, c["groups"], -1), -math.inf).view(rows, experts)
    ids = _top(choice, k)
    none = torch.isneginf(choice.gather(1, ids))
    w = torch.where(none, 0.0, score.gather(1, ids))
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    ids = torch.where(none, -1, ids)
    # the permutation: the pairs (row, slot) by expert, in order within an expert; pairs without one last
    flat = torch.where(none, experts, ids).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    place = torch.empty_like(order).scatter_(0, order, torch.arange(rows * k, device=DEV))
    used = flat < experts
    counts = (flat[:, None] == torch.arange(experts, device=DEV)).sum(0) if rows * k * experts < 1 << 22 else \
        torch.zeros(experts + 1, dtype=torch.int64, device=DEV).index_add_(0, flat, torch.ones_like(flat))[:experts]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    e2p = torch.where(used, place, -1)
    source = torch.where(used[order], order // k, -1)
    return ((w * c["scale"]).float(), ids.to(torch.int32), e2p.to(torch.int32), source.to(torch.int32),
            offsets.to(torch.int32))


def _values(q):
    """The fp32 values of an operand: bf16, or MXFP8 (bytes and tiled scales)."""
    if isinstance(q, torch.Tensor):
        return q.float()
    data, sc = q
    rows, k = data.shape
    sc = sc.view(-(-rows // 128), -(-k // 128), 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-(-rows // 128) * 128, -1)
    sc = torch.exp2(sc[:rows, : k // 32].float() - 127.0)
    return (data.view(torch.float8_e4m3fn).float().view(rows, k // 32, 32) * sc[..., None]).view(rows, k)


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _plain_linear(s):
    c = s["case"]
    y = _values(s["x"]) @ _values(s["w"]).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["activation"] == "swiglu":
        y = _silu(y[:, : c["n"]]) * y[:, c["n"]:]
    elif c["activation"] == "silu":
        y = _silu(y)
    elif c["activation"] == "relu":
        y = torch.where(y > 0, y, 0.0)
    elif c["activation"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(getattr(torch, c["out"]))


def _plain_experts(s):
    offsets, active, most = s["offsets"].long(), s["active"], s["most"]
    pairs = s["permuted_rows"].shape[0]
    inter = s["w2"].shape[2]
    at = (offsets[active][:, None] + torch.arange(most, device=DEV)).clamp_max(pairs - 1)
    x = s["x"].float()[s["permuted_rows"].long()[at]]
    y = torch.bmm(x, s["w13"][active].float().transpose(1, 2))
    y = _silu(y[..., :inter]) * y[..., inter:]
    y = torch.bmm(y, s["w2"][active].float().transpose(1, 2))
    p = torch.arange(pairs, device=DEV)
    expert = torch.searchsorted(offsets, p, right=True) - 1
    return y[torch.searchsorted(active, expert), p - offsets[expert]].to(torch.bfloat16)


# ---------------------------------------------------------------- the library's calls

def _own_route(s):
    from mhc_residual_stream_b200 import mhc as M
    c = s["case"]
    rows, experts, k = c["rows"], c["experts"], c["top_k"]
    if "workspace" not in s:
        s["workspace"] = M.new_moe_route_workspace(rows, experts, k, DEV)
    w = torch.empty(rows, k, dtype=torch.float32, device=DEV)
    ids, e2p, source, offsets = (torch.empty(z, dtype=torch.int32, device=DEV)
                                 for z in ((rows, k), rows * k, rows * k, experts + 1))
    M.mhc_moe_route(s["logits"], w, ids, e2p, source, offsets, bias=s["bias"], scoring=c["scoring"],
                    num_groups=c["groups"], top_groups=c["top_groups"], group_top=c["group_top"],
                    renormalize=c["renormalize"], weight_scale=c["scale"], workspace=s["workspace"])
    return w, ids, e2p, source, offsets


def _own_linear(s):
    from mhc_residual_stream_b200 import mhc as M
    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = M.new_linear_workspace(c["rows"], DEV)
    x, w = ((*s[q], True) if c["mxfp8"] else s[q] for q in ("x", "w"))
    out = torch.empty(c["rows"], c["n"], dtype=getattr(torch, c["out"]), device=DEV)
    M.mhc_linear(x, w, out, bias=s["bias"], activation=c["activation"], residual=s["residual"],
                 workspace=s["workspace"])
    return out


def _own_experts(s):
    from mhc_residual_stream_b200 import mhc as M
    c = s["case"]
    pairs = s["permuted_rows"].shape[0]
    if "workspace" not in s:
        s["workspace"] = M.new_moe_experts_workspace(c["rows"], pairs, c["inter"], DEV)
    out = torch.empty(pairs, c["hidden"], dtype=torch.bfloat16, device=DEV)
    M.mhc_moe_experts(s["x"], s["w13"], s["w2"], s["permuted_rows"], s["offsets"], out, workspace=s["workspace"])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "linear": _own_linear, "experts": _own_experts}[op](state)
    return {"route": _plain_route, "linear": _plain_linear, "experts": _plain_experts}[op](state)


# ---------------------------------------------------------------- work

def work(case):
    rows = case["rows"]
    if case["op"] == "route":
        e, k = case["experts"], case["top_k"]
        # logits and bias in; weights, ids and both halves of the permutation out
        return {"bytes": rows * e * 4 + (e * 4 if case["bias"] else 0) + rows * k * 16 + (e + 1) * 4,
                "flops": rows * e * 4}
    if case["op"] == "linear":
        k, n = case["k"], case["n"]
        wn = 2 * n if case["activation"] == "swiglu" else n
        per = 1 + 1 / 32 if case["mxfp8"] else 2
        out = rows * n * (4 if case["out"] == "float32" else 2)
        return {"bytes": (rows + wn) * k * per + out + (wn * 4 if case["bias"] else 0)
                + (rows * n * 2 if case["residual"] else 0), "flops": 2 * rows * wn * k}
    e, h, i, k = case["experts"], case["hidden"], case["inter"], case["top_k"]
    # the experts that have rows, of one draw of the router
    active = len(torch.unique(_routed(rows, e, k, _gen(0, "cpu"), "cpu")))
    return {"bytes": active * 3 * h * i * 2 + rows * h * 2 + rows * k * (h * 2 + 4) + (e + 1) * 4,
            "flops": 2 * rows * k * 3 * h * i}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_route(s):
    c = s["case"]
    k, groups = c["top_k"], c["groups"]
    logits = s["logits"].cpu().numpy().astype(np.float64)
    bias = 0.0 if s["bias"] is None else s["bias"].cpu().numpy().astype(np.float64)
    rows, experts = logits.shape
    weights = np.zeros((rows, k))
    ids = np.full((rows, k), -1, np.int32)
    with np.errstate(all="ignore"):
        if c["scoring"] == "softmax":
            score = np.exp(logits - logits.max(1, keepdims=True))
            score /= score.sum(1, keepdims=True)
        else:
            score = 1 / (1 + np.exp(-logits))
    for r in range(rows):
        free = [e for e in range(experts) if logits[r, e] != -math.inf]
        value = (score[r] + bias).tolist()
        if groups > 1:
            size = experts // groups
            of = [sorted((value[e] for e in free if e // size == q), reverse=True)[: c["group_top"]] for q in range(groups)]
            best = sorted((q for q in range(groups) if of[q]), key=lambda q: (-sum(of[q]), q))[: c["top_groups"]]
            free = [e for e in free if e // size in best]
        key = logits[r].tolist() if s["bias"] is None else value
        chosen = sorted(free, key=lambda e: (-key[e], e))[:k]
        ids[r, : len(chosen)] = chosen
        weights[r, : len(chosen)] = score[r, chosen]
        if c["renormalize"] and chosen:
            weights[r] /= weights[r].sum()
    return weights * c["scale"], ids, None, None, None


def _exact_values(q):
    if isinstance(q, torch.Tensor):
        return q.double()
    data, sc = q
    r, b = torch.meshgrid(torch.arange(data.shape[0], device=DEV), torch.arange(data.shape[1] // 32, device=DEV), indexing="ij")
    tiles = -(-data.shape[1] // 128)
    at = ((r // 128) * tiles + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
    scale = torch.pow(2.0, sc[at].double() - 127)
    return data.view(torch.float8_e4m3fn).double() * scale.repeat_interleave(32, dim=1)


def _exact_linear(s):
    c = s["case"]
    x, w = _exact_values(s["x"]), _exact_values(s["w"])
    bias = w.new_zeros(w.shape[0]) if s["bias"] is None else s["bias"].double()
    act = {"none": lambda v: v, "relu": lambda v: v.clamp_min(0), "silu": lambda v: v * torch.sigmoid(v),
           "gelu": lambda v: v * torch.special.ndtr(v)}
    if c["activation"] == "swiglu":
        n = c["n"]
        y = act["silu"](torch.addmm(bias[:n], x, w[:n].T)) * torch.addmm(bias[n:], x, w[n:].T)
    else:
        y = act[c["activation"]](torch.addmm(bias, x, w.T))
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_experts(s):
    out = torch.empty(len(s["permuted_rows"]), s["x"].shape[1], dtype=torch.float64, device=DEV)
    at = s["offsets"].tolist()
    for e in range(len(at) - 1):
        if at[e] == at[e + 1]:
            continue
        x = s["x"][s["permuted_rows"][at[e]:at[e + 1]].long()].double()
        gate, up = (x @ s["w13"][e].double().T).chunk(2, dim=1)
        out[at[e]:at[e + 1]] = (gate * torch.sigmoid(gate) * up) @ s["w2"][e].double().T
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "linear": _exact_linear, "experts": _exact_experts}[case["op"]](s)

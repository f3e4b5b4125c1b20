"""Cases, plain forms and 64-bit references of the operators for routed networks around the
convolution: group normalisation with an activation over the rows of each structure, the
routing of edges to branches with its balance loss, and the gradient of the convolution's
gate.

`run` computes an operator in its plain form (elementary torch operations, 32 bits) or,
with `own` set, through the package's entry points; `exact` computes it in 64 bits from
the definitions below.

Definitions.
  group norm: x [rows, width], channels last, its width cut into `groups` groups of equal
    width c; offsets [samples + 1] give each sample's rows.  Over the M = rows c values of one
    sample and group:  mu = sum(x)/M, s2 = sum((x - mu)^2)/M, rstd = 1/sqrt(s2 + eps),
    h = (x - mu) rstd, z = h weight + bias, y = act(z); act(z) = z, z sigmoid(z) ("silu") or
    z (1 + erf(z/sqrt 2))/2 ("gelu").  Rows outside every sample: y = 0, gradient 0.
    Backward, with d = grad_out act'(z) and a = d weight:
    grad_x = rstd (a - sum(a)/M - h sum(a h)/M), grad_weight = sum over rows of d h,
    grad_bias = sum over rows of d.
  routing: logits z [rows, n]; a row whose mask is 0 takes no part.  p = softmax(z); the k
    largest of a row are chosen, ties to the lowest index: ids [rows, k], largest first, -1
    for rows without part.  gates [rows, k]: p of the chosen, divided by their sum if
    renormalised; dense: [n, rows], 0 for what was not chosen.  counts[e]: rows that chose e,
    C their sum; slope[e] = n counts[e]/(C R) with R the rows that take part;
    balance = sum over e of slope[e] (sum over rows of p[e]): n sum of f_e P_e.
    Backward: gradients of the gates and of balance, counts held fixed.
  gate gradient: the convolution's message of edge e is linear in gate[e] w[e], so that with
    grad_w = dL/dw:  dL/dgate[e] = sum over c of w[e, c] grad_w[e, c] / gate[e], 0 for edges
    that are masked or have gate 0.
"""
import math
import random

import torch

own = False

EPS = 1e-5
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
BYTES = {"float32": 4, "bfloat16": 2, "float16": 2}
ACTS = ["none", "silu", "gelu"]


def listed():
    return [
        # the 32-atom workload's 418 edges through one hidden layer of a radial network, one
        # structure: the smallest call, bound by its latency
        {"name": "gn_fwd_418x64", "op": "group_norm", "pass": "forward", "rows": 418, "width": 64, "groups": 8,
         "samples": 1, "ragged": False, "tail": 0, "act": "silu", "dtype": "float32", "pad": 0},
        # a 128-wide hidden layer in bf16 over the 114688 edges of the 4096-atom Si structure:
        # one long sample
        {"name": "gn_fwd_bf16_114688x128", "op": "group_norm", "pass": "forward", "rows": 114688, "width": 128,
         "groups": 16, "samples": 1, "ragged": False, "tail": 0, "act": "silu", "dtype": "bfloat16", "pad": 0},
        # a training batch of 28 structures of about 20060 edges each, of differing sizes: the
        # largest norm
        {"name": "gn_fwd_561680x128_28", "op": "group_norm", "pass": "forward", "rows": 561680, "width": 128,
         "groups": 8, "samples": 28, "ragged": True, "tail": 0, "act": "silu", "dtype": "float32", "pad": 0},
        # backward of a batch of 48 small molecules (418 edges on average), an odd width inside
        # wider rows
        {"name": "gn_bwd_20060x481_48", "op": "group_norm", "pass": "backward", "rows": 20060, "width": 481,
         "groups": 13, "samples": 48, "ragged": True, "tail": 0, "act": "silu", "dtype": "float32", "pad": 6},
        # backward of a bf16 hidden layer over four structures in a buffer padded to a fixed
        # number of rows
        {"name": "gn_bwd_bf16_114688x128_4", "op": "group_norm", "pass": "backward", "rows": 114688, "width": 128,
         "groups": 8, "samples": 4, "ragged": True, "tail": 3000, "act": "gelu", "dtype": "bfloat16", "pad": 0},
        # 418 edges to one of four branches: latency
        {"name": "route_fwd_418x4", "op": "route", "pass": "forward", "rows": 418, "n": 4, "k": 1, "dtype": "float32",
         "masked": False, "renorm": False, "dense": True},
        # the Si structure's edges to two of eight branches, half of them masked: the gates that
        # the convolution of each branch takes
        {"name": "route_fwd_bf16_114688x8", "op": "route", "pass": "forward", "rows": 114688, "n": 8, "k": 2,
         "dtype": "bfloat16", "masked": True, "renorm": False, "dense": True},
        # and back from the gates' gradients
        {"name": "route_bwd_114688x8", "op": "route", "pass": "backward", "rows": 114688, "n": 8, "k": 2,
         "dtype": "float32", "masked": True, "renorm": False, "dense": True},
        # many branches, the nodes of a large batch: the largest routing
        {"name": "route_fwd_131072x256", "op": "route", "pass": "forward", "rows": 131072, "n": 256, "k": 8,
         "dtype": "float32", "masked": False, "renorm": True, "dense": False},
        {"name": "route_bwd_bf16_65536x64", "op": "route", "pass": "backward", "rows": 65536, "n": 64, "k": 6,
         "dtype": "bfloat16", "masked": False, "renorm": True, "dense": False},
        # the 768-atom l <= 3 workload's edges and weights, every edge gated
        {"name": "gate_bwd_20060x2176", "op": "gate", "rows": 20060, "width": 2176, "active": 1.0},
        # the Si workload's, half of the gates 0: the largest call
        {"name": "gate_bwd_114688x1312", "op": "gate", "rows": 114688, "width": 1312, "active": 0.5},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["group_norm", "group_norm", "group_norm", "route", "route", "gate"])
        if op == "group_norm":
            rows, c = _log(rng, 1, 600000), _log(rng, 1, 256)
            # groups of 16 values at least: the gradient through a group of one or two values is
            # zero but for eps, so that 32 bits leave nothing of it but their rounding
            if rows * c < 16:
                continue
            ragged = rng.random() < 0.6
            samples = _log(rng, 1, max(1, min(rows * c // 128, 2000)))
            if not ragged:
                rows = max(1, rows // samples) * samples
                if rows // samples * c < 16:
                    continue
            case = {"op": op, "pass": rng.choice(["forward", "backward"]), "rows": rows, "groups": _log(rng, 1, 64),
                    "samples": samples, "ragged": ragged, "tail": _log(rng, 1, rows) // 2 if ragged else 0,
                    "act": rng.choice(ACTS), "dtype": rng.choice(list(DTYPES)), "pad": rng.choice([0, 0, 1, 24])}
            case["width"] = c * case["groups"]
        elif op == "route":
            n = _log(rng, 2, 1024)
            case = {"op": op, "pass": rng.choice(["forward", "backward"]), "rows": _log(rng, 1, 400000), "n": n,
                    "k": _log(rng, 1, min(n, 16)), "dtype": rng.choice(list(DTYPES)), "masked": rng.random() < 0.5,
                    "renorm": rng.random() < 0.5, "dense": n <= 16 and rng.random() < 0.7}
        else:
            case = {"op": op, "rows": _log(rng, 1, 200000), "width": _log(rng, 8, 8192),
                    "active": rng.choice([0.1, 0.5, 1.0])}
        if work(case)["bytes"] <= most / 2:
            return case


def work(case):
    rows = case["rows"]
    if case["op"] == "group_norm":
        e, stats = BYTES[case["dtype"]], 8 * case["samples"] * case["groups"]
        live, f = (rows - case["tail"]) * case["width"], case["width"]
        if case["pass"] == "forward":
            return {"bytes": (live + rows * f) * e + stats + 8 * f, "flops": 14 * live}
        return {"bytes": (2 * live + rows * f) * e + stats + 16 * f, "flops": 30 * live}
    if case["op"] == "route":
        n, k, e = case["n"], case["k"], BYTES[case["dtype"]]
        gates = (n if case["dense"] else k) * 4 * rows
        if case["pass"] == "forward":
            return {"bytes": rows * (n * e + 4 * k + case["masked"]) + gates + 8 * n, "flops": rows * n * (6 + 2 * k)}
        # of dense gates' gradients only those of the chosen are needed
        return {"bytes": rows * (2 * n * e + 8 * k) + 4 * n, "flops": rows * n * (10 + k)}
    return {"bytes": int(rows * case["active"]) * case["width"] * 8 + rows * 8, "flops": rows * case["width"] * 2}


def _lengths(case, seed):
    """Rows of each sample: a fair share each, or spread over a factor of eight; a few of none
    in large ragged batches."""
    live, n = case["rows"] - case["tail"], case["samples"]
    if not case["ragged"]:
        return [live // n] * n
    r = random.Random(seed * 7919 + 13)
    share = [0.0 if n > 16 and r.random() < 0.03 else math.exp(r.uniform(0, math.log(8))) for _ in range(n)]
    share[0] = max(share[0], 1.0)
    at, total, cuts = 0.0, sum(share), [0]
    for q in share:
        at += q
        cuts.append(min(live, int(round(live * at / total))))
    cuts[-1] = live
    return [b - a for a, b in zip(cuts, cuts[1:])]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen)

    def uniform(*shape):
        return torch.rand(*shape, device=dev, generator=gen)

    s, rows = {"case": case}, case["rows"]
    if case["op"] == "group_norm":
        f, g, dt = case["width"], case["groups"], DTYPES[case["dtype"]]

        def rowwise(v):
            """v as the leading columns of rows that are `pad` wider."""
            wide = torch.zeros(rows, f + case["pad"], dtype=dt, device=dev)
            wide[:, :f] = v
            return wide[:, :f]

        lengths = _lengths(case, seed)
        s["each"], s["longest"] = lengths, max(lengths)
        s["lengths"] = torch.tensor(lengths, device=dev)
        s["offsets"] = torch.tensor([0] + lengths, device=dev).cumsum(0).int()
        # what a user passes: equal samples by their number, others by their offsets
        s["samples"] = s["offsets"] if case["ragged"] else case["samples"]
        # hidden rows: channels of differing spread and offset
        s["x"] = rowwise(normal(rows, f) * (0.3 + 1.5 * uniform(f)) + normal(f))
        s["weight"] = 1 + 0.2 * normal(f)
        s["bias"] = 0.2 * normal(f)
        if case["pass"] == "backward":
            s["grad_out"] = rowwise(normal(rows, f))
            s["stats"] = _group_stats(s)
        return s
    if case["op"] == "route":
        n, k = case["n"], case["k"]
        # a router prefers some branches over others
        s["logits"] = (1.5 * normal(rows, n) + 0.7 * normal(n)).to(DTYPES[case["dtype"]])
        s["mask"] = (uniform(rows) < 0.5).to(torch.uint8) if case["masked"] else None
        if case["pass"] == "backward":
            got = _route_forward(s)
            s["route"] = got
            s["grad_gates"] = normal(*got["gates"].shape)
            s["grad_balance"] = normal(1)
            if own:
                import clebsch_gordan_tensor_node_amd as C
                s["route"] = C.Route(got["ids"], got["gates"], got["counts"], got["balance"], got["slope"],
                                     case["renorm"], case["dense"])
        return s
    s["w"] = normal(rows, case["width"])
    s["gate"] = torch.where(uniform(rows) < case["active"], 1 - uniform(rows), 0.0)
    # the convolution's weight gradient, which carries the gate as a factor
    s["grad_w"] = normal(rows, case["width"]) * s["gate"][:, None]
    return s


# ---- plain forms -------------------------------------------------------------------

def _sample_of(s):
    """The sample of each live row."""
    n = s["lengths"].shape[0]
    live = s["case"]["rows"] - s["case"]["tail"]
    return torch.repeat_interleave(torch.arange(n, device=s["lengths"].device), s["lengths"], output_size=live)


def _per_sample(v, s):
    """Sums over each sample's rows of v [live, g], in 64 bits: one by one, or where there are
    many samples as differences of running sums."""
    if len(s["each"]) <= 64:
        return torch.stack([q.sum(0, dtype=torch.float64) for q in v.split(s["each"])])
    run = torch.nn.functional.pad(v.t().double().cumsum(1), (1, 0))
    cuts = run[:, s["offsets"].long()]
    return (cuts[:, 1:] - cuts[:, :-1]).t()


def _group_stats(s):
    case = s["case"]
    g, c = case["groups"], case["width"] // case["groups"]
    seg = _sample_of(s)
    x = s["x"][:seg.shape[0]].float().reshape(-1, g, c)
    m = (s["lengths"] * c).clamp(min=1)[:, None]
    mean = (_per_sample(x.sum(2), s) / m).float()
    var = _per_sample((x - mean[seg][:, :, None]).square().sum(2), s) / m
    return torch.stack([mean, (1 / torch.sqrt(var + EPS)).float()])


def _pointwise(z, act):
    """act(z) and act'(z)."""
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * p, p + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return z, torch.ones_like(z)


def _normed(s, stats):
    """h [live, g, c], z likewise, and the rows' rstd [live, g, 1]."""
    g = s["case"]["groups"]
    seg = _sample_of(s)
    x = s["x"][:seg.shape[0]].float().reshape(seg.shape[0], g, -1)
    rstd = stats[1][seg][:, :, None]
    h = (x - stats[0][seg][:, :, None]) * rstd
    return h, h * s["weight"].view(1, g, -1) + s["bias"].view(1, g, -1), rstd, seg


def _whole(v, s):
    """Live rows [live, g, c] as rows of x's type, zeros behind them."""
    case = s["case"]
    out = torch.zeros(case["rows"], case["width"], dtype=s["x"].dtype, device=v.device)
    out[:v.shape[0]] = v.reshape(v.shape[0], -1).to(out.dtype)
    return out


def _group_norm(s):
    case = s["case"]
    if case["pass"] == "forward":
        stats = _group_stats(s)
        _, z, _, _ = _normed(s, stats)
        return {"y": _whole(_pointwise(z, case["act"])[0], s), "stats": stats}
    h, z, rstd, seg = _normed(s, s["stats"])
    g, c = case["groups"], case["width"] // case["groups"]
    d = s["grad_out"][:seg.shape[0]].float().reshape(h.shape) * _pointwise(z, case["act"])[1]
    a = d * s["weight"].view(1, g, c)
    m = (s["lengths"] * c).clamp(min=1)[:, None]
    sa = (_per_sample(a.sum(2), s) / m).float()[seg][:, :, None]
    sh = (_per_sample((a * h).sum(2), s) / m).float()[seg][:, :, None]
    return {"grad_x": _whole((a - sa - h * sh) * rstd, s),
            "grad_weight": (d * h).double().sum(0).float().view(-1), "grad_bias": d.double().sum(0).float().view(-1)}


def _route_forward(s):
    case = s["case"]
    rows, n, k = case["rows"], case["n"], case["k"]
    z = s["logits"].float()
    live = torch.ones(rows, dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"] != 0
    e = torch.exp(z - z.max(1, keepdim=True).values)
    p = e / e.sum(1, keepdim=True) * live[:, None]
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    gates = torch.gather(p, 1, ids)
    if case["renorm"]:
        top = torch.gather(e, 1, ids)
        gates = top / top.sum(1, keepdim=True) * live[:, None]
    chosen = torch.zeros(rows, n, dtype=torch.bool, device=z.device).scatter_(1, ids, live[:, None].expand(rows, k))
    counts = chosen.sum(0)
    slope = (n * counts.double() / (counts.sum() * live.sum()).clamp(min=1)).float()
    balance = (slope * p.double().sum(0)).sum().float().view(1)
    if case["dense"]:
        gates = torch.zeros(rows, n, device=z.device).scatter_(1, ids, gates).t().contiguous()
    return {"ids": torch.where(live[:, None], ids, -1).int(), "gates": gates, "counts": counts.int(),
            "balance": balance, "slope": slope}


def _route_backward(s):
    case, r = s["case"], s["route"]
    rows = case["rows"]
    z, ids = s["logits"].float(), r["ids"].long()
    live, at = ids[:, :1] >= 0, ids.clamp(min=0)
    e = torch.exp(z - z.max(1, keepdim=True).values)
    p = e / e.sum(1, keepdim=True)
    up = s["grad_gates"]
    if case["dense"]:
        up = torch.gather(up.t(), 1, at)
    a = (s["grad_balance"] * r["slope"]).expand(rows, -1)
    if case["renorm"]:
        top = torch.gather(e, 1, at)
        q = top / top.sum(1, keepdim=True)
        grad = p * (a - (a * p).sum(1, keepdim=True))
        grad = grad.scatter_add(1, at, q * (up - (up * q).sum(1, keepdim=True)))
    else:
        a = a.scatter_add(1, at, up)
        grad = p * (a - (a * p).sum(1, keepdim=True))
    return {"grad_logits": torch.where(live, grad, 0.0).to(s["logits"].dtype)}


def _gate_backward(s):
    dot = (s["w"] * s["grad_w"]).sum(1)
    return {"grad_gate": torch.where(s["gate"] != 0, dot / s["gate"], 0.0)}


# ---- one pass ----------------------------------------------------------------------

def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "group_norm":
            return _group_norm(s)
        if case["op"] == "gate":
            return _gate_backward(s)
        if case["pass"] == "backward":
            return _route_backward(s)
        got = _route_forward(s)
        return {q: got[q] for q in ("ids", "gates", "counts", "balance")}
    import clebsch_gordan_tensor_node_amd as C
    if case["op"] == "group_norm":
        act = None if case["act"] == "none" else case["act"]
        if case["pass"] == "forward":
            y, stats = C.group_norm_forward(s["x"], case["groups"], s["weight"], s["bias"], samples=s["samples"],
                                            activation=act, eps=EPS, longest=s["longest"])
            return {"y": y, "stats": stats}
        got = C.group_norm_backward(s["grad_out"], s["x"], s["stats"], case["groups"], s["weight"], s["bias"],
                                    samples=s["samples"], activation=act, longest=s["longest"])
        return dict(zip(("grad_x", "grad_weight", "grad_bias"), got))
    if case["op"] == "gate":
        return {"grad_gate": C.conv_gate_backward(s["w"], s["grad_w"], s["gate"])}
    if case["pass"] == "backward":
        return {"grad_logits": C.route_backward(s["logits"], s["route"], s["grad_gates"], s["grad_balance"])}
    r = C.route_forward(s["logits"], case["k"], mask=s["mask"], renormalise=case["renorm"], dense=case["dense"])
    return {"ids": r.ids, "gates": r.gates, "counts": r.counts, "balance": r.balance}


# ---- 64 bits -----------------------------------------------------------------------

def _exact_act(z, act):
    z = z.detach().requires_grad_()
    y = {"none": lambda: z * 1.0, "silu": lambda: z * torch.sigmoid(z),
         "gelu": lambda: z * torch.special.ndtr(z)}[act]()
    return y.detach(), torch.autograd.grad(y.sum(), z)[0]


def _exact_group_norm(case, s):
    cuts = s["offsets"].tolist()
    g, f = case["groups"], case["width"]
    w, b = s["weight"].double(), s["bias"].double()
    x = s["x"].double()
    out = torch.zeros_like(x)
    means = torch.zeros(case["samples"], g, dtype=torch.float64, device=x.device)
    rstds = torch.full_like(means, EPS ** -0.5)
    gw, gb = torch.zeros_like(w), torch.zeros_like(b)
    for k, (lo, hi) in enumerate(zip(cuts, cuts[1:])):
        if hi == lo:
            continue
        q = x[lo:hi].view(hi - lo, g, f // g)
        if case["pass"] == "forward":
            var, mean = torch.var_mean(q, dim=(0, 2), correction=0)
            means[k], rstds[k] = mean, (var + EPS) ** -0.5
        else:
            mean, rstd = s["stats"][0, k].double(), s["stats"][1, k].double()
            means[k], rstds[k] = mean, rstd
        h = (q - means[k].view(1, g, 1)) * rstds[k].view(1, g, 1)
        y, slope = _exact_act(h.view(hi - lo, f) * w + b, case["act"])
        if case["pass"] == "forward":
            out[lo:hi] = y
            continue
        d = s["grad_out"][lo:hi].double() * slope
        gb += d.sum(0)
        gw += (d * h.view(hi - lo, f)).sum(0)
        a = (d * w).view(hi - lo, g, f // g)
        v = a - a.mean((0, 2), keepdim=True) - h * (a * h).mean((0, 2), keepdim=True)
        out[lo:hi] = (v * rstds[k].view(1, g, 1)).view(hi - lo, f)
    if case["pass"] == "forward":
        return {"y": out, "stats": torch.stack([means, rstds])}
    return {"grad_x": out, "grad_weight": gw, "grad_bias": gb}


def _exact_route(case, s):
    z = s["logits"].double()
    rows, n, k = case["rows"], case["n"], case["k"]
    p = torch.softmax(z, 1)
    if case["pass"] == "backward":
        r = s["route"]
        ids, slope = (r.ids, r.slope) if own else (r["ids"], r["slope"])
        live = ids[:, 0] >= 0
        take = torch.zeros(rows, n, dtype=torch.float64, device=z.device)
        take.scatter_(1, ids.clamp(min=0).long(), 1.0)
        up = s["grad_gates"].double()
        up = up.t() * take if case["dense"] else torch.zeros_like(take).scatter_(1, ids.clamp(min=0).long(), up)
        a = s["grad_balance"].double() * slope.double()
        grad = p * (a - p @ a[:, None])
        if case["renorm"]:
            q = p * take / (p * take).sum(1, keepdim=True)
            grad = grad + q * (up - (up * q).sum(1, keepdim=True))
        else:
            grad = grad + p * (up - (up * p).sum(1, keepdim=True))
        return {"grad_logits": grad * live[:, None]}
    live = torch.ones(rows, dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"].bool()
    # whole numbers in the order of (logit, index from the last to the first): no ties among them
    bits = (s["logits"].float() + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7fffffff), bits) * 4096 + torch.arange(n - 1, -1, -1, device=z.device)
    ids = torch.topk(key, k, dim=1).indices
    take = torch.zeros(rows, n, dtype=torch.float64, device=z.device).scatter_(1, ids, 1.0) * live[:, None]
    counts = take.sum(0)
    share = p * take
    if case["renorm"]:
        share = share / share.sum(1, keepdim=True).clamp(min=1e-300)
    balance = n * (counts / counts.sum().clamp(min=1) * (p * live[:, None]).sum(0) / live.sum().clamp(min=1)).sum()
    return {"ids": torch.where(live[:, None], ids, -1).int(),
            "gates": share.t().contiguous() if case["dense"] else torch.gather(share, 1, ids),
            "counts": counts.int(), "balance": balance.view(1)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "group_norm":
        return _exact_group_norm(case, s)
    if case["op"] == "route":
        return _exact_route(case, s)
    dot = (s["w"].double() * s["grad_w"].double()).sum(1)
    return {"grad_gate": torch.where(s["gate"] != 0, dot / s["gate"].double(), 0.0)}

"""Cases, plain forms and 64-bit references of the operators that train a network around
the convolution: layer normalisation of rows, its equivariant form over irreps, and the
AdamW step over many tensors with its gradient norm.

`run` computes an operator in its plain form (elementary torch operations, 32 bits) or,
with `own` set, through the package's entry points; `exact` computes it in 64 bits from
the definitions below.

Definitions.
  layer norm, row x of width F:  mu = sum(x)/F, s2 = sum((x - mu)^2)/F,
    rstd = 1/sqrt(s2 + eps), h = (x - mu) rstd, y = h weight + bias.
    Backward, with a = grad_out weight:  grad_x = rstd (a - sum(a)/F - h sum(a h)/F);
    grad_weight = sum over rows of grad_out h, grad_bias = sum over rows of grad_out.
  irreps norm, one term "mul x l p" of a row at a time, its block [mul][2l+1] of F values:
    0e terms as the layer norm (weight and bias per channel); other terms with mu = 0, a
    weight per channel that its 2l+1 components share, and no bias.
  AdamW, step t:  g = grad * grad_scale;  p <- p (1 - lr wd);  m <- b1 m + (1 - b1) g;
    v <- b2 v + (1 - b2) g^2;  p <- p - (lr/(1 - b1^t)) m / (sqrt(v)/sqrt(1 - b2^t) + eps).
    With clip, grad_scale = min(1, max_norm/|grad|_2) over all tensors.
  AdamW with 8-bit states holds m and r = sqrt(v) as codes over blocks of 64 elements with
    one exponent byte E, the biased fp32 exponent of the block's largest magnitude a:
    m: sign, 4 exponent and 3 mantissa bits, r: 4 exponent and 4 mantissa bits; the code is
    the top bits of the fp32 number a 2^(14 - E), whose lower bits are rounded up or down by
    16 bits of a hash of (element, seed): code = (bits + u 2^k) >> (k + 16), k = 4 for m and
    3 for r.  A positive r is stored as code 1 at least.  p is updated from the values
    before they are rounded.
"""
import math
import random

import torch

own = False

EPS = 1e-5
LR, B1, B2, ADAM_EPS, DECAY, MAX_NORM = 1e-4, 0.9, 0.999, 1e-8, 0.01, 1.0
BLOCK = 64                                   # elements that share one exponent byte
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
BYTES = {"float32": 4, "bfloat16": 2, "float16": 2}


def listed():
    si = "128x0e+64x1o+32x2e+32x3o"
    return [
        # the 32-atom workload's 418 edges through one hidden layer of a radial network: the
        # smallest call, bound by its latency
        {"name": "ln_fwd_418x64", "op": "layer_norm", "pass": "forward", "rows": 418, "width": 64,
         "dtype": "float32", "pad": 0},
        # every edge's convolution weights of the 4096-atom Si workload (114688 edges, 1312
        # columns), normalised before the convolution: the largest call
        {"name": "ln_fwd_114688x1312", "op": "layer_norm", "pass": "forward", "rows": 114688, "width": 1312,
         "dtype": "float32", "pad": 0},
        # backward of a 128-wide hidden layer in bf16 over the same edges
        {"name": "ln_bwd_bf16_114688x128", "op": "layer_norm", "pass": "backward", "rows": 114688, "width": 128,
         "dtype": "bfloat16", "pad": 0},
        # backward over the 20060 edges of the 768-atom workloads at an odd width, rows inside
        # wider ones (a column range of a fused buffer)
        {"name": "ln_bwd_20060x481", "op": "layer_norm", "pass": "backward", "rows": 20060, "width": 481,
         "dtype": "float32", "pad": 6},
        # the 32-atom workload's convolution output
        {"name": "irreps_fwd_32", "op": "irreps_norm", "pass": "forward", "rows": 32,
         "irreps": "16x0e+8x1e+16x1o", "dtype": "float32", "pad": 0},
        # the Si workload's convolution output, 4096 nodes of 5472 features
        {"name": "irreps_fwd_si_out", "op": "irreps_norm", "pass": "forward", "rows": 4096,
         "irreps": "256x0e+352x1o+384x2e+320x3o", "dtype": "float32", "pad": 0},
        # backward behind the 768-atom l <= 3 workload's convolution output
        {"name": "irreps_bwd_c2_out", "op": "irreps_norm", "pass": "backward", "rows": 768,
         "irreps": "384x0e+640x1o+640x2e+512x3o", "dtype": "float32", "pad": 0},
        # backward at the Si workload's hidden irreps, a box of 16^3 cells (32768 atoms)
        {"name": "irreps_bwd_si_hidden", "op": "irreps_norm", "pass": "backward", "rows": 32768,
         "irreps": si, "dtype": "float32", "pad": 0},
        # the step of a small potential, 24 tensors, gradients clipped by their norm: bound by
        # its launches
        {"name": "adamw32_24_small", "op": "adamw", "tensors": 24, "largest": 8192, "bits": 32,
         "param": "float32", "grad": "float32", "clip": True},
        # a large one, 160 tensors of up to 4 million elements, clipped
        {"name": "adamw32_160_large", "op": "adamw", "tensors": 160, "largest": 4194304, "bits": 32,
         "param": "float32", "grad": "float32", "clip": True},
        # 8-bit states behind bf16 gradients scaled for their range, tensors of mixed sizes
        {"name": "adamw8_96_bf16grad", "op": "adamw", "tensors": 96, "largest": 300001, "bits": 8,
         "param": "float32", "grad": "bfloat16", "clip": False},
        # 8-bit states of a large network, 300 tensors
        {"name": "adamw8_300_large", "op": "adamw", "tensors": 300, "largest": 2097152, "bits": 8,
         "param": "float32", "grad": "float32", "clip": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["layer_norm", "layer_norm", "irreps_norm", "irreps_norm", "adamw", "adamw"])
        if op == "adamw":
            bits = rng.choice([32, 8])
            # the outcome of a stochastic rounding hangs on the last bit of what is rounded, and
            # a norm's last bit on the order of its sum: clipping goes with 32-bit states
            c = {"op": op, "tensors": _log(rng, 1, 400), "largest": _log(rng, 1, 4194304), "bits": bits,
                 "param": rng.choice(["float32", "float32", "bfloat16"]) if bits == 32 else "float32",
                 "grad": rng.choice(["float32", "bfloat16", "float16"]), "clip": bits == 32 and rng.random() < 0.5}
        else:
            c = {"op": op, "pass": rng.choice(["forward", "backward"]), "dtype":
                 rng.choice(["float32", "float32", "bfloat16", "float16"]), "pad": rng.choice([0, 0, 1, 24])}
            # rows of four values at least: the gradient of a row of two is zero but for eps, so
            # that 32 bits leave nothing of it but their rounding
            if op == "layer_norm":
                c |= {"rows": _log(rng, 1, 262144), "width": _log(rng, 4, 8192)}
            else:
                lmax = rng.randint(0, 6)
                c |= {"rows": _log(rng, 1, 65536), "irreps": "+".join(
                    "%dx%d%s" % (_log(rng, 1 if l else 4, 512), l, rng.choice("eo")) for l in range(lmax + 1))}
        # the largest listed case bounds the bytes, and a backward pass costs as much again
        if work(c)["bytes"] <= most / 2:
            return c


def _terms(irreps):
    """(offset, channels, components, first weight, first bias or None) of each term."""
    out, off, w, b = [], 0, 0, 0
    for term in irreps.split("+"):
        mul, ir = term.split("x")
        mul, l, even = int(mul), int(ir[:-1]), ir[-1] == "e"
        centred = l == 0 and even
        out.append((off, mul, 2 * l + 1, w, b if centred else None))
        off, w, b = off + mul * (2 * l + 1), w + mul, b + mul * centred
    return out


def _shape(case):
    """(features, weights, biases, terms) of a norm case."""
    if case["op"] == "layer_norm":
        f = case["width"]
        return f, f, f, [(0, f, 1, 0, 0)]
    t = _terms(case["irreps"])
    return (sum(m * d for _, m, d, _, _ in t), sum(m for _, m, _, _, _ in t),
            sum(m for _, m, _, _, b in t if b is not None), t)


def _sizes(case):
    """Element counts of an AdamW case's tensors: spread over their logarithm, the largest first."""
    r = random.Random(case["tensors"] * 1000003 + case["largest"])
    return [case["largest"]] + [_log(r, 1, case["largest"]) for _ in range(case["tensors"] - 1)]


def _offsets(sizes):
    """Each tensor's place among the states (whole blocks), and their length."""
    at, offs = 0, []
    for n in sizes:
        offs.append(at)
        at += -(-n // BLOCK) * BLOCK
    return offs, at


def work(case):
    if case["op"] == "adamw":
        n, b = sum(_sizes(case)), BYTES
        p, g = b[case["param"]], b[case["grad"]]
        if case["bits"] == 32:
            return {"bytes": n * (2 * p + g + 16), "flops": n * (16 + 3 * case["clip"])}
        # codes and exponents read and written, and their values written out in 16 bits
        return {"bytes": n * (2 * p + g + 4 + 4 / BLOCK + 4), "flops": n * 30}
    f, w, bias, t = _shape(case)
    n, e = case["rows"] * f, BYTES[case["dtype"]]
    stats = 8 * case["rows"] * len(t)
    if case["pass"] == "forward":
        return {"bytes": 2 * n * e + stats + 4 * (w + bias), "flops": 8 * n}
    return {"bytes": 3 * n * e + stats + 4 * (2 * w + bias), "flops": 14 * n}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen)

    s = {"case": case}
    if case["op"] != "adamw":
        f, w, bias, t = _shape(case)
        rows, dt = case["rows"], DTYPES[case["dtype"]]

        def rowwise(v):
            """v as the leading columns of rows that are `pad` wider."""
            wide = torch.zeros(rows, f + case["pad"], dtype=dt, device=dev)
            wide[:, :f] = v
            return wide[:, :f]

        # activations: rows of differing spread, and a common offset
        x = normal(rows, f).mul_(0.2 + 2 * torch.rand(rows, 1, device=dev, generator=gen)).add_(normal(rows, 1))
        s["x"] = rowwise(x)
        s["weight"] = 1 + 0.2 * normal(w)
        s["bias"] = 0.2 * normal(bias)
        if case["pass"] == "backward":
            s["grad_out"] = rowwise(normal(rows, f))
            s["stats"] = _norm_stats(s["x"].float(), t)
            if case["op"] == "layer_norm":
                s["stats"] = s["stats"].view(2, rows)
        if own and case["op"] == "irreps_norm":
            import clebsch_gordan_tensor_node_amd as C
            s["plan"] = C.NormPlan(case["irreps"])
        return s
    sizes = _sizes(case)
    offs, total = _offsets(sizes)
    count = torch.tensor([b - a for a, b in zip(offs, offs[1:] + [total])], device=dev)
    first = torch.repeat_interleave(torch.tensor(offs, device=dev), count, output_size=total)
    long = torch.repeat_interleave(torch.tensor(sizes, device=dev), count, output_size=total)
    inside = torch.arange(total, device=dev) - first < long
    # gradients of very different size from tensor to tensor, one element in sixteen exactly
    # zero (features that no edge of this batch has)
    each = torch.rand(len(sizes), device=dev, generator=gen).mul_(-2.5).sub_(0.5)
    scale = torch.repeat_interleave(torch.pow(10.0, each), count, output_size=total) * inside
    dead = torch.rand(total, device=dev, generator=gen) < 1 / 16
    grad = torch.where(dead, 0.0, normal(total) * scale)
    m = (0.3 * normal(total)) * scale
    v = ((0.5 + torch.rand(total, device=dev, generator=gen)) * scale).square_()
    s["p"] = (0.5 * normal(total) * inside).to(DTYPES[case["param"]])
    # in 16 bits the gradients come scaled, as a scaled loss gives them
    s["grad_scale"] = torch.tensor([1.0 if case["grad"] == "float32" else 1 / 64], device=dev)
    s["grad"] = (grad / s["grad_scale"]).to(DTYPES[case["grad"]])
    s["decay"] = [DECAY if n > 1024 else 0.0 for n in sizes]
    kept = torch.tensor([1 - LR * d for d in s["decay"]], dtype=torch.float32, device=dev)
    s["kept"] = torch.repeat_interleave(kept, count, output_size=total)
    s["t"] = 1000
    if case["bits"] == 32:
        s["moments"] = (m, v)
    else:
        half = torch.full((total,), 32768, dtype=torch.int64, device=dev)
        (mc, me), (rc, re) = _encode(m, half, True), _encode(torch.sqrt(v), half, False)
        s["moments"] = (mc, rc, me, re)
    if own:
        import clebsch_gordan_tensor_node_amd as C
        s["set"] = C.ParamSet(sizes, s["decay"])
        s["params"] = s["set"].pointers([s["p"][a:a + n] for a, n in zip(offs, sizes)])
        s["grads"] = s["set"].pointers([s["grad"][a:a + n] for a, n in zip(offs, sizes)])
    return s


# ---- plain forms -------------------------------------------------------------------

def _term_stats(x, mul, d, centred):
    mean = x.sum(1) / (mul * d) if centred else torch.zeros_like(x[:, 0])
    var = (x - mean[:, None]).square().sum(1) / (mul * d)
    return mean, 1 / torch.sqrt(var + EPS)


def _norm_stats(x, terms):
    both = [_term_stats(x[:, o:o + m * d], m, d, b is not None) for o, m, d, _, b in terms]
    return torch.stack([torch.stack([a for a, _ in both], 1), torch.stack([r for _, r in both], 1)])


def _spread(w, d):
    return w[:, None].expand(w.shape[0], d).reshape(-1)


def _norm_forward(s):
    _, _, _, terms = _shape(s["case"])
    x = s["x"].float()
    stats = _norm_stats(x, terms)
    ys = [(x[:, o:o + m * d] - stats[0, :, k, None]) * stats[1, :, k, None] * _spread(s["weight"][w:w + m], d)
          + (0 if b is None else s["bias"][b:b + m]) for k, (o, m, d, w, b) in enumerate(terms)]
    return torch.cat(ys, 1).to(s["x"].dtype), stats


def _term_backward(x, g, mean, rstd, w, mul, d, centred):
    h = (x - mean[:, None]) * rstd[:, None]
    a = g * _spread(w, d)
    gx = a - h * (a * h).sum(1, keepdim=True) / (mul * d)
    if centred:
        gx = gx - a.sum(1, keepdim=True) / (mul * d)
    return gx * rstd[:, None], (g * h).sum(0).view(mul, d).sum(1), g.sum(0) if centred else g.new_zeros(0)


def _norm_backward(s):
    _, _, _, terms = _shape(s["case"])
    x, g = s["x"].float(), s["grad_out"].float()
    stats = s["stats"].view(2, x.shape[0], len(terms))
    got = [_term_backward(x[:, o:o + m * d], g[:, o:o + m * d], stats[0, :, k], stats[1, :, k],
                          s["weight"][w:w + m], m, d, b is not None) for k, (o, m, d, w, b) in enumerate(terms)]
    return torch.cat([q[0] for q in got], 1).to(s["x"].dtype), torch.cat([q[1] for q in got]), torch.cat([q[2] for q in got])


MASK32 = 0xffffffff


def _random_bits(n, seed, dev):
    """32 bits for each state element, by the seed."""
    i = torch.arange(n, device=dev)
    h = ((i & MASK32) * 0x9E3779B9 + (i >> 32) * 0x6A09E667 + ((seed * 0x3C6EF373) & MASK32)) & MASK32
    h = h ^ (h >> 15)
    h = (h * 0xBB67AE85) & MASK32
    return h ^ (h >> 16)


def _power(e):
    """2^e as fp32, from its bits (-126 <= e <= 127)."""
    return ((e + 127) << 23).view(torch.float32)


def _encode(a, u, signed):
    """Codes (uint8) and exponent bytes of a, u: 16 random bits for each element."""
    top = a.abs().view(-1, BLOCK).max(1).values.view(torch.int32) >> 23
    small = a.abs().view(-1, BLOCK) * _power(126 - top.clamp(1, 252))[:, None] * 2.0 ** -112
    shift = 20 if signed else 19
    code = (small.view(torch.int32).view(-1) + (u << (shift - 16)).int()) >> shift
    if signed:
        code = code | ((a < 0).int() << 7)
    else:
        code = torch.where(a > 0, code.clamp(min=1), code)
    return code.to(torch.uint8), top.to(torch.uint8)


def _decode(code, top, signed):
    c = code.int().view(-1, BLOCK)
    mag = ((c & 127) << 20 if signed else c << 19).view(torch.float32) * 2.0 ** 112
    val = mag * _power(top.int().clamp(1, 252) - 126)[:, None]
    return (torch.where(c > 127, -val, val) if signed else val).view(-1)


def _adamw(s):
    case, t = s["case"], s["t"]
    s["t"] = t + 1
    n, grad = s["p"].numel(), s["grad"].float()
    out, scale = {}, s["grad_scale"]
    if case["clip"]:
        norm = torch.sqrt((grad * scale).square().sum())
        scale = scale * torch.clamp(MAX_NORM / norm, max=1.0)
        out["norm"] = norm
    if case["bits"] == 32:
        m, v = s["moments"]
    else:
        mc, rc, me, re = s["moments"]
        m, v = _decode(mc, me, True), _decode(rc, re, False).square()
    g = grad * scale
    p = s["p"].float() * s["kept"]
    m = m * B1 + g * (1 - B1)
    v = v * B2 + g * g * (1 - B2)
    root = torch.sqrt(v)
    p = p - (m * (LR / (1 - B1 ** t))) / (root * (1 / math.sqrt(1 - B2 ** t)) + ADAM_EPS)
    s["p"].copy_(p)
    out["p"] = s["p"]
    if case["bits"] == 32:
        s["moments"][0].copy_(m)
        s["moments"][1].copy_(v)
        return {**out, "m": s["moments"][0], "v": s["moments"][1]}
    h = _random_bits(n, t, grad.device)
    coded = _encode(m, h & 0xffff, True), _encode(root, h >> 16, False)
    [a.copy_(b) for a, b in zip((mc, me, rc, re), coded[0] + coded[1])]
    return {**out, "m": _decode(mc, me, True).bfloat16(), "r": _decode(rc, re, False).bfloat16()}


# ---- one pass ----------------------------------------------------------------------

def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "adamw":
            return _adamw(s)
        if case["pass"] == "forward":
            y, stats = _norm_forward(s)
            return {"y": y, "stats": stats.view(2, -1) if case["op"] == "layer_norm" else stats}
        return dict(zip(("grad_x", "grad_weight", "grad_bias"), _norm_backward(s)))
    import clebsch_gordan_tensor_node_amd as C
    if case["op"] == "layer_norm":
        if case["pass"] == "forward":
            return dict(zip(("y", "stats"), C.layer_norm_forward(s["x"], s["weight"], s["bias"], EPS)))
        got = C.layer_norm_backward(s["grad_out"], s["x"], s["stats"], s["weight"])
        return dict(zip(("grad_x", "grad_weight", "grad_bias"), got))
    if case["op"] == "irreps_norm":
        if case["pass"] == "forward":
            return dict(zip(("y", "stats"), C.irreps_norm_forward(s["plan"], s["x"], s["weight"], s["bias"], EPS)))
        got = C.irreps_norm_backward(s["plan"], s["grad_out"], s["x"], s["stats"], s["weight"])
        return dict(zip(("grad_x", "grad_weight", "grad_bias"), got))
    t = s["t"]
    s["t"] = t + 1
    out, scale = {}, s["grad_scale"]
    if case["clip"]:
        norm = C.grad_norm(s["set"], s["grads"], MAX_NORM, grad_scale=scale)
        out["norm"], scale = norm[0], norm[1:]
    C.adamw_step(s["set"], s["params"], s["grads"], s["moments"], lr=LR, betas=(B1, B2), eps=ADAM_EPS, step=t,
                 grad_scale=scale, seed=t)
    out["p"] = s["p"]
    if case["bits"] == 32:
        return {**out, "m": s["moments"][0], "v": s["moments"][1]}
    return {**out, **dict(zip(("m", "r"), C.adamw_moments(s["set"], s["moments"])))}


# ---- 64 bits -----------------------------------------------------------------------

def _code64(value, bits, mantissa):
    """The values that stochastic rounding stores for `value` (fp64, >= 0 or signed)."""
    a = value.abs()
    top = torch.frexp(a.view(-1, BLOCK).max(1, keepdim=True).values)[1].sub(1).expand(-1, BLOCK).reshape(-1)
    # the grid: 2^mantissa steps per octave down to 13 octaves below the block's, even steps below
    octave = torch.maximum(torch.frexp(a)[1] - 1, top - 13)
    step = torch.ldexp(torch.ones_like(a), octave - mantissa)
    kept = torch.floor(a / step + bits.double() / 65536) * step
    return kept, step, top


def _exact_adamw(case, s):
    t = s["t"]
    sizes = _sizes(case)
    offs, total = _offsets(sizes)
    p, g = s["p"].double(), s["grad"].double() * s["grad_scale"].double()
    out = {}
    if case["clip"]:
        out["norm"] = torch.linalg.vector_norm(g)
        g = g * min(1.0, MAX_NORM / float(out["norm"]))
    if case["bits"] == 32:
        m, v = (q.double() for q in s["moments"])
    else:
        mc, rc, me, re = (q.long() for q in s["moments"])

        def value(code, top, mant):
            x, f = code >> mant, code & ((1 << mant) - 1)
            y = torch.where(x > 0, f + (1 << mant), f).double()
            e = x.clamp(min=1) - 14 - mant + top.repeat_interleave(BLOCK) - 127
            return torch.ldexp(y, e)

        m = value(mc & 127, me, 3) * torch.where(mc > 127, -1.0, 1.0)
        v = value(rc, re, 4) ** 2
    m = B1 * m + (1 - B1) * g
    v = B2 * v + (1 - B2) * g ** 2
    wd = torch.zeros(total, dtype=torch.float64, device=p.device)
    for a, n in zip(offs, sizes):
        wd[a:a + n] = DECAY if n > 1024 else 0.0
    out["p"] = p - LR * wd * p - LR * (m / (1 - B1 ** t)) / (torch.sqrt(v / (1 - B2 ** t)) + ADAM_EPS)
    if case["bits"] == 32:
        return {**out, "m": m, "v": v}
    h = _random_bits(total, t, p.device)
    r = torch.sqrt(v)
    km, _, _ = _code64(m, h & 0xffff, 3)
    kr, step, top = _code64(r, h >> 16, 4)
    least = torch.ldexp(torch.ones_like(r), top - 13 - 4)
    return {**out, "m": torch.sign(m) * km, "r": torch.where((r > 0) & (kr == 0), least, kr)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, s)
    _, _, _, terms = _shape(case)
    x, w, b = (s[k].double() for k in ("x", "weight", "bias"))
    n = x.shape[0]
    ys, gxs, gws, gbs, means, rstds = [], [], [], [], [], []
    for k, (off, mul, d, w0, b0) in enumerate(terms):
        q = x[:, off:off + mul * d].reshape(n, mul, d)
        scale = w[w0:w0 + mul].view(1, mul, 1)
        if case["pass"] == "forward":
            mean = q.mean((1, 2)) if b0 is not None else torch.zeros(n, dtype=torch.float64, device=x.device)
            rstd = (((q - mean.view(n, 1, 1)) ** 2).mean((1, 2)) + EPS) ** -0.5
            y = (q - mean.view(n, 1, 1)) * rstd.view(n, 1, 1) * scale
            if b0 is not None:
                y = y + b[b0:b0 + mul].view(1, mul, 1)
            ys.append(y.reshape(n, -1))
            means.append(mean)
            rstds.append(rstd)
        else:
            st = s["stats"].double().view(2, n, len(terms))[:, :, k]
            h = (q - st[0].view(n, 1, 1)) * st[1].view(n, 1, 1)
            g = s["grad_out"][:, off:off + mul * d].double().reshape(n, mul, d)
            a = g * scale
            gx = a - h * (a * h).mean((1, 2), keepdim=True)
            if b0 is not None:
                gx = gx - a.mean((1, 2), keepdim=True)
                gbs.append(g.sum((0, 2)))
            gxs.append((gx * st[1].view(n, 1, 1)).reshape(n, -1))
            gws.append((g * h).sum((0, 2)))
    if case["pass"] == "forward":
        stats = torch.stack([torch.stack(means, 1), torch.stack(rstds, 1)])
        return {"y": torch.cat(ys, 1), "stats": stats.view(2, n) if case["op"] == "layer_norm" else stats}
    return {"grad_x": torch.cat(gxs, 1), "grad_weight": torch.cat(gws),
            "grad_bias": torch.cat(gbs) if gbs else x.new_zeros(0)}

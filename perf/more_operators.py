"""Cases of the operators around a layer's products: the norms before and after a block with
its gate and residual, log probabilities of given tokens with entropy and alternatives, and
AdamW over many tensors with states in 8 or 32 bits.

`run` computes a case either in plain torch operations in 32 bits (`own` false) or with
this package's kernels (`own` true); `exact` computes it in 64 bits.  The widths are those
of this repository's workloads (LLaMA-7B layers, 4096 and 11008 features; micro-batches of up to
16384 tokens), vocabularies 32000 tokens and generic wide ones.
"""

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}
LAYER = [4096 * 4096] * 4 + [11008 * 4096] * 3  # one LLaMA-7B layer's matrices
NORM_ELEMS = 16384 * 4096
LOGIT_ELEMS = 8192 * 32000
TOP_ELEMS = 1 << 25  # alternatives are asked for while answering: a batch of tokens, not a micro-batch
ADAMW = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "step": 100}
DECAY = 0.1


# -- cases ------------------------------------------------------------------------

def listed():
    return [
        # one token answered: the norms between two blocks, where a launch's latency counts
        {"name": "norm 1x4096", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "alone": False, "post": True,
         "gate": "column", "block": 0},
        # a micro-batch of 8 sequences of 2048 tokens; the output's checkpoint is what the next
        # product's weight gradient reads
        {"name": "norm 16384x4096 ckpt", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16", "alone": False,
         "post": True, "gate": "column", "block": 64},
        # its backward pass, all three column sums
        {"name": "norm backward 16384x4096", "op": "norm_backward", "rows": 16384, "cols": 4096, "dtype": "bf16",
         "alone": False, "post": True, "gate": "column"},
        # a model kept in fp32 with an odd width, gated per element, a ragged number of tokens
        {"name": "norm backward 1023x2047 f32", "op": "norm_backward", "rows": 1023, "cols": 2047, "dtype": "f32",
         "alone": False, "post": False, "gate": "element"},
        # one sampled token with the alternatives that a server shows beside it
        {"name": "logprobs 1x32000 top 8", "op": "logprobs", "rows": 1, "vocab": 32000, "pad": 0, "dtype": "bf16",
         "top": 8, "entropy": True, "scale": 1.25},
        # a batch of tokens over a wide vocabulary of odd size
        {"name": "logprobs 48x131071 top 20", "op": "logprobs", "rows": 48, "vocab": 131071, "pad": 0, "dtype": "bf16",
         "top": 20, "entropy": True, "scale": 1.0},
        # the loss of a training micro-batch of 8192 tokens
        {"name": "logprobs 8192x32000", "op": "logprobs", "rows": 8192, "vocab": 32000, "pad": 0, "dtype": "bf16",
         "top": 0, "entropy": True, "scale": 1.0},
        # the gradient that starts its backward pass, with an entropy bonus
        {"name": "logprobs backward 8192x32000", "op": "logprobs_backward", "rows": 8192, "vocab": 32000, "pad": 0,
         "dtype": "bf16", "entropy": True, "scale": 1.0},
        # fp32 logits of a ragged number of tokens, in rows padded past an odd vocabulary
        {"name": "logprobs backward 333x50001 f32", "op": "logprobs_backward", "rows": 333, "vocab": 50001, "pad": 47,
         "dtype": "f32", "entropy": False, "scale": 0.5},
        # one LLaMA-7B layer's matrices: fp32 weights and states, bf16 gradients and weight copies
        {"name": "adamw layer 32-bit", "op": "adamw", "sizes": "layer", "param": "f32", "copy": True, "grad": "bf16",
         "bits": 32, "block": 256},
        # the same with states in 8 bits
        {"name": "adamw layer 8-bit", "op": "adamw", "sizes": "layer", "param": "f32", "copy": True, "grad": "bf16",
         "bits": 8, "block": 256},
        # the many small tensors of a model (norms, biases, adapters) in bf16, most of odd sizes
        {"name": "adamw 200 small tensors 8-bit", "op": "adamw", "sizes": "200 tensors of 100 to 40000", "param": "bf16",
         "copy": False, "grad": "bf16", "bits": 8, "block": 128},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _features(rng, lo, hi):
    """A count of features: mostly a multiple of 64, often of 8, sometimes any."""
    n, u = _spread(rng, lo, hi), rng.random()
    step = 64 if u < 0.55 else 8 if u < 0.8 else 1
    return max(step, n // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "logprobs", "logprobs_backward", "adamw"])
    if op in ("norm", "norm_backward"):
        while True:
            rows, cols = _spread(rng, 1, 16384), _features(rng, 64, 16384)
            if rows * cols <= NORM_ELEMS:
                break
        alone = rng.random() < 0.2
        case = {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "bf16", "f32"]), "alone": alone,
                "post": not alone and rng.random() < 0.6,
                "gate": "none" if alone else rng.choice(["none", "column", "column", "element"])}
        if op == "norm":
            case["block"] = rng.choice([0, 32, 64])
        return case
    if op in ("logprobs", "logprobs_backward"):
        top = rng.choice([0, 1, 5, 20, 32]) if op == "logprobs" else 0
        while True:
            rows, vocab = _spread(rng, 1, 8192), _features(rng, 512, 262144)
            if rows * vocab <= (TOP_ELEMS if top else LOGIT_ELEMS // 2):
                break
        case = {"op": op, "rows": rows, "vocab": vocab, "pad": rng.choice([0, 0, rng.randint(1, 127)]),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "entropy": rng.random() < 0.7,
                "scale": rng.choice([1.0, 1.0, 0.5, 1.25, 3.0])}
        return dict(case, top=top) if op == "logprobs" else case
    count = _spread(rng, 1, 250)
    hi = _spread(rng, 200, 150_000_000 // count)
    param = rng.choice(["f32", "bf16"])
    return {"op": op, "sizes": f"{count} tensors of {max(1, hi // 100)} to {hi}", "param": param,
            "copy": param == "f32" and rng.random() < 0.5, "grad": rng.choice(["bf16", "f32"]),
            "bits": rng.choice([8, 32]), "block": rng.choice([64, 128, 256, 512])}


def _tensor_sizes(text):
    """The elements of each tensor: a layer's, or so many between two bounds, spread over their
    logarithm, one in four a multiple of 64."""
    if text == "layer":
        return LAYER
    count, _, _, lo, _, hi = text.split()
    count, lo, hi = int(count), int(lo), int(hi)
    out = []
    for i in range(count):
        n = int(round(lo * (hi / lo) ** ((i * 0.6180339887498949 + 0.35) % 1.0)))
        out.append(n if i % 4 or n < 64 else n // 64 * 64)
    return out


def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        t, c, s = case["rows"], case["cols"], SIZES[case["dtype"]]
        both = not case["alone"]
        # y, residual in and h, out out; or the norm alone: x in, out out
        if op == "norm":
            planes = (4 if both else 2) + (case["gate"] == "element")
            ckpt = 2 * t * c if case["block"] else 0  # its values, read back in bf16
            return {"bytes": planes * t * c * s + 3 * c * s + 8 * t + ckpt, "flops": (12.0 if both else 5.0) * t * c}
        # dout, dh, h in and dresidual out, with y in and dy out; or dout, h in and dx out
        planes = 3
        if both:
            planes = 5 + (case["post"] or case["gate"] != "none") + 2 * (case["gate"] == "element")
        return {"bytes": planes * t * c * s + 6 * c * s + 8 * t, "flops": (24.0 if both else 12.0) * t * c}
    if op in ("logprobs", "logprobs_backward"):
        t, v, s = case["rows"], case["vocab"], SIZES[case["dtype"]]
        if op == "logprobs":
            return {"bytes": t * v * s + t * (24 + 8 * case["top"]), "flops": 6.0 * t * v}
        return {"bytes": 2 * t * v * s + 28 * t, "flops": 8.0 * t * v}
    n = sum(_tensor_sizes(case["sizes"]))
    b = SIZES[case["grad"]] + 2 * SIZES[case["param"]] + 2 * case["copy"]
    # states in 32 bits in and out; in 8 bits in and out and their values in bf16
    b += 16 if case["bits"] == 32 else 4 + 4
    return {"bytes": b * n, "flops": 18.0 * n}


# -- inputs -------------------------------------------------------------------------

def _stream(gen, rows, cols, dtype):
    """A residual stream or a block's output: normal, each column with a scale of its own and a
    few columns ten times as large."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    scale = torch.exp(0.5 * torch.randn(cols, generator=gen, device="cuda"))
    scale = torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.003, 10.0 * scale, scale)
    return x.mul_(scale).to(dtype)


def _prepare_norm(case, gen):
    t, c, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    backward = case["op"] == "norm_backward"

    def randn(*shape, scale=1.0, shift=0.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).add_(shift).to(dt)

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    s = {"case": case, "scale": 0.5, "y": None, "gate": None, "post_weight": None, "post_rstd": None, "h": None}
    s["residual"] = _stream(gen, t, c, dt)
    s["weight"] = randn(c, scale=0.2, shift=1.0)
    s["out"], s["rstd"] = empty(t, c), empty(t, dtype=torch.float32)
    if not case["alone"]:
        s["y"], s["h"] = _stream(gen, t, c, dt), empty(t, c)
        if case["post"]:
            s["post_weight"], s["post_rstd"] = randn(c, scale=0.2, shift=1.0), empty(t, dtype=torch.float32)
        if case["gate"] != "none":
            s["gate"] = randn(c, scale=0.3, shift=0.5) if case["gate"] == "column" else randn(t, c, scale=0.5)
    if not backward:
        if case["block"]:
            s["ckpt"] = (empty(t, c, dtype=torch.int8), empty(t, -(-c // case["block"]), dtype=torch.uint8))
            s["read"] = empty(t, c, dtype=torch.bfloat16)
        return s
    # what the forward pass left: the stream after the block and the norms' factors
    h = s["residual"].double()
    if not case["alone"]:
        u = s["y"].double()
        if case["post"]:
            r = ((u * u).mean(1) + EPS).rsqrt()
            s["post_rstd"] = r.float()
            u = u * r[:, None] * s["post_weight"].double()
        h = h + s["scale"] * (u if s["gate"] is None else u * s["gate"].double())
    s["h"] = h.to(dt)
    s["rstd"] = ((h * h).mean(1) + EPS).rsqrt().float()
    del h
    s["dout"], s["dresidual"], s["dweight"] = randn(t, c, scale=1e-3), s.pop("out"), empty(c)
    if not case["alone"]:
        s["dh"], s["dy"] = randn(t, c, scale=1e-3), empty(t, c)
        s["dpost_weight"] = empty(c) if case["post"] else None
        s["dgate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
    del s["residual"]
    return s


def _prepare_logprobs(case, gen):
    t, v, dt = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    x = torch.empty(t, v + case["pad"], dtype=dt, device="cuda").fill_(7.0)
    x = x[:, :v]
    # a common shape of preferences and each row's own, some rows sharp and some flat
    common = 1.5 * torch.randn(v, generator=gen, device="cuda")
    sharp = torch.exp(0.4 * torch.randn(t, 1, generator=gen, device="cuda"))
    rows_at_once = max(1, (1 << 26) // v)
    for lo in range(0, t, rows_at_once):
        part = torch.randn(min(rows_at_once, t - lo), v, generator=gen, device="cuda")
        x[lo:lo + rows_at_once] = part.mul_(1.5).add_(common).mul_(sharp[lo:lo + rows_at_once]).to(dt)
    targets = torch.randint(0, v, (t,), generator=gen, device="cuda")
    # every 16th row is held to a grammar: all but some 60 tokens are masked, half of them with
    # minus infinity, half with the type's lowest value
    for r in range(7, t, 16):
        keep = torch.randint(0, v, (60,), generator=gen, device="cuda")
        kept = x[r, keep]
        x[r] = float("-inf") if r % 32 == 7 else torch.finfo(dt).min
        x[r, keep] = kept
        targets[r] = keep[0]
    # tokens of the prompt are not scored
    unscored = torch.rand(t, generator=gen, device="cuda") < 0.05
    if t > 1:
        targets = torch.where(unscored, torch.full_like(targets, -100), targets)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    s = {"case": case, "logits": x, "targets": targets, "stats": empty(t, 2)}
    if case["op"] == "logprobs":
        s["logprob"], s["entropy"] = empty(t), empty(t) if case["entropy"] else None
        s["top_ids"] = s["top_logprobs"] = None
        if case["top"]:
            s["top_ids"], s["top_logprobs"] = empty(t, case["top"], dtype=torch.int32), empty(t, case["top"])
        return s
    # what the forward pass left, and the loss's gradient of each token
    s["dlogprob"] = torch.randn(t, generator=gen, device="cuda").sub_(1.0).div_(t)
    s["dentropy"] = torch.full((t,), -0.02 / t, device="cuda") if case["entropy"] else None
    s["entropy"] = empty(t) if case["entropy"] else None
    s["dlogits"] = torch.zeros(t, v + case["pad"], dtype=dt, device="cuda")[:, :v]
    for lo in range(0, t, rows_at_once):
        at = slice(lo, lo + rows_at_once)
        d, e, top = _exponentials64(x[at], case["scale"])
        total = e.sum(1)
        s["stats"][at, 0], s["stats"][at, 1] = top[:, 0].float(), total.float()
        if case["entropy"]:
            s["entropy"][at] = (total.log() - torch.where(e > 0, e * d, 0.0).sum(1) / total).float()
    return s


def _views(flat, sizes):
    """The tensors of a flat buffer, each from a multiple of 16 elements on."""
    out, at = [], 0
    for n in sizes:
        out.append(flat[at:at + n])
        at += -(-n // 16) * 16
    return out


def _prepare_adamw(case, gen):
    pt, gt, block = DTYPES[case["param"]], DTYPES[case["grad"]], case["block"]
    sizes = _tensor_sizes(case["sizes"])
    total = sum(-(-n // 16) * 16 for n in sizes)

    def flat(dtype):
        return torch.zeros(total, dtype=dtype, device="cuda")

    # weights, their copies and states are views of one flat buffer of each kind
    s = {"case": case, "tensors": [], "grad_scale": torch.full((1,), 0.7, device="cuda"), "param": flat(pt)}
    s["copy"] = flat(torch.bfloat16) if case["copy"] else None
    nothing = [None] * len(sizes)
    params, copies = _views(s["param"], sizes), _views(s["copy"], sizes) if case["copy"] else nothing
    if case["bits"] == 32:
        s["m"], s["v"] = flat(torch.float32), flat(torch.float32)
    else:
        s["m"], s["v"] = flat(torch.bfloat16), flat(torch.bfloat16)  # the values, read back
    reads = list(zip(_views(s["m"], sizes), _views(s["v"], sizes)))
    for i, n in enumerate(sizes):
        p = params[i].copy_(torch.randn(n, generator=gen, device="cuda").mul_(0.02))
        g = torch.randn(n, generator=gen, device="cuda")
        g = g.mul_(torch.exp(torch.randn(n, generator=gen, device="cuda"))).mul_(1e-3).to(gt)
        nb = -(-n // block)
        if case["bits"] == 32:
            m = reads[i][0].copy_(torch.randn(n, generator=gen, device="cuda").mul_(2e-4))
            v = reads[i][1].copy_(torch.exp(torch.randn(n, generator=gen, device="cuda")).mul_(1e-6))
        else:
            def step(mean):
                return (torch.randint(-1, 2, (nb,), generator=gen, device="cuda") + mean).to(torch.uint8)
            q = torch.randn(n, generator=gen, device="cuda").mul_(60.0).clamp_(-448.0, 448.0)
            m = (q.to(torch.float8_e4m3fn), step(108))
            codes = torch.randint(192, 256, (n,), generator=gen, device="cuda")
            codes[torch.rand(n, generator=gen, device="cuda") < 0.01] = 0  # no gradient so far
            v = (codes.to(torch.uint8), step(107))
        if case["copy"]:
            copies[i].copy_(p)
        # vectors (norms, biases) are not decayed; here every fifth tensor stands for one
        s["tensors"].append((p, g, m, v, copies[i], 0.0 if i % 5 == 4 else DECAY))
    s["read"] = reads if case["bits"] == 8 else []
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] in ("norm", "norm_backward"):
        return _prepare_norm(case, gen)
    return _prepare_adamw(case, gen) if case["op"] == "adamw" else _prepare_logprobs(case, gen)


# -- the plain forms ------------------------------------------------------------------

def _blocks(x, block):
    """x [..., n] as [..., blocks, block], the last block filled with zeros."""
    pad = -x.shape[-1] % block
    if pad:
        x = torch.cat([x, x.new_zeros(*x.shape[:-1], pad)], dim=-1)
    return x.reshape(*x.shape[:-1], -1, block)


def _flat(x, n):
    return x.reshape(*x.shape[:-2], -1)[..., :n]


def _plain_round_trip(x, block):
    """What the 8-bit checkpoint of x stands for: whole multiples of each block's step, the
    least power of two that keeps them below 127.5."""
    v = _blocks(x, block)
    fraction, power = torch.frexp(v.abs().amax(dim=-1, keepdim=True))
    power = power - 7 + (fraction >= 127.5 / 128).to(power.dtype)
    step = torch.ldexp(torch.ones_like(fraction), power.clamp(min=-126))
    return _flat(torch.round(v / step) * step, x.shape[-1])


def _plain_norm(s):
    case, dt = s["case"], s["residual"].dtype
    h, out = s["residual"].float(), []
    if not case["alone"]:
        u = s["y"].float()
        if case["post"]:
            r = 1.0 / torch.sqrt((u * u).mean(1) + EPS)
            u = u * r[:, None] * s["post_weight"].float()
            out.append(r)
        if s["gate"] is not None:
            u = u * s["gate"].float()
        h = h + s["scale"] * u
        out.append(h.to(dt))
    r = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
    z = h * r[:, None] * s["weight"].float()
    out += [r, z.to(dt)]
    if case["block"]:
        out.append(_plain_round_trip(z, case["block"]).to(torch.bfloat16))
    return out


def _plain_rms_backward(g, xh, r):
    """The gradient of xh = x r, r = 1/sqrt(mean x^2 + eps), for the gradient g of xh."""
    return r[:, None] * (g - xh * (g * xh).mean(1, keepdim=True))


def _plain_norm_backward(s):
    case, dt = s["case"], s["h"].dtype
    dout, xh = s["dout"].float(), s["h"].float() * s["rstd"][:, None]
    gh = _plain_rms_backward(dout * s["weight"].float(), xh, s["rstd"])
    dweight = (dout * xh).sum(0).to(dt)
    if case["alone"]:
        return [gh.to(dt), dweight]
    gh = gh + s["dh"].float()
    out = [gh.to(dt), dweight]
    du = s["scale"] * gh
    y = s["y"].float()
    yh = y * s["post_rstd"][:, None] if case["post"] else y
    u = yh * s["post_weight"].float() if case["post"] else yh
    if s["gate"] is not None:
        dgate = du * u
        out.append((dgate.sum(0) if case["gate"] == "column" else dgate).to(dt))
        du = du * s["gate"].float()
    if case["post"]:
        out.append((du * yh).sum(0).to(dt))
        du = _plain_rms_backward(du * s["post_weight"].float(), yh, s["post_rstd"])
    return out + [du.to(dt)]


def _plain_exponentials(s):
    """x - max x and its exponential in each row; masked tokens have the exponential 0 and a
    difference that products with it leave at 0."""
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    d = x - top
    e = torch.exp(s["case"]["scale"] * d)
    return torch.where(e > 0, d, torch.zeros_like(d)), e, top


def _plain_logprobs(s):
    case, scale, t = s["case"], s["case"]["scale"], s["targets"]
    d, e, top = _plain_exponentials(s)
    total = e.sum(1)
    log_total = torch.log(total)
    out = [torch.cat([top, total[:, None]], dim=1)]
    own_logit = s["logits"].float().gather(1, t.clamp(min=0)[:, None])[:, 0]
    logprob = scale * (own_logit - top[:, 0]) - log_total
    out.append(torch.where(t >= 0, logprob, torch.zeros_like(logprob)))
    if case["entropy"]:
        out.append(log_total - scale * (e * d).sum(1) / total)
    if case["top"]:
        best, ids = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
        best, ids = best[:, :case["top"]], ids[:, :case["top"]]
        out += [ids.to(torch.int32), scale * (best - top) - log_total[:, None]]
    return out


def _plain_logprobs_backward(s):
    scale, t = s["case"]["scale"], s["targets"]
    top, total = s["stats"][:, :1], s["stats"][:, 1:]
    d = s["logits"].float() - top
    p = torch.exp(scale * d) / total
    dlogprob = torch.where(t >= 0, s["dlogprob"], torch.zeros_like(s["dlogprob"]))[:, None]
    dx = -dlogprob * p
    dx.scatter_add_(1, t.clamp(min=0)[:, None], dlogprob)
    if s["dentropy"] is not None:
        logp = torch.where(p > 0, scale * d - torch.log(total), torch.zeros_like(d))
        dx = dx - s["dentropy"][:, None] * p * (logp + s["entropy"][:, None])
    s["dlogits"].copy_((scale * dx).to(s["logits"].dtype))
    return s["dlogits"]


def _plain_m(m, block, n):
    codes, exps = m
    return _flat(_blocks(codes.float(), block) * torch.ldexp(torch.ones(exps.shape, device=exps.device),
                                                             exps.to(torch.int32) - 127)[:, None], n)


def _plain_v(v, block, n):
    """Five bits of exponent below the block's and three of mantissa; the code 0 is 0."""
    codes, exps = v
    c = _blocks(codes.to(torch.int32), block)
    value = torch.ldexp(1.0 + (c & 7).float() / 8, (c >> 3) - 31 + exps.to(torch.int32)[:, None] - 127)
    return _flat(torch.where(c == 0, torch.zeros_like(value), value), n)


def _plain_store_m(m, x, block):
    """The least power of two that keeps the block's values within 448, float8's largest."""
    q = _blocks(x, block)
    fraction, power = torch.frexp(q.abs().amax(dim=1, keepdim=True))
    power = (power - 9 + (fraction > 0.875).to(power.dtype)).clamp(min=-117)
    q = q / torch.ldexp(torch.ones_like(fraction), power)
    m[0].copy_(_flat(q, x.numel()).to(torch.float8_e4m3fn))
    m[1].copy_((power[:, 0] + 127).to(torch.uint8))


def _plain_store_v(v, x, block):
    q = _blocks(x, block)
    fraction, power = torch.frexp(q)
    whole = torch.round(fraction * 16).to(torch.int32)  # 8 .. 16, times 2^(power - 4)
    power = torch.where(whole == 16, power + 1, power)
    mantissa = torch.where(whole == 16, torch.zeros_like(whole), whole - 8)
    top = torch.where(q > 0, power, torch.full_like(power, -1000)).amax(dim=1, keepdim=True)
    top = (top - 1).clamp(min=32 - 127)  # the block's exponent
    code = ((power - 1 - top + 31) * 8 + mantissa).clamp(min=1)  # never rounded to 0
    v[0].copy_(_flat(torch.where(q > 0, code, torch.zeros_like(code)), x.numel()).to(torch.uint8))
    v[1].copy_((top[:, 0] + 127).to(torch.uint8))


def _plain_adamw(s):
    case, block = s["case"], s["case"]["block"]
    lr, b1, b2, eps, step = (ADAMW[k] for k in ("lr", "beta1", "beta2", "eps", "step"))
    step_size, root = lr / (1.0 - b1 ** step), 1.0 / math.sqrt(1.0 - b2 ** step)
    for i, (p, g, m, v, copy, decay) in enumerate(s["tensors"]):
        n = p.numel()
        g = g.float() * s["grad_scale"]
        m1 = b1 * (m if case["bits"] == 32 else _plain_m(m, block, n)) + (1.0 - b1) * g
        v1 = b2 * (v if case["bits"] == 32 else _plain_v(v, block, n)) + (1.0 - b2) * (g * g)
        update = step_size * (m1 / (torch.sqrt(v1) * root + eps))
        p1 = p.float() * (1.0 - lr * decay) - update
        p.copy_(p1)
        if copy is not None:
            copy.copy_(p1)
        if case["bits"] == 32:
            m.copy_(m1)
            v.copy_(v1)
        else:
            _plain_store_m(m, m1, block)
            _plain_store_v(v, v1, block)
            s["read"][i][0].copy_(_plain_m(m, block, n))
            s["read"][i][1].copy_(_plain_v(v, block, n))
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return [s["param"]] + ([] if s["copy"] is None else [s["copy"]]) + [s["m"], s["v"]]


PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "logprobs": _plain_logprobs,
         "logprobs_backward": _plain_logprobs_backward, "adamw": _plain_adamw}


# -- the package's operators ------------------------------------------------------------

def _workspace(nbytes):
    """Scratch memory as a training loop keeps it from step to step, or None where none is needed."""
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None


def _own_norm(s, loco):
    case = s["case"]
    block = case["block"] or 64
    loco.residual_norm(s["y"], s["residual"], h=s["h"], out=s["out"], rstd=s["rstd"], weight=s["weight"],
                       post_rstd=s["post_rstd"], post_weight=s["post_weight"], gate=s["gate"], scale=s["scale"],
                       eps=EPS, checkpoint=s.get("ckpt"), block=block)
    out = [] if s["post_rstd"] is None else [s["post_rstd"]]
    out += ([] if s["h"] is None else [s["h"]]) + [s["rstd"], s["out"]]
    if case["block"]:
        loco.checkpoint_read(*s["ckpt"], block=block, out=s["read"])
        out.append(s["read"])
    return out


def _own_norm_backward(s, loco):
    case = s["case"]
    if "workspace" not in s:
        s["workspace"] = _workspace(loco.residual_norm_backward_workspace(case["rows"], case["cols"]))
    loco.residual_norm_backward(s["dout"], s["h"], rstd=s["rstd"], weight=s["weight"], dh=s.get("dh"), y=s["y"],
                                post_rstd=s["post_rstd"], post_weight=s["post_weight"], gate=s["gate"],
                                scale=s["scale"], dresidual=s["dresidual"], dy=s.get("dy"), dgate=s.get("dgate"),
                                dweight=s["dweight"], dpost_weight=s.get("dpost_weight"), workspace=s["workspace"])
    out = [s["dresidual"], s["dweight"], s.get("dgate"), s.get("dpost_weight"), s.get("dy")]
    return [t for t in out if t is not None]


def _own_logprobs(s, loco):
    case = s["case"]
    if "workspace" not in s:
        s["workspace"] = _workspace(loco.token_logprobs_workspace(case["rows"], case["vocab"], case["top"]))
    loco.token_logprobs(s["logits"], s["targets"], logprob=s["logprob"], entropy=s["entropy"], stats=s["stats"],
                        top_ids=s["top_ids"], top_logprobs=s["top_logprobs"], scale=case["scale"],
                        workspace=s["workspace"])
    out = [s["stats"], s["logprob"], s["entropy"], s["top_ids"], s["top_logprobs"]]
    return [t for t in out if t is not None]


def _own_logprobs_backward(s, loco):
    loco.token_logprobs_backward(s["logits"], s["targets"], s["stats"], dlogprob=s["dlogprob"], entropy=s["entropy"],
                                 dentropy=s["dentropy"], dlogits=s["dlogits"], scale=s["case"]["scale"])
    return s["dlogits"]


def _own_adamw(s, loco):
    case = s["case"]
    if "plan" not in s:  # a training loop's list of its tensors, kept from step to step
        s["plan"] = loco.AdamwTensors(s["tensors"], block=case["block"])
    loco.adamw(s["plan"], grad_scale=s["grad_scale"], **ADAMW)
    if case["bits"] == 8:
        if "states" not in s:
            s["states"] = loco.AdamwStates([(st, r) for t, rs in zip(s["tensors"], s["read"])
                                            for st, r in zip(t[2:4], rs)], block=case["block"])
        loco.adamw_state_read(s["states"])
    return _adamw_outputs(s)


OWN = {"norm": _own_norm, "norm_backward": _own_norm_backward, "logprobs": _own_logprobs,
       "logprobs_backward": _own_logprobs_backward, "adamw": _own_adamw}


def run(state):
    op = state["case"]["op"]
    if own:
        from bit_gradient_compression_amd import loco
        return OWN[op](state, loco)
    return PLAIN[op](state)


# -- the definition in 64 bits --------------------------------------------------------

def _stored64(x, block):
    """The values of x's 8-bit checkpoint, from the logarithm of each block's largest value."""
    at = (torch.arange(x.shape[1], device=x.device) // block).expand(x.shape)
    top = x.new_zeros(x.shape[0], -(-x.shape[1] // block)).scatter_reduce(1, at, x.abs(), "amax")
    s = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 127.5))
    s = torch.where(top >= 127.5 * torch.exp2(s), s + 1, s).clamp(min=-126)  # 127.5 itself would round to 128
    step = torch.exp2(s).gather(1, at)
    return torch.round(x / step) * step


def _exact_norm(s):
    case, out = s["case"], []
    h = s["residual"].double()
    if not case["alone"]:
        u, k = s["y"].double(), s["scale"] * torch.ones((), dtype=torch.float64, device="cuda")
        if s["gate"] is not None:
            k = k * s["gate"].double()
        if case["post"]:
            rp = (u.square().sum(1) / case["cols"] + EPS) ** -0.5
            out.append(rp)
            u = rp.unsqueeze(1) * u
            k = k * s["post_weight"].double()
        h = torch.addcmul(h, k, u)
        out.append(h)
    r = (h.square().sum(1) / case["cols"] + EPS) ** -0.5
    z = s["weight"].double() * (r.unsqueeze(1) * h)
    return out + [r, z] + ([_stored64(z, case["block"])] if case["block"] else [])


def _exact_norm_backward(s):
    case, n = s["case"], s["case"]["cols"]
    dout, h, r = s["dout"].double(), s["h"].double(), s["rstd"].double().unsqueeze(1)
    g = dout * s["weight"].double()
    # d(h r)/dh with dr/dh = -r^3 h / n
    gh = r * g - r ** 3 / n * torch.linalg.vecdot(g, h, dim=1).unsqueeze(1) * h
    dweight = torch.linalg.vecdot(dout, r * h, dim=0)
    if case["alone"]:
        return [gh, dweight]
    gh = gh + s["dh"].double()
    y, k = s["y"].double(), torch.full((), s["scale"], dtype=torch.float64, device="cuda")
    gate = torch.ones_like(k) if s["gate"] is None else s["gate"].double()
    w, rp = (s["post_weight"].double(), s["post_rstd"].double().unsqueeze(1)) if case["post"] else (torch.ones_like(k), 1)
    out = [gh, dweight]
    if case["gate"] == "column":
        out.append(s["scale"] * w * torch.linalg.vecdot(gh, rp * y, dim=0))
    elif case["gate"] == "element":
        out.append(s["scale"] * gh * (rp * y * w))
    dn = gh * gate * s["scale"]
    if not case["post"]:
        return out + [dn]
    out.append(torch.linalg.vecdot(dn, rp * y, dim=0))
    dn = dn * w
    return out + [rp * dn - rp ** 3 / n * torch.linalg.vecdot(dn, y, dim=1).unsqueeze(1) * y]


def _exponentials64(x, scale):
    x = x.double()
    top = x.max(dim=1, keepdim=True).values
    return x - top, torch.exp((x - top) * scale), top


def _exact_logprobs(s):
    case, parts = s["case"], []
    t, v, scale = case["rows"], case["vocab"], case["scale"]
    at_once = max(1, (1 << 27) // v)
    iota = torch.arange(v, device="cuda")
    for lo in range(0, t, at_once):
        x, tg = s["logits"][lo:lo + at_once], s["targets"][lo:lo + at_once]
        d, e, top = _exponentials64(x, scale)
        total = e.sum(1, keepdim=True)
        lse = scale * top + total.log()
        rows = torch.arange(x.shape[0], device="cuda")
        lp = scale * x[rows, tg.clamp(min=0)].double() - lse[:, 0]
        out = [torch.cat([top, total], 1), lp.masked_fill(tg < 0, 0.0)]
        if case["entropy"]:
            p = e / total
            out.append(-torch.where(p > 0, p * (scale * d - total.log()), 0.0).sum(1))
        if case["top"]:
            left, ids, lps = x.double().clone(), [], []
            for _ in range(case["top"]):
                best = left.max(dim=1, keepdim=True).values
                at = torch.where(left == best, iota, v).min(dim=1).values
                ids.append(at)
                lps.append(scale * best[:, 0] - lse[:, 0])
                left[rows, at] = float("-inf")
            out += [torch.stack(ids, 1).to(torch.int32), torch.stack(lps, 1)]
        parts.append(out)
    return [torch.cat(p) for p in zip(*parts)]


def _exact_logprobs_backward(s):
    case, scale = s["case"], s["case"]["scale"]
    at_once, parts = max(1, (1 << 27) // case["vocab"]), []
    for lo in range(0, case["rows"], at_once):
        at = slice(lo, lo + at_once)
        z = scale * (s["logits"][at].double() - s["stats"][at, :1].double()) - s["stats"][at, 1:].double().log()
        p, t = torch.exp(z), s["targets"][at]
        dlp = s["dlogprob"][at].double() * (t >= 0)
        picked = torch.zeros_like(p)
        picked[torch.arange(p.shape[0], device="cuda"), t.clamp(min=0)] = 1.0
        dz = dlp.unsqueeze(1) * (picked - p)
        if s["dentropy"] is not None:
            dz -= (s["dentropy"][at].double().unsqueeze(1)
                   * torch.where(p > 0, p * (z + s["entropy"][at].double().unsqueeze(1)), 0.0))
        parts.append(scale * dz)
    return torch.cat(parts)


def _significant64(x, least):
    """x rounded to four significant bits, ties to even; below 2^least to whole steps of its."""
    power = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -300)))
    power = torch.where(x.abs() >= torch.exp2(power + 1), power + 1, power)
    power = torch.where(x.abs() < torch.exp2(power), power - 1, power)
    step = torch.exp2(torch.maximum(power, torch.full_like(power, least)) - 3)
    return torch.round(x / step) * step


def _exact_adamw(s):
    case, block = s["case"], s["case"]["block"]
    lr, b1, b2, eps, step = (ADAMW[k] for k in ("lr", "beta1", "beta2", "eps", "step"))
    sizes = _tensor_sizes(case["sizes"])
    ps, ms, vs = (torch.zeros(s["param"].numel(), dtype=torch.float64, device="cuda") for _ in range(3))
    places = zip(*(_views(x, sizes) for x in (ps, ms, vs)))
    for (p, g, m, v, _, decay), (p1, m1, v1) in zip(s["tensors"], places):
        n = p.numel()
        at = torch.arange(n, device="cuda") // block
        nb = -(-n // block)
        if case["bits"] == 8:
            m = m[0].to(torch.float64) * torch.exp2(m[1].double() - 127.0)[at]
            c = v[0].double()
            high = torch.floor(c / 8)
            v = torch.where(c > 0, (8 + c - 8 * high) * torch.exp2(high - 34 + (v[1].double() - 127.0)[at]), 0.0)
        g = g.double() * s["grad_scale"].double()
        m = torch.lerp(g, m.double(), b1)
        v = torch.lerp(g * g, v.double(), b2)
        mh, vh = m / (1 - b1 ** step), v / (1 - b2 ** step)
        p1.copy_(p.double() - lr * (decay * p.double() + mh / (vh.sqrt() + eps)))
        if case["bits"] == 8:
            top = m.new_zeros(nb).scatter_reduce(0, at, m.abs(), "amax")
            scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -300) / 448)).clamp(min=-117))[at]
            m = _significant64(m / scale, -6) * scale
            v = _significant64(v, -1000)
            top = v.new_zeros(nb).scatter_reduce(0, at, v, "amax")
            floor = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -300))).clamp(min=-95) - 31)[at] * 1.125
            v = torch.where(v > 0, torch.maximum(v, floor), v)
        m1.copy_(m)
        v1.copy_(v)
    return [ps] + ([] if s["copy"] is None else [ps]) + [ms, vs]


EXACT = {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "logprobs": _exact_logprobs,
         "logprobs_backward": _exact_logprobs_backward, "adamw": _exact_adamw}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))

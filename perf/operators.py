"""The optimizer's many-tensor operators as measured: the AdamW step with fp32 states, the AdamW
step with 8-bit states, and the global gradient norm that gives both their clipping scale.

Every case is a list of tensors as a GPT-2-style model has them. The tensors of one case are views
of one flat buffer per role (a parameter buffer, a gradient buffer, ...), each tensor starting at a
multiple of 256 elements, with zeros in between; so a block of 256 elements of the buffer is a
block of one tensor, and the plain form works on the whole buffer as rows of 256.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 256
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LR, BETA1, BETA2, EPS, DECAY = 6e-4, 0.9, 0.999, 1e-8, 0.1


def f32(x):
    """The fp32 value nearest to x, as a Python float (the operators take fp32 settings)."""
    return float(np.float32(x))


# ---- the tensors of a case -------------------------------------------------------------------

def shapes_of(case):
    """(shape, decay multiplier) of each tensor. "vectors": the norms' and biases' vectors of a
    model; "tables": embedding tables and 64 scalars; "model": every tensor of a model."""
    d, v = case["d"], case["vocab"]
    if case["set"] == "tables":
        return [((v, d), 1.0)] * case["layers"] + [((64,), 0.0)]
    vectors = [((d,), 0.0)] * 4 + [((4 * d,), 0.0)] + [((d,), 0.0)] * 5
    if case["set"] == "vectors":
        return vectors * case["layers"] + [((d,), 0.0)] * 2
    matrices = [((d, d), 1.0)] * 4 + [((4 * d, d), 1.0), ((d, 4 * d), 1.0)]
    return [((v, d), 1.0), ((1024, d), 1.0)] + (matrices + vectors) * case["layers"] + [((d,), 0.0)] * 2


def numel(shape):
    return math.prod(shape)


def elements(case):
    return sum(numel(s) for s, _ in shapes_of(case))


def listed():
    return [
        # a GPT-2-124M run that keeps the norms' and biases' vectors in fp32: 122 small tensors,
        # where the call itself is what takes time
        dict(name="adamw vectors f32", op="adamw", set="vectors", d=768, layers=12, vocab=0, param="f32", grad="f32", master=False, clip=False, t=1, stochastic=False),
        # the parameters that the matrix optimizer leaves over: embedding tables and scalars
        dict(name="adamw tables bf16", op="adamw", set="tables", d=768, layers=4, vocab=50257, param="bf16", grad="bf16", master=False, clip=False, t=900, stochastic=False),
        # GPT-2-124M trained whole by AdamW in mixed precision, clipped to norm 1
        dict(name="adamw 124m master clip", op="adamw", set="model", d=768, layers=12, vocab=50257, param="bf16", grad="bf16", master=True, clip=True, t=250, stochastic=False),
        # GPT-2-1.5B, bf16 parameters whose gradients were summed in fp32: the largest
        dict(name="adamw 1.5b bf16 f32", op="adamw", set="model", d=1600, layers=48, vocab=50257, param="bf16", grad="f32", master=False, clip=False, t=20000, stochastic=False),
        # a small fp32 model of odd width: rows and tensors end inside blocks
        dict(name="adamw8 odd f32", op="adamw8", set="model", d=129, layers=2, vocab=1013, param="f32", grad="f32", master=False, clip=False, t=7, stochastic=False),
        # the same left-over tables, with a quarter of the state
        dict(name="adamw8 tables bf16", op="adamw8", set="tables", d=768, layers=4, vocab=50257, param="bf16", grad="bf16", master=False, clip=False, t=900, stochastic=True),
        # GPT-2-124M in mixed precision, clipped
        dict(name="adamw8 124m master clip", op="adamw8", set="model", d=768, layers=12, vocab=50257, param="bf16", grad="bf16", master=True, clip=True, t=250, stochastic=True),
        # GPT-2-1.5B all in bf16, where the states in 8 bits leave room on the card
        dict(name="adamw8 1.5b bf16", op="adamw8", set="model", d=1600, layers=48, vocab=50257, param="bf16", grad="bf16", master=False, clip=False, t=20000, stochastic=True),
        # the norm over small tensors: latency
        dict(name="norm vectors f32", op="norm", set="vectors", d=768, layers=12, vocab=0, param="f32", grad="f32", master=False, clip=True, t=1, stochastic=False),
        # the norm over a model of odd width
        dict(name="norm odd bf16", op="norm", set="model", d=333, layers=6, vocab=5021, param="bf16", grad="bf16", master=False, clip=True, t=1, stochastic=False),
        # GPT-2-124M's and GPT-2-1.5B's gradients
        dict(name="norm 124m bf16", op="norm", set="model", d=768, layers=12, vocab=50257, param="bf16", grad="bf16", master=False, clip=True, t=1, stochastic=False),
        dict(name="norm 1.5b f32", op="norm", set="model", d=1600, layers=48, vocab=50257, param="f32", grad="f32", master=False, clip=True, t=1, stochastic=False),
    ]


def draw(rng):
    op = rng.choice(["adamw", "adamw", "adamw8", "adamw8", "norm"])
    kind = rng.choice(["vectors", "tables", "model", "model"])
    width = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    param = rng.choice(["bf16", "f32"])
    case = dict(op=op, set=kind, d=width(5, 1600), layers=width(1, 48), vocab=width(50, 50257),
                param=param, grad=rng.choice(["bf16", "f32"]),
                master=op != "norm" and param == "bf16" and rng.random() < 0.5,
                clip=op == "norm" or rng.random() < 0.5, t=width(1, 100000),
                stochastic=op == "adamw8" and rng.random() < 0.7)
    if kind == "tables":
        case["layers"] = 1 + case["layers"] % 6
    if kind == "vectors":
        case["vocab"] = 0
    return case


# ---- inputs ----------------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    shapes = shapes_of(case)
    blocks = [-(-numel(s) // BLOCK) for s, _ in shapes]
    at, total = [0], 0
    for b in blocks:
        total += b
        at.append(total)
    inside = torch.ones(total, BLOCK, dtype=torch.bool, device=dev)
    for (shape, _), end, b in zip(shapes, at[1:], blocks):
        tail = numel(shape) - (b - 1) * BLOCK
        if tail < BLOCK:
            inside[end - 1, tail:] = False

    def noise(std):
        x = torch.randn(total, BLOCK, generator=gen, device=dev)
        return x.mul_(std).mul_(inside)

    def views(flat):
        flat = flat.view(-1)
        return [flat[a * BLOCK:a * BLOCK + numel(s)].view(s) for a, (s, _) in zip(at, shapes)]

    # gradients of one batch: normal, at a scale of its own for each tensor; a third of an
    # embedding table's rows belong to tokens that the batch does not hold and are zero
    grad = noise(1e-3)
    spread = torch.exp(0.7 * torch.randn(len(shapes), generator=gen, device=dev))
    counts = torch.tensor(blocks, device=dev)
    grad *= spread.repeat_interleave(counts)[:, None]
    for g, (shape, _) in zip(views(grad), shapes):
        if len(shape) == 2 and shape[0] == case["vocab"] and shape[0] != shape[1]:
            g *= (torch.rand(shape[0], 1, generator=gen, device=dev) > 1 / 3)
    s = {"case": case, "grad": grad.to(DT[case["grad"]]), "counts": counts, "dev": dev,
         "max_norm": 1.0 if case["clip"] else math.inf}
    s["grads"] = views(s["grad"])
    del grad
    if case["op"] == "norm":
        if own:
            from orthogonalized_momentum_optimizer_amd import GradNormPlan
            s["norm_plan"] = GradNormPlan(s["grads"])
        return s

    first = case["t"] == 1
    s["decay"] = torch.tensor([m for _, m in shapes], device=dev).repeat_interleave(counts)[:, None] * f32(DECAY)
    p = noise(0.02)
    s["param"] = p.to(DT[case["param"]])
    if case["master"]:
        s["master"] = p
    del p
    # states as a run leaves them: a mean much smaller than the root mean square
    m = noise(0.0 if first else 3e-4)
    v = noise(0.0 if first else 1e-3).square_()
    if not first:
        v.add_(1e-7 * inside)
    if case["op"] == "adamw":
        s["exp_avg"], s["exp_avg_sq"] = m, v
    else:
        s["exp_avg"], s["exp_avg_scale"] = to_blocks(m)
        s["exp_avg_sq"], s["exp_avg_sq_scale"] = to_blocks(v.sqrt_(), positive=True)
    del m, v
    s["params"] = views(s["param"])
    if own:
        from orthogonalized_momentum_optimizer_amd import AdamWPlan, GradNormPlan, make_adamw_config
        more = {}
        if case["master"]:
            more["masters"] = views(s["master"])
        if case["op"] == "adamw8":
            ends = list(zip(at, at[1:]))
            more["exp_avg_scales"] = [s["exp_avg_scale"][a:b] for a, b in ends]
            more["exp_avg_sq_scales"] = [s["exp_avg_sq_scale"][a:b] for a, b in ends]
        s["plan"] = AdamWPlan(s["params"], views(s["exp_avg"]), views(s["exp_avg_sq"]),
                              [g.dtype for g in s["grads"]], wd_muls=[m for _, m in shapes], **more)
        s["config"] = make_adamw_config(lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
                                        step=case["t"], stochastic=case["stochastic"], seed=SEED)
        if case["clip"]:
            s["norm_plan"] = GradNormPlan(s["grads"])
    return s


SEED = 1234  # of the stochastic rounding


# ---- the 8-bit form --------------------------------------------------------------------------

def two_to(byte):
    """2^(byte - 127) of an e8m0 byte (int32), exactly; byte 0 is 2^-127."""
    return torch.where(byte == 0, torch.full_like(byte, 1 << 22), byte << 23).view(torch.float32)


TOP = (2 ** 23 + 0x629146) / 2 ** 15  # 453.1...: between 448, e4m3's largest, and 464, where it would overflow


def to_blocks(x, positive=False, bits=None):
    """x (rows of 256, fp32) as e4m3 values and a power-of-two scale for each row: the smallest
    2^k with |x| <= TOP * 2^k over the row. Rounded to nearest, or with `bits` (an integer in
    [0, 2^16) for each value) up with the probability of what is cut off. `positive`: values over
    zero do not become zero."""
    mant, expo = torch.frexp(x.abs().amax(1))
    byte = (expo - 9 + (mant > TOP / 512).int() + 127).clamp_(min=0).int()
    byte = torch.where(mant == 0, torch.zeros_like(byte), byte)
    y = x * ((254 - byte) << 23).view(torch.float32)[:, None]
    y = y.clamp(-448, 448)
    if bits is not None:
        shift = (y < 2.0 ** -6).float() * 2.0 ** -6  # under 2^-6 the values are multiples of 2^-9
        z = (y + shift).view(torch.int32) + (bits * 16 + 8).int()
        y = (z & -(1 << 20)).view(torch.float32) - shift
    if positive:
        y = torch.where(x > 0, y.clamp_min(2.0 ** -9), y)
    return y.to(torch.float8_e4m3fn), byte.to(torch.uint8).view(torch.float8_e8m0fnu)


MASK = 0xFFFFFFFF


def key_of(seed, t):
    z = (seed + t * 0x1493FA689CA113AD) & (2 ** 64 - 1)
    for _ in range(2):
        z = ((z ^ (z >> 32)) * 0xE9F8AC216EBC06F5) & (2 ** 64 - 1)
    return (z ^ (z >> 32)) & MASK


def mix(x):
    """Spreads each 32-bit value of x (int64) over 32 bits."""
    x = ((x ^ (x >> 16)) * 0xEB26D985) & MASK
    x = ((x ^ (x >> 15)) * 0x4A08C6ED) & MASK
    return x ^ (x >> 16)


def bits_for(s):
    """The 16 bits of each element: elements 2j and 2j + 1 of a tensor share mix(j ^ key)."""
    counts = s["counts"]
    start = (counts.cumsum(0) - counts).repeat_interleave(counts)
    row = torch.arange(start.numel(), device=start.device) - start
    pair = row[:, None] * (BLOCK // 2) + torch.arange(BLOCK // 2, device=row.device)
    h = mix(pair ^ key_of(SEED, s["case"]["t"]))
    return torch.stack([h & 0xFFFF, h >> 16], dim=2).view(-1, BLOCK)


# ---- one pass --------------------------------------------------------------------------------

def norm_plain(s):
    """(norm, scale, norm of each tensor): squares in 64 bits, since fp32's overflow at 1.8e19."""
    rows = s["grad"].float().square().sum(1, dtype=torch.float64)
    each = torch.segment_reduce(rows, "sum", lengths=s["counts"], axis=0)
    norm = each.sum().sqrt()
    scale = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
    return norm.float(), torch.where(norm.isfinite(), scale, scale * math.nan).float(), each.sqrt().float()


def adamw_plain(s):
    case, t = s["case"], s["case"]["t"]
    b1, b2, lr = f32(BETA1), f32(BETA2), f32(LR)
    norm = scale = None
    g = s["grad"].float()
    if case["clip"]:
        norm, scale, _ = norm_plain(s)
        g = g * scale
    small = case["op"] == "adamw8"
    m, v = s["exp_avg"], s["exp_avg_sq"]
    if small:
        m = m.float() * two_to(s["exp_avg_scale"].view(torch.uint8).int())[:, None]
        v = (v.float() * two_to(s["exp_avg_sq_scale"].view(torch.uint8).int())[:, None]).square()
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    r = v.sqrt()
    p = s["master"] if case["master"] else s["param"].float()
    u = m * f32(1 / (1 - b1 ** t)) / (r * f32(1 / math.sqrt(1 - b2 ** t)) + f32(EPS))
    p = p - (u + s["decay"] * p) * lr
    s["param"].copy_(p)
    if case["master"]:
        s["master"].copy_(p)
    if small:
        bits = bits_for(s) if case["stochastic"] else None
        for name, (x, scale_of) in (("exp_avg", to_blocks(m)), ("exp_avg_sq", to_blocks(r, True, bits))):
            s[name].copy_(x)
            s[name + "_scale"].copy_(scale_of)
    else:
        s["exp_avg"].copy_(m)
        s["exp_avg_sq"].copy_(v)
    return norm


def outputs(s, norm):
    names = ("param", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
    out = {k: s[k] for k in names if k in s}
    if norm is not None:
        out["norm"] = norm
    return out


def run(s):
    case = s["case"]
    if case["op"] == "norm":
        if own:
            norm, scale, each = s["norm_plan"].norm(s["grads"], max_norm=s["max_norm"], per_tensor=True)
        else:
            norm, scale, each = norm_plain(s)
        return {"norm": norm, "scale": scale, "each": each}
    if own:
        norm = scale = None
        if case["clip"]:
            norm, scale = s["norm_plan"].norm(s["grads"], max_norm=s["max_norm"])
        s["plan"].step(s["grads"], s["config"], grad_scale=scale)
    else:
        norm = adamw_plain(s)
    return outputs(s, norm)


# ---- in 64 bits ------------------------------------------------------------------------------

def exact(case, seed):
    """Tensor by tensor, from the definitions, in float64."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    shapes, t = shapes_of(case), case["t"]
    b1, b2, lr, eps = f32(BETA1), f32(BETA2), f32(LR), f32(EPS)
    each = torch.stack([torch.linalg.vector_norm(g.double()) for g in s["grads"]])
    norm = torch.linalg.vector_norm(each)
    scale = float(min(1.0, s["max_norm"] / float(norm))) if case["clip"] else 1.0
    if case["op"] == "norm":
        return {"norm": norm, "scale": scale, "each": each}
    small = case["op"] == "adamw8"
    total = s["grad"].shape[0]
    wide = lambda: torch.zeros(total, BLOCK, dtype=torch.float64, device=s["dev"])  # noqa: E731
    out = {k: wide() for k in ("param", "master", "exp_avg", "exp_avg_sq") if k in s}
    if small:
        out["exp_avg_scale"], out["exp_avg_sq_scale"] = (torch.zeros(total, dtype=torch.float64, device=s["dev"]) for _ in "mv")
    at = 0
    for shape, mul in shapes:
        end = at - (-numel(shape) // BLOCK)
        g = s["grad"][at:end].double() * scale
        m, v = s["exp_avg"][at:end].double(), s["exp_avg_sq"][at:end].double()
        if small:
            m = m * s["exp_avg_scale"][at:end].float().double()[:, None]
            v = (v * s["exp_avg_sq_scale"][at:end].float().double()[:, None]) ** 2
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g ** 2
        p = (s["master"] if case["master"] else s["param"])[at:end].double()
        p = p - lr * ((m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + eps) + f32(DECAY) * mul * p)
        out["param"][at:end] = p
        if case["master"]:
            out["master"][at:end] = p
        if small:
            dither = None
            if case["stochastic"]:
                j = torch.arange((end - at) * BLOCK, device=s["dev"])
                h = mix((j >> 1) ^ key_of(SEED, t))
                dither = ((torch.where(j % 2 == 1, h >> 16, h & 0xFFFF).double() + 0.5) / 65536).view(-1, BLOCK)
            out["exp_avg"][at:end], out["exp_avg_scale"][at:end] = exact_blocks(m, None, False)
            out["exp_avg_sq"][at:end], out["exp_avg_sq_scale"][at:end] = exact_blocks(v.sqrt(), dither, True)
        else:
            out["exp_avg"][at:end], out["exp_avg_sq"][at:end] = m, v
        at = end
    if case["clip"]:
        out["norm"] = norm
    return out


def exact_blocks(x, dither, positive):
    top = x.abs().amax(1)
    k = torch.ceil(torch.log2((top / TOP).clamp_min(2.0 ** -127))).clamp_min(-127)
    y = (x / torch.exp2(k)[:, None]).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    n = torch.round(y / step) if dither is None else torch.floor(y / step + dither)
    y = n * step
    if positive:
        y = torch.where(x > 0, y.clamp_min(2.0 ** -9), y)
    return y, torch.exp2(k)


def work(case):
    n, size = elements(case), {"bf16": 2, "f32": 4}
    read = n * size[case["grad"]]
    if case["op"] == "norm":
        return {"bytes": read + 4 * (len(shapes_of(case)) + 2), "flops": 2 * n}
    held = 8 * n + size[case["param"]] * n if case["master"] else 2 * size[case["param"]] * n
    if case["op"] == "adamw":
        states = 16 * n
    else:
        states = 4 * n + 4 * sum(-(-numel(s) // BLOCK) for s, _ in shapes_of(case))
    return {"bytes": read + held + states, "flops": 18 * n + (2 * n if case["clip"] else 0)}

"""What the AdamW operators compute, in plain torch, and the calls a trainer makes of them.

Four operators over the tensors of one ZeRO shard: the AdamW step with 32-bit and with 8-bit states, the sum of squares
of the gradient mean (for clipping by the global norm), and the conversion of moments to and from their 8-bit form.
The tensors of a shard lie one behind the other in flat buffers, each padded to a multiple of 256 elements.
"""

import random

import torch

own = False

BLOCK = 256                      # elements that share one scale
M_MAX, V_MAX = 448.0, 57344.0    # largest e4m3 and e5m2 values
TINY = 2.0 ** -110               # a block whose largest value is below is held as zeros
BETA1, BETA2, EPS, LR = 0.9, 0.95, 1e-8, 3e-4
F8 = {"m": torch.float8_e4m3fn, "v": torch.float8_e5m2}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # a toy model's or one small layer's step: what a launch costs
        dict(name="adamw32_small", op="adamw", bits=32, total=50_000, tensors=16, p=1, grad="bf16", param="bf16",
             rounding="nearest", clip=False, shift=0, shape=1),
        # an eighth of a 124M-parameter model, 8 ranks' gradients still apart, matrices and many short vectors
        dict(name="adamw32_ranks8", op="adamw", bits=32, total=15_554_976, tensors=35, p=8, grad="bf16", param="bf16",
             rounding="nearest", clip=False, shift=0, shape=2),
        # an eighth of an 8B-parameter model after reduce-scatter and the norm, clipped
        dict(name="adamw32_large", op="adamw", bits=32, total=1_003_782_656, tensors=42, p=1, grad="bf16", param="bf16",
             rounding="nearest", clip=True, shift=0, shape=3),
        # the same steps with the moments in 8 bits
        dict(name="adamw8_small", op="adamw", bits=8, total=50_000, tensors=16, p=1, grad="bf16", param="bf16",
             rounding="nearest", clip=False, shift=0, shape=4),
        # 8 ranks, buffers that begin at an odd element, moments rounded at random
        dict(name="adamw8_ranks8_odd", op="adamw", bits=8, total=15_554_977, tensors=35, p=8, grad="bf16", param="bf16",
             rounding="stochastic", clip=True, shift=3, shape=5),
        # one of 64 shards of a 7.5B-parameter model, fp16 gradients under a loss scale
        dict(name="adamw8_mid", op="adamw", bits=8, total=117_187_500, tensors=24, p=1, grad="f16", param="f16",
             rounding="nearest", clip=True, shift=0, shape=6),
        dict(name="adamw8_large", op="adamw", bits=8, total=1_003_782_656, tensors=42, p=1, grad="bf16", param="bf16",
             rounding="stochastic", clip=False, shift=0, shape=7),
        # the gradient's norm before the step: the mean of one rank (already reduced) or of 8, which is kept
        dict(name="sumsq_small", op="sumsq", total=50_000, tensors=16, p=1, grad="bf16", store=False, shift=0, shape=8),
        dict(name="sumsq_ranks8", op="sumsq", total=15_554_976, tensors=35, p=8, grad="bf16", store=True,
             shift=0, shape=9),
        dict(name="sumsq_large", op="sumsq", total=1_003_782_656, tensors=42, p=1, grad="bf16", store=False,
             shift=0, shape=10),
        # moments out of their 8-bit form (a checkpoint written) and into it (one read)
        dict(name="to32_small", op="convert", to=32, kind="v", total=50_001, shift=1),
        dict(name="to8_mid", op="convert", to=8, kind="m", total=117_187_500, shift=0),
    ]


def draw(rng):
    op = rng.choice(["adamw", "adamw", "adamw", "sumsq", "convert"])
    total = int(20_000 * 10 ** rng.uniform(0.0, 4.0)) + rng.randrange(256)
    shift = rng.choice([0, 0, 0, 1, 2, 3, 8, 13])
    if op == "convert":
        return dict(op=op, to=rng.choice([8, 32]), kind=rng.choice(["m", "v"]), total=total, shift=shift)
    p = rng.choice([1, 1, 2, 3, 4, 8]) if 262_144 <= total <= 60_000_000 else 1
    grad = rng.choice(["bf16", "f16", "f32"])
    case = dict(op=op, total=total, tensors=rng.randint(1, 60), p=p, grad=grad, shift=shift,
                shape=rng.randrange(1 << 20))
    if op == "sumsq":
        return dict(case, store=p > 1 or rng.random() < 0.2)
    bits = rng.choice([32, 8, 8])
    return dict(case, bits=bits, param=rng.choice(["bf16", "f16"]), clip=rng.random() < 0.5,
                rounding=rng.choice(["nearest", "stochastic"]) if bits == 8 else "nearest")


def lengths(case):
    """Lengths of the case's tensors: a few large ones, many short, summing to about the total."""
    r = random.Random(case["shape"])
    weights = [10 ** r.uniform(0.0, 4.0) for _ in range(case["tensors"])]
    return [max(1, int(case["total"] * x / sum(weights))) for x in weights]


def padded(n):
    return -(-n // BLOCK) * BLOCK


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    shift = case["shift"]

    def flat(n, dtype, values=None):
        """A buffer of n elements that begins `shift` elements into its storage."""
        x = torch.zeros(n + shift, dtype=dtype, device=dev)[shift:]
        return x if values is None else x.copy_(values)

    if case["op"] == "convert":
        n = case["total"]
        x = torch.randn(n, generator=gen, device=dev)
        x = flat(n, torch.float32, x.mul_(1e-4) if case["kind"] == "m" else x.mul_(1e-3).square_())
        x[: n // 16] *= 1e-3
        if case["to"] == 8:
            s = dict(case=case, x=x, codes=flat(n, F8[case["kind"]]), scales=torch.zeros(-(-n // BLOCK), device=dev))
        else:
            wide = torch.zeros(padded(n), device=dev)
            wide[:n] = x
            codes, scales = to_codes(wide.view(-1, BLOCK), case["kind"])
            s = dict(case=case, codes=flat(n, codes.dtype, codes.view(-1)[:n]), scales=scales.view(-1),
                     x=flat(n, torch.float32))
        if own:
            from adam_zs_shard_amd import zsadamw
            s["api"] = zsadamw
        return s

    lens = lengths(case)
    sizes = [padded(n) for n in lens]
    offs = [sum(sizes[:i]) for i in range(len(sizes))]
    total, blocks = sum(sizes), sum(sizes) // BLOCK
    r = random.Random(seed)
    # which elements are a tensor's own (the rest is padding and stays zero), and each tensor's gradient size
    real = torch.ones(total, dtype=torch.bool, device=dev)
    for n, size, at in zip(lens, sizes, offs):
        real[at + n:at + size] = False
    per_block = torch.tensor([size // BLOCK for size in sizes], device=dev)

    def by_block(values):
        return torch.repeat_interleave(torch.tensor(values, dtype=torch.float32, device=dev), per_block)[:, None]

    loss_scale = 1024.0 if case["grad"] == "f16" else 1.0
    size = by_block([10 ** r.uniform(-4.5, -2.5) for _ in lens])
    grads = []
    for _ in range(case["p"]):
        g = torch.randn(total, generator=gen, device=dev)
        g.view(-1, BLOCK).mul_(size * loss_scale)
        g[total // 3: total // 3 + total // 50] = 0       # rows that this step never saw
        grads.append(flat(total, DTYPES[case["grad"]], g.mul_(real)))
        del g
    s = dict(case=case, grads=grads, lens=lens, offs=offs, step=1000)
    if case["op"] == "sumsq":
        s["mean"] = flat(total, torch.float32) if case["store"] else None
        s["sumsq"] = torch.zeros((), dtype=torch.float64, device=dev)
    else:
        s["w"] = flat(total, torch.float32, torch.randn(total, generator=gen, device=dev).mul_(0.02).mul_(real))
        m = torch.randn(total, generator=gen, device=dev)
        m.view(-1, BLOCK).mul_(size * 0.3)
        v = torch.randn(total, generator=gen, device=dev).abs_().add_(0.1)
        v.view(-1, BLOCK).mul_(size).square_()
        m, v = m.mul_(real), v.mul_(real)
        if case["bits"] == 8:
            for k, x in (("m", m), ("v", v)):
                codes, scales = to_codes(x.view(-1, BLOCK), k)
                s[k] = flat(total, codes.dtype, codes.view(-1))
                s[k + "_scale"] = scales.view(-1)
        else:
            s["m"], s["v"] = flat(total, torch.float32, m), flat(total, torch.float32, v)
        s["param"] = flat(total, DTYPES[case["param"]])
        s["lr_scale"] = [1.0 if i % 7 else 0.5 for i in range(len(lens))]
        s["decay"] = [0.1 if n > 5000 else 0.0 for n in lens]     # none on norms and biases
        s["lr"] = by_block([LR * x for x in s["lr_scale"]])
        s["lr_decay"] = by_block([LR * x * d for x, d in zip(s["lr_scale"], s["decay"])])
        s["seed"] = seed
        s["grad_scale"] = 1.0 / loss_scale
        s["max_norm"] = 1.0 if case["clip"] else 0.0
        # what the norm's operator and the sum over the ranks left: about twice the norm that is allowed
        s["sumsq"] = torch.tensor((2.0 + r.random()) ** 2 * loss_scale ** 2, dtype=torch.float64, device=dev)
    if own:
        from adam_zs_shard_amd import zsadamw as z
        esz = SIZES[case["grad"]]
        pieces = []
        for i, (n, at) in enumerate(zip(lens, offs)):
            q = dict(len=n, grads=[g.data_ptr() + esz * at for g in grads], index=at)
            if case["op"] == "sumsq":
                if case["store"]:
                    q["g_mean"] = s["mean"].data_ptr() + 4 * at
            else:
                b = 1 if case["bits"] == 8 else 4
                q.update(w=s["w"].data_ptr() + 4 * at, m=s["m"].data_ptr() + b * at, v=s["v"].data_ptr() + b * at,
                         param=s["param"].data_ptr() + 2 * at, weight_decay=s["decay"][i], lr_scale=s["lr_scale"][i])
                if case["bits"] == 8:
                    q.update(m_scale=s["m_scale"].data_ptr() + at // BLOCK * 4,
                             v_scale=s["v_scale"].data_ptr() + at // BLOCK * 4)
            pieces.append(q)
        nbytes = z.zs_adamw_workspace_bytes(lens, case["p"])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        s["table"] = z.zs_adamw_upload(pieces, case["p"], case["grad"], case.get("param"), case.get("bits", 0),
                                       s["workspace"], nbytes)
        s["api"] = z
    return s


def run(s):
    if own:
        return run_own(s)
    return {"adamw": plain_adamw, "sumsq": plain_sumsq, "convert": plain_convert}[s["case"]["op"]](s)


def run_own(s):
    case, z = s["case"], s["api"]
    if case["op"] == "convert":
        if case["to"] == 8:
            z.zs_state8_encode(s["x"], case["total"], case["kind"], s["codes"], s["scales"])
            return {"codes": s["codes"], "scales": s["scales"]}
        z.zs_state8_decode(s["codes"], s["scales"], case["total"], case["kind"], s["x"])
        return {"x": s["x"]}
    if case["op"] == "sumsq":
        z.zs_grad_sumsq_multi(s["table"], s["sumsq"], store_mean=case["store"])
        return {"sumsq": s["sumsq"], "mean": s["mean"]} if case["store"] else {"sumsq": s["sumsq"]}
    hp = z.hparams(LR, BETA1, BETA2, EPS, s["step"], grad_scale=s["grad_scale"], max_norm=s["max_norm"],
                   rounding=case["rounding"], seed=s["seed"])
    z.zs_adamw_step_multi(s["table"], hp, s["sumsq"] if case["clip"] else None)
    return {k: s[k] for k in ("w", "m", "v", "param", "m_scale", "v_scale") if k in s}


def mean_of_ranks(grads):
    """The ranks' sum in their order, rounded to fp32 at each addition, over their number."""
    total = grads[0].float()
    for g in grads[1:]:
        total = total + g
    return total if len(grads) == 1 else total / torch.full((), float(len(grads)), device=total.device)


def plain_sumsq(s):
    mean = mean_of_ranks(s["grads"])
    sumsq = mean.double().square().sum()
    if not s["case"]["store"]:
        return {"sumsq": sumsq}
    s["mean"].copy_(mean)
    return {"sumsq": sumsq, "mean": s["mean"]}


def plain_adamw(s):
    case, dev = s["case"], s["w"].device
    eight = case["bits"] == 8
    bc1, bc2 = 1.0 - BETA1 ** s["step"], 1.0 - BETA2 ** s["step"]
    g = mean_of_ranks(s["grads"])
    if case["clip"]:
        norm = s["sumsq"].sqrt() * abs(s["grad_scale"])
        coef = torch.clamp(torch.full((), s["max_norm"], dtype=torch.float64, device=dev) / (norm + 1e-6), max=1.0)
        g = g * (s["grad_scale"] * coef).float()
    else:
        g = g * s["grad_scale"]
    g = g.view(-1, BLOCK)
    m, v, w = (s[k].view(-1, BLOCK) for k in ("m", "v", "w"))
    if eight:
        m = m.float() * s["m_scale"][:, None]
        v = v.float() * s["v_scale"][:, None]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    if eight:
        u = (m * (1.0 / bc1)) / (v.sqrt() * (1.0 / bc2 ** 0.5) + EPS)
    else:
        u = (m / torch.full((), bc1, device=dev)) / ((v / torch.full((), bc2, device=dev)).sqrt() + EPS)
    w.sub_(u * s["lr"] + w * s["lr_decay"])
    s["param"].copy_(s["w"])
    if not eight:
        s["m"].copy_(m.view(-1))
        s["v"].copy_(v.view(-1))
        return {k: s[k] for k in ("w", "m", "v", "param")}
    low = high = None
    if case["rounding"] == "stochastic":
        low, high = random_halves(s["w"].numel(), s["step"], s["seed"], dev)
    for k, x, r in (("m", m, low), ("v", v, high)):
        codes, scales = to_codes(x, k, r)
        s[k].copy_(codes.view(-1))
        s[k + "_scale"].copy_(scales.view(-1))
    return {k: s[k] for k in ("w", "m", "v", "param", "m_scale", "v_scale")}


def plain_convert(s):
    case = s["case"]
    n, dev = case["total"], s["codes"].device
    if case["to"] == 8:
        x = torch.zeros(padded(n), device=dev)
        x[:n] = s["x"]
        codes, scales = to_codes(x.view(-1, BLOCK), case["kind"])
        s["codes"].copy_(codes.view(-1)[:n])
        s["scales"].copy_(scales.view(-1))
        return {"codes": s["codes"], "scales": s["scales"]}
    s["x"].copy_(s["codes"].float() * s["scales"].repeat_interleave(BLOCK)[:n])
    return {"x": s["x"]}


def to_codes(x, kind, halves=None):
    """The 8-bit codes and the scales of blocks of values, a row each; rounded to nearest, or by 16 random bits each."""
    top = M_MAX if kind == "m" else V_MAX
    most = x.abs().amax(1, keepdim=True)
    live = most >= TINY
    scales = torch.where(live, most * (1.0 / top), 0.0)
    inverse = torch.where(live, torch.full((), top, device=x.device) / most, 0.0)
    y = (x * inverse).clamp(-top, top)
    if halves is not None:
        y = to_grid(y, kind, halves.view(y.shape))
    codes = y.to(F8[kind])
    if kind == "v":  # the update divides by the root of v: what is above zero stays so
        bytes_ = codes.view(torch.uint8)
        bytes_ += ((x > 0) & live & (bytes_ == 0)).to(torch.uint8)
    return codes, scales


def to_grid(y, kind, halves):
    """y on the grid of its 8-bit type: up with the probability that its place between two neighbours says."""
    bits, least = (20, 2.0 ** -6) if kind == "m" else (21, 2.0 ** -14)
    size = y.abs()
    low = size < least      # the evenly spaced end of the grid, moved to where fp32 has that spacing
    size = torch.where(low, size + least, size)
    r = (halves << (bits - 16)) + (1 << (bits - 17))
    size = ((size.view(torch.int32) + r) & -(1 << bits)).view(torch.float32)
    return torch.copysign(torch.where(low, size - least, size), y)


def random_halves(n, step, seed, dev):
    """16 random bits twice for each element: Philox4x32 with 7 rounds, whose four words go to four elements."""
    word = 0xFFFFFFFF
    at = torch.arange(0, n, 4, device=dev)
    c0, c1 = at & word, at >> 32
    c2, c3 = torch.full_like(at, step & word), torch.full_like(at, step >> 32)
    k0, k1 = seed & word, (seed >> 32) & word
    for _ in range(7):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & word) ^ c1 ^ k0, b & word, ((a >> 32) & word) ^ c3 ^ k1, a & word
        k0, k1 = (k0 + 0x9E3779B9) & word, (k1 + 0xBB67AE85) & word
    words = torch.stack((c0, c1, c2, c3), 1).view(-1)
    return (words & 0xFFFF).int(), (words >> 16).int()


def work(case):
    n = case["total"] if case["op"] == "convert" else sum(lengths(case))
    if case["op"] == "convert":
        return {"bytes": 5 * n + 4 * padded(n) // BLOCK, "flops": 3 * n}
    read = case["p"] * SIZES[case["grad"]]
    if case["op"] == "sumsq":
        return {"bytes": n * (read + 4 * case["store"]) + 8, "flops": n * (case["p"] + 2)}
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (read + 8 + state + 2), "flops": n * (case["p"] + 20)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "convert":
        if case["to"] == 32:
            at = torch.arange(case["total"], device=s["codes"].device) // BLOCK
            return {"x": s["codes"].double() * s["scales"].double()[at]}
        blocks = torch.zeros(padded(case["total"]), dtype=torch.float64, device=s["x"].device)
        blocks[:case["total"]] = s["x"].double()
        codes, scales = exact_codes(blocks.view(-1, BLOCK), case["kind"])
        return {"codes": codes.view(-1)[:case["total"]], "scales": scales}
    mean = torch.zeros_like(s["grads"][0], dtype=torch.float64)
    for g in s["grads"]:
        mean += g.double()
    mean /= case["p"]
    if case["op"] == "sumsq":
        return {"sumsq": mean.square().sum(), "mean": mean} if case["store"] else {"sumsq": mean.square().sum()}
    if case["clip"]:
        norm = float(s["sumsq"]) ** 0.5 * s["grad_scale"]
        mean *= min(1.0, s["max_norm"] / (norm + 1e-6))
    mean *= s["grad_scale"]
    out = {}
    m, v = s["m"].double(), s["v"].double()
    if case["bits"] == 8:
        m.view(-1, BLOCK).mul_(s["m_scale"].double()[:, None])
        v.view(-1, BLOCK).mul_(s["v_scale"].double()[:, None])
    m = BETA1 * m + (1 - BETA1) * mean
    v = BETA2 * v + (1 - BETA2) * mean * mean
    del mean
    root = (v / (1 - BETA2 ** s["step"])).sqrt_()
    move = (m / (1 - BETA1 ** s["step"])).div_(root.add_(EPS))
    del root
    w = s["w"].double()
    blocks = [padded(n) // BLOCK for n in s["lens"]]
    for at, k, f, d in zip(s["offs"], blocks, s["lr_scale"], s["decay"]):
        here = slice(at, at + k * BLOCK)
        w[here] -= LR * f * (move[here] + d * w[here])
    out["w"], out["param"] = w, w
    if case["bits"] == 32:
        return dict(out, m=m, v=v)
    for k, x in (("m", m), ("v", v)):
        codes, out[k + "_scale"] = exact_codes(x.view(-1, BLOCK), k)
        # what random bits decide next to a border has no value in 64 bits
        out[k] = codes.view(-1) if case["rounding"] == "nearest" else None
    return out


def exact_codes(x, kind):
    """Blocks of 64-bit values on the grid of their 8-bit type, a sign, 2^e and 3 (m) or 2 (v) bits below."""
    top, least, bits = (448.0, -6, 3) if kind == "m" else (57344.0, -14, 2)
    most = x.abs().max(1).values
    live = most >= 2.0 ** -110
    scales = torch.where(live, most / top, torch.zeros_like(most))
    y = x * torch.where(live, top / most, torch.zeros_like(most))[:, None]
    exponent = torch.frexp(y.abs().clamp(min=2.0 ** least))[1] - 1
    spacing = torch.ldexp(torch.ones_like(y), exponent - bits)
    y = torch.round(y / spacing) * spacing
    if kind == "v":
        y = torch.where((x > 0) & live[:, None] & (y == 0), 2.0 ** (least - bits), y)
    return y, scales

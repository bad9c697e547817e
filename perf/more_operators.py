"""What the norm and embedding operators compute, in plain torch, and the calls a trainer makes of them.

Four operators whose parameters' gradients are sums over a rank's tokens: a layer norm or root-mean-square norm (with
the residual addition before it) and its backward pass, the lookup in an embedding table, scaled and with a position
table added, and the table's gradient. Weights are slices of the 16-bit working copy or fp32, gradients are written
whole or added to in f16, bf16 or f32, as the AdamW operators read them.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5


def norm_case(name, op, rows, cols, **more):
    """dtype: of activations; w: of the weights; grad: of their gradients; gap: elements between two rows."""
    case = dict(name=name, op=op, kind="layer", rows=rows, cols=cols, dtype="bf16", w="bf16", residual=False, gap=0)
    if op == "norm_grad":
        case.update(grad="bf16", add=False)
    return dict(case, **more)


def embed_case(name, op, tokens, rows, cols, **more):
    """vocab: ids are below it, `first` the first of the table's rows among them; ids: bits of an id; pad: share of -1."""
    case = dict(name=name, op=op, tokens=tokens, vocab=rows, first=0, rows=rows, cols=cols, dtype="bf16", ids=64,
                pad=0.0, scale=1.0, gap=0)
    if op == "embed":
        case.update(w="bf16", positions=0)
    else:
        case.update(grad="bf16", add=False)
    return dict(case, **more)


def listed():
    return [
        # one token of an 8B-parameter model being decoded: what a call costs
        norm_case("norm_token", "norm", 1, 4096, kind="rms", residual=True),
        # a 124M-parameter model's layer norm over a micro batch of 8 sequences
        norm_case("norm_gpt2", "norm", 8192, 768),
        # an 8B-parameter model's norm behind the residual addition, two sequences of 8192
        norm_case("norm_llama", "norm", 16384, 4096, kind="rms", residual=True),
        # a ragged batch of a small fp16 model of odd width, rows cut out of a wider buffer
        norm_case("norm_grad_odd", "norm_grad", 333, 1001, dtype="f16", w="f32", grad="f32", gap=3),
        # the backward passes of the two ordinary ones; the second adds to fp32 gradients over micro batches
        norm_case("norm_grad_gpt2", "norm_grad", 8192, 768),
        norm_case("norm_grad_llama", "norm_grad", 16384, 4096, kind="rms", residual=True, grad="f32", add=True),
        # a few tokens' lookup in an fp32 table, scaled by the root of its odd width
        embed_case("embed_few", "embed", 37, 10_007, 515, dtype="f16", w="f32", scale=515 ** 0.5, ids=32),
        # tokens and positions of a 124M-parameter model
        embed_case("embed_gpt2", "embed", 8192, 50257, 768, positions=1024),
        # the gradient of a short micro batch, added to what the output projection left in a tied table
        embed_case("embed_grad_tied", "embed_grad", 500, 50257, 768, add=True, pad=0.02),
        # one micro batch, the table's whole gradient
        embed_case("embed_grad_gpt2", "embed_grad", 8192, 50257, 768, pad=0.02),
        # an 8B-parameter model's table, two sequences of 8192
        embed_case("embed_grad_llama", "embed_grad", 16384, 128256, 4096, ids=32),
        # long sequences added to the fp32 gradient of the first of 8 parts of a vocabulary, where most tokens are
        embed_case("embed_grad_part", "embed_grad", 131072, 16032, 1024, vocab=128256, grad="f32", add=True,
                   gap=8),
    ]


def spread(rng, low, high):
    return int(low * (high / low) ** rng.random())


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "norm_grad", "embed", "embed_grad", "embed_grad"])
    dtype, w, grad = (rng.choice(["bf16", "bf16", "f16", "f32"]) for _ in range(3))
    gap = rng.choice([0, 0, 0, 1, 8, 64])
    if op in ("norm", "norm_grad"):
        cols = spread(rng, 32, 16384)
        cols = rng.choice([cols, -(-cols // 64) * 64])
        rows = spread(rng, 1, min(65536, 40_000_000 // cols))
        case = norm_case("", op, rows, cols, kind=rng.choice(["layer", "rms"]), dtype=dtype, w=w, gap=gap,
                         residual=rng.random() < 0.5)
    else:
        cols = spread(rng, 32, 8192)
        cols = rng.choice([cols, -(-cols // 64) * 64])
        rows = spread(rng, 500, min(256_000, 200_000_000 // cols))
        parts = rng.choice([1, 1, 1, 2, 8])
        tokens = spread(rng, 1, min(200_000, 60_000_000 // cols))
        case = embed_case("", op, tokens, rows, cols, vocab=rows * parts, first=rows * rng.randrange(parts), dtype=dtype,
                          ids=rng.choice([32, 64]), scale=rng.choice([1.0, cols ** 0.5]), gap=gap)
        if op == "embed":
            case.update(w=w, positions=rng.choice([0, 0, 1024, 8192]))
        else:
            case["pad"] = rng.choice([0.0, 0.02, 0.3])
    if op.endswith("_grad"):
        case.update(grad=grad, add=rng.random() < 0.4)
    del case["name"]
    return case


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype, cols = DTYPES[case["dtype"]], case["cols"]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=gen, device=dev).mul_(std).add_(mean)

    def rows_of(n, values=None):
        """n rows of activations, `gap` elements apart."""
        x = torch.zeros(n, cols + case["gap"], dtype=dtype, device=dev)[:, :cols]
        return x if values is None else x.copy_(values)

    s = dict(case=case)
    if case["op"] in ("norm", "norm_grad"):
        n, layer = case["rows"], case["kind"] == "layer"
        x = normal(n, cols) * (0.3 + 2.0 * torch.rand(n, 1, generator=gen, device=dev)) + normal(cols, std=0.2)
        x[:, :: 997] *= 20.0     # the few large channels that trained models have
        s["gamma"] = normal(cols, std=0.1, mean=1.0).to(DTYPES[case["w"]])
        s["beta"] = normal(cols, std=0.1).to(DTYPES[case["w"]]) if layer else None
        if case["op"] == "norm":
            s["x"], s["y"] = rows_of(n, x), rows_of(n)
            s["residual"], s["total"] = (rows_of(n, normal(n, cols, std=2.0)), rows_of(n)) if case["residual"] else (None, None)
            s["mean"] = torch.zeros(n, device=dev) if layer else None
            s["rstd"] = torch.zeros(n, device=dev)
            return s if not own else keep_api(s)
        s["x"], s["dx"] = rows_of(n, x), rows_of(n)
        wide = s["x"].float()
        s["mean"] = wide.mean(1) if layer else None
        s["rstd"] = ((wide - s["mean"][:, None]) if layer else wide).square().mean(1).add(EPS).rsqrt()
        s["dy"] = rows_of(n, normal(n, cols, std=1e-2))
        s["dres"] = rows_of(n, normal(n, cols, std=1e-2)) if case["residual"] else None
        grad = DTYPES[case["grad"]]
        s["dgamma"] = normal(cols, std=0.3).to(grad)
        s["dbeta"] = normal(cols, std=0.3).to(grad) if layer else None
        if own:
            keep_api(s)
            s["nbytes"] = s["api"].zs_norm_workspace_bytes(n, cols)
            s["workspace"] = torch.empty(s["nbytes"], dtype=torch.uint8, device=dev)
        return s
    n, rows = case["tokens"], case["rows"]
    # token frequencies fall as 1 / rank
    u = torch.rand(n, generator=gen, dtype=torch.float64, device=dev)
    ids = ((u * math.log(case["vocab"] + 1)).exp() - 1).long().clamp_(0, case["vocab"] - 1)
    ids[torch.rand(n, generator=gen, device=dev) < case["pad"]] = -1
    s["ids"] = ids if case["ids"] == 64 else ids.int()
    if case["op"] == "embed":
        s["table"] = normal(rows, cols, std=0.02).to(DTYPES[case["w"]])
        s["y"] = rows_of(n)
        if case["positions"]:
            s["pos"] = (torch.arange(n, device=dev) % case["positions"]).to(s["ids"].dtype)
            s["pos_table"] = normal(case["positions"], cols, std=0.02).to(DTYPES[case["w"]])
        return s if not own else keep_api(s)
    s["dy"] = rows_of(n, normal(n, cols, std=1e-2))
    s["grad"] = normal(rows, cols, std=1e-2).to(DTYPES[case["grad"]])
    if own:
        keep_api(s)
        s["nbytes"] = s["api"].zs_embed_workspace_bytes(n, rows, cols)
        s["workspace"] = torch.empty(s["nbytes"], dtype=torch.uint8, device=dev)
    return s


def keep_api(s):
    from adam_zs_shard_amd import zslayer
    s["api"] = zslayer
    return s


def run(s):
    if own:
        return run_own(s)
    return {"norm": plain_norm, "norm_grad": plain_norm_grad, "embed": plain_embed,
            "embed_grad": plain_embed_grad}[s["case"]["op"]](s)


def run_own(s):
    case, z = s["case"], s["api"]
    op, cols = case["op"], case["cols"]
    if op == "norm":
        z.zs_norm_forward(case["rows"], cols, s["x"], s["y"], s["gamma"], s["beta"], kind=case["kind"], eps=EPS,
                          residual=s["residual"], total=s["total"], mean=s["mean"], rstd=s["rstd"])
        return {k: s[k] for k in ("y", "total", "mean", "rstd") if s[k] is not None}
    if op == "norm_grad":
        z.zs_norm_backward(case["rows"], cols, s["dy"], s["x"], s["rstd"], s["dx"], mean=s["mean"], gamma=s["gamma"],
                           dres=s["dres"], dgamma=s["dgamma"], dbeta=s["dbeta"], kind=case["kind"],
                           accumulate=case["add"], workspace=s["workspace"], ws_bytes=s["nbytes"])
        return {k: s[k] for k in ("dx", "dgamma", "dbeta") if s[k] is not None}
    if op == "embed":
        z.zs_embed_forward(case["tokens"], s["ids"], case["rows"], cols, s["table"], s["y"], scale=case["scale"],
                           first_row=case["first"], pos_ids=s.get("pos"), pos_rows=case["positions"],
                           pos_table=s.get("pos_table"))
        return {"y": s["y"]}
    z.zs_embed_backward(case["tokens"], s["ids"], case["rows"], cols, s["dy"], s["grad"], s["workspace"], s["nbytes"],
                        scale=case["scale"], first_row=case["first"], accumulate=case["add"])
    return {"grad": s["grad"]}


def plain_norm(s):
    if s["residual"] is not None:
        s["total"].copy_(s["x"].float() + s["residual"].float())
    t = (s["x"] if s["residual"] is None else s["total"]).float()
    if s["mean"] is not None:
        s["mean"].copy_(t.mean(1))
        t = t - s["mean"][:, None]
    s["rstd"].copy_((t.square().mean(1) + EPS).rsqrt())
    y = t * s["rstd"][:, None] * s["gamma"].float()
    s["y"].copy_(y if s["beta"] is None else y + s["beta"].float())
    return {k: s[k] for k in ("y", "total", "mean", "rstd") if s[k] is not None}


def plain_norm_grad(s):
    dy, x = s["dy"].float(), s["x"].float()
    xh = (x if s["mean"] is None else x - s["mean"][:, None]) * s["rstd"][:, None]
    a = dy * s["gamma"].float()
    dx = a - xh * (a * xh).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - a.mean(1, keepdim=True)
    dx = dx * s["rstd"][:, None]
    s["dx"].copy_(dx if s["dres"] is None else dx + s["dres"].float())
    dgamma = (dy * xh).sum(0)
    s["dgamma"].copy_(s["dgamma"].float() + dgamma if s["case"]["add"] else dgamma)
    if s["dbeta"] is not None:
        dbeta = dy.sum(0)
        s["dbeta"].copy_(s["dbeta"].float() + dbeta if s["case"]["add"] else dbeta)
    return {k: s[k] for k in ("dx", "dgamma", "dbeta") if s[k] is not None}


def rows_among(s):
    """Each id's row of the table, and whether it has one."""
    row = s["ids"].long() - s["case"]["first"]
    return row, (row >= 0) & (row < s["case"]["rows"])


def plain_embed(s):
    row, inside = rows_among(s)
    y = s["table"][torch.where(inside, row, 0)].float() * s["case"]["scale"]
    y = torch.where(inside[:, None], y, 0.0)
    s["y"].copy_(y if "pos" not in s else y + s["pos_table"][s["pos"].long()].float())
    return {"y": s["y"]}


def plain_embed_grad(s):
    case = s["case"]
    row, inside = rows_among(s)
    sums = torch.zeros(case["rows"] + 1, case["cols"], device=row.device)
    sums.index_add_(0, torch.where(inside, row, case["rows"]), s["dy"].float())
    sums = sums[:-1] * case["scale"]
    s["grad"].copy_(s["grad"].float() + sums if case["add"] else sums)
    return {"grad": s["grad"]}


def distinct(case):
    """How many of the table's rows the case's tokens name, about."""
    r = torch.arange(case["first"], case["first"] + case["rows"], dtype=torch.float64)
    p = torch.log((r + 2) / (r + 1)) / math.log(case["vocab"] + 1)
    return int((1 - (1 - p) ** (case["tokens"] * (1 - case.get("pad", 0.0)))).sum()) + 1


def work(case):
    cols, b = case["cols"], SIZES[case["dtype"]]
    if case["op"] in ("norm", "norm_grad"):
        n, layer, res = case["rows"] * cols, case["kind"] == "layer", case["residual"]
        vectors = cols * (1 + layer)
        if case["op"] == "norm":
            return {"bytes": n * b * (4 if res else 2) + vectors * SIZES[case["w"]] + 4 * case["rows"] * (1 + layer),
                    "flops": n * 8}
        return {"bytes": n * b * (4 if res else 3) + 4 * case["rows"] * (1 + layer) + cols * SIZES[case["w"]] +
                vectors * SIZES[case["grad"]] * (1 + case["add"]), "flops": n * 12}
    n, ids = case["tokens"] * cols, case["tokens"] * case["ids"] // 8
    if case["op"] == "embed":
        pos = case["positions"]
        return {"bytes": n * b + ids * (1 + (pos > 0)) + (distinct(case) + min(pos, case["tokens"])) * cols * SIZES[case["w"]],
                "flops": n * (1 + (pos > 0))}
    part = math.log((case["first"] + 1 + case["rows"]) / (case["first"] + 1)) / math.log(case["vocab"] + 1)
    rows = 2 * distinct(case) if case["add"] else case["rows"]
    here = part * (1 - case["pad"])    # a token outside the rows has no part in the gradient
    return {"bytes": int(n * here) * b + ids + rows * cols * SIZES[case["grad"]], "flops": int(n * here)}


def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if case["op"] == "norm":
        out, t = {}, wide["x"]
        if case["residual"]:
            out["total"] = t + wide["residual"]
            t = out["total"].to(s["x"].dtype).double()     # the norm is of what is stored
        middle = torch.zeros((), dtype=torch.float64, device=t.device)
        if case["kind"] == "layer":
            out["mean"] = t.sum(1) / case["cols"]
            middle = out["mean"][:, None]
        out["rstd"] = 1.0 / torch.sqrt(((t - middle) ** 2).sum(1) / case["cols"] + EPS)
        out["y"] = (t - middle) * out["rstd"][:, None] * wide["gamma"] + wide.get("beta", 0.0)
        return out
    if case["op"] == "norm_grad":
        layer = case["kind"] == "layer"
        hat = (wide["x"] - (wide["mean"][:, None] if layer else 0.0)) * wide["rstd"][:, None]
        a = wide["dy"] * wide["gamma"]
        along = torch.einsum("rc,rc->r", a, hat)[:, None] / case["cols"]
        level = a.sum(1, keepdim=True) / case["cols"] if layer else 0.0
        out = {"dx": (a - level - hat * along) * wide["rstd"][:, None] + wide.get("dres", 0.0)}
        out["dgamma"] = (hat * wide["dy"]).sum(0) + (wide["dgamma"] if case["add"] else 0.0)
        if layer:
            out["dbeta"] = wide["dy"].sum(0) + (wide["dbeta"] if case["add"] else 0.0)
        return out
    inside = (s["ids"] >= case["first"]) & (s["ids"] < case["first"] + case["rows"])
    at = (s["ids"].long() - case["first"])[inside]
    if case["op"] == "embed":
        y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device=at.device)
        y[inside] = wide["table"][at] * case["scale"]
        return {"y": y + wide["pos_table"][s["pos"].long()] if case["positions"] else y}
    grad = wide["grad"] if case["add"] else torch.zeros_like(wide["grad"])
    return {"grad": grad.index_put_((at,), wide["dy"][inside] * case["scale"], accumulate=True)}

"""Cases of the gradient-clipping operators, for measurement.

Four operators of one path: the norm over every gradient of a model, the
gradients scaled by it, and the two optimizer steps' kernels that take the
scale from device memory (AdamW; the first kernel of the Muon step).

    N = ||(g_1, ..., g_n)||_p          s = min(1, max_norm / (N + eps))
    clip:       out_i = s g_i
    adamw:      g' = s g;  p <- p (1 - lr wd);  m <- b1 m + (1 - b1) g';  v <- b2 v + (1 - b2) g'^2;
                p <- p - lr / (1 - b1^t) * m / (sqrt(v / (1 - b2^t)) + eps)
    normalize:  g' = s g;  buf <- beta buf + g';  u = g' + beta buf;
                X0 = bf16(u / (||u||_F + 1e-7)), transposed when rows > columns

The tensors of a case are views into one flat buffer, one after the other, as
gradient buckets and flat parameter buffers lay them out: after a tensor of
odd length the next one starts at an odd element.
"""
import math

import torch

own = False

LR, B1, B2, EPS, WD, STEP0 = 6e-4, 0.9, 0.999, 1e-8, 0.1, 9
BETA, NORM_EPS, CLIP_EPS = 0.95, 1e-7, 1e-6
BF16, FP16, FP32 = "bfloat16", "float16", "float32"


# ---------------------------------------------------------------- shapes

def _hidden(layers, d):
    """The hidden matrices of `layers` GPT-2 blocks of width d, as stored."""
    return [s for _ in range(layers) for s in ((d, 3 * d), (d, d), (d, 4 * d), (4 * d, d))]


def _others(layers, d, vocab, ctx):
    """Every other GPT-2 parameter: embeddings, LayerNorm gains and biases, linear biases."""
    block = [(d,), (d,), (3 * d,), (d,), (d,), (d,), (4 * d,), (d,)]
    return [(vocab, d), (ctx, d)] + block * layers + [(d,), (d,)]


def _ragged(count, low, high):
    """`count` lengths spread over the logarithm of low..high, in a scrambled order, mostly odd."""
    steps = max(1, count - 1)
    at = [(i * 7919) % count for i in range(count)]
    return [(int(round(low * (high / low) ** (a / steps))) | (a % 4 > 0),) for a in at]


def _shapes(case):
    kind = case["tensors"]
    if kind == "matrix":
        return [(case["rows"], case["cols"])]
    if kind == "matrices":          # three of odd sizes: wide, tall and square
        r, c = case["rows"], case["cols"]
        return [(r, c), (c + 2, r), (r + 1, r + 1)]
    if kind == "hidden":
        return _hidden(case["layers"], case["d"])
    if kind == "others":
        return _others(case["layers"], case["d"], case["vocab"], case["ctx"])
    if kind == "model":
        return _hidden(case["layers"], case["d"]) + _others(case["layers"], case["d"], case["vocab"], case["ctx"])
    return _ragged(case["count"], case["low"], case["high"])


# ---------------------------------------------------------------- cases

def listed():
    gpt2 = dict(layers=12, d=768, vocab=50257, ctx=1024)
    return [
        # a single small matrix: what a call costs when there is next to nothing to read
        dict(name="norm_256", op="norm", tensors="matrix", rows=256, cols=256, dtype=FP32, p=2.0),
        # many small unaligned tensors, fp16, the largest entry instead of the sum of squares
        dict(name="norm_max_ragged", op="norm", tensors="ragged", count=193, low=1, high=200000, dtype=FP16, p=math.inf),
        # every gradient of GPT-2 124M as a bf16 backward pass leaves them
        dict(name="norm_124m_bf16", op="norm", tensors="model", dtype=BF16, p=2.0, **gpt2),
        # every gradient of the largest configuration, fp32: 1.56e9 elements in 580 tensors
        dict(name="norm_xl_fp32", op="norm", tensors="model", layers=48, d=1600, vocab=50257, ctx=1024, dtype=FP32, p=2.0),
        # one small matrix, clipped into another buffer: latency
        dict(name="clip_256", op="clip", tensors="matrix", rows=256, cols=256, dtype=FP32, out=FP32, max_norm=1.0, p=2.0),
        # ragged fp16 gradients at odd offsets, scaled into fp16
        dict(name="clip_ragged_fp16", op="clip", tensors="ragged", count=61, low=3, high=400000, dtype=FP16, out=FP16, max_norm=1.0, p=2.0),
        # GPT-2 124M: bf16 gradients clipped into the fp32 ones that the optimizer steps read
        dict(name="clip_124m_to_fp32", op="clip", tensors="model", dtype=BF16, out=FP32, max_norm=1.0, p=2.0, **gpt2),
        # GPT-2 medium, in place, on a step whose norm is under the bound: most steps of a run
        dict(name="clip_medium_under", op="clip", tensors="model", layers=24, d=1024, vocab=50257, ctx=1024,
             dtype=FP32, out="", max_norm=1e4, p=2.0),
        # a few ragged tensors of the AdamW group
        dict(name="adamw_ragged", op="adamw", tensors="ragged", count=7, low=1, high=50000, dtype=FP32),
        # the 100 AdamW tensors of GPT-2 124M (39.5e6 elements)
        dict(name="adamw_124m", op="adamw", tensors="others", dtype=FP32, **gpt2),
        # three matrices with odd sides through the Muon step's first kernel
        dict(name="normalize_odd", op="normalize", tensors="matrices", rows=129, cols=1001, dtype=FP32),
        # the 48 hidden matrices of GPT-2 124M through the same kernel
        dict(name="normalize_124m", op="normalize", tensors="hidden", layers=12, d=768, dtype=FP32),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "clip", "adamw", "normalize"])
    case = dict(op=op, dtype=FP32)
    if op in ("norm", "clip"):
        case["dtype"] = rng.choice([FP32, BF16, FP16])
        case["p"] = rng.choice([2.0, 2.0, 1.0, math.inf])
    if op == "clip":
        case["out"] = rng.choice([FP32, case["dtype"], BF16, ""])
    if op == "normalize":
        if rng.random() < 0.5:
            case.update(tensors="matrices", rows=_log(rng, 3, 2000), cols=_log(rng, 5, 6000))
        else:
            case.update(tensors="hidden", layers=rng.randint(1, 12), d=_log(rng, 64, 768))
        return case
    kind = rng.choice(["ragged", "model", "others", "matrix"])
    case["tensors"] = kind
    if kind == "ragged":
        case.update(count=_log(rng, 2, 600), low=rng.randint(1, 50), high=_log(rng, 1000, 500000))
    elif kind == "matrix":
        case.update(rows=_log(rng, 1, 8192), cols=_log(rng, 1, 8192))
    else:
        case.update(layers=rng.randint(1, 24), d=_log(rng, 64, 1024), vocab=_log(rng, 1000, 50257), ctx=rng.randint(64, 1024))
    if op == "clip":
        # a bound a little below the norm to be expected, or far above it; in place always above,
        # so that a pass finds what the last one found
        n = sum(math.prod(s) for s in _shapes(case))
        about = 5e-3 * {1.0: n, 2.0: math.sqrt(n), math.inf: 4.0}[case["p"]]
        case["max_norm"] = 1e9 if case["out"] == "" else rng.choice([0.25 * about, 0.7 * about, 1e9])
    return case


# ---------------------------------------------------------------- inputs

def _views(flat, shapes):
    out, at = [], 0
    for s in shapes:
        n = math.prod(s)
        out.append(flat[at:at + n].view(s))
        at += n
    return out


def _aligned_views(flat, shapes):
    """Each on a 16-byte boundary: the Muon step's matrices have to be."""
    out, at = [], 0
    for s in shapes:
        n = math.prod(s)
        out.append(flat[at:at + n].view(s))
        at += -(-n // 4) * 4
    return out


def prepare(case, seed):
    shapes = _shapes(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda n, std=1.0: torch.empty(n, device="cuda").normal_(0.0, std, generator=gen)  # noqa: E731
    n = sum(math.prod(s) for s in shapes)
    state = dict(case=case)
    if case["op"] == "normalize":
        n = sum(-(-math.prod(s) // 4) * 4 for s in shapes)
        state["grads"] = _aligned_views(normal(n), shapes)
        state["buf"] = normal(n, 0.1)
        state["bufs"] = _aligned_views(state["buf"], shapes)
        state["scale"] = torch.rand((), device="cuda", generator=gen) * 0.5 + 0.25
        return state
    flat = normal(n)
    views = _views(flat, shapes)
    # layers' gradients differ in size: a standard deviation of 1e-3 to 1e-2 for each tensor
    for view, std in zip(views, (10.0 ** (torch.rand(len(shapes), device="cuda", generator=gen) - 3.0)).unbind()):
        view.mul_(std)
    flat = flat.to(getattr(torch, case["dtype"]))
    state["flat"] = flat
    state["grads"] = _views(flat, shapes)
    if case["op"] == "clip" and case["out"]:
        state["out"] = torch.empty(n, device="cuda", dtype=getattr(torch, case["out"]))
        state["outs"] = _views(state["out"], shapes)
    if case["op"] == "adamw":
        state["p"], state["m"] = normal(n, 0.02), normal(n, 1e-3)
        state["v"] = normal(n, 1e-2).square_()
        state["t"] = STEP0
        state["decay"] = [len(s) > 1 or i % 2 == 0 for i, s in enumerate(shapes)]
        state["scale"] = torch.rand((), device="cuda", generator=gen) * 0.5 + 0.25
        for k in ("p", "m", "v"):
            state[k + "s"] = _views(state[k], shapes)
    if own:
        # the handle a training loop makes once for its tensors
        import newton_schulz_norm_b200 as muon
        if case["op"] == "adamw":
            state["group"] = muon.AdamWGroup(state["ps"], state["grads"], state["ms"], state["vs"], lr=LR,
                                             betas=(B1, B2), eps=EPS, weight_decay=WD, decay=state["decay"])
        else:
            state["group"] = muon.GradGroup(state["grads"], out=state.get("outs"))
    return state


# ---------------------------------------------------------------- one pass

def _plain_norm(grads, p):
    if p == math.inf:
        return torch.stack([g.float().abs().amax() for g in grads]).amax()
    if p == 1.0:
        return torch.stack([g.float().abs().sum() for g in grads]).double().sum().float()
    return torch.stack([g.float().square().sum() for g in grads]).double().sum().sqrt().float()


def _plain_clip(state, case):
    norm = _plain_norm(state["grads"], case["p"])
    scale = (case["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    for g, o in zip(state["grads"], state.get("outs", state["grads"])):
        o.copy_(g.float() * scale)
    return norm


def _plain_adamw(state, t):
    for p, g, m, v, d in zip(state["ps"], state["grads"], state["ms"], state["vs"], state["decay"]):
        g = g * state["scale"]
        p.mul_(1 - LR * WD if d else 1.0)
        m.mul_(B1).add_(g, alpha=1 - B1)
        v.mul_(B2).add_(g * g, alpha=1 - B2)
        p.sub_(LR / (1 - B1 ** t) * m / ((v / (1 - B2 ** t)).sqrt() + EPS))


def _plain_normalize(g, buf, scale):
    g = g * scale
    buf.mul_(BETA).add_(g)
    u = g + BETA * buf
    x = (u / (u.square().sum().sqrt() + NORM_EPS)).bfloat16()
    return x.t() if x.shape[0] > x.shape[1] else x


def run(state):
    case = state["case"]
    op = case["op"]
    if op == "norm":
        return state["group"].norm(case["p"]) if own else _plain_norm(state["grads"], case["p"])
    if op == "clip":
        norm = state["group"].clip(case["max_norm"], case["p"]) if own else _plain_clip(state, case)
        return dict(norm=norm, grads=state["out"] if case["out"] else state["flat"])
    if op == "adamw":
        state["t"] += 1
        if own:
            state["group"].step(state["t"], grad_scale=state["scale"])
        else:
            _plain_adamw(state, state["t"])
        return dict(p=state["p"], m=state["m"], v=state["v"])
    if own:
        import newton_schulz_norm_b200 as muon
        x0 = muon.momentum_normalize(state["grads"], state["bufs"], beta=BETA, grad_scale=state["scale"])
    else:
        x0 = [_plain_normalize(g, b, state["scale"]) for g, b in zip(state["grads"], state["bufs"])]
    return dict(x0=x0, buf=state["buf"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    n = sum(math.prod(s) for s in _shapes(case))
    size = 4 if case["dtype"] == FP32 else 2
    if case["op"] == "norm":
        return dict(bytes=n * size + 4, flops=2 * n)
    if case["op"] == "clip":
        # in place under the bound the gradients stay as they are: nothing to write
        write = 0 if case["out"] == "" else 4 if case["out"] == FP32 else 2
        return dict(bytes=n * (size + write) + 4, flops=3 * n)
    if case["op"] == "adamw":
        return dict(bytes=28 * n, flops=16 * n)        # read p, g, m, v; write p, m, v
    return dict(bytes=14 * n, flops=9 * n)             # read g, buf; write buf and bf16 X0


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    grads = state["grads"]
    if case["op"] == "normalize":
        s, bufs, x0 = state["scale"].double(), [], []
        for g, b in zip(grads, state["bufs"]):
            g = g.double() * s
            new = BETA * b.double() + g
            u = g + BETA * new
            x = u / (torch.linalg.vector_norm(u) + NORM_EPS)
            bufs.append(new)
            x0.append(x.mT if x.shape[0] > x.shape[1] else x)
        buf = state["buf"].double()
        for view, new in zip(_aligned_views(buf, _shapes(case)), bufs):
            view.copy_(new)
        return dict(x0=x0, buf=buf)
    if case["op"] == "adamw":
        t, s = STEP0 + 1, state["scale"].double()
        p, m, v = (state[k].double() for k in ("p", "m", "v"))
        g = state["flat"].double() * s
        m = B1 * m + (1 - B1) * g
        v = B2 * v + (1 - B2) * g * g
        step = (LR / (1 - B1 ** t)) * m / ((v / (1 - B2 ** t)) ** 0.5 + EPS)
        keep = torch.repeat_interleave(torch.tensor([1 - LR * WD if d else 1.0 for d in state["decay"]], device="cuda", dtype=torch.float64),
                                       torch.tensor([g.numel() for g in grads], device="cuda"))
        return dict(p=p * keep - step, m=m, v=v)
    parts = torch.stack([torch.linalg.vector_norm(g.double(), case["p"]) for g in grads])
    norm = torch.linalg.vector_norm(parts, case["p"])
    if case["op"] == "norm":
        return norm
    scale = min(1.0, case["max_norm"] / (float(norm) + CLIP_EPS))
    return dict(norm=norm, grads=state["flat"].double() * scale)

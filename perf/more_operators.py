"""Cases of the operators around the packed-MXFP4 products: the product with
bias, activation and residual in its epilogue, the products grouped by expert,
and the router and the weighted sum on either side of those.

    linear    Y = residual + act(X W^T + bias)
    grouped   Y[p] = act(X[row(p)] W_e^T + bias_e), offsets[e] <= p < offsets[e + 1]
    route     k experts a token by softmax or sigmoid scores, their weights, and the rows sorted by expert
    combine   y[t] = residual[t] + sum_j weight[t, j] Z[pos[t, j]]

W: packed MXFP4, blocks of 32 along a row share 2^e (scale byte e + 127),
elements are E2M1 values (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6), two codes a
byte, the even column in the low nibble.  X is bf16 (a16) or packed like W (a4).

`own` selects what run() calls: the package's operators, or their plain form
in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token being decoded through a router over 64 experts
        dict(name="route-token", op="route", tokens=1, experts=64, k=6, score="softmax", normalize=True, bias=False,
             scale=1.0, dtype="bf16", padded=0.0),
        # a padded batch of prompts, 256 experts chosen by biased sigmoid scores
        dict(name="route-prompt", op="route", tokens=16384, experts=256, k=8, score="sigmoid", normalize=True,
             bias=True, scale=2.5, dtype="f32", padded=0.1),
        # a decoding batch of 16: the sum over each token's experts joins the residual stream
        dict(name="combine-batch", op="combine", tokens=16, k=6, n=4096, dtype="bf16", residual="bf16", out="bf16",
             padded=0.0),
        # a padded prompt, fp32 out, odd width
        dict(name="combine-prompt", op="combine", tokens=4096, k=8, n=4100, dtype="bf16", residual="none", out="f32",
             padded=0.1),
        # a decoding batch of 16 on 64 experts, gate and up in one product
        dict(name="grouped-a16-batch", op="grouped", x="a16", tokens=16, experts=64, k=6, n=2816, kdim=2048,
             gather=True, bias="none", act="none", out="bf16"),
        # a prompt of 2048 tokens on 8 experts of a 7B-shaped MLP's up projection
        dict(name="grouped-a16-prompt", op="grouped", x="a16", tokens=2048, experts=8, k=2, n=11008, kdim=4096,
             gather=True, bias="bf16", act="silu", out="bf16"),
        # a decoding batch of 64 on 128 experts, gathered rows of packed activations
        dict(name="grouped-a4-batch", op="grouped", x="a4", tokens=64, experts=128, k=8, n=2048, kdim=4096,
             gather=True, bias="f32", act="none", out="bf16"),
        # 4096 tokens on 128 experts, the down projection on rows sorted by expert
        dict(name="grouped-a4-prompt", op="grouped", x="a4", tokens=4096, experts=128, k=8, n=4096, kdim=2048,
             gather=False, bias="none", act="none", out="bf16"),
        # the q, k and v projection with biases, one token being decoded
        dict(name="linear-a16-token", op="linear", x="a16", rows=1, n=6144, kdim=4096, bias="bf16", act="none",
             residual="none", out="bf16"),
        # the down projection of a 7B-shaped block onto its residual stream, a prompt of 2048 tokens
        dict(name="linear-a16-prompt", op="linear", x="a16", rows=2048, n=4096, kdim=11008, bias="none", act="none",
             residual="bf16", out="bf16"),
        # odd sizes, K off every stage, fp32 stream
        dict(name="linear-a4-odd", op="linear", x="a4", rows=333, n=1001, kdim=2080, bias="f32", act="gelu",
             residual="f32", out="f32"),
        # 4096 tokens through the first linear of an un-gated MLP four times as wide, with bias and activation
        dict(name="linear-a4-prompt", op="linear", x="a4", rows=4096, n=32768, kdim=8192, bias="bf16",
             act="gelu_tanh", residual="none", out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "combine", "grouped", "grouped", "linear", "linear"])
    types = ["none", "bf16", "f32"]
    if op == "route":
        experts = _log(rng, 4, 512)
        return dict(op=op, tokens=_log(rng, 1, 8192), experts=experts, k=rng.randint(1, min(8, experts)),
                    score=rng.choice(["softmax", "sigmoid"]), normalize=rng.random() < 0.7, bias=rng.random() < 0.4,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["bf16", "f32"]), padded=rng.choice([0.0, 0.1]))
    if op == "combine":
        return dict(op=op, tokens=_log(rng, 1, 4096), k=rng.randint(1, 8), n=_log(rng, 33, 4100),
                    dtype=rng.choice(["bf16", "f32"]), residual=rng.choice(types), out=rng.choice(["bf16", "f32"]),
                    padded=rng.choice([0.0, 0.1]))
    act = rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"])
    common = dict(op=op, x=rng.choice(["a16", "a4"]), bias=rng.choice(types), act=act, out=rng.choice(["bf16", "f32"]))
    if op == "grouped":
        experts = _log(rng, 2, 128)
        return dict(common, tokens=_log(rng, 1, 4096), experts=experts, k=rng.randint(1, min(8, experts)),
                    n=_log(rng, 16, 4096), kdim=32 * _log(rng, 4, 128), gather=rng.random() < 0.5)
    return dict(common, rows=_log(rng, 1, 4096), n=_log(rng, 16, 28672), kdim=32 * _log(rng, 4, 256),
                residual=rng.choice(types))


SIZE = {"bf16": 2, "f32": 4, "none": 0}


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        return dict(bytes=t * e * SIZE[case["dtype"]] + 16 * t * k + 4 * (e + 1), flops=4 * t * e)
    if op == "combine":
        t, k, n = case["tokens"], case["k"], case["n"]
        kept = round(t * (1 - case["padded"])) * k
        return dict(bytes=kept * n * SIZE[case["dtype"]] + t * n * (SIZE[case["residual"]] + SIZE[case["out"]]) + 8 * t * k,
                    flops=2 * kept * n)
    n, k = case["n"], case["kdim"]
    held = lambda rows: rows * k // 2 + rows * k // 32 if case["x"] == "a4" else 2 * rows * k  # noqa: E731
    w, b = n * k // 2 + n * k // 32, n * SIZE[case["bias"]]
    if op == "linear":
        m = case["rows"]
        return dict(bytes=held(m) + w + b + m * n * (SIZE[case["residual"]] + SIZE[case["out"]]), flops=2 * m * n * k)
    p, e = case["tokens"] * case["k"], case["experts"]
    used = min(p, e * (1 - math.exp(-p / e)))     # experts that get a row, were the choice uniform
    return dict(bytes=int(held(case["tokens"] if case["gather"] else p) + used * (w + b) + p * n * SIZE[case["out"]] +
                          4 * (e + 1) + (4 * p if case["gather"] else 0)), flops=2 * p * n * k)


# -------------------------------------------------------------- plain form
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _values(packed, scale):
    """fp32 values [N, K] of packed codes and scale bytes (none of them NaN's)."""
    code = torch.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[0], -1)
    mag = (code & 7).float()
    mag = torch.where(mag < 4, mag / 2, torch.where(mag < 6, mag - 2, 2 * mag - 8))
    v = torch.where(code > 7, -mag, mag)
    p = torch.ldexp(torch.ones_like(scale, dtype=torch.float32), scale.to(torch.int32) - 127)
    return (v.reshape(*scale.shape, 32) * p[..., None]).reshape(v.shape)


def _activate(a, act):
    if act == "relu":
        return torch.where(a < 0, torch.zeros_like(a), a)
    if act == "silu":
        return a / (1 + torch.exp(-a))
    if act == "gelu":
        return 0.5 * a * torch.erfc(-a * math.sqrt(0.5))
    if act == "gelu_tanh":
        return a / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a * a * a)))
    return a


def _plain_route(s):
    case = s["case"]
    x, k = s["logits"].double(), case["k"]
    if case["score"] == "softmax":
        top = x.max(-1, keepdim=True).values
        score = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = score.sum(-1, keepdim=True)
        score = score / torch.where(total == 0, torch.ones_like(total), total)
    else:
        score = 1 / (1 + torch.exp(-x))
    by = x if s["bias"] is None else torch.where(x == -math.inf, x, score + s["bias"].double())
    order, index = torch.sort(by, dim=-1, descending=True, stable=True)
    index, kept = index[:, :k], order[:, :k] > -math.inf
    w = torch.where(kept, score.gather(1, index), torch.zeros_like(score[:, :k]))
    if case["normalize"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total == 0, torch.ones_like(total), total)
    expert = torch.where(kept, index, torch.full_like(index, -1))
    flat = torch.where(kept, index, torch.full_like(index, case["experts"])).reshape(-1)
    group, slot = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(group, torch.arange(case["experts"] + 1, device=x.device))
    real = group < case["experts"]
    place = torch.arange(flat.numel(), device=x.device)
    token = torch.where(real, slot // k, torch.full_like(slot, -1))
    pos = torch.empty_like(slot)
    pos[slot] = torch.where(real, place, torch.full_like(place, -1))
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    return dict(expert=i32(expert), weight=(w * case["scale"]).float(), offsets=i32(offsets), token=i32(token),
                pos=i32(pos).reshape(expert.shape))


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "route":
        return _plain_route(s)
    if op == "combine":
        pos = s["pos"].long()
        kept = (pos >= 0)[..., None]
        y = torch.zeros(case["tokens"], case["n"], device="cuda") if s["residual"] is None else s["residual"].float()
        for j in range(case["k"]):
            z = s["z"][pos[:, j].clamp(min=0)].float() * s["weight"][:, j, None]
            y = y + torch.where(kept[:, j], z, torch.zeros_like(z))
        return y.to(DTYPE[case["out"]])
    if op == "linear":
        x = s["x"].float() if case["x"] == "a16" else _values(s["x"], s["x_scale"])
        y = x @ _values(s["packed"], s["scale"]).t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        y = _activate(y, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(DTYPE[case["out"]])
    x = s["x"].float() if case["x"] == "a16" else _values(s["x"], s["x_scale"])
    out = torch.empty(s["borders"][-1], case["n"], dtype=DTYPE[case["out"]], device="cuda")
    for e in range(case["experts"]):
        lo, hi = s["borders"][e], s["borders"][e + 1]
        if lo == hi:
            continue
        y = (x[s["rows"][lo:hi].long()] if case["gather"] else x[lo:hi]) @ _values(s["packed"][e], s["scale"][e]).t()
        if s["bias"] is not None:
            y = y + s["bias"][e].float()
        out[lo:hi] = _activate(y, case["act"]).to(out.dtype)
    return out


# ----------------------------------------------------------------- prepare
def _quantize(x):
    """Packed codes and scale bytes of x [M, K], fp32 and finite."""
    b = x.reshape(x.shape[0], -1, 32)
    top = b.abs().amax(-1)
    e = torch.where(top > 0, (torch.frexp(top)[1] - 3).clamp(min=-126), torch.zeros_like(top, dtype=torch.int32))
    a = torch.ldexp(b.abs(), -e[..., None])
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(a, edges, out_int32=True).to(torch.uint8)
    code = (code + 8 * ((b < 0) & (code > 0)).to(torch.uint8)).reshape(x.shape)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _activations(rand, uniform, m, k):
    """Normal values with a few channels of large magnitude, as hidden states have."""
    return rand(m, k) * (1 + 19 * (uniform(k) < 0.004).float())


def _padding(case, uniform):
    """True for the tokens that are padding."""
    return uniform(case["tokens"]) < case["padded"]


def _choose(rand, uniform, tokens, experts, k):
    """k experts a token, some of them far more popular than others."""
    gumbel = -torch.log(-torch.log(uniform(tokens, experts).clamp(1e-7, 1 - 1e-7)))
    return torch.sort(gumbel + 0.7 * rand(experts), dim=-1, descending=True)[1][:, :k]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    uniform = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    maybe = lambda t, *s: None if t == "none" else rand(*s).to(DTYPE[t])  # noqa: E731
    op = case["op"]
    s = dict(case=case)
    if op == "route":
        logits = 1.5 * rand(case["tokens"], case["experts"])
        logits[_padding(case, uniform)] = -math.inf
        s["logits"] = logits.to(DTYPE[case["dtype"]])
        s["bias"] = 0.1 * rand(case["experts"]) if case["bias"] else None
        return s
    if op == "combine":
        t, k = case["tokens"], case["k"]
        kept = ~_padding(case, uniform)[:, None].expand(t, k)
        order = torch.argsort(uniform(t * k)).reshape(t, k)           # rows of the sorted order, any
        s["pos"] = torch.where(kept, order, torch.full_like(order, -1)).to(torch.int32)
        w = torch.softmax(rand(t, k), -1)
        s["weight"] = torch.where(kept, w, torch.zeros_like(w))
        s["z"] = rand(t * k, case["n"]).to(DTYPE[case["dtype"]])
        s["residual"] = maybe(case["residual"], t, case["n"])
        return s
    n, k = case["n"], case["kdim"]
    if op == "linear":
        m = case["rows"]
        s["packed"], s["scale"] = _quantize(0.02 * rand(n, k))
        s["bias"], s["residual"] = maybe(case["bias"], n), maybe(case["residual"], m, n)
    else:
        e = case["experts"]
        parts = [_quantize(0.02 * rand(n, k)) for _ in range(e)]
        s["packed"], s["scale"] = (torch.stack(p) for p in zip(*parts))
        s["bias"] = maybe(case["bias"], e, n)
        group, slot = torch.sort(_choose(rand, uniform, case["tokens"], e, case["k"]).reshape(-1), stable=True)
        s["rows"] = (slot // case["k"]).to(torch.int32) if case["gather"] else None
        s["offsets"] = torch.searchsorted(group, torch.arange(e + 1, device="cuda")).to(torch.int32)
        s["borders"] = s["offsets"].tolist()      # the plain form's; the package's operators read them on the GPU
        m = case["tokens"] if case["gather"] else group.numel()
    x = _activations(rand, uniform, m, k)
    if case["x"] == "a16":
        s["x"] = x.bfloat16()
    else:
        s["x"], s["x_scale"] = _quantize(x)
    return s


# --------------------------------------------------------------------- run
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import post_weight_quantization_autoround_amd as ar

    case = s["case"]
    op = case["op"]
    if op == "route":
        names = ("expert", "weight", "offsets", "token", "pos")
        return dict(zip(names, ar.moe_route(s["logits"], case["k"], score=case["score"], normalize=case["normalize"],
                                            bias=s["bias"], weight_scale=case["scale"])))
    dt = DTYPE[case["out"]]
    if op == "combine":
        return ar.moe_combine(s["z"], s["pos"], s["weight"], residual=s["residual"], out_dtype=dt)
    if op == "linear":
        more = dict(bias=s["bias"], act=case["act"], residual=s["residual"], out_dtype=dt)
        if case["x"] == "a16":
            return ar.mxfp4_linear(s["x"], s["packed"], s["scale"], **more)
        return ar.mxfp4_linear_a4(s["x"], s["x_scale"], s["packed"], s["scale"], **more)
    more = dict(rows=s["rows"], bias=s["bias"], act=case["act"], out_dtype=dt)
    if case["x"] == "a16":
        return ar.mxfp4_grouped_gemm(s["x"], s["packed"], s["scale"], s["offsets"], **more)
    return ar.mxfp4_grouped_gemm_a4(s["x"], s["x_scale"], s["packed"], s["scale"], s["offsets"], **more)


# ------------------------------------------------------------------- exact
def _decode64(packed, scale):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                         device=packed.device)
    n, half = packed.shape
    v = torch.empty(n, 2 * half, dtype=torch.float64, device=packed.device)
    v[:, 0::2] = table[(packed % 16).long()]
    v[:, 1::2] = table[(packed // 16).long()]
    return v * torch.exp2(scale.double() - 127).repeat_interleave(32, dim=1)


def _act64(a, act):
    if act == "relu":
        return a.clamp(min=0)
    if act == "silu":
        return a * torch.sigmoid(a)
    if act == "gelu":
        return a * torch.special.ndtr(a)
    if act == "gelu_tanh":
        return a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a.pow(3)))) / 2
    return a


def _exact_route(s):
    case = s["case"]
    x = s["logits"].double().cpu().numpy()
    t, e, k = case["tokens"], case["experts"], case["k"]
    with np.errstate(invalid="ignore", over="ignore"):
        if case["score"] == "softmax":
            top = x.max(1)
            score = np.exp(x - np.where(np.isinf(top), 0.0, top)[:, None])
            score /= np.maximum(score.sum(1), np.finfo(np.float64).tiny)[:, None]
        else:
            score = 1 / (1 + np.exp(-x))
    by = x if s["bias"] is None else np.where(np.isinf(x), x, score + s["bias"].double().cpu().numpy())
    expert = np.argsort(-by, axis=1, kind="stable")[:, :k]
    rows = np.arange(t)[:, None]
    real = by[rows, expert] > -np.inf
    w = np.where(real, score[rows, expert], 0.0)
    if case["normalize"]:
        w /= np.maximum(w.sum(1, keepdims=True), np.finfo(np.float64).tiny)
    expert = np.where(real, expert, -1).astype(np.int32)
    groups = [np.flatnonzero(expert.reshape(-1) == i) for i in range(e)]
    slots = np.concatenate(groups)
    offsets = np.concatenate([[0], np.cumsum([len(g) for g in groups])]).astype(np.int32)
    token, pos = np.full(t * k, -1, np.int32), np.full(t * k, -1, np.int32)
    token[:len(slots)] = slots // k
    pos[slots] = np.arange(len(slots))
    out = dict(expert=expert, weight=w * case["scale"], offsets=offsets, token=token, pos=pos.reshape(t, k))
    return {name: torch.from_numpy(a).cuda() for name, a in out.items()}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "combine":
        z = torch.cat((s["z"].double(), torch.zeros(1, case["n"], dtype=torch.float64, device="cuda")))
        at = torch.where(s["pos"] < 0, z.shape[0] - 1, s["pos"].long())
        y = 0 if s["residual"] is None else s["residual"].double()
        for j in range(case["k"]):
            y = y + s["weight"][:, j:j + 1].double() * z[at[:, j]]
        return y
    x = s["x"].double() if case["x"] == "a16" else _decode64(s["x"], s["x_scale"])
    if op == "linear":
        y = torch.addmm(torch.zeros(1, dtype=torch.float64, device="cuda") if s["bias"] is None else s["bias"].double(),
                        x, _decode64(s["packed"], s["scale"]).t())
        y = _act64(y, case["act"])
        return y if s["residual"] is None else y + s["residual"].double()
    if case["gather"]:
        x = x.index_select(0, s["rows"].long())
    out = torch.empty(x.shape[0], case["n"], dtype=torch.float64, device="cuda")
    for e, part in enumerate(x.split(torch.diff(s["offsets"]).tolist())):
        y = part @ _decode64(s["packed"][e], s["scale"][e]).t()
        out[s["borders"][e]:s["borders"][e + 1]] = _act64(y if s["bias"] is None else y + s["bias"][e].double(), case["act"])
    return out

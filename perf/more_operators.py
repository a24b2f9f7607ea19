"""What is measured of the 8-bit floating-point products and of the experts' layer made of them.

linear     y = x W^T (+ bias): W in 8-bit floats (e4m3) with a scale for each block of 128 x 128,
           x coded in 8-bit floats within the call, with a power of two as scale for each row and
           group of 128 values.
route      the experts of each token from the router's logits: softmax or sigmoid scores, a bias
           that only takes part in the choice, groups of experts, the largest k, weights
           renormalised; and the tokens sorted by expert.
experts    a gated MLP whose weights are those of the chosen experts:
           y = sum over a token's experts of weight * down(q(silu(gate(x)) * up(x))), with x and the
           product behind the gate coded in 8-bit floats as above.

Ranges and forms: codes are e4m3 values, at most 448 in magnitude.  A group's scale is the smallest
power of two S for which its largest magnitude is at most 448 S, and 1 where all its values are 0.
Block scales of weights are powers of two (float8_e8m0fnu) or float32, as checkpoints hold them.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _linear(name, m, k, n, dt="bf16", scales="pow2", bias=False):
    return dict(name=name, op="linear", m=m, k=k, n=n, dt=dt, scales=scales, bias=bias)


def _route(name, tokens, experts, k, score="softmax", dt="f32", bias=False, groups=1, top_groups=1, group_score=1,
           renormalize=True, scale=1.0):
    return dict(name=name, op="route", tokens=tokens, experts=experts, k=k, score=score, dt=dt, bias=bias, groups=groups,
                top_groups=top_groups, group_score=group_score, renormalize=renormalize, scale=scale)


def _experts(name, tokens, experts, k, hidden, inner, dt="bf16", scales="pow2", **route):
    c = _route(name, tokens, experts, k, **route)
    c.update(op="experts", hidden=hidden, inner=inner, x_dt=dt, scales=scales)
    return c


def listed():
    # sizes: the decoder block of the benchmark (hidden size 4096, MLPs of 11008 and 14336) where nothing else is said
    return [
        # one user's next token through the output projection: the smallest product, all latency
        _linear("linear-1x4096", 1, 4096, 4096),
        # a decode step of two dozen users through a down projection whose block scales came with a checkpoint
        _linear("linear-24-down", 24, 11008, 4096, dt="f16", scales="f32"),
        # a few hundred tokens on a small layer of odd sizes: the last group and the last block are partial
        _linear("linear-601-ragged", 601, 1360, 1003, dt="f16", scales="f32", bias=True),
        # the benchmark's prefill product
        _linear("linear-4096-up", 4096, 4096, 11008),
        # the block's down projection over a long prompt, scales of a checkpoint
        _linear("linear-8192-down", 8192, 14336, 4096, scales="f32"),
        # one token's experts
        _route("route-1", 1, 32, 4),
        # prompts through a router with a bias for balance and limited groups, 16-bit logits
        _route("route-4097-groups", 4097, 160, 6, score="sigmoid", dt="bf16", bias=True, groups=8, top_groups=3,
               group_score=2, scale=2.5),
        # a large batch of tokens, probabilities kept as they are
        _route("route-16384", 16384, 64, 8, renormalize=False),
        # one user's next token through 4 of 32 experts
        _experts("experts-1", 1, 32, 4, 4096, 2048),
        # a decode step of 48 users, scales of a checkpoint: nearly every expert is read, for a few rows each
        _experts("experts-48", 48, 32, 4, 4096, 2048, dt="f16", scales="f32"),
        # a prompt: some hundred rows an expert, unevenly, an inner size that ends inside a block
        _experts("experts-1531", 1531, 32, 4, 4096, 1360, score="sigmoid", bias=True, scale=1.5),
        # a long prompt through the block's MLP taken eight times, two experts a token
        _experts("experts-8192", 8192, 8, 2, 4096, 14336),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_route(rng, most):
    e = _log(rng, 4, 320)
    groups = rng.choice((1, 1, 4, 8))
    e = max(e // groups, 2) * groups
    top_groups = rng.randint(1, groups)
    return dict(tokens=_log(rng, 1, most), experts=e, k=min(rng.choice((1, 2, 4, 6, 8)), e // groups * top_groups),
                score=rng.choice(("softmax", "sigmoid")), dt=rng.choice(("f32", "bf16", "f16")), bias=rng.random() < 0.5,
                groups=groups, top_groups=top_groups, group_score=rng.choice((1, 2)), renormalize=rng.random() < 0.7,
                scale=rng.choice((1.0, 2.5)))


def draw(rng):
    kind = rng.choice(("linear", "linear", "linear", "route", "experts", "experts"))
    scales = rng.choice(("pow2", "f32"))
    if kind == "linear":
        m, n, k = _log(rng, 1, 8192), _log(rng, 40, 28672), 16 * _log(rng, 6, 896)
        while m * n * k > 8192 * 4096 * 14336:
            m = (m + 1) // 2
        return dict(op="linear", m=m, k=k, n=n, dt=rng.choice(("bf16", "bf16", "f16", "f32")), scales=scales,
                    bias=rng.random() < 0.3)
    if kind == "route":
        return dict(_draw_route(rng, 16384), op="route")
    c = dict(_draw_route(rng, 8192), op="experts", hidden=16 * _log(rng, 16, 320), inner=16 * _log(rng, 10, 256),
             x_dt=rng.choice(("bf16", "f16")), scales=scales)
    while c["experts"] * c["hidden"] * c["inner"] > 8 * 4096 * 14336:  # all the experts' weights
        c["inner"] = (c["inner"] // 32 + 1) * 16
    while c["tokens"] * c["k"] * c["hidden"] * c["inner"] > 16384 * 4096 * 14336 // 4:
        c["tokens"] = (c["tokens"] + 1) // 2
    return c


def _blocks(n):
    return (n + 127) // 128


def work(case):
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        scales = _blocks(n) * _blocks(k) * (1 if case["scales"] == "pow2" else 4)
        return {"bytes": m * k * (4 if case["dt"] == "f32" else 2) + n * k + scales + 2 * m * n + (4 * n if case["bias"] else 0),
                "flops": 2.0 * m * n * k}
    t, e, k = case["tokens"], case["experts"], case["k"]
    route = t * e * (4 if case["dt"] == "f32" else 2) + (4 * e if case["bias"] else 0) + t * k * 12 + 4 * (e + 1)
    if case["op"] == "route":
        return {"bytes": route, "flops": 4.0 * t * e}
    h, i = case["hidden"], case["inner"]
    read = e * (1 - (1 - k / e) ** t)  # the experts that some token chooses, were all chosen alike
    scales = 3 * _blocks(h) * _blocks(i) * (1 if case["scales"] == "pow2" else 4)
    return {"bytes": route + read * (3 * h * i + scales) + 4 * t * h, "flops": 6.0 * t * k * h * i + 4.0 * t * e}


def _pow2_scale(top):
    """The smallest power of two S with top <= 448 S; 1 for 0."""
    m, e = torch.frexp(top)  # top = m 2^e, 1/2 <= m < 1; 448 = 7/8 * 2^9
    return torch.where(top == 0, 1.0, torch.ldexp(torch.ones_like(top), e - 9 + (m > 0.875).to(e.dtype)))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def hidden(rows, width, dt):
        # activations as a block's norm leaves them: a few channels stand out
        x = torch.randn((rows, width), generator=g, device=dev)
        x *= torch.exp(0.5 * torch.randn((1, width), generator=g, device=dev))
        return x.to(_DT[dt])

    def weight(count, n, k):
        """Codes [count, n, k] e4m3 and block scales [count, n / 128, k / 128] of weights as layers have them."""
        codes, scale = [], []
        for _ in range(count):
            w = torch.randn((n, k), generator=g, device=dev)
            w *= torch.exp(0.3 * torch.randn((n, 1), generator=g, device=dev)) * k ** -0.5
            w = torch.nn.functional.pad(w, (0, -k % 128, 0, -n % 128)).view(_blocks(n), 128, _blocks(k), 128)
            top = w.abs().amax((1, 3))
            s = _pow2_scale(top) if case["scales"] == "pow2" else top / 448.0
            q = (w / s[:, None, :, None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(_blocks(n) * 128, _blocks(k) * 128)
            codes.append(q[:n, :k].contiguous())
            scale.append(s.to(torch.float8_e8m0fnu) if case["scales"] == "pow2" else s)
        return (torch.stack([c.view(torch.uint8) for c in codes]).view(torch.float8_e4m3fn),
                torch.stack([c.view(torch.uint8) if case["scales"] == "pow2" else c for c in scale]).view(scale[0].dtype))

    s = dict(case=case)
    if case["op"] == "linear":
        s["x"] = hidden(case["m"], case["k"], case["dt"])
        codes, scale = weight(1, case["n"], case["k"])
        s["codes"], s["scale"] = codes[0], scale[0]
        s["bias"] = torch.randn(case["n"], generator=g, device=dev) if case["bias"] else None
        return s
    t, e = case["tokens"], case["experts"]
    logits = 1.3 * torch.randn((t, e), generator=g, device=dev) + 0.5 * torch.randn(e, generator=g, device=dev)
    s["logits"] = logits.to(_DT[case["dt"]])
    s["choice_bias"] = 0.1 * torch.randn(e, generator=g, device=dev) if case["bias"] else None
    if case["op"] == "experts":
        s["x"] = hidden(t, case["hidden"], case["x_dt"])
        # gate and up, one behind the other, for each expert
        codes, scale = weight(2 * e, case["inner"], case["hidden"])
        s["gate_up"], s["gate_up_scale"] = codes.unflatten(0, (e, 2)), scale.unflatten(0, (e, 2))
        s["down"], s["down_scale"] = weight(e, case["hidden"], case["inner"])
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s)
    if op == "linear":
        return {"y": _plain_linear(s)}
    r = _plain_route(s)
    return r if op == "route" else {"y": _plain_experts(s, r["ids"], r["weights"])}


def _run_own(s):
    from w8a8_int8_quantized_absmax_amd import pdq

    case = s["case"]
    if case["op"] == "linear":
        if "w" not in s:  # laid out once, as a serving program does when it loads the layer
            s["w"] = pdq.pack_weight_fp8(s["codes"], s["scale"])
        return {"y": pdq.linear_fp8(s["x"], s["w"], bias=s["bias"])["y"]}
    r = pdq.route_experts(s["logits"], case["k"], score=case["score"], bias=s["choice_bias"], groups=case["groups"],
                          top_groups=case["top_groups"], group_score=case["group_score"],
                          renormalize=case["renormalize"], scale=case["scale"])
    if case["op"] == "route":
        return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "rows": r.rows}
    if "w" not in s:
        s["w"] = (pdq.pack_weight_fp8(s["gate_up"], s["gate_up_scale"]), pdq.pack_weight_fp8(s["down"], s["down_scale"]))
    return {"y": pdq.experts_fp8(s["x"], r, *s["w"])["y"]}


# ---- the plain forms ----------------------------------------------------------------------------------------------

def _coded(x):
    """The values that the codes of x [..., k] (float32) and their groups' scales stand for."""
    k = x.shape[-1]
    v = torch.nn.functional.pad(x, (0, -k % 128)).unflatten(-1, (-1, 128))
    s = _pow2_scale(v.abs().amax(-1, keepdim=True))
    return ((v / s).to(torch.float8_e4m3fn).float() * s).flatten(-2)[..., :k]


def _values(codes, scale):
    """The weights [..., n, k] that codes and block scales stand for, float32."""
    n, k = codes.shape[-2:]
    return codes.float() * scale.float().repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]


def _plain_linear(s):
    y = _coded(s["x"].float()) @ _values(s["codes"], s["scale"]).T
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(torch.float16 if s["x"].dtype == torch.float16 else torch.bfloat16)


def _plain_route(s):
    """Scores and the choice in 64 bits, for what is next to a border."""
    case = s["case"]
    tokens, experts, k, groups = case["tokens"], case["experts"], case["k"], case["groups"]
    x = s["logits"].double()
    if case["score"] == "softmax":
        p = torch.exp(x - x.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    c = x if s["choice_bias"] is None else p + s["choice_bias"].double()  # without a bias the logits rank alike
    if groups > 1:
        each = (p if s["choice_bias"] is None else c).unflatten(1, (groups, -1))
        best = each.sort(-1, descending=True).values[..., :case["group_score"]].sum(-1)
        rank = best.sort(dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, rank, True)
        c = c.masked_fill(~kept.repeat_interleave(experts // groups, 1), -math.inf)
    ids = c.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if case["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    flat = ids.flatten()
    counts = torch.zeros(experts, dtype=torch.int64, device=x.device).index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0))
    rows = flat.sort(stable=True).indices
    return {"ids": ids.to(torch.int32), "weights": (w * case["scale"]).float(), "offsets": offsets.to(torch.int32),
            "rows": rows.to(torch.int32)}


def _plain_experts(s, ids, weights):
    """The experts that some token chose, side by side, each with its rows and zeros up to the longest."""
    tokens, k = ids.shape
    flat = ids.flatten().long()
    chosen, at = torch.unique(flat, return_inverse=True)
    order = at.sort(stable=True).indices
    count = torch.zeros_like(chosen).index_add_(0, at, torch.ones_like(at))
    slot = torch.empty_like(at)
    slot[order] = torch.arange(tokens * k, device=at.device) - (count.cumsum(0) - count)[at[order]]
    x = _coded(s["x"].float())
    held = x.new_zeros((chosen.shape[0], int(count.max()), x.shape[1]))
    held[at, slot] = x[torch.arange(tokens * k, device=at.device) // k]

    def values(codes, scale):
        return _values(codes.view(torch.uint8)[chosen].view(codes.dtype),
                       scale.view(torch.uint8)[chosen].view(scale.dtype) if scale.element_size() == 1 else scale[chosen])

    w = values(s["gate_up"], s["gate_up_scale"])
    gate, up = held @ w[:, 0].transpose(1, 2), held @ w[:, 1].transpose(1, 2)
    h = _coded(gate / (1 + torch.exp(-gate)) * up)
    y = h @ values(s["down"], s["down_scale"]).transpose(1, 2)
    y = (y[at, slot].unflatten(0, (tokens, k)) * weights[..., None]).sum(1)
    return y.to(s["x"].dtype)


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)

    def coded(x):
        """x [rows, k] float64: each group of 128 rounded to e4m3 times its power of two."""
        out = torch.zeros_like(x)
        for a in range(0, x.shape[1], 128):
            v = x[:, a:a + 128]
            top = v.abs().amax(1, keepdim=True)
            unit = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top.clamp_min(1e-300) / 448))), 1.0)
            q = v / unit
            step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)  # 3 bits behind the point, 2^-9 at least
            out[:, a:a + 128] = torch.round(q / step) * step * unit
        return out

    def product(x, codes, scale):
        n, k = codes.shape
        w = codes.double() * torch.kron(scale.double(), torch.ones((128, 128), dtype=torch.float64, device=x.device))[:n, :k]
        return x @ w.T.contiguous()

    if case["op"] == "linear":
        y = product(coded(s["x"].double()), s["codes"], s["scale"])
        return {"y": y if s["bias"] is None else y + s["bias"].double()}
    z = s["logits"].double()
    p = torch.softmax(z, 1) if case["score"] == "softmax" else torch.sigmoid(z)
    c = p.clone() if s["choice_bias"] is None else p + s["choice_bias"].double()
    size = case["experts"] // case["groups"]
    if case["groups"] > 1:
        best = torch.stack([c[:, a:a + size].topk(min(case["group_score"], size), 1).values.sum(1)
                            for a in range(0, case["experts"], size)], 1)
        for _ in range(case["groups"] - case["top_groups"]):  # the worst group goes; the last one of equals
            worst = case["groups"] - 1 - best.flip(1).argmin(1)
            best.scatter_(1, worst[:, None], math.inf)
            c[torch.arange(case["experts"], device=c.device)[None] // size == worst[:, None]] = -math.inf
    ids = []
    for _ in range(case["k"]):
        ids.append((c == c.amax(1, keepdim=True)).to(torch.uint8).argmax(1))  # the first one of equals
        c.scatter_(1, ids[-1][:, None], -math.inf)
    ids = torch.stack(ids, 1)
    w = p.gather(1, ids)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    w = w * case["scale"]
    if case["op"] == "route":
        return {"ids": None, "weights": w, "offsets": None, "rows": None}
    x = coded(s["x"].double())
    y = torch.zeros_like(x)
    for e in range(case["experts"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            gate, up = (product(x[t], s["gate_up"][e, i], s["gate_up_scale"][e, i]) for i in range(2))
            h = coded(gate * torch.sigmoid(gate) * up)
            y[t] += w[t, j, None] * product(h, s["down"][e], s["down_scale"][e])
    return {"y": y}

"""FP8 linear layers, routing and the experts' layer used together and in every way that a server calls them (MI355X):
one after the other, captured and replayed, several at once, on other streams, at sizes of every kernel variant."""
import numpy as np
import pytest
import torch

import oracle.fp8_oracle as FO
import test_gpu_route
from fp8_cases import DT, check_linear, randn, values, weight
from guards import gapped
from test_gpu_experts import check, layer
from w8a8_int8_quantized_absmax_amd import pdq

pytestmark = pytest.mark.gpu


class Block:
    """A mixture-of-experts block: router, experts, and a linear layer behind them."""

    def __init__(self, seed, hidden, inner, experts, k, scales, dt, rule):
        self.router = weight(seed, (), experts, hidden, scales)
        self.gate_up, self.down = layer(seed + 1, experts, hidden, inner, scales)
        self.out = weight(seed + 3, (), hidden, hidden, scales)
        self.bias = (0.1 * randn(seed + 4, hidden)).cuda()
        self.k, self.rule, self.dt = k, rule, DT[dt]

    def __call__(self, x):
        logits = pdq.linear_fp8(x, self.router[0])["y"]
        r = pdq.route_experts(logits, self.k, **self.rule)
        h = pdq.experts_fp8(x, r, self.gate_up[0], self.down[0])["y"]
        return logits, r, h, pdq.linear_fp8(h, self.out[0], self.bias)["y"]

    def tensors(self, x):
        logits, r, h, y = self(x)
        return [logits, r.ids, r.weights, r.offsets, r.rows, h, y]


RULES = [dict(), dict(score="sigmoid", groups=2, top_groups=1, group_score=2, scale=2.5)]


@pytest.mark.parametrize("dt,scales", [("bf16", "pow2"), ("f16", "f32")])
@pytest.mark.parametrize("tokens,rule", [(1, 0), (3, 1), (33, 0), (150, 1)])
def test_block(tokens, rule, dt, scales):
    hidden, inner, experts = 272, 144, 6
    b = Block(tokens, hidden, inner, experts, 2, scales, dt, RULES[rule])
    x = randn(tokens + 9, tokens, hidden).to(b.dt)
    logits, r, h, y = b(x.cuda())
    check_linear(logits, *FO.linear(values(x), *b.router[1:]), hidden)
    test_gpu_route.check(r, logits, 2, **RULES[rule])
    check(h, x, r, b.gate_up, b.down)
    check_linear(y, *FO.linear(values(h), *b.out[1:], values(b.bias)), hidden)
    # the INT8 layer behind it takes what the block leaves
    wq, ws, _ = pdq.quantize_weight(randn(5, 64, hidden).bfloat16().cuda())
    assert torch.isfinite(pdq.linear_prefill(y, wq, ws)["y"]).all()


@pytest.mark.parametrize("tokens", [1, 2, 40, 300])
def test_block_in_a_graph(tokens):
    """Two captured graphs of one block, each with workspaces of its own, replayed in turn on changing inputs."""
    b = Block(40, 272, 144, 6, 2, "pow2", "bf16", RULES[0])
    static = [torch.empty((tokens, 272), dtype=b.dt, device="cuda") for _ in range(2)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for x in static:
            b(x.zero_())
    torch.cuda.current_stream().wait_stream(stream)
    graphs, outs = [], []
    for x in static:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.tensors(x))
        graphs.append(g)
    for i in range(4):
        xs = [randn(50 + 2 * i + j, tokens, 272).to(b.dt).cuda() for j in range(2)]
        for x, s, g in zip(xs, static, graphs):
            s.copy_(x)
            g.replay()
        refs = [b.tensors(x) for x in xs]
        torch.cuda.synchronize()
        for out, ref in zip(outs, refs):
            for got, want in zip(out, ref):
                assert torch.equal(got, want), i


def test_blocks_on_streams_at_once():
    """Blocks of different sizes on streams of their own, interleaved: what each gives alone, bit for bit."""
    blocks = [Block(60, 272, 144, 6, 2, "pow2", "bf16", RULES[0]), Block(70, 400, 528, 10, 3, "f32", "f16", RULES[1])]
    xs = [randn(i, t, b.down[0].n).to(b.dt).cuda() for i, (b, t) in enumerate([(blocks[0], 1), (blocks[1], 30), (blocks[0], 500),
                                                                              (blocks[1], 70)])]
    pairs = [(blocks[i % 2], x) for i, x in enumerate(xs)]
    refs = [b.tensors(x) for b, x in pairs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pairs]
    got = [[] for _ in pairs]
    for _ in range(3):
        for i, (s, (b, x)) in enumerate(zip(streams, pairs)):
            with torch.cuda.stream(s):
                got[i].append(b.tensors(x))
    torch.cuda.synchronize()
    for ref, runs in zip(refs, got):
        for run in runs:
            assert all(torch.equal(a, c) for a, c in zip(run, ref))


# ---- sizes of every variant of the experts' layer ----

def skewed(seed, tokens, experts, favour):
    """Logits that send most tokens to a few experts and none to the last."""
    z = randn(seed, tokens, experts, spread=0.0)
    z[:, :favour] += 2.0
    if experts > 8:
        z[:, -1] = -float("inf")
    return z


def run_experts(seed, tokens, experts, k, hidden, inner, scales, dt, z):
    gate_up, down = layer(seed, experts, hidden, inner, scales)
    wide = randn(seed + 5, tokens, hidden + 16).to(DT[dt]).cuda()
    x = wide[:, 16:]  # a row pitch of its own
    r = pdq.route_experts(z.cuda(), k)
    y, untouched = gapped(tokens, hidden, DT[dt])
    pdq.experts_fp8(x, r, gate_up[0], down[0], out=y)
    untouched()
    check(y, x, r, gate_up, down)
    return x, r, gate_up, down, y


# (average rows of an expert: 256 or 192 rows a tile from 200, 128 from 48, 64 from 12, blocks of 16 below)
@pytest.mark.parametrize("scales", ["pow2", "f32"])
@pytest.mark.parametrize("tokens,experts,k,hidden,inner", [
    (310, 3, 2, 144, 272), (265, 1, 1, 272, 128), (601, 2, 1, 128, 144), (100, 8, 4, 144, 160), (60, 10, 4, 272, 144),
    (90, 130, 4, 64, 48), (33, 512, 8, 32, 16), (9, 70, 1, 400, 16)])
def test_experts_uneven(tokens, experts, k, hidden, inner, scales):
    run_experts(tokens, tokens, experts, k, hidden, inner, scales, "bf16", skewed(tokens, tokens, experts, max(1, experts // 3)))


@pytest.mark.parametrize("scales", ["pow2", "f32"])
@pytest.mark.parametrize("tokens", [8, 12, 60, 150, 240])
def test_experts_of_binary16_rows_are_fine(tokens, scales):
    """With binary16 rows gate and up are sums in binary32: some hundred additions of 1024 products, each off by 2^-25
    of a part of the sum by chance, less than 2^-21 of it; h of both then passes a border between two codes (2^-3
    to 2^-4 of h apart) for 2 * 2^-21 / 2^-3.5 = 2^-16.5 of the values, an error of 2^-3.5 each: 2^-8.2 2^-3.5 < 2^-11.5 of
    y's size, in quadrature with y's rounding (2^-11 / sqrt(3) at most) less than 2^-11; and the down product's
    alignment, 2^-12 (fp8_cases.check_linear)."""
    x, r, gate_up, down, y = run_experts(tokens, tokens, 3, 2, 1024, 272, scales, "f16", randn(tokens, tokens, 3, spread=0.0))
    y64, _ = FO.experts(values(x), r.ids.cpu().numpy(), values(r.weights), *gate_up[1:], *down[1:])
    assert np.linalg.norm(values(y) - y64) <= (2.0 ** -11 + 2.0 ** -12) * np.linalg.norm(y64)


# a few rows: up to 8, of which a workgroup codes 32768 values at most
@pytest.mark.parametrize("scales", ["pow2", "f32"])
@pytest.mark.parametrize("tokens,experts,k,hidden,inner", [
    (1, 8, 8, 16, 4096), (1, 8, 8, 16, 4112), (1, 1, 1, 32768, 16), (1, 1, 1, 32784, 16), (8, 3, 1, 144, 80), (9, 3, 1, 144, 80),
    (4, 2, 2, 656, 1040), (1, 512, 7, 48, 32)])
def test_experts_few_rows(tokens, experts, k, hidden, inner, scales):
    run_experts(tokens + k, tokens, experts, k, hidden, inner, scales, "f16", randn(tokens, tokens, experts, spread=0.0))


@pytest.mark.parametrize("tokens", [2, 20, 150])
def test_experts_slots_without_one(tokens):
    """Rows that see fewer experts than slots, or none; their weights sum to 1, or y is 0."""
    experts, k = 4, 3
    z = randn(tokens, tokens, experts, spread=0.0)
    z[0] = -float("inf")
    z[1:, 1:3] = -float("inf")
    z[1::2, 0] = float("-inf")
    _, r, _, _, y = run_experts(tokens, tokens, experts, k, 144, 272, "pow2", "bf16", z)
    assert (r.ids[0] == -1).all() and (y[0] == 0).all() and (r.ids[1] == torch.tensor([3, -1, -1], device="cuda")).all()


@pytest.mark.parametrize("tokens,experts", [(20, 4), (100, 4), (300, 2), (40, 130)])
def test_rows_and_offsets_of_any_content(tokens, experts):
    """Routings that no call leaves: nothing outside the outputs is touched, other tokens keep their values, and offsets
    that descend leave y without meaning (the next call is as ever)."""
    x, r, gate_up, down, y = run_experts(tokens, tokens, experts, 2, 144, 272, "pow2", "bf16",
                                         randn(tokens, tokens, experts, spread=0.0))
    rows = r.rows.clone()
    hit = rows[[3, 7]]
    rows[3], rows[7] = -5, 1 << 30
    out, untouched = gapped(tokens, 144)
    ws = torch.empty(pdq.experts_fp8_workspace_bytes(tokens, 2, experts, 144, 272) + 65536, dtype=torch.uint8, device="cuda")
    ws[-65536:] = 0x5A

    def call(routing):
        pdq.experts_fp8(x, routing, gate_up[0], down[0], out=out, workspace=ws[:-65536])
        untouched()
        assert (ws[-65536:] == 0x5A).all()

    call(pdq.Routing(r.ids, r.weights, r.offsets, rows))
    others = torch.ones(tokens, dtype=torch.bool, device="cuda")
    others[(hit // 2).long()] = False
    assert torch.equal(out[others], y[others])
    n = 2 * tokens
    for content in ([0, n], [n, 0], [0, n, 3], [-(1 << 31), (1 << 31) - 1]):
        offsets = torch.tensor((content * experts)[:experts + 1], dtype=torch.int32, device="cuda")
        call(pdq.Routing(r.ids, r.weights, offsets, r.rows))
    call(r)
    assert torch.equal(out, y)


# ---- every tile of the product, outputs in whole and in single stores ----

@pytest.mark.parametrize("gap", [24, 8, 5])
@pytest.mark.parametrize("m,n,k,scales,dt", [
    (1900, 4088, 400, "pow2", "f16"),   # 128 x 256
    (1100, 2056, 528, "pow2", "bf16"), (1100, 2056, 528, "f32", "f16"),   # 128 x 128
    (2000, 8184, 272, "pow2", "bf16"), (1500, 8184, 272, "f32", "bf16")])   # 256 x 256, 192 x 256
def test_linear_tiles(m, n, k, scales, dt, gap):
    w, wq, ws = weight(n, (), n, k, scales)
    x = randn(m, m, k).to(DT[dt])
    bias = 0.1 * randn(n + 1, n)
    assert pdq.gemm_fp8_tile(m, n, k, w.scale_type) > 0
    y, untouched = gapped(m, n, DT[dt], gap=gap)
    pdq.linear_fp8(x.cuda(), w, bias.cuda(), out=y)
    untouched()
    rows = np.unique(np.concatenate([np.arange(0, m, max(1, m // 9)), np.arange(max(0, m - 20), m)]))
    check_linear(y[torch.from_numpy(rows).cuda()], *FO.linear(values(x[rows]), wq, ws, values(bias)), k)
    assert torch.equal(pdq.linear_fp8(x.cuda(), w, bias.cuda())["y"], y)


# ---- seeded random sizes ----

@pytest.mark.parametrize("seed", range(24))
def test_linear_random(seed):
    g = np.random.default_rng(9000 + seed)
    m = int(g.integers(1, [20, 140, 700][seed % 3]))
    n, k = int(g.integers(1, 700)), 16 * int(g.integers(1, 60))
    dt, scales = str(g.choice(["f32", "bf16", "f16"])), str(g.choice(["pow2", "f32"]))
    w = weight(seed, (), n, k, scales)
    x = randn(seed + 1, m, k).to(DT[dt])
    bias = 0.1 * randn(seed + 2, n) if g.random() < 0.5 else None
    y, untouched = gapped(m, n, torch.float16 if dt == "f16" else torch.bfloat16, gap=int(g.integers(1, 30)))
    pdq.linear_fp8(x.cuda(), w[0], None if bias is None else bias.cuda(), out=y)
    untouched()
    check_linear(y, *FO.linear(values(x), *w[1:], None if bias is None else values(bias)), k)


@pytest.mark.parametrize("seed", range(24))
def test_route_random(seed):
    g = np.random.default_rng(9100 + seed)
    groups = int(g.choice([1, 1, 2, 4, 8]))
    experts = groups * int(g.integers(1, 512 // groups + 1 if seed % 3 == 0 else 20))
    k, tokens = int(g.integers(1, min(experts, 32) + 1)), int(g.integers(1, [5, 70, 600][seed % 3]))
    z = torch.from_numpy(g.normal(size=(tokens, experts)).round(int(g.integers(1, 6)))).to(DT[str(g.choice(["f32", "bf16", "f16"]))])
    z[torch.from_numpy(g.random(z.shape) < g.choice([0.0, 0.3]))] = -float("inf")
    bias = torch.from_numpy(g.normal(size=experts)).float() if g.random() < 0.5 else None
    test_gpu_route.run(z, k, bias, score=str(g.choice(["softmax", "sigmoid"])), groups=groups,
                       top_groups=int(g.integers(1, groups + 1)), group_score=int(g.integers(1, 3)),
                       renormalize=bool(g.random() < 0.5), scale=float(g.choice([1.0, 2.5])))


@pytest.mark.parametrize("seed", range(16))
def test_experts_random(seed):
    g = np.random.default_rng(9200 + seed)
    experts = int(g.integers(1, 12))
    k, tokens = int(g.integers(1, min(experts, 4) + 1)), int(g.integers(1, [8, 60, 250][seed % 3]))
    z = randn(seed, tokens, experts) * float(g.choice([0.3, 3.0]))
    run_experts(seed, tokens, experts, k, 16 * int(g.integers(1, 26)), 16 * int(g.integers(1, 26)),
                str(g.choice(["pow2", "f32"])), str(g.choice(["bf16", "f16"])), z)


# ---- what the binding refuses ----

def test_refusals():
    w = pdq.quantize_weight_fp8(torch.zeros((16, 64), dtype=torch.bfloat16, device="cuda"))
    stack = pdq.quantize_weight_fp8(torch.zeros((4, 2, 32, 64), dtype=torch.bfloat16, device="cuda"))
    down = pdq.quantize_weight_fp8(torch.zeros((4, 64, 32), dtype=torch.bfloat16, device="cuda"))
    x = torch.zeros((3, 64), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros((3, 4), device="cuda")
    r = pdq.route_experts(z, 2)
    other = pdq.route_experts(z[:2], 2)
    f32 = pdq.pack_weight_fp8(torch.zeros((4, 64, 32), device="cuda").to(torch.float8_e4m3fn),
                              torch.ones((4, 1, 1), device="cuda"))
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    many = torch.zeros((400, 64), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: pdq.linear_fp8(x[:, :32], w), lambda: pdq.linear_fp8(x.double(), w), lambda: pdq.linear_fp8(x, stack),
                 lambda: pdq.linear_fp8(x.t(), w), lambda: pdq.linear_fp8(x[0], w), lambda: pdq.linear_fp8(x, w, x[0, :16]),
                 lambda: pdq.linear_fp8(x, w, dtype=torch.float32), lambda: pdq.linear_fp8(x, w, out=x),
                 lambda: pdq.linear_fp8(x, w, torch.zeros(16)), lambda: pdq.gemm_fp8(x, w),
                 lambda: pdq.linear_fp8(x, w, workspace=x),
                 lambda: pdq.quantize_weight_fp8(x.t()), lambda: pdq.quantize_weight_fp8(x.int()),
                 lambda: pdq.pack_weight_fp8(x.to(torch.float8_e4m3fn), torch.ones((1, 2), device="cuda")),
                 lambda: pdq.pack_weight_fp8(x.to(torch.float8_e4m3fn), torch.ones((1, 1), device="cuda").half()),
                 lambda: pdq.route_experts(z, 0), lambda: pdq.route_experts(z, 5), lambda: pdq.route_experts(z, 2, score="max"),
                 lambda: pdq.route_experts(z, 2, bias=z[0, :3]), lambda: pdq.route_experts(z[0], 2),
                 lambda: pdq.route_experts(z.t(), 2), lambda: pdq.route_experts(z.long(), 2),
                 lambda: pdq.experts_fp8(x.float(), r, stack, down), lambda: pdq.experts_fp8(x, other, stack, down),
                 lambda: pdq.experts_fp8(x, r, down, stack), lambda: pdq.experts_fp8(x, r, stack, f32),
                 lambda: pdq.experts_fp8(x, r, stack, down, out=x.half()), lambda: pdq.experts_fp8(x[:, ::2], r, stack, down)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: pdq.route_experts(z, 2, groups=3), lambda: pdq.route_experts(z, 2, groups=2, top_groups=3),
                 lambda: pdq.route_experts(z, 2, scale=float("inf")), lambda: pdq.route_experts(z, 2, group_score=3),
                 lambda: pdq.route_experts(z, 2, workspace=small), lambda: pdq.linear_fp8(many, w, workspace=small),
                 lambda: pdq.experts_fp8(x, r, stack, down, workspace=small)):
        with pytest.raises(pdq.PdqError):
            call()


def test_leading_rows_of_a_shared_buffer():
    """Views into larger buffers: the rows between and behind stay as they were, and x of any row pitch counts alike."""
    w = weight(3, (), 72, 144, "pow2")
    big = randn(4, 50, 3 * 144).bfloat16().cuda()
    for m in (1, 7, 50):
        for x in (big[:m, 144:288], big[::2][:m, :144]):
            assert torch.equal(pdq.linear_fp8(x, w[0])["y"], pdq.linear_fp8(x.contiguous(), w[0])["y"])

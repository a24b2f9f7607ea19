"""The key/value cache as a decoder block uses it: INT8 projection, append, attention, INT8 projection; captured and
replayed; on several streams; on dirty workspaces."""
import numpy as np
import pytest
import torch

import oracle.kv_oracle as KO
import oracle.pdq_oracle as O
from kv_cases import Batch, host_cache, tables
from w8a8_int8_quantized_absmax_amd import pdq, synth
from gpu_helpers import dev, host
from test_gpu_kv import _f32, check_attention, check_cache, run_append, run_attention

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE, HID = 4, 2, 64, 16, 256


class Block:
    """One attention half of a decoder block with INT8 weights, and the oracle's copy of its cache."""

    def __init__(self, pages):
        self.wqkv = pdq.quantize_weight(dev(synth.weights(9100, (HQ + 2 * HKV) * D, HID, "bf16"), "bf16"))
        self.wo = pdq.quantize_weight(dev(synth.weights(9101, HID, HQ * D, "bf16"), "bf16"))
        self.cache = pdq.KVCache.empty(pages, HKV, D, PAGE)
        for t in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale):
            t.zero_()
        self.ref = host_cache(self.cache)
        cos, sin = tables(400, D)
        self.tab = cos, sin
        self.dtab = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()

    def qkv(self, x, static=None):
        y = (pdq.linear_prefill(x, *self.wqkv[:2]) if static is None else
             pdq.linear_decode(x, *static, *self.wqkv))["y"].unflatten(1, (-1, D))
        return y[:, :HQ], y[:, HQ:HQ + HKV], y[:, HQ + HKV:]

    def run(self, x, batch, static=None):
        q, k, v = self.qkv(x, static)
        q = pdq.kv_append(k, v, self.cache, batch, q=q, cos=self.dtab[0], sin=self.dtab[1])
        a = pdq.kv_attention(q, self.cache, batch, want_lse=True)
        o = pdq.linear_prefill(a["y"].flatten(1), *self.wo[:2], want_acc=True)
        return q, k, v, a, o

    def check(self, out, table, seq_len, cu_q):
        q, k, v, a, o = out
        torch.cuda.synchronize()
        KO.append(self.ref, table, seq_len, cu_q, _f32(k.cpu()), _f32(v.cpu()), cos=self.tab[0], sin=self.tab[1])
        check_cache(host_cache(self.cache), self.ref)
        want = KO.attention(self.ref, table, seq_len, cu_q, _f32(q.cpu()), D ** -0.5)
        b = type("B", (), dict(table=table, page=PAGE, dim=D))
        check_attention(b, a["y"].cpu().double().numpy(), a["lse"].cpu().double().numpy(), *want, "bf16")
        wq, ws, _ = O.quantize_weight(synth.weights(9101, HID, HQ * D, "bf16"))
        r = O.linear_prefill(_f32(a["y"].flatten(1).cpu()), wq, ws)
        assert np.array_equal(host(o["acc"]), r["acc"])
        assert np.array_equal(host(o["y"]), O.to_bf16_bits(r["y32"]))


def test_prompts_then_decode_steps():
    # three prompts of differing lengths, then steps of one token each, the first and the last over a page's end
    block = Block(40)
    new = [45, 17, 80]
    table = np.random.default_rng(1).permutation(40)[:36].reshape(3, 12).astype(np.int32)
    cu = np.cumsum([0] + new).astype(np.int32)
    dt = torch.from_numpy(table).cuda()
    x = dev(synth.round_to(synth.normal(9110, (sum(new), HID)), "bf16"), "bf16")
    seq = torch.tensor(new, dtype=torch.int32, device="cuda")
    block.check(block.run(x, pdq.KVBatch(dt, seq, torch.from_numpy(cu).cuda())), table, new, cu)
    batch = pdq.KVBatch(dt, seq)  # the steps' batch: its lengths are updated in place
    state = pdq.minmax_state("cuda")
    s, z = pdq.calibrate_static(x, state, finalize=True)
    static = float(s.item()), int(z.item())
    for step in range(5):
        seq += 1
        x = dev(synth.round_to(synth.normal(9120 + step, (3, HID)), "bf16"), "bf16")
        block.check(block.run(x, batch, static), table, [n + step + 1 for n in new], None)


def test_chunks_of_whole_pages_give_the_cache_of_the_whole_prompt():
    a, b = Block(20), Block(20)
    table = torch.arange(20, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    x = dev(synth.round_to(synth.normal(9130, (150, HID)), "bf16"), "bf16")

    def lens(n, m):
        return pdq.KVBatch(table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                           torch.tensor([0, m], dtype=torch.int32, device="cuda"))

    whole = a.run(x, lens(150, 150))
    parts = [b.run(x[lo:hi], lens(hi, hi - lo)) for lo, hi in ((0, 48), (48, 64), (64, 150))]
    torch.cuda.synchronize()
    check_cache(host_cache(a.cache), host_cache(b.cache))
    y, z = torch.cat([p[3]["y"] for p in parts]).float(), whole[3]["y"].float()
    # The same keys for each row, in tiles of other rows: each side is off by its rounding (2^-9 |y|), by 2^-11 of what the
    # weights multiply (no value is larger than `most`) for theirs, and by less than that again for the rest.
    most = 127 * float(a.cache.v_scale.max())
    assert ((y - z).abs() <= 2 * (2.0 ** -9 * z.abs() + 2 * 2.0 ** -11 * most)).all()


@pytest.mark.parametrize("length", [[30, 200, 77], [3000, 5, 1500]])
def test_decode_steps_in_a_graph(length):
    # append and attention captured once; between the replays the lengths and the inputs change in place
    b = Batch(600 + length[0], [n + 40 for n in length], None, HKV, D, PAGE, single=True)
    cos, sin = (torch.from_numpy(t).cuda() for t in tables(max(length) + 50, D))
    seq = torch.tensor(length, dtype=torch.int32, device="cuda")
    batch = pdq.KVBatch(torch.from_numpy(b.table).cuda(), seq)
    cache, eager = b.device_cache(), b.device_cache()
    x = [torch.randn((3, HQ + 2 * HKV, D), generator=torch.Generator("cuda").manual_seed(i), device="cuda").bfloat16()
         for i in range(6)]
    static = x[0].clone()
    ws = torch.empty(pdq.kv_attention_workspace_bytes(3, 3, HQ, HKV, D), dtype=torch.uint8, device="cuda")

    def call(t, c, w=None):
        q = pdq.kv_append(t[:, HQ:HQ + HKV], t[:, HQ + HKV:], c, batch, q=t[:, :HQ], cos=cos, sin=sin)
        return pdq.kv_attention(q, c, batch, want_lse=True, workspace=w)

    warm = b.device_cache()
    call(static, warm, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call(static, cache, ws)
    for i in range(6):
        seq += 1 + 3 * (i == 2)
        static.copy_(x[i])
        g.replay()
        torch.cuda.synchronize()
        want = call(x[i], eager)
        torch.cuda.synchronize()
        assert torch.equal(got["y"].view(torch.int16), want["y"].view(torch.int16)), i
        assert torch.equal(got["lse"], want["lse"]), i
        check_cache(host_cache(cache), host_cache(eager))
    del g


def test_prompt_in_a_graph():
    b = Batch(610, [300, 90], [300, 40], 2, 128, 32)
    cache, bd = b.device_cache(), b.device_batch()
    q = b.rows(8, "f16").cuda()
    ws = torch.empty(max(1, pdq.kv_attention_workspace_bytes(b.tokens, 2, 8, 2, 128)), dtype=torch.uint8, device="cuda")
    pdq.kv_attention(q, cache, bd, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = pdq.kv_attention(q, cache, bd, want_lse=True, workspace=ws)
    for i in range(4):
        q.copy_(torch.randn(q.shape, generator=torch.Generator("cuda").manual_seed(i), device="cuda").half())
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        want = pdq.kv_attention(q, cache, bd, want_lse=True)
        assert torch.equal(got["y"], want["y"]) and torch.equal(got["lse"], want["lse"])
    del g


def _calls():
    few = Batch(620, [2000, 37, 900, 4100], None, 2, 128, 16, single=True)
    some = Batch(621, [700, 40], [5, 3], 2, 64, 32)
    prompt = Batch(622, [500, 130], [400, 130], 2, 128, 64)
    wide = Batch(623, [900], [64], 1, 256, 128)
    for b, hq in ((few, 8), (some, 8), (prompt, 4), (wide, 3)):
        q, c, bd = b.rows(hq, "bf16").cuda(), b.device_cache(), b.device_batch()
        size = pdq.kv_attention_workspace_bytes(b.tokens, len(b.seq_len), hq, b.hkv, b.dim)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
        yield lambda q=q, c=c, bd=bd, ws=ws: pdq.kv_attention(q, c, bd, want_lse=True, workspace=ws), ws


def test_four_calls_on_four_streams():
    calls = [f for f, _ in _calls()]
    alone = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        got = []
        for f, st in zip(calls, streams):
            with torch.cuda.stream(st):
                got.append(f())
        torch.cuda.synchronize()
        for a, g in zip(alone, got):
            assert torch.equal(a["y"].view(torch.int16), g["y"].view(torch.int16)) and torch.equal(a["lse"], g["lse"])


def test_workspace_contents_do_not_matter():
    for f, ws in _calls():
        first = f()
        for fill in (255, 0, 127):  # NaN, zero, large numbers as floats
            if ws is not None:
                ws.fill_(fill)
            again = f()
            assert torch.equal(first["y"].view(torch.int16), again["y"].view(torch.int16))
            assert torch.equal(first["lse"], again["lse"])


def test_wide_groups_and_one_row():
    # more query heads a key/value head than a few-row tile holds: one row a sequence in the prompt kernel
    b = Batch(630, [1, 64, 65, 300, 129], None, 1, 64, 32, single=True)
    run_attention(b, 40, "f16")
    run_attention(b, 150, "bf16", window=70)
    b = Batch(631, [300, 40], None, 2, 128, 64, single=True)
    run_attention(b, 2 * 33, "bf16", softcap=8.0)


def test_few_rows_of_many_tiles():
    # sequences with far more rows than the average that the kernel was chosen by
    new = [1] * 40 + [70]
    b = Batch(632, [20] * 40 + [200], new, 1, 64, 16)
    run_attention(b, 4, "bf16")
    b = Batch(633, [20] * 12 + [150], [1] * 12 + [90], 1, 256, 16)
    run_attention(b, 2, "f16", window=40)


def test_splits_of_a_prompt():
    # few tiles of rows over a long context: the keys are cut in many parts, some of which a row does not see
    b = Batch(634, [5000], [130], 1, 128, 64)
    run_attention(b, 1, "bf16")
    run_attention(b, 1, "f16", window=300)
    b = Batch(635, [2500, 60], [70, 60], 1, 64, 64)
    run_attention(b, 2, "f16", slopes=np.array([0.5, 0.01], np.float32))


def test_empty_batches():
    c = Batch(636, [5], None, 2, 64, 16, single=True).device_cache()
    t = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    none = pdq.KVBatch(t, torch.zeros(0, dtype=torch.int32, device="cuda"))
    x = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert pdq.kv_append(x, x, c, none) is None
    assert pdq.kv_attention(x, c, none)["y"].shape == (0, 2, 64)
    # sequences without new rows, and rows of no sequence
    b = Batch(637, [5, 9], [0, 0], 2, 64, 16, tail=3)
    run_append(b, "bf16", hq=2, rot=64, positions=16)
    run_attention(b, 4, "bf16")


def test_no_pool():
    # a pool without pages: nothing is written, nothing is seen
    b = Batch(638, [5, 40], None, 2, 64, 16, single=True)
    z = torch.zeros
    c = pdq.KVCache(z((0, 2, 16, 64), dtype=torch.int8, device="cuda"), z((0, 2, 4, 64, 4), dtype=torch.int8, device="cuda"),
                    z((0, 2), device="cuda"), z((0, 2), device="cuda"))
    x = b.rows(2, "bf16").cuda()
    pdq.kv_append(x, x, c, b.device_batch())
    r = pdq.kv_attention(x, c, b.device_batch(), want_lse=True)
    assert not r["y"].any() and torch.isneginf(r["lse"]).all()
    b = Batch(639, [80, 40], [80, 40], 2, 64, 16)
    x = b.rows(2, "bf16").cuda()
    pdq.kv_append(x, x, c, b.device_batch())
    r = pdq.kv_attention(x, c, b.device_batch(), want_lse=True)
    assert not r["y"].any() and torch.isneginf(r["lse"]).all()


def test_queries_rotated_in_place():
    for single, rot, inter in ((True, 64, False), (False, 128, False), (False, 128, True)):
        length, new = [40, 7, 90], [33, 7, 1]
        b = Batch(640 + rot, length, None if single else new, 2, 128, 32, single=single, tail=0 if single else 2)
        cos, sin = (torch.from_numpy(t).cuda() for t in tables(90, rot))
        k, q = b.rows(2, "bf16").cuda(), b.rows(6, "bf16").cuda()
        bd = b.device_batch()
        kw = dict(cos=cos, sin=sin, interleaved=inter)
        apart = torch.clone(q)
        pdq.kv_append(k, k, b.device_cache(), bd, q=q, q_out=apart, **kw)
        same = pdq.kv_append(k, k, b.device_cache(), bd, q=q, q_out=q, **kw)
        assert same is q and torch.equal(q.view(torch.int16), apart.view(torch.int16))

"""Calls on the later rows of a larger buffer: cu_q[0] rows, more than a page or a tile of them, belong to no sequence.
Their outputs stay as they were and what the call does is what it does without them."""
import numpy as np
import pytest
import torch

import oracle.kv_oracle as KO
from kv_cases import Batch, host_cache, tables
from test_gpu_kv import SENTINEL, _f32, check_attention, check_cache, run_append, run_attention
from w8a8_int8_quantized_absmax_amd import pdq

pytestmark = pytest.mark.gpu


def _slopes(hq):
    return (2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)).astype(np.float32)


@pytest.mark.parametrize("page,lead", [(16, 16), (16, 75), (64, 200), (256, 513)])
@pytest.mark.parametrize("n", [1, 3, 65])
def test_append(page, lead, n):
    # fresh sequences and continued ones; pages of scale zero all around, in the table's memory before its first row too
    r = np.random.default_rng(lead + n)
    new = r.integers(0, 2 * page if n < 10 else 20, n).tolist()
    new[0] = page + 3
    length = [m + int(r.choice([0, 0, 5, page])) for m in new]
    b = Batch(800 + page + n, length, new, 2, 64, page, lead=lead, tail=2)
    b.cache["k_scale"][r.random(b.cache["k_scale"].shape) < 0.5] = 0
    b.cache["v_scale"][r.random(b.cache["v_scale"].shape) < 0.5] = 0
    run_append(b, "bf16", hq=4, rot=64)
    spare = np.setdiff1d(np.arange(b.cache["k"].shape[0]), b.table)
    b.cache["k_scale"][spare] = b.cache["v_scale"][spare] = 0
    x, c, ref = b.rows(2, "f16"), b.device_cache(), b.copy_cache()
    table = torch.full((n + 40, b.table.shape[1]), int(spare[0]), dtype=torch.int32, device="cuda")
    table[40:] = torch.from_numpy(b.table).cuda()
    bd = pdq.KVBatch(table[40:], torch.from_numpy(b.seq_len).cuda(), torch.from_numpy(b.cu_q).cuda())
    pdq.kv_append(x.cuda(), x.cuda(), c, bd)
    KO.append(ref, b.table, b.seq_len, b.cu_q, _f32(x), _f32(x))
    check_cache(host_cache(c), ref)


@pytest.mark.parametrize("group,lead", [(1, 16), (4, 4), (4, 70), (5, 33), (8, 100)])
@pytest.mark.parametrize("n", [1, 3, 65, 300])
def test_attention_few_rows(n, group, lead):
    # the rows before the first sequence raise the average that the kernel is chosen by: both kernels, by n
    r = np.random.default_rng(10 * lead + n)
    new = r.integers(0, 5, n).tolist()
    new[0] = 4
    length = [m + int(r.integers(0, 300 if n > 10 else 900)) for m in new]
    b = Batch(820 + lead + n, length, new, 2, 64, 16, lead=lead, tail=3)
    run_attention(b, 2 * group, "bf16", slopes=_slopes(2 * group))


@pytest.mark.parametrize("dim,group,lead", [(128, 4, 130), (128, 1, 600), (64, 4, 70), (256, 3, 90)])
@pytest.mark.parametrize("n", [1, 3, 65])
def test_attention_prompts(n, dim, group, lead):
    r = np.random.default_rng(20 * lead + n)
    new = [100] if n == 1 else [60, 0, 90] if n == 3 else r.integers(5, 2 * (80 // group), n).tolist()
    length = [m + int(r.integers(0, 60)) for m in new]
    b = Batch(840 + lead + n, length, new, 2, dim, 32, lead=lead, tail=3)
    run_attention(b, 2 * group, "f16", slopes=_slopes(2 * group))


@pytest.mark.parametrize("dim,group,lead", [(128, 4, 130), (64, 2, 150), (256, 4, 70)])
def test_attention_prompt_in_parts(dim, group, lead):
    # few tiles of rows over many keys: parts joined through the workspace, whatever it holds
    b = Batch(860 + dim, [2700], [80], 2, dim, 32, lead=lead, tail=2)
    hq = 2 * group
    size = pdq.kv_attention_workspace_bytes(b.tokens, 1, hq, 2, dim)
    assert size > 0
    run_attention(b, hq, "bf16", slopes=_slopes(hq))
    _dirty(b, hq, size)


def test_attention_few_rows_dirty_workspace():
    for b, hq in ((Batch(870, [900, 70, 0, 400], [3, 1, 0, 5], 2, 128, 16, lead=40, tail=2), 8),
                  (Batch(871, [30] * 90, [1] * 90, 1, 64, 16, lead=200), 4)):
        size = pdq.kv_attention_workspace_bytes(b.tokens, len(b.seq_len), hq, b.hkv, b.dim)
        assert size > 0
        run_attention(b, hq, "bf16")
        _dirty(b, hq, size)


def _dirty(b, hq, size):
    """The same bits, and rows of no sequence untouched, whatever the workspace holds."""
    q, c, bd = b.rows(hq, "bf16").cuda(), b.device_cache(), b.device_batch()
    ref = pdq.kv_attention(q, c, bd, want_lse=True)
    own = slice(int(b.cu_q[0]), int(b.cu_q[-1]))
    for fill in (0, 127, 255):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        y, lse = torch.full_like(q, SENTINEL), torch.full((b.tokens, hq), SENTINEL, device="cuda")
        pdq.kv_attention(q, c, bd, out=y, lse=lse, workspace=ws)
        assert torch.equal(y[own].view(torch.int16), ref["y"][own].view(torch.int16))
        assert torch.equal(lse[own], ref["lse"][own])
        for rest in (slice(0, own.start), slice(own.stop, None)):
            assert (y[rest] == SENTINEL).all() and (lse[rest] == SENTINEL).all()


@pytest.mark.parametrize("dim,hkv,group", [(128, 8, 4), (64, 16, 2)])
def test_attention_large_launch(dim, hkv, group):
    # more tiles than are put in order: the same bits as the call on the sequences' own rows
    new = [3300, 0, 5100, 2900] if dim == 128 else [4000, 9000, 3100]
    b = Batch(880 + dim, [0] * len(new), [0] * len(new), hkv, dim, 64)
    pages = [-(-n // 64) for n in new]
    c = Batch(881 + dim, [64 * sum(pages)], None, hkv, dim, 64, single=True).device_cache()
    table = torch.zeros((len(new), max(pages)), dtype=torch.int32)
    at = 0
    for s, p in enumerate(pages):
        table[s, :p] = torch.arange(at, at + p)
        at += p
    table, lens = table.cuda(), torch.tensor(new, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + new, dtype=torch.int32, device="cuda").cumsum(0).to(torch.int32)
    lead, rows = 700, sum(new)
    g = torch.Generator("cuda").manual_seed(dim)
    q = torch.randn((lead + rows, hkv * group, dim), generator=g, device="cuda").half()
    want = pdq.kv_attention(q[lead:], c, pdq.KVBatch(table, lens, cu), want_lse=True)
    y, lse = torch.full_like(q, SENTINEL), torch.full(q.shape[:2], SENTINEL, device="cuda")
    pdq.kv_attention(q, c, pdq.KVBatch(table, lens, cu + lead), out=y, lse=lse)
    assert torch.equal(y[lead:], want["y"]) and torch.equal(lse[lead:], want["lse"])
    assert (y[:lead] == SENTINEL).all() and (lse[:lead] == SENTINEL).all()


def test_decode_rows_and_a_chunk_in_one_buffer():
    # a serving step: 40 sequences' next tokens in the first rows, one prompt's chunk behind them, two calls on one buffer
    hq, hkv, d, page = 8, 2, 64, 16
    r = np.random.default_rng(9)
    b = Batch(890, r.integers(1, 200, 40).tolist(), None, hkv, d, page, single=True)
    chunk, n = Batch(891, [300], [150], hkv, d, page, lead=40), 40
    x = chunk.rows(hq + 2 * hkv, "bf16")
    dx, out = x.cuda(), torch.full((190, hq, d), SENTINEL, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((190, hq), SENTINEL, device="cuda")
    cos, sin = tables(310, d)
    dcos, dsin = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()
    qr = torch.zeros((190, hq, d), dtype=torch.bfloat16, device="cuda")
    for part, rows in ((chunk, slice(0, 190)), (b, slice(0, n))):  # the chunk first: its call leaves the other rows
        c, bd, ref = part.device_cache(), part.device_batch(), part.copy_cache()
        xp, ox, lx = dx[rows], out[rows], lse[rows]
        pdq.kv_append(xp[:, hq:hq + hkv], xp[:, hq + hkv:], c, bd, q=xp[:, :hq], cos=dcos, sin=dsin, q_out=qr[rows])
        before = out[:n].clone()
        pdq.kv_attention(qr[rows], c, bd, out=ox, lse=lx)
        if part is chunk:
            assert torch.equal(out[:n], before) and (lse[:n] == SENTINEL).all() and not qr[:n].any()
        xh = x[rows]
        KO.append(ref, part.table, part.seq_len, part.cu_q, _f32(xh[:, hq:hq + hkv]), _f32(xh[:, hq + hkv:]), cos=cos, sin=sin)
        check_cache(host_cache(c), ref)
        own = slice(n, None) if part is chunk else slice(0, n)
        want = KO.attention(ref, part.table, part.seq_len, part.cu_q, _f32(qr[rows].cpu()), d ** -0.5)
        check_attention(part, ox[own].cpu().double().numpy(), lx[own].cpu().double().numpy(), *(w[own] for w in want), "bf16")

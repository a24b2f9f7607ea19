"""The INT8 key/value cache on the GPU against the oracle: codes, scales and rotated queries bit for bit, attention
within the tolerance that its arithmetic gives (kv_cases.attention_tolerance)."""
import numpy as np
import pytest
import torch

import oracle.kv_oracle as KO
from kv_cases import DT, Batch, attention_tolerance, host_cache, tables
from w8a8_int8_quantized_absmax_amd import pdq

pytestmark = pytest.mark.gpu

SENTINEL = 77.0


def _f32(t):
    return t.float().numpy()


def check_cache(got, ref):
    for name in ("k_scale", "v_scale"):
        assert np.array_equal(got[name], ref[name], equal_nan=True), name
    for name in ("k", "v"):
        assert np.array_equal(got[name], ref[name]), name


def run_append(b, dtype, hq=0, rot=0, interleaved=False, fused=False, positions=None):
    """Append random rows with the library and with the oracle; everything must be equal."""
    if fused:  # the projection's output: q, k, v of a row side by side
        x = b.rows(hq + 2 * b.hkv, dtype)
        d = x.cuda()
        q, k, v = x[:, :hq], x[:, hq:hq + b.hkv], x[:, hq + b.hkv:]
        dq, dk, dv = d[:, :hq], d[:, hq:hq + b.hkv], d[:, hq + b.hkv:]
    else:
        k, v, q = b.rows(b.hkv, dtype), b.rows(b.hkv, dtype, 3.0), b.rows(hq, dtype) if hq else None
        dk, dv, dq = k.cuda(), v.cuda(), q.cuda() if hq else None
    kw, dkw = {}, {}
    q_ref = None
    if rot:
        n = positions or max(int(b.seq_len.max()), 1)
        cos, sin = tables(n, rot)
        kw = dict(cos=cos, sin=sin, interleaved=interleaved)
        dkw = dict(cos=torch.from_numpy(cos).cuda(), sin=torch.from_numpy(sin).cuda(), interleaved=interleaved)
        if hq:
            q_ref = np.full(q.shape, SENTINEL, np.float32)
            kw.update(q=_f32(q), q_out=q_ref)
            dkw.update(q=dq, q_out=torch.full(q.shape, SENTINEL, dtype=DT[dtype], device="cuda"))
    c, ref = b.device_cache(), b.copy_cache()
    got_q = pdq.kv_append(dk, dv, c, b.device_batch(), **dkw)
    torch.cuda.synchronize()
    KO.append(ref, b.table, b.seq_len, b.cu_q, _f32(k), _f32(v), **kw)
    check_cache(host_cache(c), ref)
    if q_ref is not None:
        want = torch.from_numpy(q_ref).to(DT[dtype])
        assert np.array_equal(_f32(got_q.cpu()), _f32(want), equal_nan=True)
    return c, ref


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("page,dim,hkv", [(16, 64, 3), (32, 128, 2), (64, 256, 1), (128, 128, 1), (256, 64, 2)])
def test_append_one_token_each(page, dim, hkv, dtype):
    length = [1, 2, 4, 5, page - 1, page, page + 1, 2 * page, 3 * page + 7]
    b = Batch(10 + page + dim, length, None, hkv, dim, page, single=True)
    run_append(b, dtype, hq=2 * hkv, rot=dim, interleaved=page == 32)
    b = Batch(11 + page + dim, length, None, hkv, dim, page, single=True)
    run_append(b, dtype)


@pytest.mark.parametrize("dtype,page,dim,rot,inter", [
    ("bf16", 16, 64, 64, False), ("f16", 64, 128, 64, True), ("bf16", 64, 128, 128, False), ("f16", 32, 256, 16, False),
    ("bf16", 128, 64, 32, True), ("f16", 256, 128, 0, False)])
def test_append_ragged(dtype, page, dim, rot, inter):
    new = [1, 0, page, 3, 2 * page + 5, 7, page - 1, 70]
    length = [1, 9, page, page + 2, 2 * page + 6, 7 + 3 * page - 2, 5 * page - 1, 75]
    b = Batch(20 + page, length, new, 2, dim, page, lead=3, tail=4)
    run_append(b, dtype, hq=6 if rot else 0, rot=rot, interleaved=inter, fused=rot == 128)


def test_append_many_sequences():
    # more sequences than one step of the search among 64 tells apart, empty ones among them
    r = np.random.default_rng(3)
    new = r.integers(0, 4, 300).tolist()
    length = [n + int(r.integers(0, 40)) for n in new]
    run_append(Batch(30, length, new, 1, 64, 16), "bf16", hq=1, rot=64)
    run_append(Batch(31, [1] * 4200, [1] * 4100 + [0] * 99 + [1], 1, 64, 16), "f16")


def test_append_scale_growth_and_its_absence():
    # the same tokens appended one by one, all at once, and in two calls: the scale is that of the largest value seen
    b = Batch(40, [23], [23], 2, 64, 32)
    x, y = b.rows(2, "bf16"), b.rows(2, "bf16")
    x[:, 0] *= torch.linspace(0.1, 5, 23)[:, None]  # head 0 grows, head 1 hardly
    y[0] *= 50
    c, ref = b.device_cache(), b.copy_cache()
    for n in range(1, 24):
        seq = torch.tensor([n], dtype=torch.int32)
        pdq.kv_append(x[n - 1:n].cuda(), y[n - 1:n].cuda(), c, pdq.KVBatch(torch.from_numpy(b.table).cuda(), seq.cuda()))
        KO.append(ref, b.table, [n], None, _f32(x[n - 1:n]), _f32(y[n - 1:n]))
    check_cache(host_cache(c), ref)
    d = b.device_cache()
    pdq.kv_append(x.cuda(), y.cuda(), d, b.device_batch())
    p = b.table[0, 0]
    assert np.array_equal(host_cache(d)["k_scale"][p], ref["k_scale"][p])
    assert np.array_equal(host_cache(d)["v_scale"][p], ref["v_scale"][p])


def test_append_extreme_values():
    b = Batch(50, [6, 6, 6, 6, 6], [6] * 5, 1, 64, 16)
    k, v = b.rows(1, "bf16"), b.rows(1, "bf16")
    k[0:6] = 0                  # nothing but zeros
    k[6:12] *= 1e-30            # below the smallest scale
    k[12:18] *= 1e30            # near the largest
    k[18, 0, 5] = float("nan")
    v[24, 0, 63] = float("-inf")
    c, ref = b.device_cache(), b.copy_cache()
    pdq.kv_append(k.cuda(), v.cuda(), c, b.device_batch())
    KO.append(ref, b.table, b.seq_len, b.cu_q, _f32(k), _f32(v))
    check_cache(host_cache(c), ref)
    p = b.table[:, 0]
    assert ref["k_scale"][p[0], 0] == 2.0 ** -64 and np.isnan(ref["k_scale"][p[3], 0]) and np.isnan(ref["v_scale"][p[4], 0])
    # a token behind the NaN: the page stays NaN
    nxt = pdq.KVBatch(torch.from_numpy(b.table).cuda(), torch.full((5,), 7, dtype=torch.int32, device="cuda"))
    x = b.rows(1, "bf16")[:5]
    pdq.kv_append(x.cuda(), x.cuda(), c, nxt)
    KO.append(ref, b.table, [7] * 5, None, _f32(x), _f32(x))
    check_cache(host_cache(c), ref)


def test_append_behind_scales_that_are_not_finite():
    b = Batch(55, [9, 9, 9, 9], [2] * 4, 1, 64, 16)
    for s, value in enumerate((np.inf, -np.inf, np.nan, 0.5)):
        b.cache["k_scale"][b.table[s, 0]] = b.cache["v_scale"][b.table[s, 0]] = value
    c, ref = b.device_cache(), b.copy_cache()
    x, y = b.rows(1, "bf16"), b.rows(1, "bf16")
    pdq.kv_append(x.cuda(), y.cuda(), c, b.device_batch())
    KO.append(ref, b.table, b.seq_len, b.cu_q, _f32(x), _f32(y))
    assert np.isnan(ref["k_scale"][b.table[:3, 0], 0]).all()
    check_cache(host_cache(c), ref)


def test_append_positions_outside_the_tables():
    run_append(Batch(60, [20, 40], [5, 9], 2, 64, 16), "bf16", hq=2, rot=32, positions=18)


def test_append_bad_pages_and_lengths():
    # pages outside the pool, lengths beyond the table, fewer tokens than rows: written where a page is, nowhere else
    b = Batch(70, [40, 33, 64, 5], [40, 2, 30, 9], 1, 64, 16, spare=0)
    b.table[0, 1] = -1
    b.table[1, 2] = 1 << 30
    b.seq_len[2] = 70   # rows up to position 69 of a table for 64
    run_append(b, "f16", hq=1, rot=64, positions=100)
    b = Batch(71, [5, 9, 0], None, 1, 64, 16, single=True, spare=0)
    b.seq_len[1] = (1 << 31) - 1
    c, ref = b.device_cache(), b.copy_cache()
    x = b.rows(1, "f16")
    pdq.kv_append(x.cuda(), x.cuda(), c, b.device_batch())
    KO.append(ref, b.table, b.seq_len, None, _f32(x), _f32(x))
    check_cache(host_cache(c), ref)


# ---- attention ----------------------------------------------------------------------------------------------------

def run_attention(b, hq, dtype, scale=None, strided=False, spread=1.7, **opt):
    q = b.rows(hq, dtype, spread)
    dq = q.cuda()
    if strided:
        wide = torch.zeros((b.tokens, hq + 2, b.dim), dtype=DT[dtype], device="cuda")
        wide[:, :hq] = dq
        dq = wide[:, :hq]
        out = torch.full((b.tokens, hq + 1, b.dim), SENTINEL, dtype=DT[dtype], device="cuda")[:, :hq]
    else:
        out = torch.full((b.tokens, hq, b.dim), SENTINEL, dtype=DT[dtype], device="cuda")
    lse = torch.full((b.tokens, hq), SENTINEL, device="cuda")
    slopes, prefix = opt.pop("slopes", None), opt.pop("prefix", None)
    res = pdq.kv_attention(dq, b.device_cache(), b.device_batch(), scale=scale, out=out, lse=lse,
                           alibi_slopes=None if slopes is None else torch.from_numpy(slopes).cuda(),
                           prefix_len=None if prefix is None else torch.from_numpy(prefix).cuda(), **opt)
    torch.cuda.synchronize()
    y, z = res["y"].cpu().double().numpy(), res["lse"].cpu().double().numpy()
    ref, ref_lse, mag, big = KO.attention(b.cache, b.table, b.seq_len, b.cu_q, _f32(q),
                                          b.dim ** -0.5 if scale is None else scale, slopes=slopes, prefix=prefix, **opt)
    check_attention(b, y, z, ref, ref_lse, mag, big, dtype)
    return res


def check_attention(b, y, z, ref, ref_lse, mag, big, dtype):
    none = np.isnan(ref_lse)
    assert (y[none] == SENTINEL).all() and (z[none] == SENTINEL).all()
    y, z, ref, ref_lse, mag, big = (x[~none] for x in (y, z, ref, ref_lse, mag, big))
    keys = b.table.shape[1] * b.page
    off = np.abs(y - ref)
    tol = attention_tolerance(ref, mag, big, keys, b.dim, dtype)
    assert np.isfinite(y).all()
    assert (off <= tol).all(), f"{(off / tol).max():.2f} times the tolerance"
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(z), empty) and (y[empty] == 0).all()
    d = ((b.dim + 8) * 2.0 ** -24 + 2.0 ** -22) * big + 2.0 ** -21 + keys * 2.0 ** -24
    z, ref_lse, d = z[~empty], ref_lse[~empty], d[~empty]
    assert (np.abs(z - ref_lse) <= d + 2.0 ** -23 * np.abs(ref_lse)).all()


OPTIONS = {
    "plain": {}, "cap": dict(softcap=5.0), "window": dict(window=33), "alibi": "slopes", "prefix": "prefix",
    "all": "all"}


def _options(name, b, hq):
    o = OPTIONS[name]
    slopes = (2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)).astype(np.float32)
    prefix = b.rng.integers(0, 60, len(b.seq_len)).astype(np.int32)
    if o == "slopes":
        return dict(slopes=slopes)
    if o == "prefix":
        prefix[0] = 2 ** 31 - 1
        return dict(prefix=prefix)
    if o == "all":
        return dict(softcap=9.0, window=50, slopes=slopes, prefix=prefix)
    return dict(o)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("option", list(OPTIONS))
@pytest.mark.parametrize("page,dim,hkv,group", [(16, 64, 3, 1), (32, 128, 2, 4), (64, 256, 1, 8), (128, 128, 1, 5), (256, 64, 1, 20)])
def test_attention_one_token_each(page, dim, hkv, group, option, dtype):
    length = [1, 2, 15, 16, 17, 31, 32, 33, 63, 65, 127, 128, 129, 300]
    b = Batch(100 + page + dim, length, None, hkv, dim, page, single=True)
    run_attention(b, hkv * group, dtype, **_options(option, b, hkv * group))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("option", list(OPTIONS))
@pytest.mark.parametrize("page,dim,hkv,group", [(16, 64, 2, 1), (32, 128, 1, 4), (64, 256, 1, 3), (128, 128, 2, 2)])
def test_attention_few_rows_each(page, dim, hkv, group, option, dtype):
    new = [1, 5, 0, 3, 4, 2, 7]
    length = [1, 5, 20, 40, 130, 259, 77]
    b = Batch(200 + page + dim, length, new, hkv, dim, page, lead=2, tail=3)
    run_attention(b, hkv * group, dtype, strided=True, **_options(option, b, hkv * group))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("option", list(OPTIONS))
@pytest.mark.parametrize("page,dim,hkv,group", [(16, 64, 2, 1), (32, 128, 1, 4), (64, 256, 1, 2), (128, 128, 1, 3)])
def test_attention_prompts(page, dim, hkv, group, option, dtype):
    new = [129, 1, 0, 260, 64, 33]
    length = [129, 1, 8, 260, 200, 95]
    b = Batch(300 + page + dim, length, new, hkv, dim, page, lead=1, tail=5)
    run_attention(b, hkv * group, dtype, **_options(option, b, hkv * group))


@pytest.mark.parametrize("dim,page", [(128, 64), (64, 16), (256, 128)])
def test_attention_long_context(dim, page):
    # one row, and a chunk of rows, behind a context that is split over the axis
    b = Batch(400 + dim, [9001], None, 1, dim, page, single=True)
    run_attention(b, 4, "bf16")
    run_attention(b, 4, "f16", window=5000)
    b = Batch(410 + dim, [4003], [67], 1, dim, page)
    run_attention(b, 3, "f16")


def test_attention_many_sequences():
    r = np.random.default_rng(5)
    length = r.integers(1, 90, 700).tolist()
    run_attention(Batch(420, length, None, 1, 64, 16, single=True), 2, "bf16")
    new = [min(int(n), l) for n, l in zip(r.integers(0, 3, 700), length)]
    run_attention(Batch(421, length, new, 1, 64, 16), 2, "bf16")


@pytest.mark.parametrize("n,hkv,dim", [(2, 1, 64), (9, 3, 64), (63, 2, 128), (64, 1, 64), (64, 7, 128), (65, 1, 64), (5, 2, 256)])
def test_attention_many_prompts(n, hkv, dim):
    # uneven prompts, some without rows, several of one length, rows before and behind them: every row once
    r = np.random.default_rng(430 + n)
    new = (r.choice([0, 1, 31, 32, 33, 97, 300], n) if n > 5 else r.integers(100, 400, n)).tolist()
    new[-1] = 290
    length = [int(m + k) for m, k in zip(new, r.choice([0, 0, 5, 130], n))]
    run_attention(Batch(431 + n, length, new, hkv, dim, 32, lead=2, tail=3), 2 * hkv, "bf16")
    if n < 10:
        run_attention(Batch(432 + n, length[::-1], new[::-1], hkv, dim, 32), hkv, "f16", window=70)


def test_attention_wide_scores():
    # scores of a few hundred, all weight on a key or two: the running maximum moves, nothing overflows
    b = Batch(430, [200, 130, 64], None, 1, 128, 32, single=True)
    run_attention(b, 4, "f16", scale=3.0)
    b = Batch(431, [300], [300], 1, 64, 32)
    run_attention(b, 2, "bf16", scale=3.0)
    run_attention(b, 2, "bf16", scale=-1.0)
    run_attention(b, 2, "bf16", scale=0.0)


def test_attention_uneven_value_scales():
    # pages whose value scales differ by many powers of two, the smallest the cache's own for a page of zeros
    for new in (None, [90, 41]):
        b = Batch(440, [90, 41], new, 2, 64, 16, single=new is None)
        b.cache["v_scale"] *= (2.0 ** b.rng.integers(-30, 5, b.cache["v_scale"].shape)).astype(np.float32)
        zero = b.table[0, 1]
        b.cache["v_scale"][zero] = b.cache["k_scale"][zero] = 2.0 ** -64
        b.cache["v"][zero] = b.cache["k"][zero] = 0
        run_attention(b, 4, "bf16")
        run_attention(b, 4, "f16")


def test_attention_rows_that_see_nothing():
    # pages outside the pool, lengths of zero, fewer tokens than rows, a table without columns
    b = Batch(450, [40, 0, 20, 9], [2, 1, 3, 9], 1, 64, 16)
    b.table[0, :] = -1
    b.seq_len[3] = 4
    run_attention(b, 2, "bf16")
    b = Batch(451, [40, 0, 20], None, 1, 64, 16, single=True)
    b.table[2, 0] = 1 << 30
    run_attention(b, 2, "f16")
    b = Batch(452, [0, 0], None, 1, 64, 16, single=True, spare=0)
    assert b.table.shape[1] == 0
    run_attention(b, 2, "f16")
    b = Batch(453, [260, 90], [260, 70], 1, 64, 16)
    b.table[0, 2] = b.table[0, 5] = b.table[1, 0] = 999999
    run_attention(b, 2, "f16")
    run_attention(b, 2, "f16", window=20)


def test_attention_non_finite_pages_reach_only_their_rows():
    # a page of NaN scale: rows that see it are NaN, rows whose mask hides it are as without it
    for rows in (40, 200):
        b = Batch(460, [rows], [rows], 1, 64, 16)
        q = b.rows(2, "bf16").cuda()
        kw = dict(window=8)
        ref = pdq.kv_attention(q, b.device_cache(), b.device_batch(), **kw)["y"].float().cpu().numpy()
        for which in ("k_scale", "v_scale"):
            c = b.device_cache()
            getattr(c, which)[int(b.table[0, 1])] = float("nan")  # positions 16 .. 31
            got = pdq.kv_attention(q, c, b.device_batch(), **kw)["y"].float().cpu().numpy()
            p = np.arange(rows)
            hit = (p >= 16) & (p < 31 + 8)
            assert np.isnan(got[hit]).all()
            assert np.array_equal(got[~hit], ref[~hit])


def test_attention_far_pages():
    # a pool beyond 2^31 bytes: the pages at its end
    pages, heads, page, dim = 9000, 8, 128, 256
    k = torch.zeros((pages, heads, page, dim), dtype=torch.int8, device="cuda")
    assert k.numel() > 2 ** 31
    v = torch.zeros((pages, heads, page // 4, dim, 4), dtype=torch.int8, device="cuda")
    c = pdq.KVCache(k, v, torch.zeros((pages, heads), device="cuda"), torch.zeros((pages, heads), device="cuda"))
    b = Batch(470, [200, 130], [200, 4], heads, dim, page)
    b.table[:] = [[pages - 1, pages - 3, -1, -1], [3, pages - 2, -1, -1]]
    x, y, q = b.rows(heads, "bf16"), b.rows(heads, "bf16"), b.rows(heads, "bf16")
    bd = b.device_batch()
    pdq.kv_append(x.cuda(), y.cuda(), c, bd)
    small = [pages - 1, pages - 3, pages - 2, 3]
    got = dict(k=c.k[small].cpu().numpy(), v=KO.plain_v(c.v[small].cpu().numpy()),
               k_scale=c.k_scale[small].cpu().numpy(), v_scale=c.v_scale[small].cpu().numpy())
    table = np.array([[0, 1, -1, -1], [3, 2, -1, -1]], np.int32)
    ref = dict(k=np.zeros_like(got["k"]), v=np.zeros_like(got["v"]), k_scale=np.zeros((4, heads), np.float32),
               v_scale=np.zeros((4, heads), np.float32))
    KO.append(ref, table, b.seq_len, b.cu_q, _f32(x), _f32(y))
    check_cache(got, ref)
    c.k_scale[3] = c.v_scale[3] = 2.0 ** -64  # the page of zeros before the second sequence's tokens
    ref["k_scale"][3] = ref["v_scale"][3] = 2.0 ** -64
    r = pdq.kv_attention(q.cuda(), c, bd, want_lse=True)
    want = KO.attention(ref, table, b.seq_len, b.cu_q, _f32(q), dim ** -0.5)
    check_attention(b, r["y"].cpu().double().numpy(), r["lse"].cpu().double().numpy(), *want, "bf16")


def test_attention_is_the_same_twice():
    for b in (Batch(480, [3000, 70, 1200], None, 2, 128, 32, single=True), Batch(481, [500, 2100], [400, 150], 2, 128, 32)):
        q = b.rows(8, "bf16").cuda()
        c, bd = b.device_cache(), b.device_batch()
        first = pdq.kv_attention(q, c, bd, want_lse=True)
        for _ in range(3):
            again = pdq.kv_attention(q, c, bd, want_lse=True)
            assert torch.equal(first["y"].view(torch.int16), again["y"].view(torch.int16))
            assert torch.equal(first["lse"], again["lse"])


def test_binding_refusals():
    b = Batch(490, [5, 9], [2, 3], 2, 64, 16)
    c, bd = b.device_cache(), b.device_batch()
    q, k = b.rows(4, "bf16").cuda(), b.rows(2, "bf16").cuda()
    with pytest.raises(ValueError):
        pdq.kv_append(k, k[:-1], c, bd)
    with pytest.raises(ValueError):
        pdq.kv_append(k, k.half(), c, bd)
    with pytest.raises(ValueError):
        pdq.kv_append(k, k, c, bd, q=q)
    with pytest.raises(ValueError):
        pdq.kv_append(q, q, c, bd)
    with pytest.raises(ValueError):
        pdq.kv_append(k.transpose(1, 2), k, c, bd)
    with pytest.raises(ValueError):
        pdq.kv_attention(q.float(), c, bd)
    with pytest.raises(ValueError):
        pdq.kv_attention(q, c, bd, out=torch.empty_like(q)[:-1])
    with pytest.raises(ValueError):
        pdq.kv_attention(q, c, bd, alibi_slopes=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        pdq.kv_attention(q, c, bd, prefix_len=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        pdq.KVCache(c.k, c.k, c.k_scale, c.v_scale)
    with pytest.raises(pdq.PdqError):
        pdq.kv_attention(b.rows(3, "bf16").cuda(), c, bd)  # three query heads over two
    with pytest.raises(pdq.PdqError):
        pdq.kv_attention(q, c, pdq.KVBatch(bd.page_table, bd.seq_len))  # five rows of two sequences

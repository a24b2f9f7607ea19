"""The FP8 quantizers and the linear layer against the oracle (MI355X)."""
import numpy as np
import pytest
import torch

import oracle.fp8_oracle as FO
from fp8_cases import DT, check_linear, randn, values, weight
from guards import SENTINEL, gapped
from w8a8_int8_quantized_absmax_amd import pdq

pytestmark = pytest.mark.gpu


def bits(t):
    return t.cpu().view(torch.uint8).numpy()


def image(codes):
    """The packed image of code bits [rows, k]: blocks of 16 rows x 64 K values, by chunk of 16, then row."""
    rows, k = codes.shape
    full = np.zeros((-(-rows // 16) * 16, -(-k // 128) * 128), np.uint8)
    full[:rows, :k] = codes
    return full.reshape(-1, 16, full.shape[1] // 64, 4, 16).transpose(0, 2, 3, 1, 4).reshape(-1)


def raw_quantize(x):
    """pdq_quantize_fp8 into buffers with margins, which stay as they were -> (codes, scales)."""
    m, k = x.shape
    size, pitch = pdq._fp8_sizes(m, k)
    buf = torch.full((size + 8192,), SENTINEL, dtype=torch.uint8, device="cuda")
    sc = torch.full((m * pitch + 8192,), SENTINEL, dtype=torch.uint8, device="cuda")
    pdq._kv_call("pdq_quantize_fp8", 0, x.data_ptr(), pdq._DT[x.dtype], m, k, pdq._ld(x), buf[4096:].data_ptr(),
                 sc[4096:].data_ptr())
    buf, sc = buf.cpu().numpy(), sc.cpu().numpy()
    for b, n in ((buf, size), (sc, m * pitch)):
        assert (b[:4096] == SENTINEL).all() and (b[4096 + n:] == SENTINEL).all()
    return buf[4096:4096 + size], sc[4096:4096 + m * pitch].reshape(m, pitch)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,k", [(1, 16), (1, 4096), (3, 144), (16, 128), (17, 2064), (50, 640)])
def test_quantize_codes(m, k, dt):
    x = randn(m * 7 + k, m, k).to(DT[dt])
    q, b = FO.quantize(values(x))
    codes, scale = raw_quantize(x.cuda())
    assert np.array_equal(scale[:, :b.shape[1]], b)
    assert np.array_equal(codes, image(FO.e4m3_bits(q)))
    r = pdq.quantize_fp8(x.cuda())
    assert np.array_equal(r.values().cpu().double().numpy(), FO.values(values(x)))


def test_quantize_borders():
    # every step of the scale's choice, ties of the codes, subnormal codes, zeros, the ends of binary32
    rows = []
    for e in (-149, -140, -127, -126, -119, -118, -117, -20, 0, 5, 119, 127):
        for m in (1.0, 1.75, np.nextafter(np.float32(1.75), np.float32(2)), 1.9999999):
            v = np.float64(np.float32(m)) * 2.0 ** e
            rows.append(np.float32(v) * np.linspace(-1, 1, 128).astype(np.float32))
    rows.append(np.zeros(128, np.float32))
    ties = (np.arange(128) * 0.5 + 0.5) * 2.0 ** -10  # halves of the smallest step, behind a 448
    ties[0] = 448
    rows.append(ties.astype(np.float32))
    x = np.stack(rows)
    q, b = FO.quantize(x)
    codes, scale = raw_quantize(torch.from_numpy(x).cuda())
    assert np.array_equal(scale[:, :1], b)
    assert np.array_equal(codes, image(FO.e4m3_bits(q)))


def test_quantize_strided():
    x = randn(5, 9, 400).bfloat16().cuda()
    part = x[:, 64:64 + 272]
    a, b = pdq.quantize_fp8(part), pdq.quantize_fp8(part.contiguous())
    assert torch.equal(a.data, b.data) and torch.equal(a.scale.view(torch.uint8)[:, :3], b.scale.view(torch.uint8)[:, :3])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lead,n,k", [((), 1, 16), ((), 130, 144), ((3,), 128, 256), ((2, 2), 50, 400)])
def test_quantize_weight(lead, n, k, dt):
    w = randn(n + k, *lead, n, k).to(DT[dt])
    p = pdq.quantize_weight_fp8(w.cuda())
    flat = w.reshape(-1, n, k)
    codes, scales = p.codes().reshape(-1, n, k).cpu(), p.scale.view(torch.uint8).reshape(-1, *p.scale.shape[-2:]).cpu().numpy()
    size = pdq.fp8_bytes(n, k)
    for i in range(flat.shape[0]):
        q, b = FO.quantize_weight(values(flat[i]))
        assert np.array_equal(scales[i][:, :b.shape[1]], b)
        assert np.array_equal(bits(codes[i].contiguous()), FO.e4m3_bits(q))
        assert np.array_equal(bits(p.data[i * size:(i + 1) * size]), image(FO.e4m3_bits(q)))


@pytest.mark.parametrize("scales", ["pow2", "f32"])
@pytest.mark.parametrize("lead,n,k", [((), 17, 48), ((2, 3), 130, 640)])
def test_pack_weight(lead, n, k, scales):
    g = torch.Generator().manual_seed(n)
    codes = torch.randint(0, 255, (*lead, n, k), generator=g, dtype=torch.uint8)
    s = torch.randint(1, 250, (*lead, -(-n // 128), -(-k // 128)), generator=g, dtype=torch.uint8)
    s = s.view(torch.float8_e8m0fnu) if scales == "pow2" else s.float() * 0.37
    p = pdq.pack_weight_fp8(codes.view(torch.float8_e4m3fn).cuda(), s.cuda())
    assert torch.equal(p.codes().view(torch.uint8).cpu(), codes)
    assert torch.equal(p.scales().cpu(), s.float())


SIZES = [(1, 1, 16), (1, 17, 128), (1, 300, 4112), (3, 130, 144), (16, 64, 256), (17, 128, 272), (33, 300, 640),
         (64, 48, 2064), (65, 257, 1360), (130, 513, 4112), (257, 129, 512), (300, 700, 128)]


@pytest.mark.parametrize("dt,scales,bias", [("bf16", "pow2", False), ("f16", "f32", True), ("f32", "pow2", True),
                                            ("bf16", "f32", False)])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear(m, n, k, dt, scales, bias):
    x = randn(m + n + k, m, k).to(DT[dt])
    w, wq, ws = weight(n * 3 + k, (), n, k, scales)
    b = randn(n, n) if bias else None
    y, check = gapped(m, n, torch.float16 if dt == "f16" else torch.bfloat16)
    r = pdq.linear_fp8(x.cuda(), w, bias=None if b is None else b.cuda(), out=y)
    check()
    y64, size, aligned = FO.linear(values(x), wq, ws, None if b is None else values(b))
    check_linear(r["y"], y64, size, aligned, k)
    bias_d = None if b is None else b.cuda()
    ws = torch.full((pdq.linear_fp8_workspace_bytes(m, k) + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(pdq.linear_fp8(x.cuda(), w, bias=bias_d, workspace=ws)["y"], y)  # the same on every call
    parts, check = gapped(m, n, y.dtype)
    xq = pdq.quantize_fp8(x.cuda())
    pdq.gemm_fp8(xq, w, bias=bias_d, out=parts)
    check()
    check_linear(parts, y64, size, aligned, k)
    assert torch.equal(parts, pdq.gemm_fp8(xq, w, bias=bias_d, dtype=y.dtype)["y"])


@pytest.mark.parametrize("m,n,k,scales,tile", [
    (1, 8210, 144, "pow2", 0), (3, 16400, 272, "f32", 0), (13, 8200, 1424, "pow2", 0), (20, 8210, 144, "f32", 0), (40, 11000, 144, "pow2", 0),
    (64, 6200, 272, "f32", 0), (520, 4100, 400, "pow2", 128), (1030, 4100, 144, "f32", 128), (2039, 8190, 400, "pow2", 256),
    (1529, 8190, 400, "f32", 192), (4097, 300, 1040, "pow2", None), (2047, 8150, 912, "pow2", 256), (1500, 8150, 912, "f32", 192)])
def test_linear_wide(m, n, k, scales, tile):
    # every kernel of the rule; an odd last group for the tiled ones; some rows against the oracle
    x = randn(m + n, m, k).bfloat16()
    w, wq, ws = weight(n + k, (), n, k, scales)
    if tile is not None:
        assert pdq.gemm_fp8_tile(m, n, k, w.scale_type) == tile
    y, check = gapped(m, n, torch.bfloat16)
    pdq.linear_fp8(x.cuda(), w, out=y)
    check()
    rows = np.unique(np.concatenate([np.arange(0, m, max(1, m // 7)), [m - 1]]))
    cols = np.unique(np.concatenate([np.arange(0, n, 97), np.arange(max(0, n - 40), n)]))
    y64, size, aligned = FO.linear(values(x[rows]), wq, ws)
    pick = np.ix_(np.arange(len(rows)), cols)
    check_linear(y[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()], y64[pick], size[pick], aligned[pick], k)
    # and all of them against the same codes in binary32 (whose own error is far below the roundings')
    q = pdq.quantize_fp8(x.cuda()).values()
    scale = w.scales().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    full = q @ (w.codes().float() * scale).T
    assert float((y.float() - full).norm() / full.norm()) <= 2.0 ** -8 + 2.0 ** -12
    assert bool(((y.float() - full).abs() <= 2.0 ** -8 * full.abs() + 2.0 ** -9 * full.abs().max()).all())


@pytest.mark.parametrize("m", [1, 40, 300])
def test_matrix_unit(m):
    # what the products' tolerance stands on: next to 2^16 - 2^16 a product of 2^(16 - d) is kept up to d = 13 among
    # the same eight K values, up to d = 24 among the next eight, and whole elsewhere
    k = 384
    for at in (2, 7, 8, 15, 16, 100, 200, 383):
        most = 13 if at < 8 else 24 if at < 16 else 30
        x, w = torch.zeros((m, k)), torch.zeros((31, k))
        x[:, :2] = 256.0
        x[:, 130] = 256.0  # (the groups' scales are 1)
        x[:, 260] = 256.0
        w[:, 0], w[:, 1] = 256.0, -256.0
        y = {}
        for half in (-7, -3, 0, 4, 8):  # the activation's own power of two, the weight's the rest
            x[:, at] = 2.0 ** half
            for d in range(31):
                w[d, at] = 2.0 ** (16 - d - half)
            ok = [d for d in range(31) if -9 <= 16 - d - half <= 8]
            p = pdq.pack_weight_fp8(w.clamp(max=256).to(torch.float8_e4m3fn).cuda(), torch.ones((1, 3)).cuda())
            got = pdq.linear_fp8(x.cuda(), p)["y"].cpu()
            for d in ok:
                y.setdefault(d, []).append(got[:, d])
        assert sorted(y) == list(range(31))
        for d, rows in y.items():
            for r in rows:
                assert d > most or (r == 2.0 ** (16 - d)).all(), (at, d, r)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_linear_row_of_nan(m):
    # a value that is not finite makes its own row NaN and no other; a NaN scale its channels'
    x = randn(3, m, 400).bfloat16()
    x[0, 5] = float("inf")
    if m > 1:
        x[m - 1, 399] = float("nan")
    w, wq, ws = weight(4, (), 200, 400, "pow2")
    y = pdq.linear_fp8(x.cuda(), w)["y"].cpu()
    bad = sorted({0, m - 1})
    assert torch.isnan(y[bad]).all()
    assert torch.isfinite(y[[i for i in range(m) if i not in bad]]).all()
    x = randn(3, m, 400).bfloat16()
    w.scale.view(torch.uint8)[1, 2] = 255
    y = pdq.linear_fp8(x.cuda(), w)["y"].cpu()
    assert torch.isnan(y[:, 128:]).all() and torch.isfinite(y[:, :128]).all()


@pytest.mark.parametrize("scales", ["pow2", "f32"])
def test_linear_far_scales(scales):
    # scales far apart between groups and blocks, zero groups and blocks: nothing overflows on the way
    m, n, k = 20, 150, 512
    x = randn(8, m, k)
    x[:, :128] *= 2.0 ** -60
    x[:, 128:256] = 0
    x[3] *= 2.0 ** 40
    w, wq, ws = weight(9, (), n, k, scales)
    y64, size, aligned = FO.linear(values(x), wq, ws)
    y = pdq.linear_fp8(x.cuda(), w)["y"]
    check_linear(y, y64, size, aligned, k)


def test_linear_empty():
    w = weight(1, (), 32, 64, "pow2")[0]
    assert pdq.linear_fp8(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w)["y"].shape == (0, 32)

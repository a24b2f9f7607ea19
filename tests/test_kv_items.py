"""How the key/value kernels number their work items (csrc/kv_items.h), run on the host: every item that a sequence has is
found once, and no item before the first sequence's, behind cu_q[0] > 0 rows of none, is taken for one of its."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.fixture(scope="module")
def numbering(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")):
        pytest.skip("no host compiler or no HIP headers")
    lib = str(tmp_path_factory.mktemp("kv_items") / "items.so")
    res = subprocess.run([gxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I",
                          os.path.join(ROCM, "include"), "-I",
                          os.path.join(ROOT, "w8a8_int8_quantized_absmax_amd", "csrc"),
                          os.path.join(HERE, "kv_items", "host.cpp"), "-o", lib], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    f = ctypes.CDLL(lib).items

    def items(cu_q, batch, tokens, mul, per, extra, count):
        s, k, there = np.full(count, -1, np.int32), np.full(count, -1, np.int64), np.zeros(count, np.uint8)
        f(None if cu_q is None else cu_q.ctypes.data_as(ctypes.c_void_p), batch, tokens, mul, per, extra,
          ctypes.c_int64(count), *(a.ctypes.data_as(ctypes.c_void_p) for a in (s, k, there)))
        return s, k, there.astype(bool)

    return items


def _ragged(seed):
    r = np.random.default_rng(seed)
    n = int(r.choice([1, 1, 2, 3, 9, 63, 64, 65, 130, 400]))
    new = np.where(r.random(n) < 0.3, 0, r.integers(0, int(r.choice([2, 40, 700])), n))
    lead = int(r.choice([0, 1, 3, 16, 64, 200, 1000]))
    cu = (lead + np.concatenate([[0], np.cumsum(new)])).astype(np.int32)
    return new, cu, int(cu[-1]) + int(r.choice([0, 5, 300]))


@pytest.mark.parametrize("seed", range(12))
def test_row_tiles(numbering, seed):
    # attention: tiles of `rows` of a sequence's rows x heads of a group
    new, cu, tokens = _ragged(seed)
    for group, rows in ((1, 16), (4, 32), (5, 16), (1, 128), (4, 256), (20, 128)):
        count = tokens * group // rows + len(new)
        s, k, there = numbering(cu, len(new), tokens, group, rows, 1, count)
        assert (k[there] >= 0).all()
        has = there & (k * rows < new[np.clip(s, 0, len(new) - 1)] * group)
        want = [(b, t) for b, n in enumerate(new) for t in range(-(-int(n) * group // rows))]
        assert sorted(zip(s[has].tolist(), k[has].tolist())) == want
        assert not there[:int(cu[0]) * group // rows].any()


@pytest.mark.parametrize("seed", range(12))
def test_pages(numbering, seed):
    # append: the pages that a sequence's new tokens touch
    new, cu, tokens = _ragged(100 + seed)
    r = np.random.default_rng(200 + seed)
    for page in (16, 64, 256):
        p0 = r.integers(0, 3 * page, len(new))
        count = tokens // page + 2 * len(new)
        s, k, there = numbering(cu, len(new), tokens, 1, page, 2, count)
        assert (k[there] >= 0).all()
        at = np.clip(s, 0, len(new) - 1)
        pages = np.where(new > 0, (p0 + new - 1) // page - p0 // page + 1, 0)
        has = there & (k < pages[at])
        assert sorted(zip(s[has].tolist(), k[has].tolist())) == [(b, j) for b, n in enumerate(pages) for j in range(int(n))]
        assert not there[:int(cu[0]) // page].any()


def test_one_row_a_sequence(numbering):
    for group, rows in ((1, 16), (16, 16), (17, 16), (40, 256), (300, 256)):
        each = -(-group // rows)
        s, k, there = numbering(None, 70, 70, group, rows, 1, 70 * each)
        assert there.all() and (s == np.arange(70 * each) // each).all() and (k == np.arange(70 * each) % each).all()
    s, k, there = numbering(None, 70, 70, 1, 64, 2, 70)
    assert there.all() and (s == np.arange(70)).all() and not k.any()


def test_offsets_in_no_order(numbering):
    # cannot be refused: whatever they are, a sequence of the batch and a number from 0, or none
    for seed in range(8):
        r = np.random.default_rng(300 + seed)
        n = int(r.choice([2, 5, 70]))
        cu = r.integers(-400, 1500, n + 1).astype(np.int32)
        for mul, per, extra in ((4, 32, 1), (1, 16, 2)):
            s, k, there = numbering(cu, n, 1000, mul, per, extra, 1000 * mul // per + extra * n)
            assert ((s >= 0) & (s < n)).all() and (k[there] >= 0).all()

"""Seeded random batches over the key/value cache's two calls against the oracle: every head width, page and type, ragged
and single rows, with and without each option."""
import numpy as np
import pytest

from kv_cases import Batch
from test_gpu_kv import run_append, run_attention

pytestmark = pytest.mark.gpu


def _batch(r, seed, many):
    dim, page = int(r.choice([64, 128, 256])), int(r.choice([16, 32, 64, 128, 256]))
    hkv, n = int(r.integers(1, 4)), int(r.integers(1, 7))
    single = not many and r.random() < 0.4
    most = int(r.choice([3, 40, 200])) if many else 6
    new = [int(r.integers(0, most + 1)) for _ in range(n)]
    if many:
        new[int(r.integers(0, n))] = most
    length = [(1 if single else m) + int(r.integers(0, r.choice([2, 70, 900]))) for m in new]
    return Batch(seed, length, None if single else new, hkv, dim, page, lead=0 if single else int(r.integers(0, 3)),
                 tail=0 if single else int(r.integers(0, 3)), single=single, spare=int(r.integers(0, 3)))


@pytest.mark.parametrize("seed", range(24))
def test_append(seed):
    r = np.random.default_rng(7000 + seed)
    b = _batch(r, 7100 + seed, seed % 2 == 1)
    rot = int(r.choice([0, 16, b.dim // 2, b.dim]))
    run_append(b, str(r.choice(["bf16", "f16"])), hq=int(r.integers(1, 9)) if rot else 0, rot=rot,
               interleaved=bool(r.random() < 0.5), fused=bool(rot and r.random() < 0.5))


@pytest.mark.parametrize("seed", range(48))
def test_attention(seed):
    r = np.random.default_rng(8000 + seed)
    b = _batch(r, 8100 + seed, seed % 2 == 1)
    hq = b.hkv * int(r.choice([1, 2, 3, 4, 7]))
    opt = {}
    if r.random() < 0.3:
        opt["softcap"] = float(r.choice([3.0, 20.0]))
    if r.random() < 0.4:
        opt["window"] = int(r.choice([1, 15, 64, 333]))
    if r.random() < 0.3:
        opt["slopes"] = (2.0 ** -r.uniform(0, 8, hq)).astype(np.float32)
    if r.random() < 0.3:
        opt["prefix"] = r.integers(-3, 300, len(b.seq_len)).astype(np.int32)
    run_attention(b, hq, str(r.choice(["bf16", "f16"])), strided=bool(r.random() < 0.5),
                  scale=None if r.random() < 0.7 else float(r.uniform(0.02, 0.6)), **opt)

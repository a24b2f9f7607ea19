"""Batches over a paged INT8 cache for the key/value tests: seeded host arrays."""
from __future__ import annotations

import numpy as np
import torch

import oracle.kv_oracle as KO

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


class Batch:
    """Sequences with `new[s]` new rows and `length[s]` tokens after them, on a pool of random codes and scales.

    Table entries beyond a sequence's pages name no page.  lead / tail: rows before the first and behind the last
    sequence.  single: one row a sequence, without offsets."""

    def __init__(self, seed, length, new, hkv=2, dim=64, page=16, lead=0, tail=0, single=False, spare=2):
        r = np.random.default_rng(seed)
        self.rng, self.hkv, self.dim, self.page = r, hkv, dim, page
        self.seq_len = np.array(length, np.int32)
        held = [-(-n // page) for n in length]
        pages, width = sum(held) + 3, max(held + [0]) + spare
        order = r.permutation(pages)
        self.table = np.where(r.random((len(length), width)) < 0.5, -7, pages + 5).astype(np.int32)
        at = 0
        for s, h in enumerate(held):
            self.table[s, :h] = order[at:at + h]
            at += h
        self.cu_q = None if single else (lead + np.cumsum([0] + list(new))).astype(np.int32)
        self.tokens = len(length) if single else int(self.cu_q[-1]) + tail
        self.cache = dict(
            k=np.clip(np.rint(r.normal(0, 38, (pages, hkv, page, dim))), -127, 127).astype(np.int8),
            v=np.clip(np.rint(r.normal(0, 38, (pages, hkv, page, dim))), -127, 127).astype(np.int8),
            k_scale=r.uniform(0.01, 0.05, (pages, hkv)).astype(np.float32),
            v_scale=r.uniform(0.001, 0.03, (pages, hkv)).astype(np.float32))

    def rows(self, heads, dtype, scale=1.0):
        """Random [tokens, heads, dim] of dtype as a float32 array and a device maker."""
        x = torch.from_numpy(self.rng.normal(0, scale, (self.tokens, heads, self.dim)).astype(np.float32))
        return x.to(DT[dtype])

    def device_cache(self):
        from w8a8_int8_quantized_absmax_amd import pdq

        c = self.cache
        return pdq.KVCache(torch.from_numpy(c["k"]).cuda(), torch.from_numpy(KO.device_v(c["v"])).cuda(),
                           torch.from_numpy(c["k_scale"]).cuda(), torch.from_numpy(c["v_scale"]).cuda())

    def device_batch(self):
        from w8a8_int8_quantized_absmax_amd import pdq

        cu = None if self.cu_q is None else torch.from_numpy(self.cu_q).cuda()
        return pdq.KVBatch(torch.from_numpy(self.table).cuda(), torch.from_numpy(self.seq_len).cuda(), cu)

    def copy_cache(self):
        return {n: a.copy() for n, a in self.cache.items()}


def tables(positions, rot, base=10000.0):
    half = rot // 2
    angle = np.arange(positions)[:, None] * base ** (-np.arange(half) / half)
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def host_cache(c):
    """A pdq.KVCache's tensors as the oracle's dict."""
    return dict(k=c.k.cpu().numpy(), v=KO.plain_v(c.v.cpu().numpy()), k_scale=c.k_scale.cpu().numpy(),
                v_scale=c.v_scale.cpu().numpy())


def attention_tolerance(y, mag, big, keys, dim, dtype):
    """How far an output may be from the exact y, from the arithmetic that include/pdq.h states.

    A score is off by at most d = (dim + 8) 2^-24 big (the product's additions and the factors, big the sum of
    magnitudes) + 2^-21 (|z| <= big: the exponent's rounding and the exponential's, taken together), a weight
    relatively by that, by 2^-11 for its rounding to binary16 and by keys 2^-24 for the sums it goes through, the
    denominator by the same without the rounding; mag is what the weights multiply.  Weights under 2^-19 of the
    largest are subnormal in binary16: off by 2^-30 of it, over all keys.  Then one rounding to dtype."""
    d = ((dim + 8) * 2.0 ** -24 + 2.0 ** -22) * big[..., None] + 2.0 ** -21 + keys * 2.0 ** -24
    off = mag * (2.0 ** -11 + 2 * d) * (1 + 2.0 ** -8) + keys * 2.0 ** -30
    half = torch.finfo(DT[dtype]).eps / 2
    return off + half * (np.abs(y) + off) + 2.0 ** -24

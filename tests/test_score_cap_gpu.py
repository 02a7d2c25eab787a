"""Capped scores: a row's result is a function of its own sequence alone."""
import numpy as np
import pytest
import torch

import continuous_batching_paged_gb300 as cb
import workloads
from gpu_util import DeviceBatch, oracle_append
from oracle import paged_attention as opa
from quant_util import QuantBatch

pytestmark = pytest.mark.gpu


class Cache:
    """A batch on the bf16 cache, or on the quantised one: its calls, and each sequence's keys and values."""

    def __init__(self, b, quant):
        self.b, self.quant = b, quant
        self.d = QuantBatch(b) if quant else DeviceBatch(b)
        if quant:
            self.d.append_new()
            self.d.upload()
        else:
            self.d.append()
            self.pools = oracle_append(b)

    def attend(self, q=None, **kw):
        d, b = self.d, self.b
        q = d.q if q is None else q
        if self.quant:
            r = cb.quant_attention(q, *d.pools, *d.where, b.scale, lse=True, **kw)
        else:
            r = cb.scored_attention(q, d.k_pages, d.v_pages, d.block_table, d.cu, d.kv_lens, b.block_size,
                                    b.scale, lse=True, **kw)
        assert cb.get_device_error() == cb.CB_OK
        return r

    def cached(self, s):
        b = self.b
        if self.quant:
            return self.d.cached(s)
        return [opa.gather_kv(p, b.block_table[s], int(b.kv_lens[s]), b.block_size) for p in self.pools]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("score", [dict(softcap=8.0), dict(softcap=8.0, window=60), dict(softcap=5e5)], ids=str)
def test_a_row_does_not_depend_on_others(cuda_lib, score, quant):
    """Rows whose own scores stay small, alone and beside rows, keys and sequences with large ones: the same
    bits."""
    b = workloads.build_batch([50, 90, 1, 33], [200, 90, 77, 500], 4, 2, 64, 16, seed=695)
    c = Cache(b, quant)
    q = c.d.q
    want, want_lse = (t.clone() for t in c.attend(**score))
    for keep in (slice(0, 50), slice(140, 141), slice(141, 174), slice(60, 70)):
        other = q * 512.0
        other[keep] = q[keep]
        got, lse = c.attend(q=other, **score)
        assert torch.equal(got[keep].view(torch.int16), want[keep].view(torch.int16))
        assert torch.equal(lse[keep], want_lse[keep])
    # keys that a row does not see: those behind it (the chunk's first 20 rows, and its last keys)
    kn = [t.clone() for t in (c.d.k_new, c.d.v_new)]
    kn[0][141 + 20:174] *= 256.0
    if quant:
        cb.quant_append(None, *kn, *c.d.pools, *c.d.where)
    else:
        cb.kv_append(*kn, c.d.k_pages, c.d.v_pages, c.d.block_table, c.d.cu, c.d.kv_lens, 16)
    got, lse = c.attend(**score)
    assert torch.equal(got[141:161].view(torch.int16), want[141:161].view(torch.int16))
    assert torch.equal(lse[141:161], want_lse[141:161])
    assert not torch.equal(lse[161:174], want_lse[161:174])


@pytest.mark.parametrize("quant", [False, True])
def test_same_bits_on_every_call(cuda_lib, quant):
    """Chunks with ragged ends whose scores lie around the border of the two forms, behind chunks with large
    ones: whatever the items before left in shared memory."""
    ql = [33, 190, 70, 5, 140, 1, 61] * 6
    kv = [n + x for n, x in zip(ql, [0, 300, 77, 513, 9, 400, 1000] * 6)]
    b = workloads.build_batch(ql, kv, 16, 2, 64, 16, seed=697)
    q = opa.bf16_bits_to_f64(b.q).astype(np.float32)
    for s in range(0, len(ql), 5):
        q[int(b.cu_seqlens_q[s]):int(b.cu_seqlens_q[s + 1])] *= np.float32(300.0)
    c = Cache(workloads.Batch(**{**b.__dict__, "q": workloads.f32_to_bf16_bits(q)}), quant)
    out, lse = (t.clone() for t in c.attend(softcap=4.0))
    for _ in range(30):
        o, l = c.attend(softcap=4.0)
        assert torch.equal(o.view(torch.int16), out.view(torch.int16)) and torch.equal(l, lse)

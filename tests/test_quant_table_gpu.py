"""Block tables of the quantised cache's attention with entries that name no block: below a sequence's
length they are reported, before a sliding window they are not read."""
import numpy as np
import pytest
import torch

import continuous_batching_paged_gb300 as cb
import workloads
from gpu_util import i32
from oracle import paged_attention as opa
from quant_util import P8, P16, QuantBatch, check_rows, f64

pytestmark = pytest.mark.gpu

# KV heads and block sizes: 2, 32, 64 and 256 page runs per decode tile
SHAPES = [(8, 16), (2, 4), (1, 4), (1, 5)]


def batch(ql, kv, hkv, bs, entries, D=64, seed=700):
    b = workloads.build_batch(ql, kv, 2 * hkv, hkv, D, bs, seed=seed + bs)
    d = QuantBatch(b)
    d.append_new()
    d.upload()
    table = b.block_table.copy()
    for (s, j), value in entries.items():
        table[s, j] = value
    d.table = i32(table)
    return d


def rows_right(d, out, lse, seqs, window=0):
    b = d.b
    o, l, q = f64(out), f64(lse), opa.bf16_bits_to_f64(b.q)
    for s in seqs:
        c0, c1, kv = int(b.cu_seqlens_q[s]), int(b.cu_seqlens_q[s + 1]), int(b.kv_lens[s])
        K, V = d.cached(s)
        check_rows(o[c0:c1], l[c0:c1], q[c0:c1], K, V, kv - (c1 - c0), b.scale, P16 if c1 - c0 == 1 else P8,
                   f"sequence {s}", window=window)


@pytest.mark.parametrize("entry", [-1, -2, -2 ** 31])
@pytest.mark.parametrize("hkv,bs", SHAPES)
@pytest.mark.parametrize("ql", [[1, 1], [40, 1], [1, 40]], ids=str)
def test_negative_entries_are_reported(cuda_lib, ql, hkv, bs, entry):
    """One entry, of a block before the sequence's last, is the only fault of the batch."""
    for s in (0, 1):
        d = batch(ql, [300, 290], hkv, bs, {(s, 200 // bs): entry})
        out, lse = cb.quant_attention(d.q, *d.pools, *d.where, d.b.scale, lse=True)
        assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE
        rows_right(d, out, lse, [1 - s])
        cb.quant_attention(d.q, *d.pools, *d.where, d.b.scale, softcap=20.0)
        assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE
        cb.quant_append_attention(d.q, d.k_new, d.v_new, *d.pools, *d.where, d.b.scale)
        assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE
    d = batch(ql, [300, 290], hkv, bs, {})
    cb.quant_attention(d.q, *d.pools, *d.where, d.b.scale)
    assert cb.get_device_error() == cb.CB_OK


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hkv,bs", SHAPES + [(8, 64), (3, 24)])
@pytest.mark.parametrize("entry", [-1, 2 ** 30])
def test_entries_before_the_window_are_not_read(cuda_lib, entry, hkv, bs, D):
    """A server that frees the blocks which every window has left marks them in the table."""
    ql, kv, W = [1, 70, 1, 200], [700, 500, 330, 460], 150
    first = [(k - n - W + 1) // bs for n, k in zip(ql, kv)]  # the block of the window's first key
    d = batch(ql, kv, hkv, bs, {(s, j): entry for s in range(4) for j in range(first[s])}, D)
    assert all(f > 0 for f in first)
    out, lse = cb.quant_attention(d.q, *d.pools, *d.where, d.b.scale, window=W, lse=True)
    assert cb.get_device_error() == cb.CB_OK
    rows_right(d, out, lse, range(4), W)
    # the window's own first block
    for s in range(4):
        table = d.b.block_table.copy()
        table[s, first[s]] = entry
        cb.quant_attention(d.q, *d.pools, i32(table), d.cu, d.kv, bs, d.b.scale, window=W)
        assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE

"""Capped scores: as exact as uncapped ones whatever the cap's size, and a row's result a function of its own
sequence alone."""
import numpy as np
import pytest
import torch

import continuous_batching_paged_gb300 as cb
import workloads
from gpu_util import DeviceBatch, oracle_append
from oracle import paged_attention as opa
from oracle import quant as oq
from quant_util import P8, P16, QuantBatch, f64

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


def check_capped(c, softcap):
    """Every row against the oracle.  A score x is off by 2^-20 |x| by the cap (tanh by a polynomial or from
    exp2 and a reciprocal: 2^-21 of itself, and the roundings of its factors), and by its products' rounding: D of
    them summed in fp32, 2^-24 each of the sum of |q_d k_d|, times the slope that the cap has there.  The quantised
    decode pass has its query row in fp16, off by 2^-25 of its largest power of two.  That moves a probability by e
    (and an exponential's 2^-21) and the output by 2 e times the weighted |v|; a probability is rounded once to
    p_step, the result to bf16."""
    b = c.b
    out, lse = c.attend(softcap=softcap)
    o, l, q = f64(out), f64(lse), opa.bf16_bits_to_f64(b.q)
    g = b.num_q_heads // b.num_kv_heads
    for s in range(b.num_seqs):
        c0, c1, kv = int(b.cu_seqlens_q[s]), int(b.cu_seqlens_q[s + 1]), int(b.kv_lens[s])
        n = c1 - c0
        if n == 0:
            continue
        K, V = c.cached(s)
        ref, ref_lse, size = oq.scored_attention(q[c0:c1], K, V, kv - n, b.scale, softcap)
        Kr = np.repeat(K, g, axis=1)
        mag = np.einsum("nhd,khd->nhk", np.abs(q[c0:c1]), np.abs(Kr)) * b.scale
        x = np.abs(np.einsum("nhd,khd->nhk", q[c0:c1], Kr)) * b.scale
        off = 2.0 ** -24 * (b.head_dim + 8) * mag
        if c.quant:
            off = off + b.scale * np.abs(q[c0:c1]).max(-1)[..., None] * np.abs(Kr).sum(-1).T[None] * 2.0 ** -25
        slope = np.cosh(np.minimum(np.maximum(x - off, 0.0) / softcap, 300.0)) ** -2.0  # the steepest within `off`
        e = 2.0 ** -21 + (2.0 ** -20 * softcap * np.tanh(x / softcap) + off * slope).max(-1)
        p_step = P16 if c.quant and n == 1 else P8
        assert np.isfinite(o[c0:c1]).all()
        tol = 2.0 ** -8 * np.abs(ref) + (p_step + 2 * e)[..., None] * size * (1 + 2.0 ** -8) + 1e-30
        err = np.abs(o[c0:c1] - ref)
        assert np.all(err <= tol), f"cap {softcap}, sequence {s}: worst {(err / tol).max():.3g}"
        lerr = np.abs(l[c0:c1] - ref_lse)
        assert np.all(lerr <= e + 2.0 ** -20 * (1 + np.abs(ref_lse))), f"cap {softcap}, sequence {s}: lse off by " \
                                                                       f"{lerr.max():.3g}"


CAPS = [0.3, 5.0, 50.0, 300.0, 1e3, 1e4, 1e6, 1e9, 1e15, 1e30]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 3, 1), (128, 8, 2), (128, 16, 1)])
@pytest.mark.parametrize("cap", CAPS)
def test_caps_of_all_sizes(cuda_lib, cap, D, Hq, Hkv, quant):
    check_capped(Cache(workloads.build_batch([1, 37, 1, 130, 5], [1, 37, 513, 700, 70], Hq, Hkv, D, 16,
                                             seed=670 + D + Hq), quant), cap)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("scale,cap", [(1e-4, 1e-4), (1e-4, 1e-1), (3e-3, 1e-5), (5.0, 1e-3), (40.0, 4e3), (2.0, 1e20)])
def test_scales_beside_the_usual(cuda_lib, scale, cap, quant):
    b = workloads.build_batch([1, 37, 1, 130], [1, 37, 513, 300], 4, 2, 64, 16, seed=680)
    b.scale = scale
    check_capped(Cache(b, quant), cap)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("cap", [2.0, 30.0, 1e6])
def test_small_scores_beside_large_ones(cuda_lib, cap, quant):
    """Rows and heads of one tile whose scores are 2^12 apart."""
    b = workloads.build_batch([1, 150, 1, 40], [300, 400, 65, 40], 8, 2, 128, 16, seed=690)
    q = opa.bf16_bits_to_f64(b.q).astype(np.float32)
    q[::3] *= np.float32(64.0)
    q[1::3] *= np.float32(2.0 ** -6)
    q[:, 3] *= np.float32(16.0)
    b = workloads.Batch(**{**b.__dict__, "q": workloads.f32_to_bf16_bits(q)})
    check_capped(Cache(b, quant), cap)


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


def test_caps_that_fp32_does_not_hold(cuda_lib):
    """A cap that rounds to 0 (none) or to infinity is refused, not taken for none."""
    b = workloads.build_batch([1, 3], [40, 30], 4, 2, 64, 16, seed=699)
    for quant in (False, True):
        c = Cache(b, quant)
        with pytest.raises(ValueError, match="softcap"):
            c.attend(softcap=1e-50)
        with pytest.raises((ValueError, cb.CbError), match="softcap"):
            c.attend(softcap=1e39)
        with pytest.raises(ValueError, match="softcap"):
            c.attend(softcap=-1e-50)
        c.attend(softcap=0)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("cap", [3.0, 1e7])
def test_products_beyond_fp32_and_keys_that_are_nan(cuda_lib, cap, quant):
    """Products that overflow are capped like any large one; a key that is NaN makes the rows NaN that see it, and
    no others.  (Keys are multiples of one unit vector, so that no sum of infinities is NaN.)"""
    b = workloads.build_batch([1, 70, 1], [90, 200, 40], 4, 2, 64, 16, seed=698)
    q = np.zeros(b.q.shape, dtype=np.float32)
    q[..., 5] = np.where(np.arange(q.shape[0]) % 2 == 0, 2.0 ** 100, 2.0 ** -3)[:, None]
    pool = np.zeros(b.k_pages.shape, dtype=np.float32)
    rng = np.random.default_rng(1)
    pool[..., 5] = rng.choice([-1.0, 1.0, 0.25], pool.shape[:-1]) * np.float32(2.0 ** 30)
    new = np.zeros(b.k_new.shape, dtype=np.float32)
    new[..., 5] = np.float32(2.0 ** 30)
    b = workloads.Batch(**{**b.__dict__, "q": workloads.f32_to_bf16_bits(q), "k_new": workloads.f32_to_bf16_bits(new),
                           "k_pages": workloads.f32_to_bf16_bits(pool)})
    c = Cache(b, quant)
    check_capped(c, cap)
    want, _ = c.attend(softcap=cap)
    s, p = 1, 160  # a key in the chunk: queries 30 .. 69 of it see it
    where = int(b.block_table[s, p // 16]), p % 16
    if quant:
        c.d.dk.view(torch.uint8)[where] = 0x7F
        c.d.dsc[where + (slice(None), 0)] = 255
    else:
        c.d.k_pages[where] = float("nan")
    got, _ = c.attend(softcap=cap)
    seen = torch.zeros(72, dtype=torch.bool, device="cuda")
    seen[1 + 30:1 + 70] = True
    assert torch.isnan(got[seen]).all() and torch.equal(got[~seen].view(torch.int16), want[~seen].view(torch.int16))

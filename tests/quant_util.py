"""Batches for the tests of the quantised cache and of changed scores: a seeded batch's cache in codes, the
oracle's results, and how far a kernel's may be from them."""
from __future__ import annotations

import numpy as np
import torch

import continuous_batching_paged_gb300 as cb
import workloads
from gpu_util import bf16_tensor, i32
from oracle import paged_attention as opa
from oracle import quant as oq


class QuantBatch:
    """A batch (workloads.build_batch) whose cache is quantised: host arrays k, v (codes), sc (exponent
    bytes), and the same on the device.  Slots outside a sequence's prior context hold NaN codes and
    exponent bytes of 255.  spread: the binary logarithm of the rows' sizes varies by it (the values' rows;
    the keys' by 1 at most, so that no score is so large that its rounding decides the softmax)."""

    def __init__(self, b: workloads.Batch, spread=0.0, seed=0):
        self.b = b
        rng = np.random.default_rng(seed + 17)
        self.k, ks = self._pool(b.k_pages, rng, min(spread, 1.0))
        self.v, vs = self._pool(b.v_pages, rng, spread)
        self.sc = np.stack((ks, vs), -1)
        self.dk, self.dv, self.dsc = (torch.from_numpy(x).cuda() for x in (self.k, self.v, self.sc))
        self.dk, self.dv = self.dk.view(torch.float8_e4m3fn), self.dv.view(torch.float8_e4m3fn)
        self.q, self.k_new, self.v_new = bf16_tensor(b.q), bf16_tensor(b.k_new), bf16_tensor(b.v_new)
        self.table, self.cu, self.kv = i32(b.block_table), i32(b.cu_seqlens_q), i32(b.kv_lens)

    @staticmethod
    def _pool(bits, rng, spread):
        x = opa.bf16_bits_to_f64(bits)
        if spread:  # rows of very different sizes
            x = x * 2.0 ** np.round(rng.normal(0, spread, x.shape[:-1]))[..., None]
        dead = np.isnan(x).any(-1)
        codes, sc = oq.quantise(np.where(dead[..., None], 0.0, x))
        codes[dead], sc[dead] = 0x7F, 255
        return codes, sc

    @property
    def pools(self):
        return self.dk, self.dv, self.dsc

    @property
    def where(self):
        return self.table, self.cu, self.kv, self.b.block_size

    def slots(self):
        """Each packed token's (block, offset)."""
        b = self.b
        out = []
        for s in range(b.num_seqs):
            n = int(b.cu_seqlens_q[s + 1] - b.cu_seqlens_q[s])
            for i in range(n):
                p = int(b.kv_lens[s]) - n + i
                out.append((int(b.block_table[s, p // b.block_size]), p % b.block_size))
        return out

    def append(self, k_new, v_new):
        """The oracle's append of float64 rows into the host pools; upload() moves them."""
        for x, pool, w in ((k_new, self.k, 0), (v_new, self.v, 1)):
            codes, sc = oq.quantise(x)
            for t, (blk, off) in enumerate(self.slots()):
                pool[blk, off] = codes[t]
                self.sc[blk, off, :, w] = sc[t]

    def append_new(self):
        self.append(opa.bf16_bits_to_f64(self.b.k_new), opa.bf16_bits_to_f64(self.b.v_new))

    def upload(self):
        self.dk.view(torch.uint8).copy_(torch.from_numpy(self.k))
        self.dv.view(torch.uint8).copy_(torch.from_numpy(self.v))
        self.dsc.copy_(torch.from_numpy(self.sc))

    def cached(self, s, first=0, last=None):
        """Keys and values of sequence s as the host pools hold them."""
        b = self.b
        last = int(b.kv_lens[s]) if last is None else last
        pos = np.arange(first, last)
        blk, off = b.block_table[s, pos // b.block_size], pos % b.block_size
        return (oq.values(self.k[blk, off], self.sc[blk, off, :, 0]),
                oq.values(self.v[blk, off], self.sc[blk, off, :, 1]))

    def workspace(self):
        b = self.b
        n = cb.workspace_size(b.num_seqs, b.num_q_heads, b.num_kv_heads, b.head_dim, self.q.shape[0])
        return torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")


def check_rows(out, lse, q, K, V, ctx, scale, p_step, what, softcap=0.0, slopes=None, visible=0, window=0):
    """One sequence's rows against the oracle (out and lse: float64 arrays of the kernel's results).

    A probability is rounded once to 2^-8 (bf16, the chunk pass) or 2^-11 (fp16, the quantised decode
    pass) of itself: p_step, which moves the output by p_step times the weighted |v| at most.  A score is
    off by `e`: D products summed in fp32 (2^-24 each, of the sum of |q_d k_d|), a cap computed to 2^-21
    of it, a bias rounded twice, an exponential of 2^-22; that moves each p by e, and the output by 2 e
    times the weighted |v|.  The query row in fp16 is off by 2^-25 of its largest power of two.  The
    result is rounded to bf16: 2^-8 of itself."""
    ref, ref_lse, size = oq.scored_attention(q, K, V, ctx, scale, softcap, slopes, visible, window)
    n, hq, d = q.shape
    g = hq // K.shape[1]
    Kf = np.where(np.isfinite(K), np.abs(K), 0)
    mag = np.einsum("nhd,khd->nhk", np.abs(q), np.repeat(Kf, g, axis=1)).max(-1) * scale
    fp16 = scale * np.abs(q).max(-1) * np.repeat(Kf.sum(-1).max(0), g)[None] * 2.0 ** -25
    far = K.shape[0]
    e = 2.0 ** -24 * (d + 8) * mag + fp16 + 2.0 ** -21 + 2.0 ** -21 * softcap
    if slopes is not None:
        e = e + 2.0 ** -23 * np.abs(np.asarray(slopes, dtype=np.float64))[None] * far
    assert np.isfinite(out).all(), f"{what}: not finite"
    tol = 2.0 ** -8 * np.abs(ref) + (p_step + 2 * e)[..., None] * size * (1 + 2.0 ** -8) + 1e-30
    err = np.abs(out - ref)
    assert np.all(err <= tol), f"{what}: {np.count_nonzero(err > tol)} of {err.size}, worst {(err / tol).max():.3g} " \
                               f"at {np.unravel_index((err / tol).argmax(), err.shape)}"
    if lse is not None:
        # its own rounding, the logarithm's, and a sum of rounded terms
        lerr = np.abs(lse - ref_lse)
        assert np.all(lerr <= e + 2.0 ** -20 * (1 + np.abs(ref_lse))), f"{what}: lse off by {lerr.max():.3g}"


P16, P8 = 2.0 ** -11, 2.0 ** -8   # a probability in fp16, in bf16


def f64(t):
    return t.double().cpu().numpy()

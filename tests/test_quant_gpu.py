"""The quantised cache: the append bit for bit, the read-back, and attention over it, against the float64
oracle."""
import numpy as np
import pytest
import torch

import continuous_batching_paged_gb300 as cb
import workloads
from gpu_util import bf16_tensor, bits_of, i32
from oracle import paged_attention as opa
from oracle import quant as oq
from oracle import rope as orope
from quant_util import P8, P16, QuantBatch, check_rows, f64

pytestmark = pytest.mark.gpu

# ragged mix: decodes, chunks crossing block boundaries, an empty sequence, a first token
RAGGED = ([1, 37, 0, 5, 1, 130, 1], [1, 37, 9, 70, 513, 300, 65])


def rotated_fp32(bits, pos, cs, interleaved):
    """bf16 rows turned in fp32, each product and sum rounded, and no rounding behind them."""
    x = (bits.astype(np.uint32) << 16).view(np.float32).copy()
    rot = cs.shape[1]
    c, s = cs[pos][:, None, :rot // 2], cs[pos][:, None, rot // 2:]
    a, b = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
            else (slice(0, rot // 2), slice(rot // 2, rot)))
    xa, xb = x[..., a].copy(), x[..., b].copy()
    x[..., a] = xa * c - xb * s
    x[..., b] = xb * c + xa * s
    return x


def check_append(b, rot=0, interleaved=False, packed=False, in_place=False, keys_only=False, stream=None):
    d = QuantBatch(b)
    q, kn, vn = d.q, d.k_new, d.v_new
    if packed:
        row = torch.cat((q, kn, vn), 1)
        h, k = q.shape[1], kn.shape[1]
        q, kn, vn = row[:, :h], row[:, h:h + k], row[:, h + k:]
    cs = orope.table(int(b.kv_lens.max(initial=1)), rot) if rot else None
    torch.cuda.synchronize()
    if not rot:
        assert cb.quant_append(None, kn, vn, *d.pools, *d.where, stream=stream) is None
    else:
        got = cb.quant_append(None if keys_only else q, kn, vn, *d.pools, *d.where,
                              cos_sin=torch.from_numpy(cs).cuda(), interleaved=interleaved,
                              q_out=q if in_place else None, stream=stream)
    assert cb.get_device_error(stream) == cb.CB_OK
    pos = orope.positions_of(b.cu_seqlens_q, b.kv_lens)
    k = rotated_fp32(b.k_new, pos, cs, interleaved) if rot else opa.bf16_bits_to_f64(b.k_new)
    d.append(k.astype(np.float64), opa.bf16_bits_to_f64(b.v_new))
    assert np.array_equal(d.dk.view(torch.uint8).cpu().numpy(), d.k)
    assert np.array_equal(d.dv.view(torch.uint8).cpu().numpy(), d.v)
    assert np.array_equal(d.dsc.cpu().numpy(), d.sc)
    if rot and not keys_only:
        want = b.q.copy()
        want[..., :rot] = workloads.f32_to_bf16_bits(rotated_fp32(b.q, pos, cs, interleaved)[..., :rot])
        assert np.array_equal(bits_of(got), want)


@pytest.mark.parametrize("D", [64, 128])
def test_append(cuda_lib, D):
    check_append(workloads.build_batch(*RAGGED, 8, 4, D, 16, seed=800 + D))
    check_append(workloads.build_batch(*RAGGED, 8, 4, D, 16, seed=801 + D), packed=True)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 48)])
def test_append_rotated(cuda_lib, D, rot, interleaved):
    check_append(workloads.build_batch(*RAGGED, 8, 4, D, 16, seed=810 + rot), rot, interleaved)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (15, 5), (32, 8), (40, 40), (16, 1), (6, 3)])
def test_append_head_layouts(cuda_lib, Hq, Hkv):
    b = workloads.build_batch(*RAGGED, Hq, Hkv, 64 if Hq % 2 else 128, 20, seed=820 + Hq)
    check_append(b, 32, packed=True)
    check_append(b, 32, True, keys_only=True)
    check_append(b)


@pytest.mark.parametrize("bs", [4, 5, 256])
def test_append_block_sizes(cuda_lib, bs):
    check_append(workloads.build_batch(*RAGGED, 4, 2, 64, bs, seed=830 + bs), 64)


@pytest.mark.parametrize("T", [1, 2, 31, 257, 3000])
def test_append_token_counts(cuda_lib, T):
    check_append(workloads.build_batch([T], [T + 13], 8, 2, 128, 32, seed=840 + T), 128, in_place=True)


def test_append_extreme_rows(cuda_lib):
    """Zeros, infinities, NaN, subnormals, the largest values, rows at the edges of the exponents."""
    b = workloads.build_batch([12, 1], [40, 7], 4, 2, 64, 16, seed=850)
    x = opa.bf16_bits_to_f64(b.k_new).astype(np.float32)
    x[0] = 0
    x[1, 0, 3], x[1, 1, 5], x[1, 1, 6] = np.inf, np.nan, -np.inf
    x[2] = np.nan
    x[3, :, 0] = 3.0e38
    x[4] *= np.float32(2.0 ** -130)
    x[5] *= np.float32(2.0 ** -60)
    x[6, :, :] = 1.0
    x[6, 0, 0], x[6, 1, 0] = 448, 450
    x[7] *= np.float32(2.0 ** 33)
    x[8] *= np.float32(2.0 ** -24)
    x[9, :, 1:] = np.float32(2.0 ** -20)
    x[10] = -np.inf
    bits = workloads.f32_to_bf16_bits(x)
    b = workloads.Batch(**{**b.__dict__, "k_new": bits, "v_new": bits[::-1].copy()})
    check_append(b)


def test_append_padding_rows_bad_metadata_and_empty(cuda_lib):
    b = workloads.build_batch([1, 3, 1], [40, 70, 9], 4, 2, 64, 16, seed=853)
    d = QuantBatch(b)
    pad = lambda t: torch.cat((t, torch.full((11,) + t.shape[1:], 3.0, dtype=t.dtype, device="cuda")))
    cb.quant_append(None, pad(d.k_new), pad(d.v_new), *d.pools, *d.where)
    assert cb.get_device_error() == cb.CB_OK
    d.append_new()
    assert np.array_equal(d.dk.view(torch.uint8).cpu().numpy(), d.k)
    assert np.array_equal(d.dsc.cpu().numpy(), d.sc)
    # a bad block, a length below the query's, a decreasing cu: skipped and reported
    table = b.block_table.copy()
    table[1, 4] = b.num_pages + 3
    for name, value in (("table", i32(table)), ("kv", i32([40, 2, 9])), ("cu", i32([0, 1, 4, 3]))):
        d = QuantBatch(b)
        setattr(d, name, value)
        before = d.k.copy(), d.sc.copy()
        cb.quant_append(None, d.k_new, d.v_new, *d.pools, *d.where)
        assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE, name
        ok = {d.slots()[0], d.slots()[4], d.slots()[1]} | set(d.slots())
        for a, c in zip(before, (d.dk.view(torch.uint8).cpu().numpy(), d.dsc.cpu().numpy())):
            changed = {tuple(x[:2]) for x in np.argwhere(a != c).tolist()}
            assert changed <= ok, name
    d = QuantBatch(b)
    z = d.k_new[:0]
    cb.quant_append(None, z, z, *d.pools, d.table[:0], i32([0]), i32([]), 16)
    assert np.array_equal(d.dk.view(torch.uint8).cpu().numpy(), d.k)


# ------------------------------------------------------------------------------------ read back
@pytest.mark.parametrize("Hkv,D,bs", [(1, 64, 16), (2, 128, 16), (5, 64, 5), (8, 128, 32), (16, 64, 4), (40, 128, 64)])
def test_gather(cuda_lib, Hkv, D, bs):
    kv = [1, 37, 9, 300, 513, 65, 40]
    b = workloads.build_batch([0] * 7, kv, Hkv, Hkv, D, bs, seed=860 + Hkv)
    d = QuantBatch(b, spread=6)
    for starts in (None, [0, 37, 3, 250, 1, 64, 5]):
        lens = [k - (starts[i] if starts else 0) for i, k in enumerate(kv)]
        lens[2] = 0 if starts else lens[2]
        cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
        n = int(cu[-1]) + 5
        ko = torch.full((n, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
        vo = ko.clone()
        got = cb.quant_gather(*d.pools, d.table, i32(cu), bs, n, key_starts=None if starts is None else i32(starts),
                              k_out=ko, v_out=vo)
        assert got[0] is ko and got[1] is vo
        assert cb.get_device_error() == cb.CB_OK
        for s in range(7):
            a = starts[s] if starts else 0
            K, V = d.cached(s, a, a + lens[s])
            assert np.array_equal(f64(ko[cu[s]:cu[s + 1]]), K)
            assert np.array_equal(f64(vo[cu[s]:cu[s + 1]]), V)
        assert (ko[-5:].float() == 7).all() and (vo[-5:].float() == 7).all()


def test_gather_large_and_misused(cuda_lib):
    b = workloads.build_batch([0, 0], [20000, 9000], 2, 2, 64, 16, seed=870)
    d = QuantBatch(b)
    ko, vo = cb.quant_gather(*d.pools, d.table, i32([0, 20000, 29000]), 16, 29000)
    K, V = (np.concatenate(x) for x in zip(d.cached(0), d.cached(1)))
    assert np.array_equal(f64(ko), K) and np.array_equal(f64(vo), V)
    assert cb.get_device_error() == cb.CB_OK
    # positions past the table, a negative start, a bad block id, a bad cu: reported, nothing else written
    table = b.block_table.copy()
    table[1, 2] = -1
    for tab, cu, starts, n in ((b.block_table, [0, 1, 60], [b.max_blocks * 16 - 10, b.max_blocks * 16 - 10], 60),
                               (b.block_table, [0, 4, 8], [-3, 0], 8), (table, [0, 4, 80], None, 80),
                               (b.block_table, [0, 9, 5], None, 9), (b.block_table, [1, 5, 8], None, 8)):
        out = torch.full((n + 3, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        v = out.clone()
        cb.quant_gather(*d.pools, i32(tab), i32(cu), 16, n, key_starts=None if starts is None else i32(starts),
                        k_out=out[:n], v_out=v[:n])
        assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE, cu
        assert (out[n:].float() == 7).all() and (v[n:].float() == 7).all()


# ------------------------------------------------------------------------------------ attention
def check_attention(b, spread=0.0, seed=0, decode_ctas=0, serial=False, stream=None, edit=None, p8=False,
                    upload=True, **score):
    """quant_attention on the batch against the oracle; returns the batch and the results."""
    d = QuantBatch(b, spread, seed)
    if upload:
        d.append_new()
    if edit is not None:
        edit(d)
    d.upload()
    slopes, visible = score.get("slopes"), score.get("visible")
    dev = dict(softcap=score.get("softcap", 0.0), window=score.get("window", 0))
    if slopes is not None:
        dev["slopes"] = torch.tensor(slopes, dtype=torch.float32, device="cuda")
        slopes = np.asarray(slopes, dtype=np.float32)
    if visible is not None:
        dev["visible_lens"] = i32(visible)
    out = torch.full_like(d.q, float("nan"))
    lse = torch.full(d.q.shape[:2], float("nan"), dtype=torch.float32, device="cuda")
    torch.cuda.synchronize()
    cb.quant_attention(d.q, *d.pools, *d.where, b.scale, out=out, lse=lse, workspace=d.workspace(),
                       decode_ctas=decode_ctas, serial=serial, stream=stream, **dev)
    assert cb.get_device_error(stream) == cb.CB_OK
    check_results(d, out, lse, slopes, visible, score)
    return d, out, lse


def check_results(d, out, lse, slopes=None, visible=None, score={}, q=None):
    b = d.b
    o, l, q = f64(out), f64(lse), opa.bf16_bits_to_f64(b.q) if q is None else q
    for s in range(b.num_seqs):
        c0, c1 = int(b.cu_seqlens_q[s]), int(b.cu_seqlens_q[s + 1])
        if c1 == c0:
            continue
        n, kv = c1 - c0, int(b.kv_lens[s])
        K, V = d.cached(s)
        check_rows(o[c0:c1], l[c0:c1], q[c0:c1], K, V, kv - n, b.scale, P16 if n == 1 else P8,
                   f"sequence {s} ({n} of {kv})", score.get("softcap", 0.0), slopes,
                   0 if visible is None else visible[s], score.get("window", 0))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (16, 1), (7, 1), (4, 2), (32, 2), (6, 3), (48, 3), (4, 4),
                                    (64, 4), (10, 5), (35, 7), (8, 8), (32, 8), (64, 8), (16, 16), (128, 8)])
def test_decode_head_layouts(cuda_lib, Hq, Hkv, D):
    kv = [1, 31, 32, 33, 300, 513, 65, 1100]
    check_attention(workloads.build_batch([1] * 8, kv, Hq, Hkv, D, 16, seed=900 + Hq + Hkv))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [4, 5, 6, 8, 12, 24, 32, 64, 100, 256])
def test_decode_block_sizes(cuda_lib, bs, D):
    kv = [1, 16, 40, 257, 700, 65]
    for hkv in (1, 3, 8):
        check_attention(workloads.build_batch([1] * 6, kv, 2 * hkv, hkv, D, bs, seed=910 + bs + hkv))


def test_decode_split_and_merged(cuda_lib):
    """Sequences cut over many CTAs, none, and a given number of CTAs."""
    b = workloads.build_batch([1] * 5, [9000, 17, 800, 4096, 1], 16, 2, 128, 32, seed=920)
    for n in (0, 1, 7, 512):
        check_attention(b, decode_ctas=n)


def test_decode_ranges_left_to_the_last_cta(cuda_lib):
    """Beside chunk work the decode CTAs take their ranges by the SM they are on; where too few are on the
    chosen ones (here 2 to 7 of 152), the last one takes what is left."""
    for n, kv in ((2, [20, 35]), (4, [70, 30, 35]), (7, [90, 65, 20, 35])):
        b = workloads.build_batch([1] * (len(kv) - 1) + [30], kv, 8, 8, 128, 16, seed=919 + n)
        for _ in range(3):
            check_attention(b, decode_ctas=n)
    check_attention(workloads.build_batch([1, 1, 40], [3000, 500, 300], 32, 16, 64, 16, seed=929), decode_ctas=5)
    check_attention(workloads.build_batch([1, 1, 40], [3000, 500, 300], 32, 16, 64, 16, seed=929), decode_ctas=400)


def test_decode_many_short_sequences(cuda_lib):
    rng = np.random.default_rng(5)
    kv = rng.integers(1, 70, 700).tolist()
    check_attention(workloads.build_batch([1] * 700, kv, 4, 2, 64, 16, seed=921))


def test_rows_of_very_different_sizes(cuda_lib):
    """Keys' and values' scales differ by 2^40 and more between tokens."""
    b = workloads.build_batch([1, 1, 40, 1], [600, 33, 300, 1500], 8, 2, 128, 16, seed=922)
    check_attention(b, spread=8)
    check_attention(b, spread=14, decode_ctas=3)


def test_tiny_and_huge_values(cuda_lib):
    """Values at both ends of the scales, with the probability at the small ones."""
    def edit(d):
        for s in range(d.b.num_seqs):
            pos = np.arange(int(d.b.kv_lens[s]))
            blk, off = d.b.block_table[s, pos // 16], pos % 16
            d.sc[blk, off, :, 1] = np.where(pos % 3 == 0, 95, 158)[:, None]
            d.sc[blk, off, :, 0] = np.where(pos % 3 == 0, 124, 110)[:, None]
    check_attention(workloads.build_batch([1, 1, 30], [200, 65, 90], 4, 2, 64, 16, seed=923), edit=edit)


def test_zero_queries_and_zero_rows(cuda_lib):
    b = workloads.build_batch([1, 20, 1], [100, 50, 3], 4, 2, 64, 16, seed=924)
    q = b.q.copy()
    q[0], q[5] = 0, 0
    kn = b.k_new.copy()
    kn[:] = 0
    check_attention(workloads.Batch(**{**b.__dict__, "q": q, "k_new": kn}))


def test_large_scores(cuda_lib):
    b = workloads.build_batch([1, 1, 150, 1], [600, 33, 300, 1500], 8, 2, 128, 64, seed=925, k_scale=16.0)
    check_attention(b)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (5, 1), (8, 4), (32, 8), (16, 1), (9, 3)])
def test_chunks(cuda_lib, Hq, Hkv, D):
    """Chunks alone and beside decodes: lengths around the 128-row tiles, prior context or none."""
    ql, kl = [2, 127, 128, 129, 300, 1, 1, 0, 33], [2, 500, 128, 1000, 300, 77, 1, 9, 1033]
    check_attention(workloads.build_batch(ql, kl, Hq, Hkv, D, 16, seed=930 + Hq))


@pytest.mark.parametrize("bs", [4, 5, 7, 48, 100, 256])
def test_chunk_block_sizes(cuda_lib, bs):
    check_attention(workloads.build_batch([70, 1, 200], [500, 40, 201], 4, 2, 128, bs, seed=940 + bs))


def test_chunks_long_context_and_serial(cuda_lib):
    b = workloads.build_batch([256, 1, 64], [5000, 3000, 64], 8, 2, 128, 32, seed=941)
    _, out, lse = check_attention(b)
    _, out2, lse2 = check_attention(b, serial=True, stream=torch.cuda.Stream())
    assert torch.equal(out[-64:].view(torch.int16), out2[-64:].view(torch.int16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("score", [dict(), dict(window=40, softcap=20.0)], ids=str)
def test_chunks_of_one_to_three_tiles(cuda_lib, D, score):
    """Many short items in a row on every CTA: one tile, two, three, and ends at and beside a tile's."""
    rng = np.random.default_rng(949)
    ql = [int(x) for x in rng.integers(2, 70, 90)]
    kv = [q + int(x) for q, x in zip(ql, rng.choice([0, 0, 1, 58, 60, 128, 186, 250], 90))]
    ql[:4], kv[:4] = [128, 129, 64, 2], [128, 129, 128, 257]
    check_attention(workloads.build_batch(ql, kv, 16, 8, D, 16, seed=949), **score)


@pytest.mark.parametrize("D,Hq,Hkv,bs", [(128, 8, 2, 16), (64, 15, 5, 7), (128, 16, 1, 64)])
def test_only_decodes_only_chunks_and_one_pass_after_the_other(cuda_lib, D, Hq, Hkv, bs):
    """Batches without work for one of the passes, and both passes in a row (serial): the same bits."""
    for ql, kv in (([1] * 5, [700, 1, 64, 2000, 33]), ([70, 2, 300], [70, 900, 1500]), ([1, 200, 1, 1], [4000, 900, 80, 7])):
        b = workloads.build_batch(ql, kv, Hq, Hkv, D, bs, seed=946)
        for score in (dict(), dict(window=100, softcap=9.0), dict(visible=[9999] * len(ql))):
            _, out, lse = check_attention(b, **score)
            _, out2, lse2 = check_attention(b, serial=True, stream=torch.cuda.Stream(), **score)
            assert torch.equal(out.view(torch.int16), out2.view(torch.int16)) and torch.equal(lse, lse2)
            check_attention(b, decode_ctas=1, **score)


@pytest.mark.parametrize("scale,cap", [(9e11, 1e8), (3e3, 1e-3)])
def test_scales_and_caps_far_apart(cuda_lib, scale, cap):
    """Zero queries: every score is 0, whatever the scale and the cap."""
    b = workloads.build_batch([1, 130, 3], [90, 300, 3], 4, 2, 64, 16, seed=947)
    b.q[...] = 0
    b.scale = scale
    d, out, _ = check_attention(b, softcap=cap)
    _, plain, _ = check_attention(b)  # (both off by 2^-8 in p and 2^-8 in the result)
    top = max(np.abs(d.cached(s)[1]).max() for s in range(3))
    assert (out.float() - plain.float()).abs().max() <= 4 * 2.0 ** -8 * top


def test_order_behind_other_work(cuda_lib):
    """On a stream whose earlier kernels still write what each call reads (the append's rows, the cache, the
    queries), calls and the results they leave for later ones, each call's own workspace and outputs new."""
    b = workloads.build_batch([1, 64, 1], [900, 700, 300], 8, 2, 128, 16, seed=948)
    d = QuantBatch(b)
    d.upload()
    big = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    want = [t.clone() for t in step_of(d, d.q, d.k_new, d.v_new)]
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.Stream()):
        d.upload()
        src = [d.q.clone(), d.k_new.clone(), d.v_new.clone()]
        late = [torch.full_like(t, float("nan")) for t in src]
        torch.cuda.synchronize()
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            for _ in range(4):
                big.add_(1)
            for t, x in zip(late, src):
                t.copy_(x)
            got = step_of(d, *late)
            keep = [t.clone() for t in got]
            for t in late:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        assert cb.get_device_error() == cb.CB_OK
        for x, y in zip(keep, want):
            assert torch.equal(x.float(), y.float())


def step_of(d, q, k, v):
    """Append, attention, read-back, and the step over the same rows: their outputs."""
    b = d.b
    cb.quant_append(None, k, v, *d.pools, *d.where)
    o1 = cb.quant_attention(q, *d.pools, *d.where, b.scale)
    cu = i32([0] + list(np.cumsum(b.kv_lens)))
    k1, v1 = cb.quant_gather(*d.pools, d.where[0], cu, b.block_size, int(sum(b.kv_lens)))
    o2 = cb.quant_append_attention(q, k, v, *d.pools, *d.where, b.scale)
    return o1, k1, v1, o2


def test_nan_rows(cuda_lib):
    """A key or value row with a value that is not finite is NaN as a whole; it makes the rows NaN that see
    it and no others (and the pools hold NaN rows in every slot that no sequence owns)."""
    b = workloads.build_batch([1, 140, 1, 1], [90, 200, 90, 40], 4, 2, 128, 16, seed=942)
    d = QuantBatch(b)
    d.append_new()
    for s, p, h, w in ((0, 50, 1, 0), (1, 130, 0, 0), (1, 40, 1, 1), (2, 89, 1, 1)):
        (d.v if w else d.k)[b.block_table[s, p // 16], p % 16, h] = 0x7F
        d.sc[b.block_table[s, p // 16], p % 16, h, w] = 255
    d.upload()
    out, lse = cb.quant_attention(d.q, *d.pools, *d.where, b.scale, lse=True)
    assert cb.get_device_error() == cb.CB_OK
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros_like(nan)
    want[0, 2:] = True                       # a key
    want[1 + 70:141, :2] = True              # of the queries that see it (the first is at position 60)
    want[1:141, 2:] = True                   # a value
    want[141, 2:] = True
    assert np.array_equal(nan, want)
    keys = want[..., 0].copy()
    keys[1:142, 2:] = False                  # (a value does not count for lse)
    assert np.array_equal(torch.isnan(lse).cpu().numpy(), keys)
    # stored by the append, read back
    x = opa.bf16_bits_to_f64(b.k_new).astype(np.float32)
    x[3, 0, 5], x[4, 1, 7] = np.inf, np.nan
    kn = bf16_tensor(workloads.f32_to_bf16_bits(x))
    cb.quant_append(None, kn, d.v_new, *d.pools, *d.where)
    ko, vo = cb.quant_gather(*d.pools, d.table, d.cu, 16, 143, key_starts=i32(b.kv_lens - b.q_lens))
    bad = np.zeros((143, 2), dtype=bool)
    bad[3, 0] = bad[4, 1] = True
    assert np.array_equal(torch.isnan(ko).all(-1).cpu().numpy(), bad)
    assert np.array_equal(torch.isnan(ko).any(-1).cpu().numpy(), bad) and not torch.isnan(vo).any()


# the changed scores
SLOPES = lambda h: [2.0 ** (-8.0 * (i + 1) / h) for i in range(h)]
MIXED = ([1, 37, 1, 130, 5, 1], [1, 37, 513, 700, 70, 1300])


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 8, 2), (128, 3, 1), (128, 32, 2)])
@pytest.mark.parametrize("score", [dict(softcap=2.0), dict(softcap=30.0), dict(slopes=True), dict(visible=True),
                                   dict(window=50), dict(softcap=5.0, slopes=True, visible=True),
                                   dict(softcap=5.0, slopes=True, window=200)], ids=str)
def test_changed_scores(cuda_lib, score, D, Hq, Hkv):
    score = dict(score)
    if "slopes" in score:
        score["slopes"] = SLOPES(Hq)
    if "visible" in score:
        score["visible"] = [1, 20, 100, 650, 0, 5000]
    check_attention(workloads.build_batch(*MIXED, Hq, Hkv, D, 16, seed=950 + D + Hq), **score)


# ------------------------------------------------------------------------------------ steps
@pytest.mark.parametrize("rot", [0, 64])
@pytest.mark.parametrize("D,Hq,Hkv,bs", [(64, 4, 2, 16), (128, 32, 8, 32), (128, 5, 5, 20)])
def test_step(cuda_lib, D, Hq, Hkv, bs, rot):
    """Append, attend and read back, in parts and in one call: the same bits, and the oracle's values."""
    b = workloads.build_batch([1, 37, 0, 5, 1, 130, 1], [1, 37, 9, 70, 513, 300, 65], Hq, Hkv, D, bs, seed=960 + D)
    a, c = QuantBatch(b), QuantBatch(b)
    cs = orope.table(600, rot) if rot else None
    csd = torch.from_numpy(cs).cuda() if rot else None
    q_rot = cb.quant_append(a.q if rot else None, a.k_new, a.v_new, *a.pools, *a.where, cos_sin=csd)
    q = q_rot if rot else a.q
    out, lse = cb.quant_attention(q, *a.pools, *a.where, b.scale, lse=True)
    out2, lse2 = cb.quant_append_attention(c.q, c.k_new, c.v_new, *c.pools, *c.where, b.scale, cos_sin=csd, lse=True)
    assert cb.get_device_error() == cb.CB_OK
    assert torch.equal(a.dk.view(torch.uint8), c.dk.view(torch.uint8))
    assert torch.equal(a.dv.view(torch.uint8), c.dv.view(torch.uint8)) and torch.equal(a.dsc, c.dsc)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
    assert torch.equal(lse.view(torch.int32), lse2.view(torch.int32))
    a.k, a.v, a.sc = (t.cpu().numpy() for t in (a.dk.view(torch.uint8), a.dv.view(torch.uint8), a.dsc))
    check_results(a, out, lse, q=f64(q))
    # read back what the step stored: the rotated keys, to the rounding of the codes
    n = b.q_lens
    ko, vo = cb.quant_gather(*a.pools, a.table, a.cu, bs, int(a.q.shape[0]), key_starts=i32(b.kv_lens - n))
    pos = orope.positions_of(b.cu_seqlens_q, b.kv_lens)
    k = opa.bf16_bits_to_f64(b.k_new)
    k = orope.rotate(k, pos, cs, False) if rot else k
    for got, x in ((f64(ko), k), (f64(vo), opa.bf16_bits_to_f64(b.v_new))):
        top = np.abs(x).max(-1, keepdims=True)
        # half a step, 2^-4 of the value, or 2^-10 of the scale (448 scales are below twice the largest)
        assert np.all(np.abs(got - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * top / 224) * (1 + 1e-4) + 1e-6 * top)


def test_steps_in_a_row_captured_and_replayed(cuda_lib):
    """Decode steps of a growing batch: eager, and captured once and replayed, give the same bits; two
    captured graphs share a workspace."""
    b = workloads.build_batch([1, 1, 1], [33, 289, 993], 8, 2, 128, 16, seed=970)  # (8 more fit their blocks)
    e, g = QuantBatch(b), QuantBatch(b)
    e.append_new(), g.append_new()
    e.upload(), g.upload()
    cs = torch.from_numpy(orope.table(1100, 128)).cuda()
    ws, out, rot = g.workspace(), torch.empty_like(g.q), torch.empty_like(g.q)
    call = lambda: cb.quant_append_attention(g.q, g.k_new, g.v_new, *g.pools, *g.where, b.scale, cos_sin=cs,
                                             q_out=rot, out=out, workspace=ws)
    call()                                   # (both caches hold the first step's rotated keys)
    cb.quant_append_attention(e.q, e.k_new, e.v_new, *e.pools, *e.where, b.scale, cos_sin=cs)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for x in graphs:
        with torch.cuda.graph(x):
            call()
    rng = torch.Generator(device="cuda").manual_seed(3)
    for step in range(6):
        new = [torch.randn(t.shape, generator=rng, device="cuda").bfloat16() for t in (e.q, e.k_new, e.v_new)]
        for d in (e, g):
            for t, x in zip((d.q, d.k_new, d.v_new), new):
                t.copy_(x)
            d.kv += 1
        want = cb.quant_append_attention(e.q, e.k_new, e.v_new, *e.pools, *e.where, b.scale, cos_sin=cs)
        graphs[step % 2].replay()
        assert cb.get_device_error() == cb.CB_OK
        assert torch.equal(want.view(torch.int16), out.view(torch.int16))
        assert torch.equal(e.dk.view(torch.uint8), g.dk.view(torch.uint8)) and torch.equal(e.dsc, g.dsc)


def test_attention_bad_metadata(cuda_lib):
    """Bad block ids and lengths are reported; the other sequences' rows are right."""
    b = workloads.build_batch([1, 1, 40, 1], [300, 90, 200, 40], 8, 2, 128, 16, seed=980)
    table = b.block_table.copy()
    table[0, 3], table[2, 5] = b.num_pages + 7, -5
    d = QuantBatch(b)
    d.append_new()
    d.upload()
    d.table = i32(table)
    out, lse = cb.quant_attention(d.q, *d.pools, *d.where, b.scale, lse=True)
    assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE
    o, l, q = f64(out), f64(lse), opa.bf16_bits_to_f64(b.q)
    for s, t in ((1, 1), (3, 42)):
        K, V = d.cached(s)
        check_rows(o[t:t + 1], l[t:t + 1], q[t:t + 1], K, V, int(b.kv_lens[s]) - 1, b.scale, P16, f"sequence {s}")
    d.table = i32(b.block_table)
    for name, value in (("kv", i32([300, 90, 20, 40])), ("cu", i32([0, 1, 2, 42, 50])),
                        ("kv", i32([300, 90000, 200, 40]))):
        keep = getattr(d, name)
        setattr(d, name, value)
        cb.quant_attention(d.q, *d.pools, *d.where, b.scale)
        assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE
        setattr(d, name, keep)


def test_padding_rows_are_left(cuda_lib):
    b = workloads.build_batch([1, 30, 1], [300, 90, 40], 8, 2, 64, 16, seed=981)
    d = QuantBatch(b)
    d.append_new()
    d.upload()
    q = torch.cat((d.q, torch.full((140, 8, 64), float("nan"), dtype=torch.bfloat16, device="cuda")))
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    cb.quant_attention(q, *d.pools, *d.where, b.scale, out=out, lse=lse)
    assert cb.get_device_error() == cb.CB_OK
    check_results(d, out[:32], lse[:32])
    assert (out[32:].float() == 7).all() and (lse[32:] == 7).all()


def test_far_slots(cuda_lib):
    """A pool of more than 2^31 bytes of codes: blocks at its end."""
    P, bs, hkv, D = 70000, 32, 8, 128
    k = torch.zeros((P, bs, hkv, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v, sc = k.clone(), torch.zeros((P, bs, hkv, 2), dtype=torch.uint8, device="cuda")
    kn, vn = (torch.randn(41, hkv, D, device="cuda").bfloat16() for _ in "kv")
    table, cu, kv = i32([[P - 1, P - 3]] * 1 + [[P - 2, P - 5]]), i32([0, 40, 41]), i32([40, 1])
    q = torch.randn(41, 2 * hkv, D, device="cuda").bfloat16()
    out = cb.quant_append_attention(q, kn, vn, k, v, sc, table, cu, kv, bs, D ** -0.5)
    ko, vo = cb.quant_gather(k, v, sc, table, cu, bs, 41)
    assert cb.get_device_error() == cb.CB_OK
    codes, s = oq.quantise(f64(kn))
    assert np.array_equal(f64(ko), oq.values(codes, s))
    K, V = f64(ko), f64(vo)
    check_rows(f64(out[:40]), None, f64(q[:40]), K[:40], V[:40], 0, D ** -0.5, P8, "chunk")
    assert np.abs(f64(out[40]) - np.repeat(V[40], 2, axis=0)).max() == 0


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(cuda_lib, seed):
    rng = np.random.default_rng(9000 + seed)
    hkv = int(rng.choice([1, 2, 3, 4, 5, 6, 8, 16]))
    g = int(rng.choice([1, 2, 3, 4, 7, 8])) if hkv != 4 else int(rng.choice([1, 9, 16]))
    S = int(rng.integers(1, 30))
    ql = [int(x) for x in rng.choice([0, 1, 1, 1, 1, 2, 9, 140], S)]
    kl = [n + int(rng.integers(0 if n else 1, 900)) for n in ql]
    b = workloads.build_batch(ql, kl, hkv * g, hkv, int(rng.choice([64, 128])), int(rng.choice([4, 7, 16, 40, 64])),
                              seed=seed)
    if sum(ql) == 0:
        return
    check_attention(b, spread=float(rng.choice([0, 2])), seed=seed, decode_ctas=int(rng.choice([0, 0, 3])))


def test_same_bits_on_every_call(cuda_lib):
    """Which CTA computes what depends on the GPU's state, the results do not."""
    b = workloads.build_batch([1] * 20 + [200, 1, 77], list(range(100, 2100, 100)) + [900, 5000, 333], 16, 2, 128, 32,
                              seed=990)
    d, out, lse = check_attention(b)
    for _ in range(10):
        o, l = cb.quant_attention(d.q, *d.pools, *d.where, b.scale, lse=True)
        assert torch.equal(o.view(torch.int16), out.view(torch.int16)) and torch.equal(l, lse)


def test_two_streams_at_once(cuda_lib):
    """Two batches on two streams, each with its workspace, over and over: as alone."""
    calls = []
    for i, (hq, hkv) in enumerate(((8, 2), (32, 8))):
        b = workloads.build_batch([1] * 8 + [90, 1], [700, 33, 1500, 64, 900, 10, 2000, 128, 400, 77], hq, hkv, 128, 16,
                                  seed=991 + i)
        d, out, _ = check_attention(b)
        calls.append((b, d, out, torch.cuda.Stream(), d.workspace(), torch.empty_like(out)))
    torch.cuda.synchronize()
    for _ in range(20):
        for b, d, out, stream, ws, o in calls:
            cb.quant_attention(d.q, *d.pools, *d.where, b.scale, out=o, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for b, d, out, _, _, o in calls:
        assert torch.equal(o.view(torch.int16), out.view(torch.int16))
    assert cb.get_device_error() == cb.CB_OK


def test_many_sequences_heads_and_keys(cuda_lib):
    rng = np.random.default_rng(7)
    ql = rng.choice([0, 1, 1, 2], 2500).tolist()
    kl = [n + int(x) for n, x in zip(ql, rng.integers(1, 30, 2500))]
    check_attention(workloads.build_batch(ql, kl, 2, 1, 64, 8, seed=993))
    check_attention(workloads.build_batch([1, 1, 20], [300, 40, 60], 80, 40, 64, 16, seed=994))
    check_attention(workloads.build_batch([1, 3], [70000, 66000], 2, 1, 64, 128, seed=995))


def test_served_by_the_scheduler(cuda_lib):
    """Requests served step by step over the 8-bit cache (the scheduler's lengths and block tables): every
    step's rows against the oracle's cache."""
    from continuous_batching_paged_gb300.runtime import BlockAllocator, Scheduler
    P, bs, hq, hkv, D, mb = 64, 16, 8, 2, 128, 12
    sched = Scheduler(BlockAllocator(P, bs, mb), max_batch_tokens=64, max_requests_per_batch=8)
    for i, (n, m) in enumerate(((70, 4), (5, 6), (33, 3))):
        sched.add_request(i, prompt_len=n, max_new_tokens=m)
    k = np.full((P, bs, hkv, D), 0x7F, dtype=np.uint8)
    v, sc = k.copy(), np.full((P, bs, hkv, 2), 255, dtype=np.uint8)
    dk, dv, dsc = (torch.from_numpy(x).cuda() for x in (k, v, sc))
    pools = dk.view(torch.float8_e4m3fn), dv.view(torch.float8_e4m3fn), dsc
    gen = torch.Generator(device="cuda").manual_seed(5)
    steps = 0
    while sched.num_active():
        step = sched.step()
        S = len(step["seq_ids"])
        if S == 0:
            continue
        T, cu, kv, table = int(step["num_tokens"]), step["cu_seqlens_q"], step["kv_lens"], step["block_table"]
        q, kn, vn = (torch.randn(T, h, D, generator=gen, device="cuda").bfloat16() for h in (hq, hkv, hkv))
        out, lse = cb.quant_append_attention(q, kn, vn, *pools, i32(table.copy()), i32(cu.copy()), i32(kv.copy()), bs,
                                             D ** -0.5, lse=True)
        assert cb.get_device_error() == cb.CB_OK
        codes = [oq.quantise(f64(x)) for x in (kn, vn)]
        for s in range(S):
            for t in range(int(cu[s]), int(cu[s + 1])):
                p = int(kv[s]) - int(cu[s + 1]) + t
                at = int(table[s, p // bs]), p % bs
                for w, pool in ((0, k), (1, v)):
                    pool[at], sc[at + (slice(None), w)] = codes[w][0][t], codes[w][1][t]
        for s in range(S):
            c0, c1 = int(cu[s]), int(cu[s + 1])
            if c1 > c0:
                pos = np.arange(int(kv[s]))
                blk, off = table[s, pos // bs], pos % bs
                K, V = oq.values(k[blk, off], sc[blk, off, :, 0]), oq.values(v[blk, off], sc[blk, off, :, 1])
                check_rows(f64(out[c0:c1]), f64(lse[c0:c1]), f64(q[c0:c1]), K, V, int(kv[s]) - (c1 - c0), D ** -0.5,
                           P16 if c1 - c0 == 1 else P8, f"step {steps}, sequence {s}")
        steps += 1
    assert steps >= 5
    assert np.array_equal(dk.cpu().numpy(), k) and np.array_equal(dsc.cpu().numpy(), sc)


def test_binding_refusals(cuda_lib):
    b = workloads.build_batch([1, 3], [40, 30], 4, 2, 64, 16, seed=996)
    d = QuantBatch(b)
    ok = dict(q=d.q, pools=d.pools, where=d.where)
    bad_sc = d.dsc[..., 0].contiguous()
    f = torch.float32
    attend = lambda q=d.q, pools=d.pools, where=d.where, **kw: cb.quant_attention(q, *pools, *where, 0.125, **kw)
    for match, call in [
            ("kv_scales must be", lambda: attend(pools=(d.dk, d.dv, bad_sc))),
            ("float8_e4m3fn", lambda: attend(pools=(d.dk.view(torch.uint8), d.dv, d.dsc))),
            ("match k_pages", lambda: attend(pools=(d.dk, d.dv[:3].contiguous(), d.dsc))),
            ("block_size", lambda: attend(where=(d.table, d.cu, d.kv, 8))),
            ("num_seqs \\+ 1", lambda: attend(where=(d.table, d.cu[:-1].contiguous(), d.kv, 16))),
            ("bfloat16", lambda: attend(q=d.q.float())),
            ("contiguous", lambda: attend(q=d.q.transpose(0, 1))),
            ("slopes must be", lambda: attend(slopes=torch.zeros(3, device="cuda"))),
            ("slopes must be", lambda: attend(slopes=torch.zeros(4, device="cuda", dtype=torch.float64))),
            ("visible_lens", lambda: attend(visible_lens=torch.zeros(3, device="cuda", dtype=torch.int32))),
            ("visible_lens", lambda: attend(visible_lens=torch.zeros(2, device="cuda"))),
            ("softcap", lambda: attend(softcap="5")),
            ("out must be", lambda: attend(out=torch.empty(4, 4, 128, device="cuda", dtype=torch.bfloat16))),
            ("lse must be", lambda: attend(lse=torch.empty(3, 4, device="cuda"))),
            ("workspace must be", lambda: attend(workspace=torch.empty(9, device="cuda"))),
            ("window", lambda: attend(window=2 ** 40)),
            ("q_out without q", lambda: cb.quant_append(None, d.k_new, d.v_new, *d.pools, *d.where, q_out=d.q)),
            ("k_new must be", lambda: cb.quant_append(None, d.k_new[:, :1], d.v_new[:, :1], *d.pools, *d.where)),
            ("v_new must match", lambda: cb.quant_append(None, d.k_new, d.v_new[:2], *d.pools, *d.where)),
            ("contiguous token rows", lambda: cb.quant_append(None, d.k_new[:1].expand(4, 2, 64), d.v_new, *d.pools, *d.where)),
            ("cos_sin must be", lambda: cb.quant_append(d.q, d.k_new, d.v_new, *d.pools, *d.where, cos_sin=torch.zeros(64, 64, device="cuda").double())),
            ("q_out without cos_sin", lambda: cb.quant_append_attention(d.q, d.k_new, d.v_new, *d.pools, *d.where, 0.125, q_out=d.q)),
            ("num_rows", lambda: cb.quant_gather(*d.pools, d.table, d.cu, 16, -1)),
            ("num_rows", lambda: cb.quant_gather(*d.pools, d.table, d.cu, 16, 2.5)),
            ("key_starts", lambda: cb.quant_gather(*d.pools, d.table, d.cu, 16, 4, key_starts=d.cu)),
            ("k_out must be", lambda: cb.quant_gather(*d.pools, d.table, d.cu, 16, 4, k_out=torch.empty(3, 2, 64, device="cuda", dtype=torch.bfloat16))),
            ("block_size", lambda: cb.quant_gather(*d.pools, d.table, d.cu, 8, 4))]:
        with pytest.raises(ValueError, match=match):
            call()
    for call in (lambda: cb.quant_append(d.q, d.k_new, d.v_new, *d.pools, *d.where),       # a q that nothing turns
                 lambda: attend(softcap=-1.0), lambda: attend(out=d.q),
                 lambda: attend(visible_lens=d.kv, window=4), lambda: attend(window=-3)):
        with pytest.raises(cb.CbError):
            call()
    assert cb.get_device_error() == cb.CB_OK
    # accepted: numpy integers, a view of wider rows, given outputs
    d.append_new()
    d.upload()
    out = torch.empty_like(d.q)
    assert attend(out=out, decode_ctas=np.int64(4), softcap=np.float32(0)) is out
    cb.quant_gather(*d.pools, d.table, d.cu, np.int32(16), np.int64(4))

"""The rotary append (cb_rope_append) against the float64 oracle and, bit for bit, against the same
fp32 arithmetic written with numpy; slots, padding rows, strides, device errors."""
import numpy as np
import pytest
import torch

import continuous_batching_paged_gb300 as cb
import workloads
from gpu_util import DeviceBatch, bf16_tensor, bits_of, i32, oracle_append
from oracle import paged_attention as opa
from oracle import rope as orope

pytestmark = pytest.mark.gpu


def rotate_fp32(bits, pos, cs, interleaved):
    """The operator's own arithmetic on bf16 bits: fp32 products and sums, each rounded, then bf16."""
    x = (bits.astype(np.uint32) << 16).view(np.float32).copy()
    rot = cs.shape[1]
    c, s = cs[pos][:, None, :rot // 2], cs[pos][:, None, rot // 2:]
    a, b = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
            else (slice(0, rot // 2), slice(rot // 2, rot)))
    xa, xb = x[..., a].copy(), x[..., b].copy()
    x[..., a] = xa * c - xb * s
    x[..., b] = xb * c + xa * s
    out = bits.copy()
    out[..., :rot] = workloads.f32_to_bf16_bits(x[..., :rot])
    return out


def bound_of(x, pos, cs, interleaved):
    """How far one rounded result may be from the exact one: half a bf16 step (2^-8 relative) and
    three fp32 roundings (2^-24 each) of terms no larger than |x c| + |y s|, the half step taken of
    the value so perturbed."""
    mag = np.abs(x).astype(np.float64)
    terms = mag.copy()
    for j, (a, b) in enumerate(orope.pairs(cs.shape[1], interleaved)):
        c, s = np.abs(cs[pos, j])[:, None], np.abs(cs[pos, cs.shape[1] // 2 + j])[:, None]
        terms[:, :, a] = mag[:, :, a] * c + mag[:, :, b] * s
        terms[:, :, b] = mag[:, :, b] * c + mag[:, :, a] * s
    return terms * (3 * 2.0 ** -24) * (1 + 2.0 ** -8)


def check(b, rot, interleaved, packed=False, in_place=False, keys_only=False, table_rows=None,
          stream=None):
    cs = orope.table(table_rows or int(b.kv_lens.max(initial=1)), rot)
    pos = orope.positions_of(b.cu_seqlens_q, b.kv_lens)
    db = DeviceBatch(b)
    q, kn, vn = db.q, db.k_new, db.v_new
    if packed:
        row = torch.cat((q, kn, vn), 1)
        q, kn, vn = row[:, :q.shape[1]], row[:, q.shape[1]:q.shape[1] + kn.shape[1]], \
            row[:, q.shape[1] + kn.shape[1]:]
    cs_dev = torch.from_numpy(cs).cuda()
    torch.cuda.synchronize()
    q_out = cb.rope_append(None if keys_only else q, kn, vn, db.k_pages, db.v_pages,
                           db.block_table, db.cu, db.kv_lens, b.block_size, cs_dev,
                           interleaved=interleaved, q_out=q if in_place else None, stream=stream)
    assert cb.get_device_error(stream) == cb.CB_OK
    # keys: the append oracle on the rotated rows; values: the append oracle
    rotated = workloads.Batch(**{**b.__dict__, "k_new": rotate_fp32(b.k_new, pos, cs, interleaved)})
    k_ref, v_ref = oracle_append(rotated)
    assert np.array_equal(bits_of(db.k_pages), k_ref)
    assert np.array_equal(bits_of(db.v_pages), v_ref)
    exact_k = orope.rotate(opa.bf16_bits_to_f64(b.k_new), pos, cs, interleaved)
    got_k = opa.bf16_bits_to_f64(rotated.k_new)     # what the pages hold, per token
    lim = 2.0 ** -8 * np.abs(exact_k) + bound_of(opa.bf16_bits_to_f64(b.k_new), pos, cs, interleaved)
    assert np.all(np.abs(got_k - exact_k) <= lim)
    if keys_only:
        assert q_out is None
        return
    got = bits_of(q_out)
    assert q_out.is_contiguous() and np.array_equal(got, rotate_fp32(b.q, pos, cs, interleaved))
    x = opa.bf16_bits_to_f64(b.q)
    exact = orope.rotate(x, pos, cs, interleaved)
    lim = 2.0 ** -8 * np.abs(exact) + bound_of(x, pos, cs, interleaved)
    assert np.all(np.abs(opa.bf16_bits_to_f64(got) - exact) <= lim)


# ragged mix: decodes, chunks crossing block boundaries, an empty sequence, a first token
RAGGED = ([1, 37, 0, 5, 1, 130, 1], [1, 37, 9, 70, 513, 300, 65])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 16),
                                   (128, 112)])
def test_rotations(cuda_lib, D, rot, interleaved):
    check(workloads.build_batch(*RAGGED, 8, 4, D, 16, seed=700 + rot), rot, interleaved)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (15, 5), (32, 8), (64, 8), (40, 40), (16, 1)])
@pytest.mark.parametrize("packed", [False, True])
def test_head_layouts_and_strides(cuda_lib, Hq, Hkv, packed):
    check(workloads.build_batch(*RAGGED, Hq, Hkv, 64 if Hq % 2 else 128, 32, seed=720 + Hq), 32,
          packed, packed=packed)


@pytest.mark.parametrize("bs", [4, 16, 64, 256, 12])
def test_block_sizes(cuda_lib, bs):
    check(workloads.build_batch(*RAGGED, 4, 2, 64, bs, seed=730 + bs), 64, False)


@pytest.mark.parametrize("T", [1, 2, 7, 31, 64, 257, 2048, 6000])
def test_token_counts(cuda_lib, T):
    # from one token (all warps on its heads) to one warp per token
    check(workloads.build_batch([T], [T + 13], 8, 2, 128, 32, seed=740 + T), 128, False, packed=True)


def test_many_sequences(cuda_lib):
    rng = np.random.default_rng(61)
    q_lens = [int(x) for x in rng.integers(0, 4, 3000)]
    kv_lens = [q + int(rng.integers(0, 40)) for q in q_lens]
    check(workloads.build_batch(q_lens, kv_lens, 4, 2, 64, 16, seed=62), 64, True)


def test_in_place_and_keys_only(cuda_lib):
    b = workloads.build_batch(*RAGGED, 8, 4, 128, 16, seed=750)
    check(b, 128, False, in_place=True)
    check(b, 64, True, in_place=True)
    check(b, 128, False, keys_only=True)
    check(b, 128, True, keys_only=True, packed=True)


def test_far_positions(cuda_lib):
    # positions around 200 000: the table's rows past 2^31 bytes are not reached here, but offsets
    # of position * rot_dim are 64-bit
    b = workloads.build_batch([1, 9], [200001, 150000], 2, 1, 64, 128, seed=751)
    check(b, 64, False)


def test_other_stream(cuda_lib):
    b = workloads.build_batch(*RAGGED, 8, 4, 128, 16, seed=752)
    check(b, 128, False, stream=torch.cuda.Stream())


def test_padding_rows_and_empty_batches(cuda_lib):
    b = workloads.build_batch([1, 3, 1], [40, 70, 9], 4, 2, 64, 16, seed=753)
    cs = torch.from_numpy(orope.table(128, 64)).cuda()
    db = DeviceBatch(b)
    pad = lambda t: torch.cat((t, torch.full((11,) + t.shape[1:], 3.0, dtype=t.dtype, device="cuda")))
    q_out = torch.full((16, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    cb.rope_append(pad(db.q), pad(db.k_new), pad(db.v_new), db.k_pages, db.v_pages, db.block_table,
                   db.cu, db.kv_lens, 16, cs, q_out=q_out)
    assert cb.get_device_error() == cb.CB_OK
    pos = orope.positions_of(b.cu_seqlens_q, b.kv_lens)
    assert np.array_equal(bits_of(q_out[:5]), rotate_fp32(b.q, pos, orope.table(128, 64), False))
    assert (q_out[5:].float() == 7.0).all()
    k_ref, _ = oracle_append(workloads.Batch(**{**b.__dict__, "k_new": rotate_fp32(
        b.k_new, pos, orope.table(128, 64), False)}))
    assert np.array_equal(bits_of(db.k_pages), k_ref)
    # no tokens, and tokens without a sequence: nothing happens
    e = workloads.build_batch([0, 0], [5, 9], 4, 2, 64, 16, seed=3)
    de = DeviceBatch(e)
    before = bits_of(de.k_pages).copy()
    out = cb.rope_append(de.q, de.k_new, de.v_new, de.k_pages, de.v_pages, de.block_table, de.cu,
                         de.kv_lens, 16, cs)
    assert out.shape == (0, 4, 64)
    out = torch.full((2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    cb.rope_append(torch.zeros_like(out), z, z, de.k_pages, de.v_pages, de.block_table[:0],
                   i32([0]), i32([]), 16, cs, q_out=out)
    assert cb.get_device_error() == cb.CB_OK
    assert (out.float() == 7.0).all() and np.array_equal(bits_of(de.k_pages), before)


def test_position_past_the_table_is_reported_and_skipped(cuda_lib):
    b = workloads.build_batch([2, 1], [20, 5], 4, 2, 64, 16, seed=5)
    cs = torch.from_numpy(orope.table(19, 64)).cuda()         # position 19 has no row
    db = DeviceBatch(b)
    before = bits_of(db.k_pages).copy()
    q_out = torch.full_like(db.q, 7.0)
    cb.rope_append(db.q, db.k_new, db.v_new, db.k_pages, db.v_pages, db.block_table, db.cu,
                   db.kv_lens, 16, cs, q_out=q_out)
    assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE
    assert cb.get_device_error() == cb.CB_OK
    changed = np.argwhere(np.any(bits_of(db.k_pages) != before, axis=(2, 3))).tolist()
    assert sorted(changed) == sorted([[int(b.block_table[0, 1]), 2], [int(b.block_table[1, 0]), 4]])
    assert (q_out[1].float() == 7.0).all() and not (q_out[0].float() == 7.0).any()


def test_bad_metadata_is_reported_and_skipped(cuda_lib):
    b = workloads.build_batch([2, 1], [20, 5], 4, 2, 64, 16, seed=5)
    cs = torch.from_numpy(orope.table(64, 64)).cuda()
    table = b.block_table.copy()
    table[0, 1] = b.num_pages + 3
    for field, value in (("block_table", i32(table)), ("kv_lens", i32([1, 5])),
                         ("cu", i32([0, 2, 1]))):
        db = DeviceBatch(b)
        setattr(db, field, value)
        before = bits_of(db.v_pages).copy()
        cb.rope_append(db.q, db.k_new, db.v_new, db.k_pages, db.v_pages, db.block_table, db.cu,
                       db.kv_lens, 16, cs)
        assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE, field
        changed = np.argwhere(np.any(bits_of(db.v_pages) != before, axis=(2, 3))).tolist()
        assert all(c in ([int(b.block_table[1, 0]), 4], [int(b.block_table[0, 1]), 2])
                   for c in changed), field


def test_captured_and_replayed(cuda_lib):
    b = workloads.build_batch([1, 40, 1], [33, 60, 500], 8, 2, 128, 16, seed=754)
    cs_np = orope.table(600, 128)
    cs = torch.from_numpy(cs_np).cuda()
    db = DeviceBatch(b)
    q_out = torch.empty_like(db.q)
    call = lambda: cb.rope_append(db.q, db.k_new, db.v_new, db.k_pages, db.v_pages,
                                  db.block_table, db.cu, db.kv_lens, 16, cs, q_out=q_out)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    b2 = workloads.build_batch([1, 40, 1], [34, 61, 501], 8, 2, 128, 16, seed=755)
    d2 = DeviceBatch(b2)
    for name in ("q", "k_new", "v_new", "kv_lens", "cu"):
        getattr(db, name).copy_(getattr(d2, name))
    db.block_table.copy_(d2.block_table)
    g.replay()
    assert cb.get_device_error() == cb.CB_OK
    pos = orope.positions_of(b2.cu_seqlens_q, b2.kv_lens)
    assert np.array_equal(bits_of(q_out), rotate_fp32(b2.q, pos, cs_np, False))


@pytest.mark.parametrize("which", ["q", "k_new", "v_new"])
def test_broadcast_rows_are_refused(cuda_lib, which):
    b = workloads.build_batch(*RAGGED, 8, 4, 128, 16, seed=770)
    db = DeviceBatch(b)
    rows = dict(q=db.q, k_new=db.k_new, v_new=db.v_new)
    rows[which] = rows[which][:1].expand_as(rows[which])
    cs = torch.from_numpy(orope.table(600, 128)).cuda()
    where = (db.k_pages, db.v_pages, db.block_table, db.cu, db.kv_lens, b.block_size)
    before = bits_of(db.k_pages)
    with pytest.raises(ValueError, match=f"{which} must have contiguous token rows"):
        cb.rope_append(*rows.values(), *where, cs)
    with pytest.raises(ValueError, match=f"{which} must have contiguous token rows"):
        cb.rope_append_attention(*rows.values(), *where, b.scale, cs)
    assert cb.get_device_error() == cb.CB_OK
    assert np.array_equal(bits_of(db.k_pages), before)

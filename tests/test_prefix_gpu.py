"""Attention over shared prefixes (cb_shared_prefix_attention) and the whole step
(cb_rope_append_attention) against the float64 oracle, which knows nothing of groups: it computes
every sequence alone over the keys its own block table names.

Elementwise bound on |gpu - ref|.  out = sum p v / sum p with p in (0, 1] rounded to bf16 for the
product (half a step: 2^-8 relative) and out rounded to bf16 (2^-8 of itself): 2^-8 |ref| +
2^-8 A (1 + 2^-8) with A = sum p |v| / sum p.  What fp32 adds is below a tenth of that: scores of
D <= 128 products, each |q k| summed in fp32 with relative error under 2^-20 of sum |q k| scale
(about 12 here, 48 with keys x4): 5e-5 absolute in the exponent at most, 1 % of 2^-8; the sums
and the merge a few 2^-24.  lse: that same 5e-5, and 2e-6 relative for the exponentials, the sum
and the logarithm."""
import numpy as np
import pytest
import torch

import continuous_batching_paged_gb300 as cb
import workloads
from gpu_util import bf16_tensor, bits_of, i32
from oracle import paged_attention as opa
from oracle import rope as orope

pytestmark = pytest.mark.gpu


def grouped_batch(q_lens, own, group, prefix, Hq, Hkv, D, bs, seed, k_scale=1.0, copies=False):
    """A batch whose sequence s holds its group's first prefix[g] keys, then own[s] >= q_lens[s] keys
    of its own (the last q_lens[s] appended already).  Members share the prefix's whole blocks, and
    hold a copy of its last, partial one (copies: of every block).  Slots past kv_len and unused
    blocks are NaN."""
    rng = np.random.default_rng(seed)
    kv = [o + (prefix[g] if g >= 0 else 0) for o, g in zip(own, group)]
    S, nblk = len(q_lens), [-(-k // bs) for k in kv]
    whole = [0 if copies else p // bs for p in prefix]
    pages = sum(whole) + sum(n - (whole[g] if g >= 0 else 0) for n, g in zip(nblk, group)) + 3
    ids = list(rng.permutation(pages))
    kp = np.full((pages, bs, Hkv, D), workloads.BF16_NAN, dtype=np.uint16)
    vp = kp.copy()
    draw = lambda n, sc=1.0: workloads.f32_to_bf16_bits(
        rng.standard_normal((n, Hkv, D), dtype=np.float32) * np.float32(sc))
    pk, pv = [draw(p, k_scale) for p in prefix], [draw(p) for p in prefix]
    common = [[ids.pop() for _ in range(n)] for n in whole]
    table = np.full((S, max(nblk, default=1) + 2), -1, dtype=np.int32)
    for s in range(S):
        g = group[s]
        row = (common[g] if g >= 0 else [])[:nblk[s]]
        row = row + [ids.pop() for _ in range(nblk[s] - len(row))]
        table[s, :len(row)] = row
        k, v = draw(kv[s], k_scale), draw(kv[s])
        if g >= 0:
            k[:prefix[g]], v[:prefix[g]] = pk[g], pv[g]
        for j, blk in enumerate(row):
            n = min(bs, kv[s] - j * bs)
            kp[blk, :n], vp[blk, :n] = k[j * bs:j * bs + n], v[j * bs:j * bs + n]
    cu = np.concatenate(([0], np.cumsum(q_lens))).astype(np.int32)
    q = workloads.f32_to_bf16_bits(rng.standard_normal((int(cu[-1]), Hq, D), dtype=np.float32))
    return dict(q=q, kp=kp, vp=vp, table=table, cu=cu, kv=np.array(kv, dtype=np.int32),
                group=np.array(group, dtype=np.int32), prefix=np.array(prefix, dtype=np.int32),
                bs=bs, scale=D ** -0.5)


class Dev:
    def __init__(self, b):
        self.b = b
        self.q, self.kp, self.vp = bf16_tensor(b["q"]), bf16_tensor(b["kp"]), bf16_tensor(b["vp"])
        self.table, self.cu, self.kv = i32(b["table"]), i32(b["cu"]), i32(b["kv"])
        self.group, self.prefix = i32(b["group"]), i32(b["prefix"])

    def workspace(self):
        """Exactly the size asked for, every byte 0xFF: a read of what was never written shows."""
        n = cb.prefix_workspace_size(self.kv.numel(), self.q.shape[1], self.kp.shape[2],
                                     self.q.shape[2], self.q.shape[0], self.prefix.numel())
        return torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def attend(self, **kw):
        kw.setdefault("lse", True)
        kw.setdefault("workspace", self.workspace())
        return cb.shared_prefix_attention(self.q, self.kp, self.vp, self.table, self.cu, self.kv,
                                          self.b["bs"], self.b["scale"], self.group, self.prefix, **kw)


def reference(b, rows=None):
    """Oracle output, A (its |V| average) and lse; NaN slots are never read by it."""
    args = (b["table"], b["cu"], b["kv"], b["bs"], b["scale"])
    ref, lse = opa.ragged_paged_attention(b["q"], b["kp"], b["vp"], *args)
    mag, _ = opa.ragged_paged_attention(b["q"], b["kp"], b["vp"] & np.uint16(0x7FFF), *args)
    return ref, mag, lse


def assert_matches(out, lse, b, what=""):
    ref, mag, ref_lse = reference(b)
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all(), what
    lim = 2.0 ** -8 * np.abs(ref) + 1.1 * 2.0 ** -8 * mag
    bad = np.abs(got - ref) > lim
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float((np.abs(got - ref) / lim).max()))
    if lse is not None:
        err = np.abs(lse.cpu().numpy().astype(np.float64) - ref_lse)
        assert np.all(err <= 5e-5 + 2e-6 * np.abs(ref_lse)), (what, float(err.max()))


def check(b, **kw):
    d = Dev(b)
    out, lse = d.attend(**kw)
    assert cb.get_device_error() == cb.CB_OK
    assert_matches(out, lse, b)
    return d, out, lse


# 11 sequences: two groups, two loners, in no order
Q11 = [1] * 11
OWN11 = [5, 1, 33, 140, 17, 2, 64, 9, 300, 1, 48]
GRP11 = [0, 1, -1, 0, 1, 0, 0, -1, 1, 0, 0]


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (6, 2), (5, 5), (8, 2), (10, 2), (14, 2), (32, 8),
                                    (64, 8), (24, 2), (16, 1), (32, 16), (36, 12)])
@pytest.mark.parametrize("D", [64, 128])
def test_head_layouts(cuda_lib, Hq, Hkv, D):
    if Hkv == 12:
        Hq, Hkv = 144, 12                              # 12 query heads each, 12 KV heads (3 x 4)
    check(grouped_batch(Q11, OWN11, GRP11, [200, 333], Hq, Hkv, D, 16, seed=800 + Hq))


@pytest.mark.parametrize("bs", [4, 8, 12, 16, 32, 64, 128, 256])
def test_block_sizes(cuda_lib, bs):
    check(grouped_batch(Q11, OWN11, GRP11, [200, 333], 8, 2, 128, bs, seed=820 + bs))


@pytest.mark.parametrize("prefix", [0, 1, 127, 128, 129, 255, 256, 257, 511, 512, 640])
def test_prefix_lengths(cuda_lib, prefix):
    # below 128 keys nothing is shared; own = 1: the prefix is the whole prior context
    check(grouped_batch([1] * 5, [1, 1, 7, 100, 1], [0] * 5, [prefix], 8, 2, 64, 16,
                        seed=840 + prefix))


def test_query_lengths(cuda_lib):
    # members of no, 1 .. 8 (shared) and more query tokens (the chunk pass), one short of a tile and
    # more than one tile among them
    q = [0, 1, 2, 3, 8, 9, 130, 5, 1, 0, 7, 4]
    own = [4, 1, 2, 30, 8, 20, 131, 50, 17, 0, 90, 4]
    grp = [0, 0, 0, 1, 1, 1, 0, -1, 0, 1, 1, -1]
    check(grouped_batch(q, own, grp, [260, 150], 8, 2, 128, 16, seed=860))
    check(grouped_batch(q, own, grp, [260, 150], 3, 1, 64, 32, seed=861))
    check(grouped_batch(q, own, grp, [260, 150], 16, 1, 64, 8, seed=862))


@pytest.mark.parametrize("Hq,Hkv,n", [(8, 2, 31), (8, 2, 32), (8, 2, 33), (8, 2, 64), (8, 2, 65),
                                      (8, 2, 300), (3, 1, 43), (16, 1, 17), (1, 1, 300)])
def test_tile_borders(cuda_lib, Hq, Hkv, n):
    # around one and two tiles of query rows, and many tiles
    rng = np.random.default_rng(n)
    own = [1 + int(x) for x in rng.integers(0, 40, n)]
    check(grouped_batch([1] * n, own, [0] * n, [300], Hq, Hkv, 64, 16, seed=870 + n))


@pytest.mark.parametrize("decode_ctas,serial", [(0, False), (1, False), (7, False), (512, False),
                                                (0, True), (3, True)])
def test_split_prefixes(cuda_lib, decode_ctas, serial):
    # few rows and long prefixes: parts of the prefix, and of the own keys, merged by whoever is last
    b = grouped_batch([1, 1, 1, 2, 1, 1], [900, 3, 1500, 40, 1, 20], [0, 0, 1, 1, -1, 0],
                      [9000, 5001], 8, 2, 128, 32, seed=880)
    check(b, decode_ctas=decode_ctas, serial=serial)


def test_long_prefix_of_64k(cuda_lib):
    check(grouped_batch([1] * 5, [3, 50, 1, 900, 12], [0] * 5, [65536 + 77], 4, 1, 64, 64, seed=881))


def test_many_groups(cuda_lib):
    n, rng = 120, np.random.default_rng(5)
    order = [int(x) for x in rng.permutation([g for g in range(n) for _ in range(2)])]
    prefix = [int(x) for x in rng.integers(100, 400, n)]
    check(grouped_batch([1] * 240, [1 + int(x) for x in rng.integers(0, 30, 240)], order, prefix, 4,
                        2, 64, 16, seed=882))


def test_more_sequences_and_groups_than_planner_threads(cuda_lib):
    n, rng = 1100, np.random.default_rng(6)
    group = [i % n for i in range(2 * n + 50)]
    prefix = [int(x) for x in rng.integers(120, 140, n)]
    check(grouped_batch([1] * len(group), [1 + (i % 5) for i in range(len(group))], group, prefix, 2,
                        1, 64, 16, seed=883))


def test_groups_that_share_nothing(cuda_lib):
    own = [40, 200, 3, 77]
    q = [1, 1, 1, 70]
    for group, prefix in (([-1] * 4, [100]), ([0, 1, 2, 3], [150, 200, 128, 500]), ([-1] * 4, []),
                          ([3, 3, -1, -1], [-5, 1 << 30, 0, 129])):
        full = [p if 0 <= p < 1000 else 0 for p in prefix]
        b = grouped_batch(q, own, group, full, 8, 2, 128, 16, seed=884)
        b["prefix"] = np.array(prefix, dtype=np.int32)      # a group without members may say anything
        check(b)


def test_members_with_copies_of_the_prefix(cuda_lib):
    check(grouped_batch([1] * 6, [3, 1, 40, 9, 200, 5], [0] * 6, [400], 8, 2, 128, 16, seed=885,
                        copies=True))


def test_large_scores(cuda_lib):
    check(grouped_batch(Q11, OWN11, GRP11, [200, 1333], 8, 2, 128, 16, seed=886, k_scale=4.0))


def test_rescaled_running_maximum(cuda_lib):
    # scores that grow along the prefix and into the own keys, by far more than the lazy rescale's
    # step, and own keys far above or below the prefix's
    b = grouped_batch([1] * 4, [30, 30, 30, 30], [0] * 4, [1000], 4, 1, 64, 16, seed=887)
    kp = opa.bf16_bits_to_f64(b["kp"])
    for s in range(4):
        for j, blk in enumerate(b["table"][s][b["table"][s] >= 0]):
            if s == 0 or j >= 1000 // 16:
                pos = np.arange(j * 16, j * 16 + 16)[:, None, None]
                grow = np.where(pos < 1000, 0.02 + pos / 250.0, [0.01, 8.0, 1.0, 4.0][s])
                kp[blk] = kp[blk] * grow
    # only whole shared blocks were scaled the same for all; make the partial block a copy again
    last = [int(t[1000 // 16]) for t in b["table"]]
    for blk in last[1:]:
        kp[blk, :1000 % 16] = kp[last[0], :1000 % 16]
    bits = workloads.f32_to_bf16_bits(kp.astype(np.float32))
    b["kp"] = bits
    ref, mag, ref_lse = reference(b)
    d = Dev(b)
    out, lse = d.attend()
    assert cb.get_device_error() == cb.CB_OK
    got = out.float().cpu().numpy().astype(np.float64)
    # scores here reach |q||k| = 8 * 8 * 8: the fp32 part of the bound grows by that over 12
    lim = 2.0 ** -8 * np.abs(ref) + 1.6 * 2.0 ** -8 * mag
    assert np.all(np.abs(got - ref) <= lim), float((np.abs(got - ref) / lim).max())
    assert np.all(np.abs(lse.cpu().numpy() - ref_lse) <= 5e-4 + 2e-6 * np.abs(ref_lse))


def test_same_results_every_time_and_in_any_order(cuda_lib):
    b = grouped_batch([1] * 40, [1 + 13 * i % 90 for i in range(40)], [i % 2 for i in range(40)],
                      [700, 2100], 8, 2, 128, 16, seed=888)
    d, out, lse = check(b)
    for _ in range(5):
        out2, lse2 = d.attend()
        assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
        assert torch.equal(lse, lse2)
    alone = cb.ragged_paged_attention(d.q, d.kp, d.vp, d.table, d.cu, d.kv, b["bs"], b["scale"])
    assert_matches(alone, None, b)


def test_lse_left_out_and_outputs_given(cuda_lib):
    b = grouped_batch(Q11, OWN11, GRP11, [200, 333], 8, 2, 128, 16, seed=889)
    d, out, _ = check(b)
    mine = torch.full_like(out, 7.0)
    got = d.attend(lse=None, out=mine)
    assert got is mine and torch.equal(mine.view(torch.int16), out.view(torch.int16))


def test_padding_rows_and_sequences(cuda_lib):
    b = grouped_batch(Q11, OWN11, GRP11, [200, 333], 8, 2, 128, 16, seed=890)
    d, out, lse = check(b)
    pad = dict(b)
    pad["q"] = np.concatenate((b["q"], np.full((9,) + b["q"].shape[1:], workloads.BF16_NAN, np.uint16)))
    pad["cu"] = np.concatenate((b["cu"], np.full(5, b["cu"][-1], np.int32)))
    pad["kv"] = np.concatenate((b["kv"], np.zeros(5, np.int32)))
    pad["group"] = np.concatenate((b["group"], np.array([0, 99, -7, 1, -1], np.int32)))  # not looked at
    pad["table"] = np.concatenate((b["table"], np.full((5, b["table"].shape[1]), -1, np.int32)))
    p = Dev(pad)
    o, l = torch.full_like(p.q, 7.0), torch.full(p.q.shape[:2], 7.0, device="cuda")
    p.attend(out=o, lse=l)
    assert cb.get_device_error() == cb.CB_OK
    assert_matches(o[:11], l[:11], b)
    assert (o[11:].float() == 7.0).all() and (l[11:] == 7.0).all()


@pytest.mark.parametrize("field,index,value", [("group", 3, 2), ("group", 3, -2), ("prefix", 0, 336),
                                               ("prefix", 1, -1)])
def test_bad_groups_are_reported(cuda_lib, field, index, value):
    # sequence 9 has a prior context of 200 keys: a prefix of 336 is too long for it
    b = grouped_batch(Q11, OWN11, GRP11, [200, 333], 8, 2, 128, 16, seed=891)
    b[field][index] = value
    d = Dev(b)
    out, lse = d.attend()
    assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE
    assert cb.get_device_error() == cb.CB_OK
    assert_matches(out, lse, b)        # (such a batch is computed without sharing)


def test_bad_lengths_and_blocks_are_reported(cuda_lib):
    b = grouped_batch(Q11, OWN11, GRP11, [200, 333], 8, 2, 128, 16, seed=892)
    for field, at, value in (("kv", 4, 0), ("kv", 4, 1 << 20), ("cu", 3, 30), ("cu", 5, -3),
                             ("table", (0, 2), 1 << 20), ("table", (9, 12), -1)):
        bad = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in b.items()}
        bad[field][at] = value
        d = Dev(bad)
        d.attend()
        assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE, field
    check(b)


def test_two_streams_with_a_workspace_each(cuda_lib):
    batches = [grouped_batch([1] * 30, [1 + 7 * i for i in range(30)], [0] * 30, [2000 + 500 * k], 8,
                             2, 128, 16, seed=893 + k) for k in range(2)]
    devs = [Dev(b) for b in batches]
    ws, streams = [d.workspace() for d in devs], [torch.cuda.Stream() for _ in devs]
    torch.cuda.synchronize()
    res = [None, None]
    for _ in range(5):
        for k in range(2):
            res[k] = devs[k].attend(workspace=ws[k], stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert_matches(*res[k], batches[k])
    # and with memory of the call's own
    res = [d.attend(workspace=None, stream=s) for d, s in zip(devs, streams)]
    torch.cuda.synchronize()
    assert cb.get_device_error() == cb.CB_OK
    for k in range(2):
        assert_matches(*res[k], batches[k])


def test_captured_and_replayed_with_other_groups(cuda_lib):
    # one graph serves any lengths and groups of its shape: the plan is made on the device
    b = grouped_batch(Q11, OWN11, GRP11, [200, 333], 8, 2, 128, 16, seed=895)
    d = Dev(b)
    ws, out = d.workspace(), torch.empty_like(d.q)
    lse = torch.empty(d.q.shape[:2], dtype=torch.float32, device="cuda")
    d.attend(workspace=ws, out=out, lse=lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.attend(workspace=ws, out=out, lse=lse)
    wide = d.table.shape[1]
    for k, (own, grp, prefix) in enumerate([(OWN11, GRP11, [200, 333]),
                                            ([1] * 11, [1] * 11, [0, 300]),
                                            ([9] * 11, [-1] * 11, [0, 0]),
                                            ([30] * 11, [0, 1] * 5 + [0], [129, 300])]):
        b2 = grouped_batch(Q11, own, grp, prefix, 8, 2, 128, 16, seed=896 + k)
        n = b2["kp"].shape[0]
        assert n <= d.kp.shape[0]
        t = np.full((11, wide), -1, np.int32)
        t[:, :b2["table"].shape[1]] = b2["table"]
        d.kp[:n].copy_(bf16_tensor(b2["kp"]))
        d.vp[:n].copy_(bf16_tensor(b2["vp"]))
        for dst, src in ((d.table, t), (d.kv, b2["kv"]), (d.group, b2["group"]),
                         (d.prefix, b2["prefix"])):
            dst.copy_(i32(src))
        d.q.copy_(bf16_tensor(b2["q"]))
        g.replay()
        assert cb.get_device_error() == cb.CB_OK
        assert_matches(out, lse, b2, f"replay {k}")


@pytest.mark.parametrize("groups", [True, False])
@pytest.mark.parametrize("serial", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (16, 1, 64)])
def test_step_equals_its_parts(cuda_lib, groups, serial, Hq, Hkv, D):
    # rotate + append + attend in one call: bit for bit the two calls one after the other
    q = [1, 2, 1, 40, 1, 1, 8, 1]
    own = [5, 2, 33, 41, 17, 2, 64, 9]
    b = grouped_batch(q, own, [0, 1, -1, 0, 1, 0, 0, 1], [200, 333], Hq, Hkv, D, 16, seed=897)
    d = Dev(b)
    rng = np.random.default_rng(898)
    T = d.q.shape[0]
    qkv = bf16_tensor(workloads.f32_to_bf16_bits(
        rng.standard_normal((T, Hq + 2 * Hkv, D), dtype=np.float32)))
    qv, kn, vn = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cs_np = orope.table(int(b["kv"].max()), 64)
    cs = torch.from_numpy(cs_np).cuda()
    pools = [(d.kp.clone(), d.vp.clone()) for _ in range(2)]
    where = lambda p: (*p, d.table, d.cu, d.kv, 16)
    rot = cb.rope_append(qv, kn, vn, *where(pools[0]), cs)
    kw = dict(lse=True, serial=serial)
    if groups:
        out, lse = cb.shared_prefix_attention(rot, *where(pools[0]), b["scale"], d.group, d.prefix,
                                              **kw)
        kw.update(prefix_group=d.group, prefix_lens=d.prefix)
    else:
        out, lse = cb.ragged_paged_attention(rot, *where(pools[0]), b["scale"], **kw)
    q_out = torch.empty_like(rot)
    out2, lse2 = cb.rope_append_attention(qv, kn, vn, *where(pools[1]), b["scale"], cs, q_out=q_out,
                                          **kw)
    assert cb.get_device_error() == cb.CB_OK
    for x, y in ((rot, q_out), (out, out2), *zip(*pools)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert torch.equal(lse, lse2)
    # and against the oracle on what the pages hold now
    assert_matches(out2, lse2, {**b, "q": bits_of(rot), "kp": bits_of(pools[1][0]),
                                "vp": bits_of(pools[1][1])})


def test_window_with_step_but_not_with_groups(cuda_lib):
    b = grouped_batch([1, 20, 1], [300, 100, 9], [-1, -1, -1], [], 8, 2, 128, 16, seed=899)
    d = Dev(b)
    kn = torch.randn(22, 2, 128, device="cuda").bfloat16()
    cs = torch.from_numpy(orope.table(301, 128)).cuda()
    args = (d.q, kn, kn.clone(), d.kp, d.vp, d.table, d.cu, d.kv, 16, b["scale"], cs)
    out = cb.rope_append_attention(*args, window=50)
    rot = cb.rope_append(*args[:9], cs)
    ref = cb.ragged_paged_attention(rot, d.kp, d.vp, d.table, d.cu, d.kv, 16, b["scale"], window=50)
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    with pytest.raises(cb.CbError, match="window"):
        cb.rope_append_attention(*args, window=50, prefix_group=i32([0, 0, -1]),
                                 prefix_lens=i32([8]))
    assert cb.get_device_error() == cb.CB_OK


def test_empty_batches(cuda_lib):
    d = Dev(grouped_batch([0, 0], [5, 9], [0, 0], [130], 4, 2, 64, 16, seed=3))
    out, lse = d.attend()
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert cb.get_device_error() == cb.CB_OK


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (4, 1), (8, 2), (5, 1), (8, 1), (12, 1)])
def test_verified_tokens_share_records(cuda_lib, Hq, Hkv):
    # up to 8 query tokens of a member: 8 / G of them in one record of the decode pass, whose tokens
    # see different numbers of own keys; own lengths put those edges inside a 16-key tile, at its
    # border, and into a tile of which the first tokens see nothing
    rng = np.random.default_rng(Hq)
    q = [1 + i % 8 for i in range(48)]
    own = [n + int(x) for n, x in zip(q, rng.integers(0, 40, 48))]
    own[:8] = [1, 2, 3, 4, 5, 6, 7, 8]                       # nothing but this step's tokens
    group = [i % 2 for i in range(48)]
    # prefix ends at tile borders and beside them
    for prefix in ([256, 144], [131, 271]):
        for ctas in (0, 40):
            b = grouped_batch(q, own, group, prefix, Hq, Hkv, 64, 16, seed=910 + Hq)
            check(b, decode_ctas=ctas)
    # (slots behind kv_len are NaN)
    check(grouped_batch([8, 7, 8], [8, 39, 41], [0, 0, 0], [144], Hq, Hkv, 128, 16, seed=911))


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (3, 1, 64), (16, 1, 64), (5, 5, 128)])
@pytest.mark.parametrize("prefix", [128, 200, 384, 1000])
def test_chunks_of_a_group(cuda_lib, Hq, Hkv, D, prefix):
    # members with more than 8 query tokens: the prefix with the group's other tokens, the own keys in
    # the chunk pass from the prefix's end on; own lengths from the chunk itself to several tiles more
    q = [9, 1, 128, 129, 300, 1, 40, 8]
    own = [9, 4, 128, 400, 300, 30, 41, 8]
    b = grouped_batch(q, own, [0, 0, 0, 0, 0, -1, -1, 0], [prefix], Hq, Hkv, D, 16, seed=920 + prefix)
    check(b)
    check(b, serial=True)


def test_chunks_too_many_to_share(cuda_lib):
    # enough chunk items to fill the GPU: the chunks are computed alone, the other members share
    b = grouped_batch([700, 1, 600, 3, 1], [800, 4, 600, 9, 70], [0, 0, 0, 0, 0], [300], 64, 8, 64, 32,
                      seed=930)
    check(b)
    # one chunk alone in its group, and a group of nothing but chunks
    check(grouped_batch([200, 1, 30, 45], [201, 9, 30, 60], [0, -1, 1, 1], [260, 400], 8, 2, 64, 16,
                        seed=931))


def test_nothing_left_for_the_decode_pass(cuda_lib):
    # every token is one of several of its sequence: own keys are groups of their own, in and outside
    # of the groups, and no sequence has a decode record
    q = [3, 8, 2, 5, 40, 8, 2]
    own = [3, 30, 200, 129, 300, 8, 500]
    for Hq, Hkv, D in ((8, 2, 128), (8, 1, 64), (5, 5, 64), (12, 1, 64)):
        for grp in ([0, 0, 0, 0, 0, -1, -1], [-1] * 7, [0, 1, 0, 1, -1, 0, 1]):
            check(grouped_batch(q, own, grp, [300, 140], Hq, Hkv, D, 16, seed=940 + Hq))


def test_more_sequences_than_the_planner_sees_at_once(cuda_lib):
    # beyond 256 sequences several tokens of a member take several records
    rng = np.random.default_rng(9)
    q = [int(x) for x in rng.integers(1, 9, 300)]
    own = [n + int(x) for n, x in zip(q, rng.integers(0, 30, 300))]
    grp = [int(x) for x in rng.integers(-1, 3, 300)]
    check(grouped_batch(q, own, grp, [200, 150, 400], 4, 1, 64, 16, seed=950))
    check(grouped_batch(q[:256], own[:256], grp[:256], [200, 150, 400], 4, 1, 64, 16, seed=951))


@pytest.mark.parametrize("n", [40, 200, 600])
def test_tiles_of_a_group_are_the_same_on_every_call(cuda_lib, n):
    # 2 to 19 tiles of a group: were a token now in a unit of two tiles, now in the last one, its
    # parts would be rounded differently
    rng = np.random.default_rng(n)
    q = [int(x) for x in rng.integers(1, 4, n)]
    own = [k + int(x) for k, x in zip(q, rng.integers(0, 20, n))]
    b = grouped_batch(q, own, [int(x < 0.8) for x in rng.random(n)], [150, 900], 8, 2, 64, 16, seed=960)
    d, out, lse = check(b)
    busy = torch.randn(4096, 4096, device="cuda")
    for i in range(12):
        if i % 2:
            busy @ busy  # (another neighbour on the stream)
        out2, lse2 = d.attend()
        assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
        assert torch.equal(lse, lse2)


def test_pages_past_32_bit_offsets(cuda_lib):
    # the last pages of pools of 2^32 elements and more: same bits as in a small pool
    b = grouped_batch([1, 3, 1, 1, 40, 1], [30, 9, 200, 1, 45, 17], [0, 0, 0, -1, 0, 0], [300], 8, 8, 128,
                      64, seed=961)
    d = Dev(b)
    out, lse = d.attend()
    n = d.kp.shape[0]
    far = 2 ** 32 // (64 * 8 * 128) + n
    pools = []
    for near in (d.kp, d.vp):
        pool = torch.empty((far, 64, 8, 128), dtype=torch.bfloat16, device="cuda")
        pool[far - n:] = near
        pools.append(pool)
    table = torch.where(d.table >= 0, d.table + (far - n), d.table)
    out2, lse2 = cb.shared_prefix_attention(d.q, *pools, table, d.cu, d.kv, 64, b["scale"], d.group,
                                            d.prefix, lse=True)
    assert cb.get_device_error() == cb.CB_OK
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16)) and torch.equal(lse, lse2)
    # and the rotary append into them
    kn = torch.randn(d.q.shape[0], 8, 128, device="cuda").bfloat16()
    cs = torch.from_numpy(orope.table(int(b["kv"].max()), 128)).cuda()
    rot = cb.rope_append(d.q, kn, kn.flip(0), d.kp, d.vp, d.table, d.cu, d.kv, 64, cs)
    rot2 = cb.rope_append(d.q, kn, kn.flip(0), *pools, table, d.cu, d.kv, 64, cs)
    assert cb.get_device_error() == cb.CB_OK
    assert torch.equal(rot.view(torch.int16), rot2.view(torch.int16))
    for near, pool in zip((d.kp, d.vp), pools):
        assert torch.equal(near.view(torch.int16), pool[far - n:].view(torch.int16))


def test_steps_in_a_row_and_the_same_sequence_twice(cuda_lib):
    # layer after layer without a wait between them, into the same workspace: each call starts early
    # behind the one before; and two entries of the batch that are the same sequence
    b = grouped_batch([1] * 30, [1 + 7 * i for i in range(30)], [i % 3 - 1 for i in range(30)],
                      [400, 333], 8, 2, 128, 16, seed=962)
    b["table"][5], b["kv"][5] = b["table"][2], b["kv"][2]  # (both of group 1)
    b["q"][5] = b["q"][2]
    d = Dev(b)
    ws = d.workspace()
    q = [d.q, d.q.flip(0).contiguous()]
    alone = []
    for x in q:
        alone.append(cb.shared_prefix_attention(x, d.kp, d.vp, d.table, d.cu, d.kv, 16, b["scale"], d.group,
                                                d.prefix))
        torch.cuda.synchronize()
    assert_matches(alone[0], None, b)
    outs = [cb.shared_prefix_attention(q[i % 2], d.kp, d.vp, d.table, d.cu, d.kv, 16, b["scale"], d.group,
                                       d.prefix, workspace=ws) for i in range(40)]
    for i, o in enumerate(outs):
        assert torch.equal(o.view(torch.int16), alone[i % 2].view(torch.int16)), i
    assert cb.get_device_error() == cb.CB_OK


@pytest.mark.parametrize("first,step", [(0.0, 0.3), (0.0, 0.1), (90.0, -0.3), (-40.0, 0.36), (5.0, 1.0)])
@pytest.mark.parametrize("decode_ctas", [0, 1])
def test_own_scores_that_climb_and_fall(cuda_lib, first, step, decode_ctas):
    # the score of own key j is first + step j: per tile of 16 keys the running maximum grows by less and
    # by more than the 2^8 at which it is followed (0.3 x 16 log2(e) = 6.9, 0.36: 8.3), or never again
    b = grouped_batch([1] * 3, [300, 77, 16], [0] * 3, [208], 1, 1, 64, 16, seed=970)
    q = opa.bf16_bits_to_f64(b["q"])
    kp = opa.bf16_bits_to_f64(b["kp"])
    for s in range(3):
        along = q[s, 0] / (q[s, 0] @ q[s, 0]) / b["scale"]
        for j in range(208 // 16, int(b["kv"][s] + 15) // 16):
            n = min(16, int(b["kv"][s]) - j * 16)
            score = first + step * (j * 16 - 208 + np.arange(n))
            kp[b["table"][s][j], :n, 0] = score[:, None] * along
    b["kp"] = workloads.f32_to_bf16_bits(kp.astype(np.float32))
    # (scores reach 300: the fp32 sums are off by 300 x 2^-20 = 2.9e-4, 7 % of 2^-8)
    ref, mag, ref_lse = reference(b)
    out, lse = Dev(b).attend(decode_ctas=decode_ctas)
    assert cb.get_device_error() == cb.CB_OK
    got = out.float().cpu().numpy().astype(np.float64)
    lim = 2.0 ** -8 * np.abs(ref) + 1.1 * 2.0 ** -8 * mag
    assert np.all(np.abs(got - ref) <= lim), float((np.abs(got - ref) / lim).max())
    assert np.all(np.abs(lse.cpu().numpy() - ref_lse) <= 3e-4 + 2e-6 * np.abs(ref_lse))


@pytest.mark.parametrize("bs", [5, 6, 9, 10, 14])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (1, 1, 64)])
def test_block_sizes_with_odd_factors(cuda_lib, bs, Hq, Hkv, D):
    # blocks that a tile of 128 keys is cut into runs of one or two keys for: a group with one tile of
    # rows, one with two and one with three, keys that end inside a tile and at its border ...
    rng = np.random.default_rng(bs)
    n = [9, 130 // (Hq // Hkv) + 3, 2 * 128 // (Hq // Hkv) + 5]
    group = [g for g in range(3) for _ in range(n[g])] + [-1, -1]
    own = [1 + int(x) for x in rng.integers(0, 30, len(group))]
    check(grouped_batch([1] * len(group), own, group, [515, 384, 201], Hq, Hkv, D, bs, seed=1010 + bs))
    # ... and own keys of several tokens as groups with a causal edge, drafts and chunks
    b = grouped_batch([8, 3, 1, 40, 130, 8, 2], [300, 700, 4, 90, 400, 200, 8], [0, 0, 0, 0, -1, -1, 0],
                      [260], Hq, Hkv, D, bs, seed=1020 + bs)
    check(b)
    check(b, serial=True)


@pytest.mark.parametrize("bs", [5, 6])
def test_bad_blocks_in_runs_of_one_or_two_keys(cuda_lib, bs):
    b = grouped_batch(Q11, OWN11, GRP11, [200, 333], 8, 2, 128, bs, seed=1030)
    b["table"][0, 3], b["table"][1, 20] = 1 << 20, -1
    Dev(b).attend()
    assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE
    assert cb.get_device_error() == cb.CB_OK


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (2, 1), (3, 1), (4, 1), (8, 1), (16, 1)])
@pytest.mark.parametrize("n", [1, 5, 40, 256, 257, 300])
def test_a_call_stays_inside_its_workspace(cuda_lib, Hq, Hkv, n):
    # every sequence with 8 tokens, which take as many records or chains as there can be, with the own
    # keys short (records) and long (groups of their own), and chunks beside them
    for own, extra in ((9, []), (400, []), (30, [200, 90])):
        q = [8] * n + extra
        b = grouped_batch(q, [own + i % 7 for i in range(n)] + [x + 20 for x in extra],
                          [i % 2 for i in range(n)] + [-1] * len(extra), [140, 260], Hq, Hkv, 64, 16,
                          seed=1040 + n)
        d = Dev(b)
        need = d.workspace().numel()
        ws = torch.full((need + (1 << 20),), 255, dtype=torch.uint8, device="cuda")
        out, lse = d.attend(workspace=ws)
        assert cb.get_device_error() == cb.CB_OK
        assert (ws[need:] == 255).all()
        assert_matches(out, lse, b)

"""Attention with changed scores and masks on the bf16 cache (cb_scored_attention) against the float64
oracle, and without changes against the plain call."""
import numpy as np
import pytest
import torch

import continuous_batching_paged_gb300 as cb
import workloads
from gpu_util import DeviceBatch, i32, oracle_append
from oracle import paged_attention as opa
from quant_util import P8, check_rows, f64

pytestmark = pytest.mark.gpu

MIXED = ([1, 37, 1, 130, 5, 1, 0], [1, 37, 513, 700, 70, 1300, 12])
VISIBLE = [1, 20, 100, 650, 0, 5000, 3]


def slopes_of(h):
    return [2.0 ** (-8.0 * (i + 1) / h) for i in range(h)]


def check(b, stream=None, serial=False, decode_ctas=0, **score):
    d = DeviceBatch(b)
    d.append()
    kw = dict(score)
    if "slopes" in kw:
        kw["slopes"] = torch.tensor(kw["slopes"], dtype=torch.float32, device="cuda")
    if "visible_lens" in kw:
        kw["visible_lens"] = i32(kw["visible_lens"])
    out = torch.full_like(d.q, float("nan"))
    lse = torch.full(d.q.shape[:2], float("nan"), dtype=torch.float32, device="cuda")
    ws = torch.full((max(256, cb.workspace_size(b.num_seqs, b.num_q_heads, b.num_kv_heads, b.head_dim,
                                                b.num_tokens)),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    cb.scored_attention(d.q, d.k_pages, d.v_pages, d.block_table, d.cu, d.kv_lens, b.block_size, b.scale,
                        out=out, lse=lse, workspace=ws, stream=stream, serial=serial,
                        decode_ctas=decode_ctas, **kw)
    assert cb.get_device_error(stream) == cb.CB_OK
    kp, vp = oracle_append(b)
    o, l, q = f64(out), f64(lse), opa.bf16_bits_to_f64(b.q)
    for s in range(b.num_seqs):
        c0, c1, kv = int(b.cu_seqlens_q[s]), int(b.cu_seqlens_q[s + 1]), int(b.kv_lens[s])
        if c1 > c0:
            K, V = (opa.gather_kv(p, b.block_table[s], kv, b.block_size) for p in (kp, vp))
            check_rows(o[c0:c1], l[c0:c1], q[c0:c1], K, V, kv - (c1 - c0), b.scale, P8, f"sequence {s}",
                       score.get("softcap", 0.0),
                       np.asarray(score["slopes"], dtype=np.float32) if "slopes" in score else None,
                       score["visible_lens"][s] if "visible_lens" in score else 0, score.get("window", 0))
    return d, out, lse


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 8, 2), (128, 3, 1), (128, 32, 2), (64, 15, 5)])
@pytest.mark.parametrize("score", [dict(softcap=2.0), dict(softcap=50.0), dict(slopes=True),
                                   dict(visible_lens=True), dict(softcap=5.0, slopes=True, visible_lens=True),
                                   dict(softcap=5.0, slopes=True, window=200), dict(window=50)], ids=str)
def test_changes(cuda_lib, score, D, Hq, Hkv):
    score = dict(score)
    if "slopes" in score:
        score["slopes"] = slopes_of(Hq)
    if "visible_lens" in score:
        score["visible_lens"] = VISIBLE
    check(workloads.build_batch(*MIXED, Hq, Hkv, D, 16, seed=600 + D + Hq), **score)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 32, 8), (128, 16, 1)])
def test_without_changes_it_is_the_plain_call(cuda_lib, D, Hq, Hkv):
    b = workloads.build_batch(*MIXED, Hq, Hkv, D, 16, seed=610)
    d, out, lse = check(b)
    want, want_lse = d.attend(lse=True)
    # (the scores are scaled before, not within, the exponent's multiply-add)
    assert torch.allclose(out.float(), want.float(), rtol=2.0 ** -7, atol=2.0 ** -9)
    assert torch.allclose(lse, want_lse, rtol=1e-6, atol=2e-6)


def test_large_scores_are_capped(cuda_lib):
    """Scores far beyond the cap, where tanh is 1, and large ones without a cap."""
    b = workloads.build_batch(*MIXED, 8, 2, 128, 16, seed=620, k_scale=64.0)
    check(b, softcap=10.0)
    check(b, softcap=0.5)
    check(b, softcap=1e6)


@pytest.mark.parametrize("scale,cap", [(9e11, 1e8), (1e30, 1e30), (1e-30, 1e-3), (1e-6, 1e20), (3e3, 1e-3)])
def test_scales_and_caps_far_apart(cuda_lib, scale, cap):
    """Zero queries: every score is 0, whatever the scale and the cap, and a row is the mean of its values."""
    b = workloads.build_batch([1, 130, 3], [90, 300, 3], 4, 2, 64, 16, seed=625)
    b.q[...] = 0
    b.scale = scale
    _, out, _ = check(b, softcap=cap)
    vp = oracle_append(b)[1]
    top = max(np.abs(opa.gather_kv(vp, b.block_table[s], int(b.kv_lens[s]), 16)).max() for s in range(3))
    _, plain, _ = check(b, softcap=0.0)  # (both off by 2^-8 in p and 2^-8 in the result)
    assert (out.float() - plain.float()).abs().max() <= 4 * 2.0 ** -8 * top


def test_only_decodes_only_chunks_and_one_pass_after_the_other(cuda_lib):
    """Batches without work for one of the passes, and both passes in a row (serial): the same bits."""
    for ql, kv in (([1] * 5, [700, 1, 64, 2000, 33]), ([70, 2, 300], [70, 900, 1500]), ([1, 200, 1, 1], [4000, 900, 80, 7])):
        b = workloads.build_batch(ql, kv, 8, 2, 128, 16, seed=626)
        for score in (dict(softcap=3.0), dict(slopes=slopes_of(8), window=100), dict(visible_lens=[9999] * len(ql))):
            _, out, lse = check(b, **score)
            _, out2, lse2 = check(b, serial=True, stream=torch.cuda.Stream(), **score)
            assert torch.equal(out.view(torch.int16), out2.view(torch.int16)) and torch.equal(lse, lse2)
            check(b, decode_ctas=1, **score)


def test_positive_and_zero_slopes(cuda_lib):
    b = workloads.build_batch(*MIXED, 8, 2, 64, 16, seed=630)
    check(b, slopes=[0.0, 0.5, -0.5, 0.01, -0.01, 1.0, -1.0, 0.125])


def test_visible_lens_cover_tiles_and_ends(cuda_lib):
    """Prefixes that end before, in and after the chunk, at tile borders, and beyond the sequence."""
    for ctx in (0, 200):
        ql = [300] * 7
        kv = [300 + ctx] * 7
        vis = [-5, 0, 1, ctx + 128, ctx + 129, ctx + 300, 100000]
        for hq in (2, 3):
            check(workloads.build_batch(ql, kv, hq, 1, 64, 16, seed=640 + ctx), visible_lens=vis)


def test_long_context_and_other_stream(cuda_lib):
    b = workloads.build_batch([200, 1, 1], [4000, 9000, 64], 8, 2, 128, 32, seed=650)
    check(b, softcap=30.0, slopes=slopes_of(8), stream=torch.cuda.Stream())


def test_padding_rows_and_graph(cuda_lib):
    b = workloads.build_batch([1, 30, 1], [300, 90, 40], 8, 2, 64, 16, seed=660)
    d = DeviceBatch(b)
    d.append()
    q = torch.cat((d.q, torch.full((140, 8, 64), float("nan"), dtype=torch.bfloat16, device="cuda")))
    out = torch.full_like(q, 7.0)
    sl, vis = torch.tensor(slopes_of(8), device="cuda"), i32([5, 80, 0])
    ws = torch.empty(cb.workspace_size(3, 8, 2, 64, 172), dtype=torch.uint8, device="cuda")
    call = lambda: cb.scored_attention(q, d.k_pages, d.v_pages, d.block_table, d.cu, d.kv_lens, 16, b.scale,
                                       softcap=4.0, slopes=sl, visible_lens=vis, out=out, workspace=ws)
    call()
    assert cb.get_device_error() == cb.CB_OK
    assert (out[32:].float() == 7).all()
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    out.fill_(7.0)
    g.replay()
    assert torch.equal(first.view(torch.int16), out.view(torch.int16))
    vis.fill_(0)                              # the lengths are read when the graph runs
    g.replay()
    torch.cuda.synchronize()
    changed = (first != out).any(-1).any(-1).cpu()
    assert changed[1:30].any() and not changed[[0, 31]].any()


def test_bad_metadata_is_reported(cuda_lib):
    b = workloads.build_batch([1, 30, 1], [300, 90, 40], 8, 2, 64, 16, seed=661)
    d = DeviceBatch(b)
    d.append()
    table = b.block_table.copy()
    table[1, 1] = b.num_pages
    cb.scored_attention(d.q, d.k_pages, d.v_pages, i32(table), d.cu, d.kv_lens, 16, b.scale, softcap=3.0)
    assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE
    assert cb.get_device_error() == cb.CB_OK

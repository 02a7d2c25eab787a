"""Block moves of the quantised cache: codes and scales bit for bit, what attends to them before and after, and
requests that share blocks served step by step."""
import random

import numpy as np
import pytest
import torch

import continuous_batching_paged_gb300 as cb
import workloads
from continuous_batching_paged_gb300.runtime import BlockAllocator, Scheduler
from gpu_util import i32
from oracle import blocks as ob
from oracle import quant as oq
from quant_util import P8, P16, QuantBatch, check_rows, f64

pytestmark = pytest.mark.gpu

# block size, KV heads, head_dim: a block's scales are 8, 10, 12, 30, 256 and 128 bytes
SHAPES = [(4, 1, 64), (5, 1, 128), (6, 1, 64), (5, 3, 64), (16, 8, 128), (64, 1, 128)]


def pools(P, bs, H, D, seed):
    rng = np.random.default_rng(seed)
    host = [rng.integers(0, 256, (P, bs, H, n), dtype=np.uint8) for n in (D, D, 2)]
    dev = [torch.from_numpy(x).cuda() for x in host]
    return host, (dev[0].view(torch.float8_e4m3fn), dev[1].view(torch.float8_e4m3fn), dev[2])


def same(dev, host):
    return all(np.array_equal(t.view(torch.uint8).cpu().numpy(), x) for t, x in zip(dev, host))


@pytest.mark.parametrize("bs,H,D", SHAPES)
def test_copy(cuda_lib, bs, H, D):
    P = 97
    host, (k, v, sc) = pools(P, bs, H, D, seed=bs + H + D)
    perm = np.random.default_rng(7).permutation(P)
    src, dst = np.append(perm[:30], perm[70]), np.append(perm[30:60], perm[70])  # (the last pair: a no-op)
    cb.copy_blocks(k, v, i32(src), i32(dst), bs, kv_scales=sc)
    assert cb.get_device_error() == cb.CB_OK
    want = [ob.copy_blocks(x, src, dst) for x in host]
    assert same((k, v, sc), want)
    # a bad id: reported, and its pair alone left out
    cb.copy_blocks(k, v, i32([1, 2, 3]), i32([5, P + 4, 6]), bs, kv_scales=sc)
    assert cb.get_device_error() == cb.CB_ERR_OUT_OF_RANGE
    assert same((k, v, sc), [ob.copy_blocks(x, [1, 3], [5, 6]) for x in want])


@pytest.mark.parametrize("bs,H,D", SHAPES)
def test_offload_and_restore(cuda_lib, bs, H, D):
    P, n = 300, 77
    host, (k, v, sc) = pools(P, bs, H, D, seed=11)
    blocks = np.random.default_rng(12).permutation(P)[:n]
    others = np.setdiff1d(np.arange(P), blocks)[:n]
    hk, hv = (torch.empty(n, bs, H, D, dtype=torch.float8_e4m3fn).pin_memory() for _ in "kv")
    hs = torch.empty(n, bs, H, 2, dtype=torch.uint8).pin_memory()
    cb.kv_offload(k, v, i32(blocks), bs, hk, hv, kv_scales=sc, host_scales=hs)
    assert cb.get_device_error() == cb.CB_OK
    out = [ob.gather_blocks(x, blocks) for x in host]
    assert all(np.array_equal(t.view(torch.uint8).numpy(), x) for t, x in zip((hk, hv, hs), out))
    cb.kv_restore(k, v, i32(others), bs, hk, hv, kv_scales=sc, host_scales=hs)
    assert cb.get_device_error() == cb.CB_OK
    assert same((k, v, sc), [ob.scatter_blocks(x, others, y) for x, y in zip(host, out)])


def test_a_moved_request_gives_the_same_bits(cuda_lib):
    b = workloads.build_batch([1, 60, 1], [300, 200, 90], 8, 2, 128, 16, seed=997)
    d = QuantBatch(b, spread=3)
    d.append_new()
    d.upload()
    attend = lambda table: cb.quant_attention(d.q, *d.pools, i32(table), d.cu, d.kv, 16, b.scale, softcap=30.0, lse=True)
    want = attend(b.block_table)
    used = np.concatenate([b.block_table[s, :-(-int(b.kv_lens[s]) // 16)] for s in range(3)])
    free = np.setdiff1d(np.arange(b.num_pages), used)
    table = b.block_table.copy()
    src = table[0, :2].copy()
    table[0, :2] = free[:2]                                 # copied on write
    cb.copy_blocks(d.dk, d.dv, i32(src), i32(free[:2]), 16, kv_scales=d.dsc)
    got = attend(table)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # a request's blocks out, their place overwritten, and back into the same places
    mine = table[1, :13]
    hk, hv = (torch.empty(13, 16, 2, 128, dtype=torch.float8_e4m3fn).pin_memory() for _ in "kv")
    hs = torch.empty(13, 16, 2, 2, dtype=torch.uint8).pin_memory()
    cb.kv_offload(d.dk, d.dv, i32(mine), 16, hk, hv, kv_scales=d.dsc, host_scales=hs)
    torch.cuda.synchronize()
    for t in (d.dk, d.dv, d.dsc):
        t.view(torch.uint8)[torch.from_numpy(mine.astype(np.int64)).cuda()] = 0x33
    cb.kv_restore(d.dk, d.dv, i32(mine), 16, hk, hv, kv_scales=d.dsc, host_scales=hs)
    got = attend(table)
    assert cb.get_device_error() == cb.CB_OK
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_served_with_shared_blocks(cuda_lib):
    """Requests that are forked while they run: the scheduler's copy-on-write pairs, the step, and the oracle's
    cache after every step."""
    P, bs, hq, hkv, D, mb = 200, 16, 8, 2, 64, 16
    rng = random.Random(17)
    sched = Scheduler(BlockAllocator(P, bs, mb), max_batch_tokens=96, max_requests_per_batch=8)
    for r in range(6):
        sched.add_request(r, rng.randint(1, 90), rng.randint(4, 14))
    (k, v, sc), dev = pools(P, bs, hkv, D, seed=19)
    gen = torch.Generator(device="cuda").manual_seed(5)
    next_id, steps, copies = 100, 0, 0
    while sched.num_active():
        step = sched.step()
        steps += 1
        S = len(step["seq_ids"])
        if S:
            src, dst = step["cow_src"].copy(), step["cow_dst"].copy()
            if len(src):
                copies += len(src)
                cb.copy_blocks(dev[0], dev[1], i32(src), i32(dst), bs, kv_scales=dev[2])
                k, v, sc = (ob.copy_blocks(x, src, dst) for x in (k, v, sc))
            T, cu, kv, table = (int(step["num_tokens"]), step["cu_seqlens_q"].copy(), step["kv_lens"].copy(),
                                step["block_table"].copy())
            q, kn, vn = (torch.randn(T, h, D, generator=gen, device="cuda").bfloat16() for h in (hq, hkv, hkv))
            out, lse = cb.quant_append_attention(q, kn, vn, *dev, i32(table), i32(cu), i32(kv), bs, D ** -0.5, lse=True)
            assert cb.get_device_error() == cb.CB_OK
            for w, (x, pool) in enumerate(((kn, k), (vn, v))):
                codes, e = oq.quantise(f64(x))
                for s in range(S):
                    for t in range(int(cu[s]), int(cu[s + 1])):
                        p = int(kv[s]) - int(cu[s + 1]) + t
                        at = int(table[s, p // bs]), p % bs
                        pool[at], sc[at + (slice(None), w)] = codes[t], e[t]
            for s in range(S):
                c0, c1 = int(cu[s]), int(cu[s + 1])
                pos = np.arange(int(kv[s]))
                blk, off = table[s, pos // bs], pos % bs
                K, V = oq.values(k[blk, off], sc[blk, off, :, 0]), oq.values(v[blk, off], sc[blk, off, :, 1])
                if c1 > c0:
                    check_rows(f64(out[c0:c1]), f64(lse[c0:c1]), f64(q[c0:c1]), K, V, int(kv[s]) - (c1 - c0), D ** -0.5,
                               P16 if c1 - c0 == 1 else P8, f"step {steps}, sequence {s}")
            ids = [int(x) for x, n in zip(step["seq_ids"], np.diff(cu)) if n == 1]
            if steps % 4 == 2 and ids:
                try:
                    sched.fork_request(ids[0], next_id, rng.randint(3, 9))
                    next_id += 1
                except cb.CbError:
                    pass  # (the parent is at its last token)
        assert steps < 300
    assert copies > 0 and same(dev, (k, v, sc))


def test_refusals(cuda_lib):
    _, (k, v, sc) = pools(20, 16, 2, 64, seed=1)
    ids, bf = i32([1, 2]), torch.zeros(20, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    hk = torch.empty(2, 16, 2, 64, dtype=torch.float8_e4m3fn).pin_memory()
    hs = torch.empty(2, 16, 2, 2, dtype=torch.uint8).pin_memory()
    for match, call in [
            ("kv_scales must be given", lambda: cb.copy_blocks(k, v, ids, ids, 16)),
            ("bfloat16", lambda: cb.copy_blocks(bf, v, ids, ids, 16)),
            ("float8_e4m3fn", lambda: cb.copy_blocks(k, bf, ids, ids, 16, kv_scales=sc)),
            ("float8_e4m3fn", lambda: cb.copy_blocks(bf, bf, ids, ids, 16, kv_scales=sc)),
            ("kv_scales must be", lambda: cb.copy_blocks(k, v, ids, ids, 16, kv_scales=sc[:3])),
            ("same length", lambda: cb.copy_blocks(k, v, ids, i32([1]), 16, kv_scales=sc)),
            ("host_scales must be", lambda: cb.kv_offload(k, v, ids, 16, hk, hk, kv_scales=sc)),
            ("host_scales must be", lambda: cb.kv_offload(k, v, ids, 16, hk, hk, kv_scales=sc, host_scales=hs[:1])),
            ("host_k must be", lambda: cb.kv_restore(k, v, ids, 16, hk[:1], hk, kv_scales=sc, host_scales=hs)),
            ("host_scales without", lambda: cb.kv_restore(bf, bf, i32([1]), 16, hk, hk, host_scales=hs)),
            ("block_size", lambda: cb.copy_blocks(k, v, ids, ids, 8, kv_scales=sc))]:
        with pytest.raises(ValueError, match=match):
            call()
    assert cb.get_device_error() == cb.CB_OK

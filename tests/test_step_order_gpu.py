"""The per-step calls behind other work: their launches may start before the launch ahead of them ends,
and must see what came before all the same, whatever it is (a copy, a memset, another stream's work that
the stream waits for, the call before), eager and captured."""
import numpy as np
import pytest
import torch

import continuous_batching_paged_gb300 as cb
import workloads
from gpu_util import DeviceBatch, bits_of, i32
from oracle import rope as orope

pytestmark = pytest.mark.gpu

SLOW = 2_000_000                                        # cycles: about 1 ms


class Step:
    def __init__(self, seed):
        self.b = workloads.build_batch([1, 40, 1, 3], [200, 60, 170, 300], 8, 2, 128, 16, seed=seed)
        d = self.d = DeviceBatch(self.b)
        d.block_table[2, :8] = d.block_table[0, :8]     # the first 128 keys in common
        self.cs = torch.from_numpy(orope.table(512, 128)).cuda()
        self.group, self.lens = i32([0, -1, 0, -1]), i32([128])
        self.fresh = torch.randn_like(d.q)
        self.out, self.rot = torch.empty_like(d.q), torch.empty_like(d.q)
        self.ws = torch.empty(cb.prefix_workspace_size(4, 8, 2, 128, d.q.shape[0], 1), dtype=torch.uint8,
                              device="cuda")
        self.call("rope_append")                        # (the pages hold this step's keys and values)

    def call(self, name):
        d = self.d
        where = (d.k_pages, d.v_pages, d.block_table, d.cu, d.kv_lens, 16)
        kw = dict(out=self.out, workspace=self.ws)
        if name == "rope_append":
            return cb.rope_append(d.q, d.k_new, d.v_new, *where, self.cs, q_out=self.out)
        if name == "shared_prefix_attention":
            return cb.shared_prefix_attention(d.q, *where, self.b.scale, self.group, self.lens, **kw)
        groups = dict(prefix_group=self.group, prefix_lens=self.lens) if "groups" in name else {}
        return cb.rope_append_attention(d.q, d.k_new, d.v_new, *where, self.b.scale, self.cs,
                                        q_out=self.rot, **kw, **groups)


CALLS = ["rope_append", "shared_prefix_attention", "step", "step with groups"]


def _before(s, how, side, host):
    """Queue work that ends with q == s.fresh."""
    q = s.d.q
    if how == "copy":
        torch.cuda._sleep(SLOW)
        q.copy_(s.fresh)
    elif how == "copy from the host":
        torch.cuda._sleep(SLOW)
        q.copy_(host, non_blocking=True)
    elif how == "kernel":
        torch.cuda._sleep(SLOW)
        torch.add(s.fresh, 0, out=q)
    elif how == "memset behind a kernel":               # (of the output: rows that the call writes whole)
        torch.cuda._sleep(SLOW)
        torch.add(s.fresh, 0, out=q)
        s.out.zero_()
    else:                                               # another stream, with a call just before
        if how == "other stream behind a call":
            s.call("rope_append")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(SLOW)
            torch.add(s.fresh, 0, out=q)
        torch.cuda.current_stream().wait_stream(side)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("how", ["copy", "copy from the host", "kernel", "memset behind a kernel",
                                 "other stream", "other stream behind a call"])
@pytest.mark.parametrize("name", CALLS)
def test_sees_the_work_before_it(cuda_lib, name, how, captured):
    s = Step(1100)
    host, stale = s.fresh.cpu().pin_memory(), torch.zeros_like(s.fresh)
    s.d.q.copy_(s.fresh)
    expect = bits_of(s.call(name))
    assert s.out.isfinite().all()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph() if captured else None
    torch.cuda.synchronize()
    if captured:
        with torch.cuda.graph(graph):
            _before(s, how, side, host)
            s.call(name)
    for _ in range(3):
        s.d.q.copy_(stale)
        s.out.fill_(7.0)
        torch.cuda.synchronize()
        if captured:
            graph.replay()
        else:
            _before(s, how, side, host)
            s.call(name)
        after = s.out.clone()                           # (and work behind the call waits for it)
        torch.cuda.synchronize()
        assert cb.get_device_error() == cb.CB_OK
        same = np.array_equal(bits_of(after), expect)
        assert same


@pytest.mark.parametrize("name", CALLS)
def test_other_stream_waits_for_the_call(cuda_lib, name):
    # an event behind the call: what another stream does after it sees the results
    s, side = Step(1101), torch.cuda.Stream()
    s.d.q.copy_(s.fresh)
    expect = bits_of(s.call(name))
    assert s.out.isfinite().all()
    for _ in range(5):
        s.out.fill_(7.0)
        torch.cuda.synchronize()
        torch.cuda._sleep(SLOW)
        s.call(name)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = s.out.clone()
        torch.cuda.synchronize()
        same = np.array_equal(bits_of(got), expect)
        assert same
    assert cb.get_device_error() == cb.CB_OK

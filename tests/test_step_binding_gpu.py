"""The C++ binding of the per-step calls: streams by their handles, and arguments as users hand them
over (integers of other types, integers that no length can be)."""
import numpy as np
import pytest
import torch

import continuous_batching_paged_gb300 as cb
import workloads
from gpu_util import DeviceBatch, bits_of, i32
from oracle import rope as orope

pytestmark = pytest.mark.gpu


class Step:
    """A ragged batch of three sequences, two of them a group, and the three calls on it."""

    def __init__(self, seed):
        self.b = workloads.build_batch([1, 5, 1], [200, 60, 170], 8, 2, 128, 16, seed=seed)
        self.d = DeviceBatch(self.b)
        self.cs = torch.from_numpy(orope.table(256, 128)).cuda()
        self.group, self.lens = i32([0, -1, 0]), i32([128])
        self.d.block_table[2, :8] = self.d.block_table[0, :8]      # the first 128 keys in common
        self.call("rope_append")                                   # (the pages hold this step's rows)

    def call(self, name, block_size=16, **kw):
        d = self.d
        where = (d.k_pages, d.v_pages, d.block_table, d.cu, d.kv_lens, block_size)
        if name == "rope_append":
            return cb.rope_append(d.q, d.k_new, d.v_new, *where, self.cs, **kw)
        if name == "shared_prefix_attention":
            return cb.shared_prefix_attention(d.q, *where, self.b.scale, self.group, self.lens, **kw)
        return cb.rope_append_attention(d.q, d.k_new, d.v_new, *where, self.b.scale, self.cs,
                                        prefix_group=self.group, prefix_lens=self.lens, **kw)


CALLS = ["rope_append", "shared_prefix_attention", "rope_append_attention"]


class _Handle:
    cuda_stream = 0


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [0, _Handle()])
def test_default_stream_by_its_handle(cuda_lib, name, stream):
    # the default stream's handle is 0: the call waits for what is queued there, q's last change here
    s = Step(1000)
    fresh = torch.randn_like(s.d.q)
    s.d.q.copy_(fresh)
    expect = s.call(name)
    assert expect.isfinite().all()
    expect = bits_of(expect)
    s.d.q.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                      # about 0.1 s
    s.d.q.copy_(fresh)
    got = s.call(name, stream=stream)
    torch.cuda.synchronize()
    assert cb.get_device_error() == cb.CB_OK
    assert np.array_equal(bits_of(got), expect)
    with cb._on_stream(stream):
        assert torch.cuda.current_stream().cuda_stream == 0


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("size", [1 << 70, -(1 << 70), 1 << 40, 1 << 31, -16, 0, 17])
def test_block_sizes_of_no_pool_are_refused(cuda_lib, name, size):
    s = Step(1001)
    with pytest.raises(ValueError, match="block_size"):
        s.call(name, block_size=size)
    assert s.call(name) is not None                     # nothing is left behind for the next call
    assert cb.get_device_error() == cb.CB_OK


@pytest.mark.parametrize("name", CALLS)
def test_integers_of_other_types(cuda_lib, name):
    s = Step(1002)
    expect = bits_of(s.call(name))
    for kind in (np.int32, np.int64, np.uint8):
        assert np.array_equal(bits_of(s.call(name, block_size=kind(16))), expect)
    with pytest.raises(ValueError, match="block_size must be an integer"):
        s.call(name, block_size=16.0)
    if name == "rope_append":
        return
    expect = bits_of(s.call(name, decode_ctas=7))
    assert np.array_equal(bits_of(s.call(name, decode_ctas=np.int64(7))), expect)
    for bad in (7.0, 1 << 70, 1 << 31):
        with pytest.raises(ValueError, match="decode_ctas must be"):
            s.call(name, decode_ctas=bad)
    if name == "rope_append_attention":
        with pytest.raises(ValueError, match="window must be"):
            s.call(name, window=2.5)
    assert cb.get_device_error() == cb.CB_OK

"""cb_rope_append refuses bad arguments on the host, before any CUDA call, and the binding refuses
host tensors and wrong shapes."""
import ctypes

import pytest
import torch

import continuous_batching_paged_gb300 as cb
from continuous_batching_paged_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return cb.library()


Q, KV, OUT = 1 << 20, 1 << 24, 1 << 28       # addresses far apart; never dereferenced


def _status(lib, q=Q, k=KV, v=KV, q_out=OUT, kp=KV, table=256, rope=True, dims=None, bs=16, **kw):
    d = dict(num_seqs=4, num_tokens=35, num_q_heads=4, num_kv_heads=2, head_dim=64, num_pages=24,
             max_blocks_per_seq=9)
    d.update(dims or {})
    r = cb.CbRope(256, 128, 64, 0, 0, 0, 0, 0)
    for name, value in kw.items():
        setattr(r, name, value)
    return lib.cb_rope_append(q, k, v, q_out, kp, KV, table, 256, 256, bs,
                              ctypes.byref(r) if rope else None, ctypes.byref(cb.CbDims(**d)), None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(rope=False), cb.CB_ERR_INVALID_ARG, b"rope is NULL"),
    (dict(q=None), cb.CB_ERR_INVALID_ARG, b"null"),
    (dict(q_out=None), cb.CB_ERR_INVALID_ARG, b"null"),
    (dict(k=None), cb.CB_ERR_INVALID_ARG, b"null"),
    (dict(table=None), cb.CB_ERR_INVALID_ARG, b"null"),
    (dict(cos_sin=None), cb.CB_ERR_INVALID_ARG, b"null"),
    (dict(cos_sin=264), cb.CB_ERR_INVALID_ARG, b"16-byte"),
    (dict(q=Q + 8), cb.CB_ERR_INVALID_ARG, b"16-byte"),
    (dict(q_out=OUT + 2), cb.CB_ERR_INVALID_ARG, b"16-byte"),
    (dict(kp=KV + 4), cb.CB_ERR_INVALID_ARG, b"16-byte"),
    (dict(max_positions=0), cb.CB_ERR_INVALID_ARG, b"max_positions"),
    (dict(rot_dim=0), cb.CB_ERR_INVALID_ARG, b"rot_dim"),
    (dict(rot_dim=8), cb.CB_ERR_INVALID_ARG, b"rot_dim"),
    (dict(rot_dim=24), cb.CB_ERR_INVALID_ARG, b"rot_dim"),
    (dict(rot_dim=80), cb.CB_ERR_INVALID_ARG, b"rot_dim"),
    (dict(interleaved=2), cb.CB_ERR_INVALID_ARG, b"interleaved"),
    (dict(q_stride=255), cb.CB_ERR_INVALID_ARG, b"stride"),
    (dict(q_stride=260), cb.CB_ERR_INVALID_ARG, b"stride"),
    (dict(k_stride=64), cb.CB_ERR_INVALID_ARG, b"stride"),
    (dict(v_stride=-128), cb.CB_ERR_INVALID_ARG, b"stride"),
    (dict(q_out=Q + 512), cb.CB_ERR_INVALID_ARG, b"overlaps"),
    (dict(q_out=Q, q_stride=512), cb.CB_ERR_INVALID_ARG, b"overlaps"),
    (dict(q_out=Q - 16), cb.CB_ERR_INVALID_ARG, b"overlaps"),
    (dict(bs=3), cb.CB_ERR_INVALID_ARG, b"at least 4"),
    (dict(dims=dict(head_dim=96)), cb.CB_ERR_UNSUPPORTED, b"head_dim"),
    (dict(dims=dict(num_q_heads=3)), cb.CB_ERR_INVALID_ARG, b"multiple"),
])
def test_refusals(lib, kw, status, text):
    assert _status(lib, **kw) == status
    assert text in lib.cb_last_error_message()


def test_empty_batches_are_no_ops(lib):
    assert _status(lib, dims=dict(num_tokens=0)) == cb.CB_OK
    assert _status(lib, dims=dict(num_seqs=0)) == cb.CB_OK
    assert _status(lib, q=None, q_out=None, dims=dict(num_seqs=0)) == cb.CB_OK
    assert _status(lib, table=None, dims=dict(num_seqs=0)) == cb.CB_OK        # an empty table


def test_struct_matches_the_header():
    assert ctypes.sizeof(cb.CbRope) == 8 + 4 * 4 + 5 * 8
    assert cb.CbRope.q_stride.offset == 24


def test_binding_refuses_host_tensors_and_bad_rows():
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    q, kn, kp = t(3, 4, 64), t(3, 2, 64), t(8, 16, 2, 64)
    meta = (t(2, 4, dtype=torch.int32), t(3, dtype=torch.int32), t(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        cb.rope_append(q, kn, kn, kp, kp, *meta, 16, t(32, 64, dtype=torch.float32))
    with pytest.raises(ValueError, match="cos_sin"):
        cb.rope_append(q, kn, kn, kp, kp, *meta, 16, t(32, 64))
    with pytest.raises(ValueError, match="contiguous token rows"):
        cb._explain_rows("q", _FakeCuda(t(3, 64, 4).transpose(1, 2)))


class _FakeCuda:
    """A host tensor that answers is_cuda with True, for checks that touch no memory."""

    def __init__(self, t):
        self._t = t
        self.is_cuda = True

    def __getattr__(self, name):
        return getattr(self._t, name)


def test_rows_of_views():
    qkv = torch.zeros(5, 8, 64, dtype=torch.bfloat16)
    for rows in (qkv, qkv[:, :4], qkv[:, 4:6], qkv[:1, :4], qkv[:, 3:4], qkv[:0]):
        assert cb._rows_ok(*rows.shape, rows.stride())
        cb._explain_rows("q", _FakeCuda(rows))
    for rows in (qkv.transpose(0, 1), qkv[:, ::2], qkv[:, :, ::2]):
        assert not cb._rows_ok(*rows.shape, rows.stride()) or rows.shape[0] == 0


@pytest.mark.parametrize("kw", [dict(k=OUT), dict(v=OUT - 16), dict(k=OUT + 35 * 512 - 16),
                                dict(v=OUT - 34 * 2048 - 16, v_stride=1024)])
def test_rotated_queries_must_not_overlap_the_new_rows(lib, kw):
    assert _status(lib, **kw) == cb.CB_ERR_INVALID_ARG
    assert b"overlaps k_new or v_new" in lib.cb_last_error_message()


def test_binding_refuses_broadcast_rows():
    # a stride of 0 is the library's word for contiguous rows: a broadcast row would be read past its end
    row = torch.zeros(1, 2, 64)
    assert not cb._rows_ok(*row.expand(5, 2, 64).shape, row.expand(5, 2, 64).stride())
    assert cb._rows_ok(*row.expand(1, 2, 64).shape, row.expand(1, 2, 64).stride())
    assert not cb._rows_ok(5, 2, 64, (64, 64, 1))

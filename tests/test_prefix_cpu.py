"""cb_shared_prefix_attention and cb_rope_append_attention refuse bad arguments on the host, before
any CUDA call; the workspace size is host arithmetic; the binding refuses host tensors."""
import ctypes

import pytest
import torch

import continuous_batching_paged_gb300 as cb
from continuous_batching_paged_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return cb.library()


P, QO = 1 << 20, 1 << 28      # addresses far apart; never dereferenced


def _dims(**kw):
    d = dict(num_seqs=4, num_tokens=35, num_q_heads=4, num_kv_heads=2, head_dim=64, num_pages=24,
             max_blocks_per_seq=9)
    d.update(kw)
    return cb.CbDims(**d)


def _attend(lib, q=P, out=P, ws=P, ws_bytes=1 << 40, prefix=True, group=256, lens=256, ng=2, scale=0.1,
            dims=None, bs=16, window=0):
    p = cb.CbPrefix(group, lens, ng)
    o = cb.CbOptions(0, 0)
    o.window = window
    return lib.cb_shared_prefix_attention(q, P, P, 256, 256, 256, bs, scale,
                                          ctypes.byref(p) if prefix else None, out, None, ws, ws_bytes,
                                          ctypes.byref(dims or _dims()), ctypes.byref(o), None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(prefix=False), cb.CB_ERR_INVALID_ARG, b"prefix is NULL"),
    (dict(group=None), cb.CB_ERR_INVALID_ARG, b"null"),
    (dict(lens=None), cb.CB_ERR_INVALID_ARG, b"null"),
    (dict(ng=-1), cb.CB_ERR_INVALID_ARG, b"num_groups"),
    (dict(window=5), cb.CB_ERR_UNSUPPORTED, b"window"),
    (dict(q=None), cb.CB_ERR_INVALID_ARG, b"null"),
    (dict(out=P + 8), cb.CB_ERR_INVALID_ARG, b"16-byte"),
    (dict(ws=P + 16), cb.CB_ERR_INVALID_ARG, b"256-byte"),
    (dict(ws_bytes=1 << 16), cb.CB_ERR_INVALID_ARG, b"workspace too small"),
    (dict(scale=0.0), cb.CB_ERR_INVALID_ARG, b"scale"),
    (dict(scale=float("nan")), cb.CB_ERR_INVALID_ARG, b"scale"),
    (dict(bs=3), cb.CB_ERR_INVALID_ARG, b"at least 4"),
    (dict(dims=_dims(head_dim=96)), cb.CB_ERR_UNSUPPORTED, b"head_dim"),
    (dict(dims=_dims(num_q_heads=34)), cb.CB_ERR_UNSUPPORTED, b"16 query heads"),
    (dict(dims=_dims(num_q_heads=9, num_kv_heads=9)), cb.CB_ERR_UNSUPPORTED, b"multiple of 8"),
])
def test_refusals(lib, kw, status, text):
    assert _attend(lib, **kw) == status
    assert text in lib.cb_last_error_message()


def test_empty_batches_are_no_ops(lib):
    assert _attend(lib, dims=_dims(num_tokens=0)) == cb.CB_OK
    assert _attend(lib, dims=_dims(num_seqs=0)) == cb.CB_OK


def test_step_refusals(lib):
    r = cb.CbRope(256, 128, 64, 0, 0, 0, 0, 0)

    def step(q=P, k=P, q_out=QO, rope=r, prefix=None, ws_bytes=1 << 40):
        return lib.cb_rope_append_attention(
            q, k, P, q_out, P, P, 256, 256, 256, 16, 0.1, None if rope is None else ctypes.byref(rope),
            prefix, P, None, P, ws_bytes, ctypes.byref(_dims()), None, None)

    for kw, text in ((dict(q=None), b"null"), (dict(q_out=None), b"null"),
                     (dict(q=None, q_out=None), b"null"), (dict(k=None), b"null"),
                     (dict(rope=None), b"rope is NULL"), (dict(q_out=P + 16), b"overlaps"),
                     (dict(rope=cb.CbRope(256, 128, 20, 0)), b"rot_dim"),
                     (dict(ws_bytes=100), b"workspace too small"),
                     (dict(prefix=ctypes.byref(cb.CbPrefix(256, None, 1))), b"null")):
        assert step(**kw) == cb.CB_ERR_INVALID_ARG, kw
        assert text in lib.cb_last_error_message(), (kw, lib.cb_last_error_message())


def test_workspace_size(lib):
    size = lambda ng, **kw: lib.cb_prefix_workspace_size(ctypes.byref(_dims(**kw)), ng)
    plain = lib.cb_attention_workspace_size(ctypes.byref(_dims()))
    assert size(0) == plain and size(1) > plain and size(1) % 256 == 0
    assert size(5000) > size(1)
    assert size(1, num_seqs=400, num_tokens=400) > size(1)
    assert size(1, num_pages=999, max_blocks_per_seq=999) == size(1)
    assert size(-1) == 0 and size(1, head_dim=96) == 0 and size(1, num_q_heads=3) == 0
    assert size(1, num_q_heads=64) == 0                       # 32 query heads per KV head
    assert lib.cb_prefix_workspace_size(None, 1) == 0
    # only so many tokens of chunks share: more of them do not grow the prefixes' part
    grow = size(1, num_tokens=200000) - size(1, num_tokens=100000)
    assert grow < 64 * 1024
    assert cb.prefix_workspace_size(4, 4, 2, 64, 35, 1) == size(1)


def test_struct_matches_the_header():
    assert ctypes.sizeof(cb.CbPrefix) == 2 * 8 + 2 * 4 + 2 * 8


def test_binding_refuses_host_tensors():
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    q, kn, kp = t(3, 4, 64), t(3, 2, 64), t(8, 16, 2, 64)
    meta = (t(2, 4, dtype=torch.int32), t(3, dtype=torch.int32), t(2, dtype=torch.int32))
    grp = (t(2, dtype=torch.int32), t(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        cb.shared_prefix_attention(q, kp, kp, *meta, 16, 0.125, *grp)
    with pytest.raises(ValueError, match="CUDA tensor"):
        cb.rope_append_attention(q, kn, kn, kp, kp, *meta, 16, 0.125, t(9, 64, dtype=torch.float32),
                                 prefix_group=grp[0], prefix_lens=grp[1])
    with pytest.raises(ValueError, match="bfloat16"):
        cb.shared_prefix_attention(q.float(), kp, kp, *meta, 16, 0.125, *grp)


@pytest.mark.parametrize("out", [P, P + 16, P + 35 * 512 - 16, P - 35 * 512 + 16])
def test_output_must_not_overlap_the_queries(lib, out):
    assert _attend(lib, out=out) == cb.CB_ERR_INVALID_ARG
    assert b"overlaps the queries" in lib.cb_last_error_message()
    r = cb.CbRope(256, 128, 64, 0, 0, 0, 0, 0)
    assert lib.cb_rope_append_attention(QO, QO + (1 << 24), QO, P, P, P, 256, 256, 256, 16, 0.1,
                                        ctypes.byref(r), None, out, None, P, 1 << 40,
                                        ctypes.byref(_dims()), None, None) == cb.CB_ERR_INVALID_ARG
    assert b"overlaps the queries" in lib.cb_last_error_message()


@pytest.mark.parametrize("S,T,Hq,Hkv,D", [(256, 2048, 32, 32, 128), (512, 4096, 64, 64, 128),
                                          (1024, 9000, 64, 8, 128), (257, 2304, 64, 8, 128),
                                          (128, 512, 32, 8, 64), (300, 40000, 16, 1, 64), (64, 64, 32, 8, 128)])
def test_workspace_holds_what_a_batch_can_need(lib, S, T, Hq, Hkv, D):
    # partial rows (D + 2 fp32 values a query head): the decode pass's records of up to `pack` tokens,
    # of sequences with at most 8 tokens, and a slot per decode CTA; the listed tokens (8 a sequence,
    # and those of fewer than 152 chunk items), twice where a token can have two chains; 160 CTAs' own
    pack = max(1, 8 // (Hq // Hkv))
    records = min(S * -(-8 // pack), (T + S * (pack - 1)) // pack)
    short = min(T, 8 * S)
    listed = short if S > 256 else min(T, 8 * S + 152 * 256 // Hq) + short
    rows = (512 + max(records, S)) * pack * Hq + listed * Hq + 160 * 256
    # the lists: under 128 bytes for a record, a token or a group, and a counter per record and head
    lists = 128 * (records + S + listed + 300) + 4 * (records + S) * Hq
    size = lib.cb_prefix_workspace_size(ctypes.byref(_dims(num_seqs=S, num_tokens=T, num_q_heads=Hq,
                                                           num_kv_heads=Hkv, head_dim=D)), 1)
    assert rows * (4 * D + 8) <= size <= rows * (4 * D + 8) + lists + 16384

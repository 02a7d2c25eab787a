"""The calls on the quantised cache and with changed scores refuse bad arguments on the host, before any
CUDA call, and the binding refuses host tensors and wrong types."""
import ctypes

import pytest
import torch

import continuous_batching_paged_gb300 as cb
from continuous_batching_paged_gb300 import _build

INVALID, UNSUPPORTED, OK = cb.CB_ERR_INVALID_ARG, cb.CB_ERR_UNSUPPORTED, cb.CB_OK


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return cb.library()


# addresses far apart; never dereferenced
Q, KV, OUT, SC, WS, META = 1 << 20, 1 << 24, 1 << 28, 1 << 30, 1 << 31, 256


def _dims(**kw):
    d = dict(num_seqs=4, num_tokens=35, num_q_heads=4, num_kv_heads=2, head_dim=64, num_pages=24,
             max_blocks_per_seq=9)
    d.update(kw)
    return ctypes.byref(cb.CbDims(**d))


def _rope(**kw):
    r = cb.CbRope(256, 128, 64, 0, 0, 0, 0, 0)
    for name, value in kw.items():
        setattr(r, name, value)
    return ctypes.byref(r)


def _append(lib, q=Q, k=KV, v=KV, q_out=OUT, kp=KV, sc=SC, table=META, bs=16, rope={}, dims={}):
    return lib.cb_quant_append(q, k, v, q_out, kp, KV, sc, table, META, META, bs,
                               None if rope is None else _rope(**rope), _dims(**dims), None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(sc=None), INVALID, b"null"), (dict(sc=SC + 8), INVALID, b"kv_scales"),
    (dict(k=None), INVALID, b"null"), (dict(kp=KV + 4), INVALID, b"16-byte"),
    (dict(q_out=None), INVALID, b"null"), (dict(table=None), INVALID, b"null"),
    (dict(rope=None), INVALID, b"without cos_sin"),                       # q, and nothing that turns it
    (dict(rope=dict(cos_sin=None, rot_dim=0)), INVALID, b"without cos_sin"),
    (dict(q=None, q_out=None, rope=dict(cos_sin=None)), INVALID, b"rot_dim"),
    (dict(q=None, q_out=None, rope=dict(cos_sin=None, rot_dim=0, interleaved=1)), INVALID, b"rot_dim"),
    (dict(rope=dict(rot_dim=24)), INVALID, b"rot_dim"), (dict(rope=dict(max_positions=0)), INVALID, b"max_pos"),
    (dict(rope=dict(k_stride=64)), INVALID, b"stride"), (dict(q_out=Q + 512), INVALID, b"overlaps"),
    (dict(k=OUT), INVALID, b"overlaps"), (dict(bs=3), INVALID, b"at least 4"),
    (dict(dims=dict(head_dim=96)), UNSUPPORTED, b"head_dim"),
    (dict(dims=dict(num_q_heads=3)), INVALID, b"multiple")])
def test_append_refusals(lib, kw, status, text):
    assert _append(lib, **kw) == status
    assert text in lib.cb_last_error_message()


def test_empty_batches_are_no_ops(lib):
    for dims in (dict(num_tokens=0), dict(num_seqs=0)):
        assert _append(lib, dims=dims) == OK
        assert _append(lib, q=None, q_out=None, rope=None, dims=dims) == OK
        assert _gather(lib, dims=dims) == OK
        assert _attend(lib, dims=dims) == OK
        assert _step(lib, dims=dims) == OK


def _gather(lib, kp=KV, sc=SC, table=META, cu=META, starts=None, bs=16, ko=OUT, vo=OUT + (1 << 20), dims={}):
    return lib.cb_quant_gather(kp, KV, sc, table, cu, starts, bs, ko, vo, _dims(**dims), None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(kp=None), INVALID, b"null"), (dict(sc=None), INVALID, b"null"), (dict(cu=None), INVALID, b"null"),
    (dict(ko=None), INVALID, b"null"), (dict(ko=OUT + 8), INVALID, b"16-byte"),
    (dict(sc=SC + 2), INVALID, b"kv_scales"), (dict(vo=OUT + 16), INVALID, b"overlaps"),
    (dict(bs=2), INVALID, b"at least 4"), (dict(dims=dict(head_dim=32)), UNSUPPORTED, b"head_dim")])
def test_gather_refusals(lib, kw, status, text):
    assert _gather(lib, **kw) == status
    assert text in lib.cb_last_error_message()


def _score(**kw):
    s = cb.CbScore()
    for name, value in kw.items():
        setattr(s, name, value)
    return ctypes.byref(s)


def _attend(lib, q=Q, sc=SC, out=OUT, ws=WS, size=1 << 30, scale=0.125, score={}, options={}, bs=16, dims={}):
    o = cb.CbOptions()
    for name, value in options.items():
        setattr(o, name, value)
    return lib.cb_quant_attention(q, KV, KV, sc, META, META, META, bs, scale,
                                  None if score is None else _score(**score), out, None, ws, size,
                                  _dims(**dims), ctypes.byref(o), None)


def _scored(lib, q=Q, out=OUT, scale=0.125, score={}, window=0, dims={}, size=1 << 30):
    o = cb.CbOptions()
    o.window = window
    return lib.cb_scored_attention(q, KV, KV, META, META, META, 16, scale,
                                   None if score is None else _score(**score), out, None, WS, size,
                                   _dims(**dims), ctypes.byref(o), None)


BAD_SCORES = [(dict(softcap=-1.0), INVALID, b"softcap"), (dict(softcap=float("nan")), INVALID, b"softcap"),
              (dict(softcap=float("inf")), INVALID, b"softcap"), (dict(slopes=258), INVALID, b"aligned"),
              (dict(visible_lens=1), INVALID, b"aligned"), (dict(softcap=1e-36), INVALID, b"range")]


@pytest.mark.parametrize("score,status,text", BAD_SCORES)
def test_bad_scores(lib, score, status, text):
    for call in (_attend, _scored, _step):
        assert call(lib, score=score) == status
        assert text in lib.cb_last_error_message()


@pytest.mark.parametrize("kw,status,text", [
    (dict(sc=None), INVALID, b"null"), (dict(sc=SC + 1), INVALID, b"kv_scales"), (dict(q=None), INVALID, b"null"),
    (dict(ws=WS + 16), INVALID, b"256-byte"), (dict(size=256), INVALID, b"workspace too small"),
    (dict(scale=0.0), INVALID, b"scale"), (dict(out=Q), INVALID, b"overlaps"), (dict(out=Q - 16), INVALID, b"overlaps"),
    (dict(dims=dict(num_q_heads=34)), UNSUPPORTED, b"16 query heads"),
    (dict(dims=dict(num_q_heads=9, num_kv_heads=9)), UNSUPPORTED, b"multiple of 8"),
    (dict(score=dict(visible_lens=META), options=dict(window=5)), UNSUPPORTED, b"sliding window"),
    (dict(bs=3), INVALID, b"at least 4")])
def test_attention_refusals(lib, kw, status, text):
    assert _attend(lib, **kw) == status
    assert text in lib.cb_last_error_message()


def test_scored_refusals(lib):
    assert _scored(lib, score=None) == INVALID and b"score is NULL" in lib.cb_last_error_message()
    assert _scored(lib, out=Q + 16) == INVALID and b"overlaps" in lib.cb_last_error_message()
    assert _scored(lib, score=dict(visible_lens=META), window=3) == UNSUPPORTED
    assert _scored(lib, size=64) == INVALID and b"workspace" in lib.cb_last_error_message()


def _step(lib, q=Q, q_out=OUT + (1 << 22), rope={}, score={}, out=OUT, k=KV, sc=SC, dims={}):
    return lib.cb_quant_append_attention(q, k, KV, q_out, KV, KV, sc, META, META, META, 16, 0.125,
                                         None if rope is None else _rope(**rope), _score(**score), out, None, WS,
                                         1 << 30, _dims(**dims), None, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(q=None), INVALID, b"null"), (dict(q_out=None), INVALID, b"null"), (dict(k=None), INVALID, b"null"),
    (dict(sc=None), INVALID, b"null"), (dict(rope=None), INVALID, b"q_out without cos_sin"),
    (dict(q_out=OUT), INVALID, b"overlaps"), (dict(rope=None, q_out=None, out=Q), INVALID, b"overlaps")])
def test_step_refusals(lib, kw, status, text):
    assert _step(lib, **kw) == status
    assert text in lib.cb_last_error_message()


def test_struct_matches_the_header():
    assert ctypes.sizeof(cb.CbScore) == 8 + 2 * 8 + 2 * 8
    assert cb.CbScore.slopes.offset == 8 and cb.CbScore.visible_lens.offset == 16


def test_binding_refuses_host_tensors_and_wrong_types():
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=torch.float32).to(dtype)
    q, kn = t(3, 4, 64), t(3, 2, 64)
    codes, sc = t(8, 16, 2, 64, dtype=torch.float8_e4m3fn), t(8, 16, 2, 2, dtype=torch.uint8)
    meta = (t(2, 4, dtype=torch.int32), t(3, dtype=torch.int32), t(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        cb.quant_append(None, kn, kn, codes, codes, sc, *meta, 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        cb.quant_attention(q, codes, codes, sc, *meta, 16, 0.125)
    with pytest.raises(ValueError, match="CUDA tensor"):
        cb.quant_append_attention(q, kn, kn, codes, codes, sc, *meta, 16, 0.125)
    with pytest.raises(ValueError, match="CUDA tensor"):
        cb.quant_gather(codes, codes, sc, meta[0], meta[1], 16, 3)
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        cb.quant_gather(t(8, 16, 2, 64), codes, sc, meta[0], meta[1], 16, 3)
    with pytest.raises(ValueError, match="CUDA tensor"):
        cb.scored_attention(q, t(8, 16, 2, 64), t(8, 16, 2, 64), *meta, 16, 0.125, softcap=5.0)
    with pytest.raises(ValueError, match="kv_scales must be given"):
        cb.quant_attention(q, codes, codes, None, *meta, 16, 0.125)

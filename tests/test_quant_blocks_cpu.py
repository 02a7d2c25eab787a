"""The block moves of the quantised cache refuse bad arguments on the host, before any CUDA call."""
import ctypes

import pytest

import continuous_batching_paged_gb300 as cb
from continuous_batching_paged_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return cb.library()


KV, SC, HOST, IDS = 1 << 24, 1 << 30, 1 << 28, 256  # (never dereferenced)


def calls(lib, kp=KV, sc=SC, ids=IDS, n=3, bs=16, hk=HOST, hs=HOST + (1 << 20), **dims):
    d = ctypes.byref(cb.CbDims(**dict(dict(num_seqs=0, num_tokens=0, num_q_heads=2, num_kv_heads=2, head_dim=64,
                                           num_pages=24, max_blocks_per_seq=1), **dims)))
    return [lambda: lib.cb_quant_copy_blocks(kp, KV, sc, ids, IDS, n, bs, d, None),
            lambda: lib.cb_quant_offload(kp, KV, sc, ids, n, bs, d, hk, HOST, hs, None),
            lambda: lib.cb_quant_restore(kp, KV, sc, ids, n, bs, d, hk, HOST, hs, None)]


@pytest.mark.parametrize("kw,status,text", [
    (dict(kp=None), cb.CB_ERR_INVALID_ARG, b"null"), (dict(sc=None), cb.CB_ERR_INVALID_ARG, b"null"),
    (dict(ids=None), cb.CB_ERR_INVALID_ARG, b"null"), (dict(n=-1), cb.CB_ERR_INVALID_ARG, b"negative"),
    (dict(kp=KV + 8), cb.CB_ERR_INVALID_ARG, b"16-byte"), (dict(sc=SC + 2), cb.CB_ERR_INVALID_ARG, b"16-byte"),
    (dict(bs=3), cb.CB_ERR_INVALID_ARG, b"at least 4"), (dict(head_dim=96), cb.CB_ERR_UNSUPPORTED, b"head_dim"),
    (dict(bs=1 << 29), cb.CB_ERR_UNSUPPORTED, b"2^30"), (dict(num_pages=0), cb.CB_ERR_INVALID_ARG, b"num_pages")])
def test_refusals(lib, kw, status, text):
    for call in calls(lib, **kw):
        assert call() == status
        assert text in lib.cb_last_error_message()


def test_host_buffers(lib):
    for kw in (dict(hs=None), dict(hk=None), dict(hs=HOST + 2)):
        for call in calls(lib, **kw)[1:]:
            assert call() == cb.CB_ERR_INVALID_ARG


def test_nothing_to_move(lib):
    for call in calls(lib, n=0, kp=None, sc=None):
        assert call() == cb.CB_OK

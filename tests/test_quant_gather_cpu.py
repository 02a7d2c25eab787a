"""The read-back refuses outputs that lie in the cache it reads, on the host."""
import ctypes

import pytest

import continuous_batching_paged_gb300 as cb
from continuous_batching_paged_gb300 import _build

K, V, SC, OUT, META = 1 << 24, 1 << 25, 1 << 26, 1 << 28, 256  # (never dereferenced)
CODES, SCALES, ROWS = 24 * 16 * 2 * 64, 24 * 16 * 2 * 2, 35 * 2 * 64 * 2  # bytes: a pool, the scales, an output


@pytest.mark.parametrize("at", [K, K + CODES - 16, K - ROWS + 16, V, V + CODES - 16, V - ROWS + 16, SC,
                                SC + SCALES - 16, SC - ROWS + 16])
def test_outputs_in_the_cache(at):
    _build.build()
    lib = cb.library()
    dims = ctypes.byref(cb.CbDims(num_seqs=4, num_tokens=35, num_q_heads=2, num_kv_heads=2, head_dim=64,
                                  num_pages=24, max_blocks_per_seq=9))
    for ko, vo in ((at, OUT), (OUT, at)):
        assert lib.cb_quant_gather(K, V, SC, META, META, None, 16, ko, vo, dims, None) == cb.CB_ERR_INVALID_ARG
        assert b"overlaps the cache" in lib.cb_last_error_message()

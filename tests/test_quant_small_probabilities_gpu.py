"""Decode over the quantised cache where most keys have small probabilities."""
import numpy as np
import pytest
import torch

import continuous_batching_paged_gb300 as cb
from gpu_util import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("behind", [16, 22, 26, 30])
@pytest.mark.parametrize("D,Hkv", [(64, 1), (128, 8)])
def test_keys_beside_one_that_takes_all(cuda_lib, D, Hkv, behind):
    """The first key takes nearly all of a head's probability, the others have 2^-behind of it each; half of the
    first value row is 0, so half of the output is the others' alone.

    Their values are 1 and their probabilities powers of two (the score's rounding, 2^-23 of it, moves them by
    30 ln 2 2^-23 at most, less than fp16 shows), exact in fp16 where 2^-24 and above stands for them.  l sums n
    terms in fp32 beside 1, each sum off by 2^-24 of it at most, and so does o: n 2^-24 each.  The result is rounded
    to bf16."""
    n, bs = 4096, 32
    P = n // bs
    k = torch.zeros(P, bs, Hkv, D, device="cuda")
    v = torch.ones(P, bs, Hkv, D, device="cuda")
    k[0, 0, :, 0] = 1.0
    v[0, 0, :, D // 2:] = 0.0
    pools = (torch.zeros(P, bs, Hkv, D, device="cuda").to(torch.float8_e4m3fn),
             torch.zeros(P, bs, Hkv, D, device="cuda").to(torch.float8_e4m3fn),
             torch.zeros(P, bs, Hkv, 2, dtype=torch.uint8, device="cuda"))
    table = i32(np.arange(P)[None])
    rows = lambda x: x.reshape(n, Hkv, D).bfloat16()
    cb.quant_append(None, rows(k), rows(v), *pools, table, i32([0, n]), i32([n]), bs)
    q = torch.zeros(1, Hkv, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 1.0
    out, lse = cb.quant_attention(q, *pools, table, i32([0, 1]), i32([n]), bs, behind * float(np.log(2.0)),
                                  lse=True, decode_ctas=1)
    assert cb.get_device_error() == cb.CB_OK
    o = out.double().cpu().numpy()[0]
    others = (n - 1) * 2.0 ** -behind
    tol = 2.0 ** -8 + 2 * n * 2.0 ** -24
    assert np.all(np.abs(o[:, :D // 2] - 1.0) <= tol)
    want = others / (1.0 + others)
    assert np.all(np.abs(o[:, D // 2:] - want) <= tol * want), o[0, -1] / want
    assert np.all(np.abs(lse.double().cpu().numpy() - behind * np.log(2.0) - np.log1p(others))
                  <= 2.0 ** -20 * (1 + behind) + n * 2.0 ** -24)

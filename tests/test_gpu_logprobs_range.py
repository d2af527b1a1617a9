"""Token log probabilities on the GPU where logits, masks or the temperature are large: results as in 64 bits
(check of test_gpu_logprobs, its tolerances)."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_vocab_gb300 import binding as ssd
from test_gpu_logprobs import DT, _lib, check, logits, outputs  # noqa: F401 (the fixture builds the library)

pytestmark = pytest.mark.gpu


@DT
@pytest.mark.parametrize("T", [1.0, 0.3, 1e-6, 2e-7, 0.0])
def test_large_row_maximum(dtype, T):
    """Rows whose largest logit is far from 0 for their temperature: a forced token, all of a row at one value or near it."""
    n = 20
    for V in (9001, 128256):
        for big in (400.0, 3e7, 3e9, 1e10, 1e15, 1e20):
            z = logits(1, 5, V, dtype, 21)
            z[0, 0, V // 3] = big
            z[0, 1, :V] = -big
            z[0, 2, :V] = big
            z[0, 3, :V] = -big * (1 + torch.rand(V, generator=torch.Generator().manual_seed(3)) * 1e-2)
            z[0, 4, :V] = big * (1 + torch.rand(V, generator=torch.Generator().manual_seed(4)) * 1e-6)
            check(z, V, T, np.array([[V // 3, V - 1, 0, 17, V // 2]], np.int32), n)


@DT
@pytest.mark.parametrize("mask", [-1e9, -2e9, -1e10, -1e12, -1e15, -1e20, -1e28])
def test_finite_masks(dtype, mask):
    """A grammar's mask by a finite value: most of a row, whole stages, all but one token, a few scattered ones; the
    token allowed or masked."""
    n = 20
    for V in (9001, 32000, 128256):
        z = logits(1, 6, V, dtype, 22)
        rng = np.random.default_rng(V)
        few = torch.as_tensor(rng.permutation(V)[:10].copy(), device="cuda")
        keep = z[0, 0, few].clone()
        z[0, 0, :V] = mask
        z[0, 0, few] = keep
        z[0, 1, :V - 10] = mask         # the allowed tokens last
        z[0, 2, 10:V] = mask            # first
        z[0, 3, :V], z[0, 3, 4000] = mask, 1.5
        z[0, 4, :V // 2] += mask        # added to the logits
        z[0, 5, 3:V:2] = mask
        tokens = np.array([[int(few[3]), 5, 3, 4000, V - 1, 4]], np.int32)
        for T in (1.0, 0.7, 0.6, 0.3, 0.1, 0.05, 0.01, 0.0):
            check(z, V, T, tokens, n)


@DT
@pytest.mark.parametrize("T", [1e20, 1e26, 1e27, 1e28, 1e29, 1e30, 3e38])
def test_large_temperature(dtype, T):
    """Tokens of -inf have probability 0 at any temperature; what lies behind a row's end counts nothing."""
    for V in (3, 9001, 32777):
        z = logits(1, 4, V, dtype, 23)
        z[0, 0, 1:V:2] = -math.inf
        z[0, 1, 1:V] = -math.inf
        z[0, 2, :V] *= 1e28
        z[0, 3, :V] = z[0, 3, :V] * 1e29 - 2e29
        check(z, V, T, np.array([[0, 1, V - 1, V // 2]], np.int32), min(V, 20))


@DT
@pytest.mark.parametrize("T", [1e3, 1e30, 1e37, 3e38])
def test_logits_whose_difference_passes_fp32(dtype, T):
    """ln p where a logit less the row's largest is no fp32 number, but over T it is."""
    V = 1003
    z = logits(1, 3, V, dtype, 24)
    top = torch.finfo(dtype).max
    z[0, 0, :V], z[0, 0, 9] = -top, top
    z[0, 1, :V:2], z[0, 1, 1:V:2] = top, -top
    z[0, 2, :V] = z[0, 2, :V] * (top / 32)
    check(z, V, T, np.array([[8, 9, V - 1]], np.int32), 20)


@DT
@pytest.mark.parametrize("n", [0, 5])
def test_no_probability_above_one(dtype, n):
    """ln p <= 0 and entropy >= 0, also where one token has all of a row's probability."""
    V, R = 3001, 512
    z = logits(2, R, V, dtype, 25)
    g = torch.Generator().manual_seed(5)
    tokens = torch.randint(0, V, (2, R), generator=g, dtype=torch.int32).cuda()
    tall = (30 + 70 * torch.rand(2, R, generator=g)).to("cuda", dtype)
    z.scatter_(2, tokens.long()[..., None], tall[..., None])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for T in (1.0, 0.7, 0.3, 1e-2):
        o = outputs(2, R, n)
        ssd.ssd_token_logprobs(z, V, T, tokens=tokens, status=st, **o)
        assert (o["logprob"] <= 0).all() and (o["logprob"] >= -1e-5).all(), (T, o["logprob"].max())
        assert (o["entropy"] >= 0).all() and (o["entropy"] <= 1e-3).all(), (T, o["entropy"].min())
        assert (o["top_logprob"] <= 0).all()
    assert int(st.item()) == 0


@DT
def test_long_rows_summed_by_differences(dtype):
    """Rows of many equal terms, whose additions round the same way each time, at the largest sizes."""
    top = 1 << (20 if dtype == torch.float32 else 21)
    for V in (195115, top):
        z = logits(1, 3, V, dtype, 26)
        z[0, :, :V] = -1e30
        z[0, 0, 100], z[0, 1, 100], z[0, 2, V - 1] = 0.7e30, 3e30, 9e30
        for T in (2.9e29, 7e29):
            check(z, V, T, np.array([[100, 5, V - 1]], np.int32), 20)

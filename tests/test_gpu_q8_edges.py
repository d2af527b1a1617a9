"""Edges of the 8-bit cache calls: sequences of a batch that take no part."""
import math

import numpy as np
import pytest
import torch

import q8_ref as ref
from speculative_decoding_vocab_gb300 import binding as ssd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_vocab_gb300 import build
    build.build()
    ssd.load()


def dev(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x)).to("cuda", dtype)


@pytest.mark.parametrize("d", [64, 128])
def test_append_leaves_empty_sequences_alone(d):
    """count = 0 (or below, clamped) behind rows of a block: nothing is read, written or reported, whatever the
    block's id and scale are: no block, one past the pool, a page past the table, scales 0, NaN, negative, tiny."""
    rng = np.random.default_rng(d)
    B, S, H, nb = 9, 20, 2, 12
    table = np.full((B, 3), -1, np.int32)
    table[:, 2] = np.arange(B)
    table[1, 2] = nb + 5
    prefix = np.full(B, 37, np.int32)              # page 2, five rows held
    prefix[2] = 53                                 # page 3: past the table
    x = torch.as_tensor(rng.standard_normal((B, S, 2 * H, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    codes = rng.integers(0, 256, (2, nb, H, 16, d)).astype(np.uint8)
    scale = np.full((2, nb, H), 2.0 ** -110, np.float32)
    scale[:, 3], scale[:, 4], scale[:, 5], scale[:, 6] = 0.0, math.nan, -1.0, math.inf
    g = [dev(codes[0]), dev(codes[1]), dev(scale[0]), dev(scale[1])]
    for count, flags in ((np.zeros(B), 0), (np.full(B, -3), ref.BAD_PREFIX)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ssd.ssd_kv_append_q8(x[:, :, :H], x[:, :, H:], *g, dev(table), dev(prefix), 0, count=dev(count.astype(np.int32)),
                             status=status)
        for got, want in zip(g, (codes[0], codes[1], scale[0], scale[1])):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        assert int(status.item()) == flags

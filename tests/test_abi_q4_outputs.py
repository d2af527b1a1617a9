"""Outputs that the binding of the 4-bit cache's reading back takes or refuses (no GPU: what is taken ends at the
device check)."""
import pytest
import torch

from speculative_decoding_vocab_gb300 import binding as ssd
from test_abi_q4 import cache, place

B, S, H, D = 2, 3, 2, 64


def test_read_without_outputs():
    """As in the C call, nothing is asked for; the other arguments are checked all the same."""
    good = {**cache(), **place(), "k_out": None, "v_out": None, "node0": 0}
    with pytest.raises(ValueError, match="CUDA device"):
        ssd.ssd_kv_read_q4(**good)
    with pytest.raises(ValueError, match="prefix_len"):
        ssd.ssd_kv_read_q4(**{**good, "prefix_len": torch.zeros(B, dtype=torch.int64)})

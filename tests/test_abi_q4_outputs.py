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


def read_into(k_out, v_out):
    ssd.ssd_kv_read_q4(*cache().values(), *list(place().values())[:2], 0, k_out, v_out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_read_outputs_that_meet(dtype):
    n = H * D
    flat = torch.zeros(4 * B * S * n, dtype=dtype)

    def rows(at, ss=S * n, ts=n):
        return flat.as_strided((B, S, H, D), (ss, ts, D, 1), at)
    k = rows(0)
    wide = rows(0, 2 * S * n, 2 * n)
    far = rows(0, 4 * n, n)           # sequences with room of a token behind them
    meet = [(k, k), (k, rows(n)), (k, rows(S * n)), (k, rows(B * S * n - D)), (wide, rows(n - D, 2 * S * n, 2 * n)),
            (wide, rows(n + D, 2 * S * n, 2 * n)), (wide, rows(n)), (far, rows(3 * n - D, 4 * n, n)),
            (k[:, :1], rows(n)[:, :1].as_strided((B, 1, H, D), (S * n, n, D, 1), n - D))]
    for a, b in meet:
        for x, y in ((a, b), (b, a)):
            with pytest.raises(ValueError, match="overlap"):
                read_into(x, y)
    apart = [(k, rows(B * S * n)), (wide, rows(n, 2 * S * n, 2 * n)), (k, None),
             (far[:, :2], rows(2 * n, 4 * n, n)[:, :2]),
             (torch.zeros(B, S, 3 * H, D, dtype=dtype)[:, :, H:2 * H], torch.zeros(B, S, H, D, dtype=dtype))]
    fused = torch.zeros(B, S, 2 * H, D, dtype=dtype)
    apart += [(fused[:, :, :H], fused[:, :, H:]), (fused.view(B, S, 2, H, D)[:, :, 1], fused.view(B, S, 2, H, D)[:, :, 0])]
    stacked = torch.zeros(B, 2, S, H, D, dtype=dtype)
    apart.append((stacked[:, 0], stacked[:, 1]))
    for x, y in apart:
        with pytest.raises(ValueError, match="CUDA device"):
            read_into(x, y)

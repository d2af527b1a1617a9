"""4-bit attention on the GPU at the ends of v's scales, with long uncut key ranges."""
import numpy as np
import pytest
import torch

from speculative_decoding_vocab_gb300 import binding as ssd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_vocab_gb300 import build
    build.build()
    ssd.load()


@pytest.mark.parametrize("use_ws", [True, False], ids=["split", "unsplit"])
@pytest.mark.parametrize("keys", [1, 40, 50021, 808543, 1369569])
@pytest.mark.parametrize("d,Hq,Hkv,Nq", [(64, 1, 1, 1), (128, 8, 1, 6), (64, 16, 1, 4), (128, 16, 1, 8)],
                         ids=["16rows", "48rows", "64rows", "128rows"])
@pytest.mark.parametrize("byte", [27, 30, 127, 252])
def test_equal_scores_at_the_ends_of_v_scales(byte, d, Hq, Hkv, Nq, keys, use_ws):
    """All keys score 0 and all of v is code 3 or 5 (1.5, 3), so out is that value.  P t = 2^11 and v / t are exact, the
    sums of up to 2^21 equal powers of two (times 3 with the code's fraction: below 2^24) are exact in fp32, a row's
    factor rounds three times at 2^-24 and ex2 is off by less than 2^-21: the value before rounding is off by
    less than 2^-20 of itself and, being a bf16 number, comes out as it is."""
    maxb = (keys + Nq + 15) // 16
    u8, i32 = dict(dtype=torch.uint8, device="cuda"), dict(dtype=torch.int32, device="cuda")
    # one block stands for all (it is only read)
    kc = torch.zeros(1, Hkv, 16, d // 2, **u8)
    ks = torch.full((1, Hkv, 16, d // 32), 127, **u8)
    vs = torch.full((1, Hkv, 16, d // 32), byte, **u8)
    vc = torch.full((1, Hkv, 8, d), 0x33, **u8)
    vc[..., d // 2:] = 0x55
    q = torch.randn(1, Nq, Hq, d, generator=torch.Generator().manual_seed(1)).to("cuda", torch.bfloat16)
    table, parent = torch.zeros(1, maxb, **i32), torch.arange(-1, Nq - 1, **i32)[None].contiguous()
    prefix, status, out = torch.tensor([keys], **i32), torch.zeros(1, **i32), torch.empty_like(q)
    lse = torch.empty(1, Nq, Hq, device="cuda")
    ws = None
    if use_ws:
        ws = torch.empty(ssd.ssd_attention_q4_workspace_size(1, Nq, Hq, Hkv, d), **u8)
    ssd.ssd_branch_attention_q4(q, kc, vc, ks, vs, table, prefix, parent, out, lse=lse, status=status, ws=ws)
    scale = 2.0 ** (byte - 127)
    want = torch.full((d,), 1.5 * scale, dtype=torch.float64)
    want[d // 2:] = 3 * scale
    assert int(status.item()) == 0
    got = out.double().cpu()
    assert (got == want).all(), (got / want).aminmax()
    ln = np.log(keys + 1 + np.arange(Nq))[None, :, None]
    np.testing.assert_allclose(lse.double().cpu().numpy(), np.broadcast_to(ln, lse.shape), rtol=0, atol=2.0 ** -19 * 16)


@pytest.mark.parametrize("use_ws", [True, False], ids=["split", "unsplit"])
@pytest.mark.parametrize("d,Hq,Hkv,Nq", [(64, 1, 1, 1), (128, 8, 1, 6), (64, 16, 1, 4), (128, 16, 1, 8)],
                         ids=["16rows", "48rows", "64rows", "128rows"])
@pytest.mark.parametrize("order", ["rising", "falling", "equal"])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_near_their_limit(sign, order, d, Hq, Hkv, Nq, use_ws):
    """Scores up to 0.99 * 2^24 in magnitude, pages of one score each: the largest score's pages have all the weight, and
    out is their value, a bf16 number (the weights are equal, so it comes out as it is); lse is off by the roundings of m, of
    its product with ln 2 and of the score, 4 * 2^-24 of 2^24, beside ln of the keys' number (below 10)."""
    values = [0.5, 1, 1.5, 2, 3, 4, 6]          # of code i + 1
    pages = 7 * 60
    codes = np.repeat(np.arange(1, 8), 60)
    if order == "equal":
        codes[:] = 5
    elif (order == "falling") == (sign > 0):
        codes = codes[::-1].copy()
    u8, i32 = dict(dtype=torch.uint8, device="cuda"), dict(dtype=torch.int32, device="cuda")
    c = torch.arange(1, 8, **u8).view(7, 1, 1, 1)
    kc = (c * 17).expand(7, Hkv, 16, d // 2).contiguous()
    vc = (c * 17).expand(7, Hkv, 8, d).contiguous()
    ks = torch.full((7, Hkv, 16, d // 32), 127, **u8)
    q = torch.full((1, Nq, Hq, d), float(sign), dtype=torch.bfloat16, device="cuda")
    table = torch.as_tensor(codes - 1, dtype=torch.int32, device="cuda")[None].contiguous()
    parent = torch.arange(-1, Nq - 1, **i32)[None].contiguous()
    prefix, status = torch.tensor([pages * 16 - Nq], **i32), torch.zeros(1, **i32)
    out, lse = torch.empty_like(q), torch.empty(1, Nq, Hq, device="cuda")
    ws = torch.empty(ssd.ssd_attention_q4_workspace_size(1, Nq, Hq, Hkv, d), **u8) if use_ws else None
    scale = 0.99 * 2.0 ** 24 / (6 * d)
    ssd.ssd_branch_attention_q4(q, kc, vc, ks, ks.clone(), table, prefix, parent, out, lse=lse, scale=scale,
                                status=status, ws=ws)
    held = [values[x - 1] for x in codes]
    best = max(held) if sign > 0 else min(held)
    assert int(status.item()) == 0
    assert (out.double() == best).all(), out.double().aminmax()
    assert (lse.double() - sign * best * d * scale).abs().max().item() <= 4 + 10

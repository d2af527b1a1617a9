"""Token log probabilities on the GPU against their definition in 64 bits (q4_ref.token_logprobs)."""
import math

import numpy as np
import pytest
import torch

import q4_ref as ref
from speculative_decoding_vocab_gb300 import binding as ssd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_vocab_gb300 import build
    build.build()
    ssd.load()


def outputs(B, R, n, fill=7):
    f32, i32 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    return dict(logprob=torch.full((B, R), float(fill), **f32), rank=torch.full((B, R), fill, **i32),
                entropy=torch.full((B, R), float(fill), **f32), top_ids=torch.full((B, R, n), fill, **i32),
                top_logprob=torch.full((B, R, n), float(fill), **f32))


def check(z, V, T, tokens, n, expect=0):
    """z [B, R, V'] on the GPU.  Roundings counted: y = (z - m) / T is off by 2^-23 of itself (the difference is
    one rounding, 1/T and the product another each: 3 * 2^-24 below 2^-22); an exponential by that times |y| plus
    2^-21 of itself, so the sum of exponentials, whose terms are positive and which is added in fp32 (2^-20 of it,
    trees of at most 2^4 partial chains), by E|y| 2^-22 + 2^-19 relative; the logarithm of it rounds once."""
    B, R = z.shape[:2]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = outputs(B, R, n)
    gt = None if tokens is None else torch.as_tensor(tokens, dtype=torch.int32, device="cuda")
    if tokens is None:
        del o["logprob"], o["rank"]
    ssd.ssd_token_logprobs(z, V, T, tokens=gt, status=st, **o)
    torch.cuda.synchronize()
    want, flags = ref.token_logprobs(z[:, :, :V].double().cpu().numpy(), T, tokens, n)
    assert int(st.item()) == flags == expect
    live = want.pop("wanted")
    for k, g in o.items():
        g, x = g.cpu().numpy(), want[k]
        assert (g[~live] == 7).all(), k  # rows that are not wanted stay as they were
        g, x = g[live].astype(np.float64), x[live].astype(np.float64)
        if k in ("rank", "top_ids"):
            np.testing.assert_array_equal(g, x, err_msg=k)
            continue
        np.testing.assert_array_equal(np.isnan(g), np.isnan(x), err_msg=k)
        fine = np.isfinite(x)
        np.testing.assert_array_equal(g[~fine], x[~fine], err_msg=k)
        # entropy <= ln V < 15: its second term E|y| <= entropy + 1
        tol = 2.0 ** -22 * np.abs(x) + 2.0 ** -19 * 16
        assert (np.abs(g - x) <= tol)[fine].all(), (k, np.abs(g - x)[fine].max())
    return o


def logits(B, R, V, dtype, seed, sigma=2.5, pad=0):
    g = torch.Generator().manual_seed(seed)
    width = -(-V // 8) * 8 + pad
    z = torch.randn(B, R, width, generator=g) * sigma
    z[:, :, V:] = math.inf  # behind a row: not read
    return z.to("cuda", dtype)


DT = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])


@DT
@pytest.mark.parametrize("B,R,V,n", [(1, 1, 1, 1), (2, 3, 7, 7), (1, 2, 64, 64), (3, 2, 1001, 20), (2, 6, 4099, 5),
                                     (1, 5, 32000, 20), (2, 2, 128256, 64), (1, 2, 151937, 1), (1, 1, 300001, 33)])
def test_sizes(dtype, B, R, V, n):
    rng = np.random.default_rng(V)
    z = logits(B, R, V, dtype, V + n)
    tokens = rng.integers(0, V, (B, R)).astype(np.int32)
    tokens[0, 0] = int(z[0, 0, :V].float().argmax())
    for T in (1.0, 0.6):
        check(z, V, T, tokens, n)
    check(z, V, 1.0, None, 0)
    check(z, V, 0.0, tokens, n)


def test_largest_row():
    z = logits(1, 1, 1 << 21, torch.bfloat16, 5)
    check(z, 1 << 21, 1.0, np.array([[(1 << 21) - 1]], np.int32), 64)
    z = logits(1, 1, 1 << 20, torch.float32, 5)
    check(z, 1 << 20, 1.3, np.array([[77]], np.int32), 64)


@DT
def test_tail_and_bad_tokens(dtype):
    """-1 leaves its row alone (its logits may hold anything); other ids outside the vocabulary are reported."""
    V, n = 5003, 9
    z = logits(3, 4, V, dtype, 1)
    tokens = np.array([[5, 6, -1, -1], [V - 1, V, 0, -1], [1, -2, 2 ** 31 - 1, 3]], np.int32)
    z[0, 2:] = math.nan
    check(z, V, 1.0, tokens, n, expect=ref.BAD_TOKEN)


@DT
@pytest.mark.parametrize("n", [1, 20, 64])
def test_ties(dtype, n):
    """Equal logits rank by index: all of a row, two levels, zeros of both signs, ties across the n-th place."""
    V = 40007
    z = logits(1, 6, V, dtype, 2)
    z[0, 0, :V] = 1.5
    z[0, 1, :V] = torch.where(torch.arange(V) % 3 == 0, 2.0, -3.0)
    z[0, 2, :V] = torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)
    z[0, 3, :V] = z[0, 3, :V].round()
    z[0, 4, :V] = -5.0
    z[0, 4, [V - 1, 17, 9000, 20001]] = 3.0
    z[0, 5, :V] = torch.linspace(-8, 8, V)       # sorted: the likeliest all in one place
    tokens = np.array([[V - 1, 3, 1, 12345, V - 1, V - 40]], np.int32)
    check(z, V, 1.0, tokens, n)
    check(z, V, 0.0, tokens, n)


@DT
def test_masked_and_extreme(dtype):
    """-inf (also all but one, and as the token), the type's lowest value, large and equal logits, sharp rows."""
    V, n = 9001, 20
    z = logits(1, 8, V, dtype, 3)
    z[0, 0, :V] = -math.inf
    z[0, 0, 7000] = 2.0
    z[0, 1, 5:V] = -math.inf
    z[0, 2, 100:V] = torch.finfo(dtype).min
    z[0, 3, :V] = torch.finfo(dtype).max
    z[0, 4, 77] = 1e4
    z[0, 5, :V] = 1e30
    z[0, 6, :V] *= 1e-20
    z[0, 7, ::2] = -math.inf
    tokens = np.array([[7000, 6, 99, 5, 78, 0, 9000, 0]], np.int32)
    check(z, V, 1.0, tokens, n)
    check(z, V, 0.0, tokens, n)
    check(z, V, 2.0 ** -20, tokens, n)


@DT
@pytest.mark.parametrize("n", [1, 3, 20])
def test_ties_behind_the_last_whole_vector(dtype, n):
    """Equal logits on both sides of a row's last whole vector rank by index like any others, also in rising rows."""
    for V in (9, 4099, 16389, 200001):
        z = logits(1, 3, V, dtype, V + n)
        z[0, 0, V - 12:V] = 50.0
        z[0, 1, :V] = torch.sort(z[0, 1, :V])[0].round()
        z[0, 2, V - 1], z[0, 2, V // 2] = 50.0, 50.0
        check(z, V, 1.0, np.array([[V - 1, V - 2, V // 2]], np.int32), min(n, V))


@DT
@pytest.mark.parametrize("T", [1.0, 1.5, 1e4])
def test_lowest_value_as_the_token(dtype, T):
    """ln p of a token at the type's lowest value is finite where T leaves it in fp32's range, given and among the first."""
    V = 1003
    z = logits(2, 3, V, dtype, 11)
    low = torch.finfo(dtype).min
    z[0, :, 5:V] = low                          # 5 tokens before them
    z[1, 0, :V], z[1, 0, 7] = low, -1e30        # the largest logit far below 0
    z[1, 1, 3::4] = low / 2
    tokens = np.array([[5, 900, 1002], [8, 7, 12]], np.int32)
    check(z, V, T, tokens, 20)


@DT
def test_rows_without_a_distribution(dtype):
    V, n = 3001, 5
    z = logits(2, 3, V, dtype, 4)
    z[0, 0, :V] = -math.inf
    z[0, 1, V - 1] = math.nan
    z[1, 0, 0] = math.inf
    tokens = np.array([[1, 2, 3], [4, V, 6]], np.int32)
    check(z, V, 1.0, tokens, n, expect=ref.BAD_VALUE | ref.BAD_TOKEN)
    check(z, V, 0.0, tokens, n, expect=ref.BAD_VALUE | ref.BAD_TOKEN)


def test_strides_streams_and_graph():
    """Rows inside a wider buffer, a broadcast batch, two streams at once, and a captured call replayed."""
    V, n = 20011, 8
    wide = logits(4, 5, V, torch.bfloat16, 6, pad=64)
    z = wide[1::2, 1:4]
    tokens = np.array([[1, 2, 3], [4, 5, -1]], np.int32)
    first = check(z, V, 1.0, tokens, n)
    check(z[:1].expand(2, 3, z.shape[2]), V, 1.0, tokens, n)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gt = torch.as_tensor(tokens, device="cuda")
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [outputs(2, 3, n) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o in zip(streams, outs):
            ssd.ssd_token_logprobs(z, V, 1.0, tokens=gt, status=st, stream=s, **o)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(o[k], first[k]) for k in o)
    o = outputs(2, 3, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.ssd_token_logprobs(z, V, 1.0, tokens=gt, status=st, **o)
    other = logits(4, 5, V, torch.bfloat16, 7, pad=64)
    want = outputs(2, 3, n)
    ssd.ssd_token_logprobs(other[1::2, 1:4], V, 1.0, tokens=gt, status=st, **want)
    wide.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], want[k]) for k in o)

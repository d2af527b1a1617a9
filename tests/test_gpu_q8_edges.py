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


@pytest.mark.parametrize("d,Hq,Hkv,chains", [(64, 8, 2, 3), (128, 16, 1, 6)], ids=["32-rows", "112-rows"])
def test_step_with_finished_requests(d, Hq, Hkv, chains):
    """A fixed batch of which two requests have ended (length and prefix -1; their table rows, tree and queries hold
    anything): the step's calls leave them out without a flag, and the others get what they get alone."""
    rng = np.random.default_rng(d)
    B, N, nb, maxb, idle = 5, 1 + chains, 60, 12, [1, 4]
    live = [b for b in range(B) if b not in idle]
    lengths = np.array([33, 70, 5, 150, 16], np.int32)
    g = dict(table=torch.full((B, maxb), -1, dtype=torch.int32, device="cuda"),
             pages=torch.zeros(B, dtype=torch.int32, device="cuda"), ring=torch.arange(nb, dtype=torch.int32, device="cuda"),
             pool=torch.tensor([0, nb, 0, 0], dtype=torch.int32, device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.empty(B, N, dtype=torch.int32, device="cuda")

    def tables(length, reserve, s=None):
        ssd.ssd_block_table_update(dev(length), reserve, g["table"], g["pages"], g["ring"], g["pool"], slots=s, status=status)
    tables(lengths, N)
    lengths[idle] = -1
    for _ in range(2):  # the round in which they end, and the next
        tables(lengths, N, slots)
        assert (g["table"][idle] == -1).all() and (slots[idle] == -1).all()
    codes = rng.integers(0, 0x7F, (2, nb, Hkv, 16, d)).astype(np.uint8)
    scale = (2.0 ** rng.integers(-8, -4, (2, nb, Hkv))).astype(np.float32)
    parent = np.zeros((B, N), np.int32)
    parent[:, 0] = -1
    parent[idle] = 999
    x = torch.as_tensor(rng.standard_normal((B, N, Hq + 2 * Hkv, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    x[idle, :, :Hq] = math.nan
    turns = ssd.ssd_rope_frequencies(d)[0].cuda()

    def step(sel):
        t, prefix, par = g["table"][sel].contiguous(), dev(lengths[sel]), dev(parent[sel])
        y = x[sel].contiguous()
        q, k, v = y[:, :, :Hq], y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:]
        qo, ko = torch.full((len(sel), N, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(
            (len(sel), N, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
        c = [dev(codes[0]), dev(codes[1]), dev(scale[0]), dev(scale[1])]
        out, lse = torch.full_like(qo, 7.0), torch.full((len(sel), N, Hq), 7.0, device="cuda")
        ssd.ssd_tree_rope(q, k, turns, d, prefix, qo, ko, parent=par, status=status)
        ssd.ssd_kv_append_q8(ko, v, *c, t, prefix, 0, status=status)
        ssd.ssd_branch_attention_q8(qo, *c, t, prefix, par, out, lse=lse, status=status)
        return qo, ko, out, lse, c
    whole, alone = step(list(range(B))), step(live)
    for a, b in zip(whole[:4], alone[:4]):
        assert torch.equal(a[live], b)
    for a, b in zip(whole[4], alone[4]):
        assert torch.equal(a, b)
    assert (whole[0][idle] == 7).all() and (whole[1][idle] == 7).all()
    assert (whole[2][idle] == 0).all() and (whole[3][idle] == -math.inf).all()
    assert int(status.item()) == 0


def test_rope_chain_behind_the_largest_node():
    """A chain's node numbers pass 32 bits with the tokens: positions go on."""
    S, d, node0 = 5, 64, 2 ** 31 - 3
    x = torch.as_tensor(np.random.default_rng(1).standard_normal((1, S, 2, d)).astype(np.float32)).cuda()
    turns = ssd.ssd_rope_frequencies(d)[0]
    out, status = torch.empty_like(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    ssd.ssd_tree_rope(x, None, turns.cuda(), d, dev(np.array([9], np.int32)), out, None, node0=node0, status=status)
    frac = np.array([[((9 + node0 + s) * int(t)) % 2 ** 64 / 2 ** 64 for t in turns.tolist()] for s in range(S)])
    z = np.exp(2j * math.pi * frac)[None, :, None]
    y = x.cpu().numpy().astype(np.float64)
    w = (y[..., :32] + 1j * y[..., 32:]) * z
    want = np.concatenate([w.real, w.imag], -1)
    # the angle in half-turns rounded to 24 bits, sincospi, two products and a sum: below 2^-20 (|a| + |b|)
    tol = 2.0 ** -20 * np.tile(np.abs(y[..., :32]) + np.abs(y[..., 32:]), 2)
    assert (np.abs(out.cpu().numpy() - want) <= tol).all()
    assert int(status.item()) == 0


@pytest.mark.parametrize("grow", [3, 8, 14])
def test_append_after_a_rejected_row(grow):
    """A row that is large by 2^grow is appended behind accepted rows, rejected, and written over by a small one: the
    block keeps the grown scale, and its accepted rows are what rounding them to that scale leaves: unchanged while they
    are e4m3's normal values there (2^-6 of the scale and more), else off by up to 2^-10 of it."""
    rng = np.random.default_rng(grow)
    H, d = 2, 64
    rows = rng.uniform(0.25, 1, (1, 6, H, d)).astype(np.float32) * np.where(rng.random((1, 6, H, d)) < 0.5, -1, 1)
    rows[0, 0, :, 0] = 1.75   # the scale: 448 = 1.75 * 2^8
    x = torch.as_tensor(rows).to(torch.bfloat16)
    big = (x[:, :1].float() * 2.0 ** grow).to(torch.bfloat16)
    table, status = dev(np.array([[1]], np.int32)), torch.zeros(1, dtype=torch.int32, device="cuda")
    c = [torch.zeros(2, H, 16, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.zeros(2, H, device="cuda") for _ in range(2)]

    def append(rows, at):
        y = rows.cuda()
        ssd.ssd_kv_append_q8(y, y, *c, *s, table, dev(np.array([at], np.int32)), 0, status=status)
    append(x[:, :5], 0)
    before = ref.VALUES[c[0][1].cpu().numpy()][:, :5]
    assert (s[0][1] == 2.0 ** -8).all()
    append(big, 5)                # the draft
    append(x[:, 5:], 5)           # it was rejected: the accepted token takes its place
    assert int(status.item()) == 0
    scale = 2.0 ** (grow - 8)
    assert (s[0][1] == scale).all() and (s[1][1] == scale).all()
    was, now = before * 2.0 ** -8, ref.VALUES[c[0][1].cpu().numpy()][:, :5] * scale
    normal = np.abs(was) >= 2.0 ** -6 * scale
    np.testing.assert_array_equal(now[normal], was[normal])
    assert (np.abs(now - was) <= 2.0 ** -10 * scale).all()
    assert normal.all() == (grow <= 12) and ((now == was).mean() < 0.6) == (grow > 12)
    np.testing.assert_array_equal(c[0].cpu().numpy(), c[1].cpu().numpy())


@pytest.mark.parametrize("Nq", [2, 5], ids=["32-rows", "80-rows"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_scale_at_the_end_of_fp32(d, Nq):
    """A key scale near fp32's largest: a query of zeros has equal scores (0 times a factor past fp32's range is not 0)."""
    rng = np.random.default_rng(d)
    L, N, Hq = 90, Nq, 16
    codes = rng.integers(0, 0x7F, (2, 6, 1, 16, d)).astype(np.uint8)
    table, parent = np.arange(6, dtype=np.int32)[None], np.arange(-1, N - 1, dtype=np.int32)[None]
    q = torch.zeros(1, N, Hq, d, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(1, N, Hq, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssd.ssd_branch_attention_q8(q, dev(codes[0]), dev(codes[1]), torch.full((6, 1), 3e38, device="cuda"),
                                torch.full((6, 1), 0.25, device="cuda"), dev(table), dev(np.array([L], np.int32)), dev(parent),
                                out, lse=lse, scale=2.0, status=status)
    v = ref.VALUES[codes[1][:, 0].reshape(-1, d)] * 0.25
    for i in range(N):
        want = v[:L + i + 1].mean(0)
        # P to 2^-11, the output to 2^-8, sums to 2^-20
        assert (np.abs(out[0, i].double().cpu().numpy() - want) <= (2.0 ** -8 + 2.0 ** -10) * want).all()
        assert (lse[0, i] - math.log(L + i + 1)).abs().max() <= 2.0 ** -18
    assert int(status.item()) == 0

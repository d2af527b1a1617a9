"""The 4-bit cache calls on the GPU against plain 64-bit forms (q4_ref): the
append and the rows read back exactly, attention within tolerances counted
from its roundings, each alone and as one verification pass."""
import math

import numpy as np
import pytest
import torch

import q4_ref as ref
from speculative_decoding_vocab_gb300 import binding as ssd
from speculative_decoding_vocab_gb300 import workloads as w

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_vocab_gb300 import build
    build.build()
    ssd.load()


def dev(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x)).to("cuda", dtype)


def new_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def bf16(x):
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16)


def cache(rng, nb, H, d, lo=-6, hi=3):
    """Random codes and scales."""
    return ref.Cache(rng.integers(0, 16, (nb, H, 16, d)).astype(np.uint8),
                     (127 + rng.integers(lo, hi, (nb, H, 16, d // 32))).astype(np.uint8))


def on_gpu(kc, vc):
    return dev(kc.packed("k")), dev(vc.packed("v")), dev(kc.scale), dev(vc.scale)


# ---------------------------------------------------------------------------
# the append, and the rows read back
# ---------------------------------------------------------------------------
def run_append(kn, vn, kc, vc, table, prefix, node0, count=None):
    """Both sides (torch bf16 rows, Caches changed in place by the reference); flags."""
    g = on_gpu(kc, vc)
    st = new_status()
    ssd.ssd_kv_append_q4(kn.cuda(), vn.cuda(), *g, dev(table), dev(prefix), node0,
                         count=None if count is None else dev(count), status=st)
    flags = 0
    for x, c, which, gc, gs in ((kn, kc, "k", g[0], g[2]), (vn, vc, "v", g[1], g[3])):
        flags |= ref.kv_append(x.double().numpy(), c, table, prefix, node0, count)
        np.testing.assert_array_equal(gs.cpu().numpy(), c.scale)
        np.testing.assert_array_equal(gc.cpu().numpy(), c.packed(which))
    assert int(st.item()) == flags
    return flags


def run_read(kc, vc, table, prefix, node0, S, count=None, dtype=torch.float32, strided=False):
    H, d = kc.codes.shape[1], kc.codes.shape[3]
    B = len(prefix)
    if strided:  # inside a fused buffer
        x = torch.full((B, S, 2 * H + 3, d), 7.0, dtype=dtype, device="cuda")
        outs = x[:, :, 1:1 + H], x[:, :, 2 + H:2 + 2 * H]
    else:
        x = torch.full((2, B, S, H, d), 7.0, dtype=dtype, device="cuda")
        outs = x[0], x[1]
    st = new_status()
    ssd.ssd_kv_read_q4(*on_gpu(kc, vc), dev(table), dev(prefix), node0, *outs,
                       count=None if count is None else dev(count), status=st)
    flags = 0
    for o, c in zip(outs, (kc, vc)):
        want = np.full((B, S, H, d), 7.0)
        flags |= ref.kv_read(c, table, prefix, node0, count, want)
        np.testing.assert_array_equal(o.double().cpu().numpy(), want)
        o.fill_(7.0)
    assert (x == 7.0).all()  # nothing else was written
    assert int(st.item()) == flags
    return flags


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,node0", [(1, 0), (1, 15), (2, 1), (16, 0), (16, 5), (17, 16), (33, 9), (100, 3)])
def test_append_and_read(d, S, node0):
    rng = np.random.default_rng(S * 7 + node0 + d)
    B, H = 4, 3
    maxb = (60 + node0 + S + 15) // 16
    nb = B * maxb + 3
    table = rng.permutation(nb)[:B * maxb].astype(np.int32).reshape(B, maxb)
    kc, vc = cache(rng, nb, H, d), cache(rng, nb, H, d)
    mag = np.exp(rng.normal(0, 3, (B, S, H, d // 32, 1)).repeat(32, -1).reshape(B, S, H, d))
    kn, vn = (bf16(rng.standard_normal((B, S, H, d)) * mag) for _ in range(2))
    prefix = np.array([0, 5, 16, 60], np.int32)
    assert run_append(kn, vn, kc, vc, table, prefix, node0) == 0
    for dtype in (torch.float32, torch.bfloat16):
        assert run_read(kc, vc, table, prefix, node0, S, dtype=dtype, strided=S % 2 == 0) == 0


def test_append_padded_and_strided():
    """A padded batch out of a fused projection: rows past a sequence's count are not written."""
    rng = np.random.default_rng(5)
    B, S, H, d, maxb = 6, 40, 2, 64, 8
    nb = B * maxb
    table = rng.permutation(nb).astype(np.int32).reshape(B, maxb)
    kc, vc = cache(rng, nb, H, d), cache(rng, nb, H, d)
    x = bf16(rng.standard_normal((B, S, 2 * H + 5, d)))
    count = np.array([0, 1, 40, 17, 23, 9], np.int32)
    prefix = np.array([3, 15, 60, 32, 0, -1], np.int32)
    assert run_append(x[:, :, 3:3 + H], x[:, :, 3 + H:3 + 2 * H], kc, vc, table, prefix, 2, count) == 0
    assert run_read(kc, vc, table, prefix, 2, S, count, torch.bfloat16) == 0
    count[2], count[0] = 41, -1
    assert run_append(x[:, :, 3:3 + H], x[:, :, 3 + H:3 + 2 * H], kc, vc, table, prefix, 2, count) == ref.BAD_PREFIX
    assert run_read(kc, vc, table, prefix, 2, S, count) == ref.BAD_PREFIX


def test_append_values():
    """Zeros of both signs, the type's extremes, values that are not finite, every border between two codes."""
    rng = np.random.default_rng(6)
    B, S, H, d, maxb = 8, 20, 2, 64, 3
    nb = B * maxb
    table = rng.permutation(nb).astype(np.int32).reshape(B, maxb)
    kc, vc = cache(rng, nb, H, d), cache(rng, nb, H, d)
    kn, vn = bf16(rng.standard_normal((B, S, H, d))), bf16(rng.standard_normal((B, S, H, d)))
    kn[0] = 0                                   # the smallest scale
    kn[0, :, 0] = -0.0
    vn[1] = vn[1] * 1e38                        # near the largest: some clamped
    vn[1, 0] = torch.finfo(torch.bfloat16).max
    kn[2] = kn[2].sign() * 2.0 ** -133          # subnormal
    kn[1] = kn[1].sign() * 2.0 ** -101          # just below the smallest scale
    vn[2] = 6.0                                 # 6 = 6 * 1: no larger scale
    kn[3, :, 0] = 6.03125                       # just over
    kn[4, 3, 1, 5], kn[4, 4, 0, 0], vn[4, 0, 0, 40] = math.inf, math.nan, -math.inf
    vn[5] = math.nan
    steps = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    borders = np.concatenate([steps, steps * (1 - 2 ** -7), steps * (1 + 2 ** -7), [6.0]])
    kn[6, :, :, :] = bf16(np.resize(np.concatenate([borders, -borders]), 64))
    kn[6, :, :, [0, 32]] = 6.0
    kn[7] = kn[6] * 2.0 ** 20
    prefix = np.array([3, 3, 0, 9, 9, 9, 9, 9], np.int32)
    assert run_append(kn, vn, kc, vc, table, prefix, 0) == ref.BAD_VALUE
    for dtype in (torch.float32, torch.bfloat16):
        run_read(kc, vc, table, prefix, 0, S, dtype=dtype)


def test_read_any_scale():
    """Every scale byte, also those that the append does not write: exact in both types, NaN for 255."""
    rng = np.random.default_rng(8)
    kc, vc = cache(rng, 64, 2, 64), cache(rng, 64, 2, 64)
    kc.scale[:] = np.resize(np.arange(256), kc.scale.shape)
    vc.scale[:] = np.resize(np.arange(256)[::-1], vc.scale.shape)
    table = rng.permutation(64).astype(np.int32).reshape(1, 64)
    # 3, 4 and 6 pass the largest number of both types above 2^125 (byte 252): infinite
    for c in (kc, vc):
        c.codes[np.repeat(c.scale, 32, axis=-1) > 252] &= 9
    for dtype in (torch.float32, torch.bfloat16):
        assert run_read(kc, vc, table, np.array([0], np.int32), 0, 1024, dtype=dtype) == 0


def test_append_and_read_flags():
    rng = np.random.default_rng(7)
    B, S, H, d = 4, 6, 2, 128
    kc, vc = cache(rng, 6, H, d), cache(rng, 6, H, d)
    table = np.array([[0, 1], [2, 9], [3, -1], [4, 5]], np.int32)
    kn, vn = bf16(rng.standard_normal((B, S, H, d))), bf16(rng.standard_normal((B, S, H, d)))
    vn[1, 5] = math.inf                         # a row of a bad block: not written, not reported as a value
    prefix = np.array([28, 12, 30, -2], np.int32)
    assert run_append(kn, vn, kc, vc, table, prefix, 0) == ref.BAD_PREFIX | ref.BAD_BLOCK
    assert run_read(kc, vc, table, prefix, 0, S) == ref.BAD_PREFIX | ref.BAD_BLOCK
    prefix = np.array([2 ** 31 - 3, 12, -1, 5], np.int32)  # positions that pass 31 bits
    assert run_append(kn, vn, kc, vc, table, prefix, 5) == ref.BAD_PREFIX | ref.BAD_BLOCK


def test_append_in_steps_is_append_at_once():
    """Token by token, in pieces or at once: the same cache."""
    rng = np.random.default_rng(9)
    H, d, n = 3, 128, 37
    table = dev(rng.permutation(8).astype(np.int32).reshape(1, 8))
    kn, vn = (bf16(rng.standard_normal((1, n, H, d))).cuda() for _ in range(2))
    prefix, st = dev(np.array([11], np.int32)), new_status()
    got = []
    for step in (1, 2, 5, n):
        g = ssd.q4_cache(8, H, d)
        for o in range(0, n, step):
            ssd.ssd_kv_append_q4(kn[:, o:o + step], vn[:, o:o + step], *g, table, prefix, o, status=st)
        got.append(g)
    for g in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(g, got[0]))
    assert int(st.item()) == 0


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attention_inputs(B, Hq, Hkv, d, lengths, parent, Nq, seed, spread=2, extra_blocks=2):
    """A filled cache over a shuffled pool; what no sequence may see has NaN scales."""
    rng = np.random.default_rng(seed)
    N = len(parent)
    need = [-(-(L + N) // 16) for L in lengths]
    maxb = max(need) + 1
    nb = sum(need) + extra_blocks
    order = rng.permutation(nb).astype(np.int32)
    table = np.full((B, maxb), -1, np.int32)
    kc, vc = cache(rng, nb, Hkv, d, -3 - spread, -2 + spread), cache(rng, nb, Hkv, d, -2 - spread, -1 + spread)
    hidden = np.ones((nb, 16), bool)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        hidden[table[b, :need[b]]] = (np.arange(need[b] * 16) >= lengths[b] + N).reshape(-1, 16)
    for c in (kc, vc):
        c.scale.transpose(0, 2, 1, 3)[hidden] = 255
    q = bf16(rng.standard_normal((B, Nq, Hq, d))).float().numpy()
    return dict(q=q, kc=kc, vc=vc, table=table, prefix=np.array(lengths, np.int32),
                parent=np.broadcast_to(np.asarray(parent, np.int32), (B, N)).copy())


def gpu_attention(a, scale, use_ws=True, want_lse=True, stream=None):
    B, Nq, Hq, d = a["q"].shape
    Hkv = a["kc"].codes.shape[1]
    q = bf16(a["q"]).cuda()
    out = torch.full_like(q, 7.0)
    lse = torch.full((B, Nq, Hq), 7.0, device="cuda") if want_lse else None
    st = new_status()
    n = ssd.ssd_attention_q4_workspace_size(B, Nq, Hq, Hkv, d)
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda") if use_ws else None
    ssd.ssd_branch_attention_q4(q, *on_gpu(a["kc"], a["vc"]), dev(a["table"]), dev(a["prefix"]), dev(a["parent"]), out,
                                lse=lse, scale=scale, status=st, ws=ws, stream=stream)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), None if lse is None else lse.cpu().numpy(), int(st.item())


def check_attention(a, use_ws=True, scale=None, expect=0):
    """Roundings counted.  A score is a fp32 sum (2^-20 of its terms' magnitudes: products and sums truncated
    below 2^-24 of the largest, d <= 128 of them in 4 groups) of a query that may be held as 2^e (q1 + q2), two
    e4m3 terms with max|q| in 2^e [2^7, 2^8): q1 leaves at most 4 bits, which q2 holds but for those below its
    half step 2^-10, so q is off by at most 2^-10 2^e <= 2^-17 max|q| in each element.  A probability p times its
    key's largest v scale t is held in a half: off by 2^-11 of itself, or by 2^-25 where it is subnormal, the
    row's largest lying in [2^11, 2^15]: 2^-36 of that.  A value over t is held in a half, exactly but below
    2^-24 of 2^13: off by at most 2^-38.  Sums of products are fp32 (2^-20), p moves with its score, and the
    output rounds by 2^-8."""
    scale = a["q"].shape[3] ** -0.5 if scale is None else scale
    out, lse, flags = gpu_attention(a, scale, use_ws)
    o, l, weight, (xabs, xcut), (share, cut), rf = ref.attention(
        a["q"], a["kc"], a["vc"], a["table"], a["prefix"], a["parent"], scale, device="cuda")
    assert flags == rf == expect
    dx = 2.0 ** -20 * xabs + 2.0 ** -17 * xcut + 2.0 ** -20
    tol = (2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -20 + 2 * dx[..., None]) * weight + 2.0 ** -36 * share
           + 2.0 ** -38 * cut[..., None] + 1e-30)
    nan = np.isnan(o)
    np.testing.assert_array_equal(np.isnan(out), nan)
    err = np.where(nan, 0, np.abs(out - o))
    bad = err > np.where(nan, 0, tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size}: error {err.max()}, at {np.argwhere(bad)[:3]}"
    fine = np.isfinite(l)
    np.testing.assert_array_equal(np.isfinite(lse), fine)
    np.testing.assert_array_equal(np.isnan(lse), np.isnan(l))
    # lse = ln 2 (m + log2 sum): the score, the sum's 2^-20, and the last rounding
    assert (np.abs(lse[fine] - l[fine]) <= (dx + 2.0 ** -20 + 2.0 ** -22 * np.abs(l))[fine]).all()
    return out, lse


CHAIN = lambda n: list(range(-1, n - 1))  # noqa: E731


@pytest.mark.parametrize("use_ws", [True, False], ids=["split", "unsplit"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,lengths,parent,Nq", [
    (1, 1, [0], CHAIN(1), 1),
    (8, 2, [1, 127, 128], CHAIN(1), 1),
    (16, 1, [500, 3, 15, 16], CHAIN(4), 4),                     # 64 rows
    (6, 1, [255, 256, 257], CHAIN(8), 8),                       # 48 rows
    (12, 4, [70, 200], list(w.branch_tree(3, (3, 2, 1, 1), [4] * 7)), 28),   # 84 rows, group 3
    (4, 4, [33, 90, 129], list(w.branch_tree(4, (8, 4, 2, 1, 1), [1 + i % 4 for i in range(16)])), 36),
    (32, 2, [260, 61], CHAIN(9), 9),                            # 144 rows: two row tiles
    (7, 1, [3000, 10], CHAIN(5), 3),
    (8, 1, [9000], CHAIN(2), 1),
], ids=["one-key", "single", "gqa16", "rows48", "tree", "ragged-tree", "two-tiles", "long-short", "long"])
def test_attention(use_ws, d, Hq, Hkv, lengths, parent, Nq):
    check_attention(attention_inputs(len(lengths), Hq, Hkv, d, lengths, parent, Nq, seed=Hq + len(lengths)),
                    use_ws=use_ws)


@pytest.mark.parametrize("use_ws", [True, False], ids=["split", "unsplit"])
@pytest.mark.parametrize("d,Hq,Hkv,Nq", [(64, 2, 2, 1), (128, 16, 1, 8), (128, 4, 1, 9), (64, 16, 1, 4)])
@pytest.mark.parametrize("B,long", [(151, ()), (153, (0,)), (700, (13, 350, 699)), (320, (100, 101, 102))])
def test_attention_many_short_sequences(use_ws, d, Hq, Hkv, Nq, B, long):
    """Hundreds of sequences of one tile and a few of many."""
    rng = np.random.default_rng(B + d)
    lengths = [int(x) for x in rng.integers(0, 40, B)]
    for b in long:
        lengths[b] = 2500 + b
    check_attention(attention_inputs(B, Hq, Hkv, d, lengths, CHAIN(Nq), Nq, seed=B), use_ws=use_ws)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 5, 16])
def test_attention_largest_trees(d, group):
    """128 nodes, all of them queries: a random tree, nodes across key tiles."""
    rng = np.random.default_rng(group)
    parent = [-1] + [int(rng.integers(-1, m)) for m in range(1, 128)]
    check_attention(attention_inputs(2, group, 1, d, [100, 1], parent, 128, seed=group))


# (query heads of one KV head, nodes before the queries, queries): rows on either side of 64
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,spine,Nq", [(8, 2, 22, 2), (16, 1, 60, 5), (3, 1, 2, 65)])
def test_attention_query_after_spine(d, Hq, Hkv, spine, Nq):
    """Nodes before the queries are keys alone; lengths at every place of a tile."""
    parent = CHAIN(spine) + [spine // 3 if i % 3 else i + spine - 1 for i in range(Nq)]
    check_attention(attention_inputs(17, Hq, Hkv, d, [111 + i for i in range(17)], parent, Nq, seed=4))


ROWS = [(4, 1, 2), (16, 1, 5)]  # Hq, Hkv, Nq: 8 and 80 rows


@pytest.mark.parametrize("Hq,Hkv,Nq", ROWS)
@pytest.mark.parametrize("d", [64, 128])
def test_attention_sharp_and_flat(d, Hq, Hkv, Nq):
    """Scores far apart (one key takes all), a late maximum, equal scores, and an attention sink whose value is 0."""
    a = attention_inputs(3, Hq, Hkv, d, [700, 3000, 700], CHAIN(Nq), Nq, seed=9, spread=0)
    check_attention(a, scale=1.0)
    a["q"][1] = 0

    def key(pos, size):
        a["kc"].codes[a["table"][2, pos // 16], 0, pos % 16] = ref.e2m1_round(np.sign(a["q"][2, 0, 0]) * 6.0)
        a["kc"].scale[a["table"][2, pos // 16], 0, pos % 16] = 127 + size
    check_attention(a)
    key(0, 1)
    a["vc"].codes[a["table"][2, 0], 0, 0] = 0
    a["vc"].scale[a["table"][2, 0], 0, 0] = 27
    check_attention(a)
    key(0, -3)
    key(647, 2)
    check_attention(a)


@pytest.mark.parametrize("Hq,Hkv,Nq", [(4, 2, 3), (32, 2, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_scales(d, Hq, Hkv, Nq):
    """Scales that are tiny, huge, far apart between keys and between the groups of a key."""
    a = attention_inputs(4, Hq, Hkv, d, [300, 300, 300, 40], CHAIN(Nq), Nq, seed=21)
    t, ks, vs = a["table"], a["kc"].scale, a["vc"].scale
    rng = np.random.default_rng(3)
    vs[t[0, :18]] = 27                            # no value to speak of but at the end
    some = t[1, ::2][t[1, ::2] >= 0]
    vs[some] -= 30
    some = t[2, :18]
    vs[some] = 127 + rng.integers(-20, 20, vs[some].shape)   # groups of a key by up to 2^40 apart
    some = t[3, :2]
    ks[some] = 0                                  # all scores equal but for the last block's
    check_attention(a)
    vs[t[3, :2]] = 27 + 10
    vs[t[1, :18]] += 90
    vs[t[0, :18]] = rng.integers(0, 60, vs[t[0, :18]].shape)  # around the smallest that counts
    check_attention(a)
    vs[t[0, :18]] = 250                           # around the largest
    vs[t[0, 1:18:2]] = 220
    check_attention(a)


@pytest.mark.parametrize("Hq,Hkv,Nq", [(4, 2, 2), (32, 2, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_bad_blocks(d, Hq, Hkv, Nq):
    """Bad ids and short tables hide keys; a row may be left without any; slots without a request."""
    a = attention_inputs(5, Hq, Hkv, d, [200, 60, 14, 40, 100], CHAIN(Nq), Nq, seed=30)
    a["table"][0, 3] = 10 ** 6
    a["table"][1, :] = -1                         # nothing left: 0 and -inf
    out, lse = check_attention(a, expect=ssd.FLAG_BAD_BLOCK)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    a["prefix"][2], a["prefix"][3], a["prefix"][4] = 16 * a["table"].shape[1] - 1, -7, -1
    a["parent"][0, 1] = 1
    a["parent"][4, 0] = 77                        # of the slot without a request: not looked at
    out, lse = check_attention(a, expect=ssd.FLAG_BAD_BLOCK | ssd.FLAG_BAD_PREFIX | ssd.FLAG_BAD_TREE)
    assert (out[4] == 0).all() and (lse[4] == -math.inf).all()


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (32, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_nan(d, Hq, Hkv):
    """A NaN scale reaches the rows that see it, and no other: in k the whole row, in v its group, in q its row."""
    G = Hq // Hkv
    parent = [-1, 0, 0, 1, 2]                     # 1 and 2 are siblings
    for length in (5, 126, 300, 1500):
        a = attention_inputs(2, Hq, Hkv, d, [length, 40], parent, 5, seed=40 + length)

        def at(b, pos, h, group):
            return a["table"][b, pos // 16], h, pos % 16, group
        a["vc"].scale[at(0, length + 1, 0, 0)] = 255        # a tree node: seen by itself and node 3
        a["kc"].scale[at(0, length + 2, 1, 1)] = 255        # a tree node: seen by itself and node 4
        a["vc"].scale[at(1, 7, 1, d // 32 - 1)] = 255       # the prefix: seen by all
        out, _ = check_attention(a)
        assert np.isnan(out).sum() == 2 * G * 32 + 2 * G * d + 5 * G * 32
        a["q"][0, 3, 1, 0] = math.inf
        o, l, st = gpu_attention(a, 0.1)
        assert np.isnan(o[0, 3, 1]).all() and np.isnan(l[0, 3, 1]) and not np.isnan(o[0, 3, 0, 32:]).any()


def test_attention_two_streams_and_graph():
    """Two calls at once with workspaces of their own, and a captured call replayed on new inputs."""
    sets = [attention_inputs(3, 8, 2, 128, [4000, 50, 900], CHAIN(4), 4, seed=50 + i) for i in range(3)]
    B, Nq, Hq, d = sets[0]["q"].shape
    base = [gpu_attention(a, 0.1) for a in sets]
    g = [dict(qb=bf16(a["q"]).cuda(), cache=on_gpu(a["kc"], a["vc"]),
              **{k: dev(a[k]) for k in ("table", "prefix", "parent")}) for a in sets[:2]]
    for x in g:
        x["out"] = torch.empty(B, Nq, Hq, d, dtype=torch.bfloat16, device="cuda")
        x["lse"], x["st"] = torch.empty(B, Nq, Hq, device="cuda"), new_status()
        x["ws"] = torch.empty(max(256, ssd.ssd_attention_q4_workspace_size(B, Nq, Hq, 2, d)), dtype=torch.uint8,
                              device="cuda")
        x["s"] = torch.cuda.Stream()
    torch.cuda.synchronize()

    def launch(x, stream=None):
        ssd.ssd_branch_attention_q4(x["qb"], *x["cache"], x["table"], x["prefix"], x["parent"],
                                    x["out"], lse=x["lse"], scale=0.1, status=x["st"], ws=x["ws"], stream=stream)
    for _ in range(20):
        for x in g:
            launch(x, x["s"])
    torch.cuda.synchronize()
    for x, (o, l, _) in zip(g, base):
        np.testing.assert_array_equal(x["out"].float().cpu().numpy(), o)
        np.testing.assert_array_equal(x["lse"].cpu().numpy(), l)
    x = g[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        launch(x)
    for to, new in zip(x["cache"], on_gpu(sets[2]["kc"], sets[2]["vc"])):
        to.copy_(new)
    for k in ("table", "prefix", "parent"):
        x[k].copy_(dev(sets[2][k]))
    x["qb"].copy_(bf16(sets[2]["q"]))
    graph.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(x["out"].float().cpu().numpy(), base[2][0])
    np.testing.assert_array_equal(x["lse"].cpu().numpy(), base[2][1])


def test_attention_without_lse_and_repeated():
    """The same call twice gives the same bits; without the log-sum-exp too."""
    for d in (64, 128):
        a = attention_inputs(2, 8, 2, d, [1500, 700], CHAIN(6), 6, seed=60)
        o1, l1, _ = gpu_attention(a, 0.125)
        o2, l2, _ = gpu_attention(a, 0.125)
        o3, _, _ = gpu_attention(a, 0.125, want_lse=False)
        np.testing.assert_array_equal(o1, o2)
        np.testing.assert_array_equal(l1, l2)
        np.testing.assert_array_equal(o1, o3)

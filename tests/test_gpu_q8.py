"""The 8-bit cache calls on the GPU against plain 64-bit forms (q8_ref):
block tables and the append exactly, rotary positions and attention within
tolerances counted from their roundings, each alone and as one decode step."""
import math

import numpy as np
import pytest
import torch

import q8_ref as ref
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


# ---------------------------------------------------------------------------
# block tables
# ---------------------------------------------------------------------------
def table_state(rng, B, maxb, n, free, head=None):
    """Empty tables and a ring of `free` shuffled free blocks (the others are someone else's)."""
    ring = np.full(n, -1, np.int32)
    head = int(rng.integers(0, n)) if head is None else head
    ring[(head + np.arange(free)) % n] = rng.permutation(n)[:free]
    return dict(table=np.full((B, maxb), -1, np.int32), pages=np.zeros(B, np.int32), ring=ring,
                pool=np.array([head, free, 0, 0], np.int32))


def run_tables(st, length, reserve, S):
    """One call on both sides; compares everything and keeps the new state."""
    g = {k: dev(v) for k, v in st.items()}
    slots = torch.full((len(length), S), -9, dtype=torch.int32, device="cuda") if S else None
    status = new_status()
    ssd.ssd_block_table_update(dev(length), reserve, g["table"], g["pages"], g["ring"], g["pool"], slots=slots,
                               status=status)
    want, flags = ref.block_table_update(length, reserve, st["table"], st["pages"], st["ring"], st["pool"], S)
    for k in st:
        np.testing.assert_array_equal(g[k].cpu().numpy(), st[k], err_msg=k)
    if S:
        np.testing.assert_array_equal(slots.cpu().numpy(), want)
    assert int(status.item()) == flags
    return flags


@pytest.mark.parametrize("B", [1, 2, 63, 64, 65, 200, 1025, 2100])
@pytest.mark.parametrize("S", [0, 1, 21])
def test_block_tables_over_rounds(B, S):
    rng = np.random.default_rng(B * 31 + S)
    maxb = 40
    st = table_state(rng, B, maxb, B * 30 + 7, B * 30 + 7)
    length = rng.integers(0, 200, B).astype(np.int32)
    for step in range(5):
        run_tables(st, length, S, S)                         # room for the tree
        length = np.where(rng.random(B) < 0.1, -1, length + rng.integers(0, S + 2, B)).astype(np.int32)
        run_tables(st, length, 0, 0)                         # the accepted tokens alone
        length = np.where(length < 0, rng.integers(0, 150, B), length).astype(np.int32)
    assert st["pool"][1] + st["pages"].sum() == B * 30 + 7   # no block lost


@pytest.mark.parametrize("B", [3, 130])
def test_block_tables_run_out(B):
    rng = np.random.default_rng(B)
    st = table_state(rng, B, 64, 10 * B, 5 * B + 2)
    assert run_tables(st, rng.integers(100, 160, B).astype(np.int32), 0, 17) == ref.NO_BLOCKS
    run_tables(st, np.full(B, -1, np.int32), 5, 3)
    assert st["pool"][1] == 5 * B + 2 and (st["table"] == -1).all()


def test_block_tables_bad_input():
    rng = np.random.default_rng(0)
    st = table_state(rng, 4, 8, 64, 40)
    st["pages"][:] = [9, -3, 0, 2]
    st["table"][0] = [0, 1, 2, 3, 4, 5, 6, 7]
    st["table"][3, :2] = [8, 9]
    flags = run_tables(st, np.array([5, 17, 129, 2 ** 31 - 1], np.int32), 2 ** 31 - 1 - 2 ** 30, 4)
    assert flags == ref.BAD_PREFIX
    flags = run_tables(st, np.array([5, 17, 129, 30], np.int32), 0, 4)
    assert flags == ref.BAD_PREFIX
    for head, free in ((64, 3), (-1, 3), (0, 65), (0, -1)):
        st = table_state(rng, 2, 8, 64, 40)
        st["pool"][:2] = head, free
        assert run_tables(st, np.array([0, 20], np.int32), 0, 2) & ref.BAD_PREFIX


def test_block_tables_captured():
    """A captured pair of updates replayed over changing lengths."""
    rng = np.random.default_rng(3)
    B, S, n = 100, 6, 2000
    st = table_state(rng, B, 24, n, n)
    g = {k: dev(v) for k, v in st.items()}
    length, after = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    slots, status = torch.zeros(B, S, dtype=torch.int32, device="cuda"), new_status()

    def step():
        ssd.ssd_block_table_update(length, S, g["table"], g["pages"], g["ring"], g["pool"], slots=slots, status=status)
        ssd.ssd_block_table_update(after, 0, g["table"], g["pages"], g["ring"], g["pool"], status=status)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ln = rng.integers(0, 60, B).astype(np.int32)
    for _ in range(6):
        nx = (ln + rng.integers(0, S + 1, B)).astype(np.int32)
        length.copy_(dev(ln))
        after.copy_(dev(nx))
        graph.replay()
        want, f0 = ref.block_table_update(ln, S, st["table"], st["pages"], st["ring"], st["pool"], S)
        _, f1 = ref.block_table_update(nx, 0, st["table"], st["pages"], st["ring"], st["pool"], 0)
        for k in st:
            np.testing.assert_array_equal(g[k].cpu().numpy(), st[k], err_msg=k)
        np.testing.assert_array_equal(slots.cpu().numpy(), want)
        ln = nx
    assert int(status.item()) == 0 and f0 == f1 == 0


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def rope_close(got, x, want, rot, mscale, bf16):
    """fp32: the angle in half-turns is rounded to 24 bits (at most 2^-25 half-turns = 2^-25 pi rad), sincospi
    is good to 2 units in the last place of 1 (2^-23), the factor mscale, two products and a sum round by 2^-24
    each: below 2^-20 mscale (|a| + |b|) together.  bf16 then rounds the result by half a step, 2^-8."""
    x = np.abs(x.astype(np.float64))
    pair = np.zeros_like(x)
    pair[..., :rot] = x[..., :rot].max(axis=-1, keepdims=True) * 2  # no element's pair is larger
    tol = 2.0 ** -20 * mscale * pair + (2.0 ** -8 * np.abs(want) if bf16 else 0)
    err = np.abs(got.astype(np.float64) - want)
    assert (err <= tol).all(), f"error {err.max()} at {np.unravel_index((err - tol).argmax(), err.shape)}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("B,S,Hq,Hkv,d,rot", [
    (1, 1, 1, 1, 64, 64), (3, 5, 8, 2, 64, 32), (2, 17, 4, 4, 128, 128), (2, 3, 7, 1, 80, 24), (1, 300, 3, 3, 64, 2),
    (2, 4, 2, 1, 10, 6), (1, 2, 2, 2, 512, 512)])
def test_rope_chain(dtype, interleaved, B, S, Hq, Hkv, d, rot):
    """Tokens of a chain (prompts): far positions, all widths of access, parts of the head."""
    g = torch.Generator().manual_seed(B * S + d)
    q = torch.randn(B, S, Hq, d, generator=g).to("cuda", dtype)
    k = torch.randn(B, S, Hkv, d, generator=g).to("cuda", dtype)
    turns, mscale = ssd.ssd_rope_frequencies(rot, 10000.0, 8.0, 4096.0)
    prefix = np.array([0, 131071, 2 ** 31 - 400][:B], np.int32)
    qo, ko, st = torch.empty_like(q), torch.empty_like(k), new_status()
    ssd.ssd_tree_rope(q, k, turns.cuda(), rot, dev(prefix), qo, ko, node0=7, interleaved=interleaved, mscale=mscale,
                      status=st)
    theta = turns.numpy().astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    pos = prefix.astype(np.int64)[:, None] + 7 + np.arange(S)
    # the angle modulo a turn from the integers, so that the reference keeps its bits at far positions
    frac = np.array([[[((int(p) * int(t)) % 2 ** 64) / 2 ** 64 for t in turns.tolist()] for p in row] for row in pos])
    for x, o in ((q, qo), (k, ko)):
        xs = x.float().cpu().numpy()
        want = ref.rope(xs, theta, rot, np.zeros_like(pos), interleaved, 1.0)  # shape and copied part
        ang = frac * 2 * math.pi
        c, s = np.cos(ang)[:, :, None] * mscale, np.sin(ang)[:, :, None] * mscale
        i0, i1 = ((np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved
                  else (np.arange(rot // 2), np.arange(rot // 2, rot)))
        a, b = xs[..., i0].astype(np.float64), xs[..., i1].astype(np.float64)
        want[..., i0], want[..., i1] = a * c - b * s, a * s + b * c
        rope_close(o.float().cpu().numpy(), xs, want, rot, mscale, dtype == torch.bfloat16)
    assert int(st.item()) == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_tree_in_place_strided(interleaved):
    """The fed nodes of a branch tree, inside a fused projection, in place; the value heads stay as they are."""
    B, Hq, Hkv, d, K, F, steps = 3, 6, 2, 64, 4, (4, 2, 1, 1, 1), 3
    S = sum(F)
    parent = w.fill_tree(K, F, steps)
    node0 = len(parent) - S
    g = torch.Generator().manual_seed(1)
    x = torch.randn(B, S, Hq + 2 * Hkv, d, generator=g).to("cuda", torch.bfloat16)
    before = x.float().cpu().numpy()
    prefix = np.array([0, 77, 100000], np.int32)
    turns, _ = ssd.ssd_rope_frequencies(48)
    st = new_status()
    q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
    par = dev(np.broadcast_to(parent, (B, len(parent))))
    ssd.ssd_tree_rope(q, k, turns.cuda(), 48, dev(prefix), q, k, parent=par, node0=node0, interleaved=interleaved,
                      status=st)
    theta = turns.numpy().astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    pos = prefix[:, None].astype(np.int64) + np.array(ref.depths(parent, node0, S))
    after = x.float().cpu().numpy()
    want = ref.rope(before, theta, 48, pos, interleaved, 1.0)
    rope_close(after[:, :, :Hq + Hkv], before[:, :, :Hq + Hkv], want[:, :, :Hq + Hkv], 48, 1.0, True)
    np.testing.assert_array_equal(after[:, :, Hq + Hkv:], before[:, :, Hq + Hkv:])
    assert int(st.item()) == 0
    # one operand alone, flags: a bad parent ends the path, a negative prefix counts as 0
    ko = torch.empty(B, S, Hkv, d, dtype=torch.bfloat16, device="cuda")
    par[0, node0] = node0
    ssd.ssd_tree_rope(None, k, turns.cuda(), 48, dev(np.array([0, 77, -4], np.int32)), None, ko, parent=par,
                      node0=node0, interleaved=interleaved, status=st)
    pos[0, 0], pos[2] = 0, pos[2] - 100000
    kb = after[:, :, Hq:Hq + Hkv]
    rope_close(ko.float().cpu().numpy(), kb, ref.rope(kb, theta, 48, pos, interleaved, 1.0), 48, 1.0, True)
    assert int(st.item()) == ssd.FLAG_BAD_TREE | ssd.FLAG_BAD_PREFIX


# ---------------------------------------------------------------------------
# the quantising append
# ---------------------------------------------------------------------------
def cache(rng, nb, H, d, lo=-6, hi=3):
    """Random finite codes (no NaN) and power-of-two scales."""
    c = rng.integers(0, 256, (nb, H, 16, d)).astype(np.uint8)
    c[(c & 0x7F) == 0x7F] = 0x3A
    return c, (2.0 ** rng.integers(lo, hi, (nb, H))).astype(np.float32)


def bf16(x):
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16)


def run_append(kn, vn, kc, ks, vc, vs, table, prefix, node0, count=None, u8=True):
    """Both sides (torch bf16 rows on the CPU, numpy caches changed in place by the reference); flags."""
    gk, gv, gks, gvs = dev(kc), dev(vc), dev(ks), dev(vs)
    st = new_status()
    a, b = (gk, gv) if u8 else (gk.view(torch.float8_e4m3fn), gv.view(torch.float8_e4m3fn))
    ssd.ssd_kv_append_q8(kn.cuda(), vn.cuda(), a, b, gks, gvs, dev(table), dev(prefix), node0,
                         count=None if count is None else dev(count), status=st)
    flags = 0
    for x, c, s, gc, gs in ((kn, kc, ks, gk, gks), (vn, vc, vs, gv, gvs)):
        flags |= ref.kv_append(x.double().numpy(), c, s, table, prefix, node0, count)
        np.testing.assert_array_equal(gs.cpu().numpy(), s)
        got = gc.cpu().numpy()
        bad = got != c
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], c[bad][:4])
    assert int(st.item()) == flags
    return flags


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,node0", [(1, 0), (1, 15), (16, 0), (16, 5), (17, 16), (33, 9), (100, 3)])
def test_append(d, S, node0):
    rng = np.random.default_rng(S * 7 + node0 + d)
    B, H = 4, 3
    maxb = (60 + node0 + S + 15) // 16
    nb = B * maxb + 3
    table = rng.permutation(nb)[:B * maxb].astype(np.int32).reshape(B, maxb)
    kc, ks = cache(rng, nb, H, d)
    vc, vs = cache(rng, nb, H, d)
    mag = np.exp(rng.normal(0, 3, (B, S, H, 1)))  # rows of unequal size: scales grow, or stay
    kn, vn = (bf16(rng.standard_normal((B, S, H, d)) * mag) for _ in range(2))
    assert run_append(kn, vn, kc, ks, vc, vs, table, np.array([0, 5, 16, 60], np.int32), node0, u8=S % 2 == 0) == 0


def test_append_padded_and_strided():
    """A padded batch out of a fused projection: rows past a sequence's count are not written."""
    rng = np.random.default_rng(5)
    B, S, H, d, maxb = 5, 40, 2, 64, 8
    nb = B * maxb
    table = rng.permutation(nb).astype(np.int32).reshape(B, maxb)
    kc, ks = cache(rng, nb, H, d)
    vc, vs = cache(rng, nb, H, d)
    x = bf16(rng.standard_normal((B, S, 2 * H + 5, d)))
    count = np.array([0, 1, 40, 17, 23], np.int32)
    prefix = np.array([3, 15, 60, 32, 0], np.int32)
    run_append(x[:, :, 3:3 + H], x[:, :, 3 + H:3 + 2 * H], kc, ks, vc, vs, table, prefix, 2, count)
    count[2], count[0] = 41, -1
    assert run_append(x[:, :, 3:3 + H], x[:, :, 3 + H:3 + 2 * H], kc, ks, vc, vs, table, prefix, 2,
                      count) == ref.BAD_PREFIX


def test_append_values():
    """Zeros, the type's extremes, non-finite values, exact 448 borders, scales that another program wrote."""
    rng = np.random.default_rng(6)
    B, S, H, d, maxb = 8, 20, 2, 64, 3
    nb = B * maxb
    table = rng.permutation(nb).astype(np.int32).reshape(B, maxb)
    kc, ks = cache(rng, nb, H, d)
    vc, vs = cache(rng, nb, H, d)
    kn, vn = bf16(rng.standard_normal((B, S, H, d))), bf16(rng.standard_normal((B, S, H, d)))
    kn[0] = 0                                   # the smallest scale
    vn[1] = vn[1] * 1e38                        # near the largest
    kn[2] = kn[2].sign() * 2.0 ** -133          # subnormal
    vn[2] = 448.0                               # 448 = 448 * 1: no larger scale
    kn[3, :, 0] = 450.0                         # just over
    kn[4, 3, 1, 5], kn[4, 4, 0, 0], vn[4, 0, 0, 9] = math.inf, math.nan, -math.inf
    vn[5] = math.nan
    prefix = np.array([3, 3, 0, 9, 9, 9, 9, 9], np.int32)
    ks[table[6, 0]] = 0.3                       # not a power of two: kept where it suffices
    vs[table[6, 0]] = 0.003                     # and where it grows
    ks[table[7, 0]] = [0.0, 1e30]
    assert run_append(kn, vn, kc, ks, vc, vs, table, prefix, 0) == ref.BAD_VALUE
    vs[table[7, 0]] = [math.nan, -1.0]          # bad scales count as 0
    ks[table[7, 0]] = [math.inf, 1.0]
    assert run_append(kn[7:], vn[7:], kc, ks, vc, vs, table[7:], prefix[7:], 0) == ref.BAD_VALUE


def test_append_flags():
    rng = np.random.default_rng(7)
    B, S, H, d = 4, 6, 2, 128
    kc, ks = cache(rng, 6, H, d)
    vc, vs = cache(rng, 6, H, d)
    table = np.array([[0, 1], [2, 9], [3, -1], [4, 5]], np.int32)
    kn, vn = bf16(rng.standard_normal((B, S, H, d))), bf16(rng.standard_normal((B, S, H, d)))
    prefix = np.array([28, 12, 30, -2], np.int32)
    assert run_append(kn, vn, kc, ks, vc, vs, table, prefix, 0) == ref.BAD_PREFIX | ref.BAD_BLOCK


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attention_inputs(B, Hq, Hkv, d, lengths, parent, Nq, seed, spread=3, extra_blocks=2):
    """A filled cache over a shuffled pool; what no sequence may see holds NaN codes."""
    rng = np.random.default_rng(seed)
    N = len(parent)
    need = [-(-(L + N) // 16) for L in lengths]
    maxb = max(need) + 1
    nb = sum(need) + extra_blocks
    order = rng.permutation(nb).astype(np.int32)
    table = np.full((B, maxb), -1, np.int32)
    at = 0
    kc, ks = np.full((nb, Hkv, 16, d), 0x7F, np.uint8), np.full((nb, Hkv), np.nan, np.float32)
    vc, vs = kc.copy(), ks.copy()
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        n = lengths[b] + N
        for c, s in ((kc, ks), (vc, vs)):
            x = rng.standard_normal((need[b] * 16, Hkv, d)) * np.exp(0.3 * rng.standard_normal((1, Hkv, d)))
            x[:, :, :] *= np.repeat(2.0 ** rng.integers(-spread, spread + 1, (need[b], Hkv, 1)), 16, axis=0)
            x = x.reshape(need[b], 16, Hkv, d).transpose(0, 2, 1, 3)
            sc = 2.0 ** np.ceil(np.log2(np.abs(x).max(axis=(2, 3)) / 448))
            codes = ref.e4m3_round((x / sc[:, :, None, None]).astype(np.float32).astype(np.float64))
            flat = codes.transpose(0, 2, 1, 3).reshape(-1, Hkv, d)
            flat[n:] = 0x7F  # the last block's slots behind the sequence
            c[table[b, :need[b]]] = flat.reshape(need[b], 16, Hkv, d).transpose(0, 2, 1, 3)
            s[table[b, :need[b]]] = sc
    q = bf16(rng.standard_normal((B, Nq, Hq, d))).float().numpy()
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, prefix=np.array(lengths, np.int32),
                parent=np.broadcast_to(np.asarray(parent, np.int32), (B, N)).copy())


def gpu_attention(a, scale, use_ws=True, want_lse=True, stream=None):
    B, Nq, Hq, d = a["q"].shape
    Hkv = a["ks"].shape[1]
    g = {k: dev(v) for k, v in a.items()}
    q = g["q"].to(torch.bfloat16)
    out = torch.full_like(q, 7.0)
    lse = torch.full((B, Nq, Hq), 7.0, device="cuda") if want_lse else None
    st = new_status()
    n = ssd.ssd_attention_q8_workspace_size(B, Nq, Hq, Hkv, d)
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda") if use_ws else None
    ssd.ssd_branch_attention_q8(q, g["kc"], g["vc"], g["ks"], g["vs"], g["table"], g["prefix"], g["parent"], out,
                                lse=lse, scale=scale, status=st, ws=ws, stream=stream)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), None if lse is None else lse.cpu().numpy(), int(st.item())


def check_attention(a, use_ws=True, scale=None, expect=0):
    """Roundings counted.  A probability is held as two e4m3 terms, half a step of the first taken up by the
    second to half a step: 2^-4 * 2^-4 = 2^-8, and where the second, 32 (p - p1), underflows (half a step of 2^-9)
    2^-15, the row's largest p v_scale lying in [2^4, 2^8]: 2^-19 of it.  A
    score is a fp32 sum (2^-20 of its terms' magnitudes: products and sums truncated below 2^-24 of the largest,
    d <= 128 of them in 4 groups) of a query held as 2^e (q1 + q2) with max|q| in 2^e [2^7, 2^8): q1 leaves at
    most 4 bits, which q2 holds but for those below its half step 2^-10, so q is off by at most 2^-10 2^e <=
    2^-17 max|q| in each element; both move p by as much.  The output rounds by 2^-8."""
    scale = a["q"].shape[3] ** -0.5 if scale is None else scale
    out, lse, flags = gpu_attention(a, scale, use_ws)
    o, l, weight, (xabs, xcut), share, rf = ref.attention(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["prefix"],
                                                  a["parent"], scale, device="cuda")
    assert flags == rf == expect
    dx = 2.0 ** -20 * xabs + 2.0 ** -17 * xcut + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * dx[..., None]) * weight + 2.0 ** -19 * share + 1e-30
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
    (12, 4, [70, 200], list(w.branch_tree(3, (3, 2, 1, 1), [4] * 7)), 28),   # 84 rows, group 3
    (4, 4, [33, 90, 129], list(w.branch_tree(4, (8, 4, 2, 1, 1), [1 + i % 4 for i in range(16)])), 36),
    (32, 2, [260, 61], CHAIN(9), 9),                            # 144 rows: two row tiles
    (7, 1, [3000, 10], CHAIN(5), 3),
    (8, 1, [9000], CHAIN(2), 1),
], ids=["one-key", "single", "gqa16", "tree", "ragged-tree", "two-tiles", "long-short", "long"])
def test_attention(use_ws, d, Hq, Hkv, lengths, parent, Nq):
    check_attention(attention_inputs(len(lengths), Hq, Hkv, d, lengths, parent, Nq, seed=Hq + len(lengths)),
                    use_ws=use_ws)


@pytest.mark.parametrize("use_ws", [True, False], ids=["split", "unsplit"])
@pytest.mark.parametrize("d,Hq,Hkv,Nq", [(64, 2, 2, 1), (128, 16, 1, 8), (128, 4, 1, 9)])
@pytest.mark.parametrize("B,long", [(151, ()), (153, (0,)), (700, (13, 350, 699)), (320, (100, 101, 102))])
def test_attention_many_short_sequences(use_ws, d, Hq, Hkv, Nq, B, long):
    """Hundreds of sequences of one tile and a few of many: pieces begin and end at any place of an item, its end
    included, and a CTA runs many items."""
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


@pytest.mark.parametrize("d", [64, 128])
def test_attention_query_after_spine(d):
    """Few queries behind a long tree (the nodes before them are keys alone), lengths at every place of a tile."""
    parent = CHAIN(20) + [3, 3, 20, 21]
    check_attention(attention_inputs(17, 8, 2, d, [111 + i for i in range(17)], parent, 2, seed=4))


def test_attention_sharp_and_flat():
    """Scores far apart (one key takes all), a late maximum, equal scores, and an attention sink."""
    a = attention_inputs(3, 4, 1, 128, [700, 700, 700], CHAIN(2), 2, seed=9, spread=0)
    check_attention(a, scale=1.0)
    a["q"][1] = 0
    one = a["kc"][a["table"][2, 0], 0, 0].copy()
    a["kc"][a["table"][2, 0], 0, 0] = ref.e4m3_round(np.sign(a["q"][2, 0, 0]) * 20.0)
    check_attention(a)
    a["kc"][a["table"][2, 0], 0, 0] = one
    a["kc"][a["table"][2, 40], 0, 7] = ref.e4m3_round(np.sign(a["q"][2, 0, 0]) * 60.0)
    check_attention(a)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_scales(d):
    """Block scales that are zero, tiny, huge, not powers of two, far apart."""
    a = attention_inputs(4, 4, 2, d, [300, 300, 300, 40], CHAIN(3), 3, seed=21)
    t = a["table"]
    a["vs"][t[0, :19]] = 0.0                      # no value anywhere but in the last block
    a["vs"][t[1, ::2][t[1, ::2] >= 0]] *= 2.0 ** -30
    a["vs"][t[2][t[2] >= 0]] *= 0.3
    a["ks"][t[2][t[2] >= 0]] *= 0.7
    a["ks"][t[3][t[3] >= 0]] = 0.0                # all scores equal
    check_attention(a)
    a["vs"][t[3][t[3] >= 0]] = 2.0 ** -90
    a["vs"][t[1][t[1] >= 0]] *= 2.0 ** 90
    check_attention(a)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_bad_blocks(d):
    """Bad ids, bad scales and short tables hide keys; a row may be left without any."""
    a = attention_inputs(4, 4, 2, d, [200, 60, 14, 40], CHAIN(2), 2, seed=30)
    a["table"][0, 3] = 10 ** 6
    a["table"][1, :] = -1                         # nothing left: 0 and -inf
    out, lse = check_attention(a, expect=ssd.FLAG_BAD_BLOCK)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    a["ks"][a["table"][0, 5], 1], a["vs"][a["table"][2, 0], 0] = -1.0, math.inf
    check_attention(a, expect=ssd.FLAG_BAD_BLOCK | ssd.FLAG_BAD_VALUE)
    a["prefix"][2], a["prefix"][3] = 16 * a["table"].shape[1] - 1, -7
    a["parent"][0, 1] = 1
    check_attention(a, expect=ssd.FLAG_BAD_BLOCK | ssd.FLAG_BAD_VALUE | ssd.FLAG_BAD_PREFIX | ssd.FLAG_BAD_TREE)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_nan(d):
    """A NaN reaches the rows that see it, and no other: in k the whole row, in v one element, in q its row."""
    parent = [-1, 0, 0, 1, 2]                     # 1 and 2 are siblings
    for length in (5, 126, 300):
        a = attention_inputs(2, 4, 2, d, [length, 40], parent, 5, seed=40 + length)

        def at(b, pos, h):
            return a["table"][b, pos // 16], h, pos % 16
        a["vc"][at(0, length + 1, 0)][3] = 0xFF   # a tree node: seen by itself and node 3
        a["kc"][at(0, length + 2, 1)][5] = 0x7F   # a tree node: seen by itself and node 4
        a["vc"][at(1, 7, 1)][d - 1] = 0x7F        # the prefix: seen by all
        out, _ = check_attention(a)
        assert np.isnan(out).sum() == 2 * 2 + 2 * 2 * d + 5 * 2
        a["q"][0, 3, 1, 0] = math.inf
        o, l, st = gpu_attention(a, 0.1)
        assert np.isnan(o[0, 3, 1]).all() and np.isnan(l[0, 3, 1]) and not np.isnan(o[0, 3, 0, :3]).any()


# The same edges with more than 64 rows per KV head (a lane per row): 16 heads per KV head, 5 to 9 queries.
@pytest.mark.parametrize("d", [64, 128])
def test_attention_many_rows_after_spine(d):
    parent = CHAIN(60) + [3, 3, 60, 61, 0]
    check_attention(attention_inputs(17, 16, 1, d, [47 + i for i in range(17)], parent, 5, seed=60 + d))
    check_attention(attention_inputs(9, 3, 1, d, [120 + i for i in range(9)], parent, 65, seed=61 + d))


@pytest.mark.parametrize("d", [64, 128])
def test_attention_many_rows_sharp_and_flat(d):
    a = attention_inputs(3, 16, 1, d, [700, 3000, 700], CHAIN(9), 9, seed=62, spread=0)
    check_attention(a, scale=1.0)
    a["q"][1] = 0
    one = a["kc"][a["table"][2, 0], 0, 0].copy()
    a["kc"][a["table"][2, 0], 0, 0] = ref.e4m3_round(np.sign(a["q"][2, 0, 0]) * 20.0)
    check_attention(a)
    a["kc"][a["table"][2, 0], 0, 0] = one
    a["kc"][a["table"][2, 40], 0, 7] = ref.e4m3_round(np.sign(a["q"][2, 0, 0]) * 60.0)
    check_attention(a)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_many_rows_scales(d):
    a = attention_inputs(4, 32, 2, d, [300, 300, 300, 40], CHAIN(5), 5, seed=63)
    t = a["table"]
    a["vs"][t[0, :19]] = 0.0                      # no value anywhere but in the last block
    a["vs"][t[1, ::2][t[1, ::2] >= 0]] *= 2.0 ** -30
    a["vs"][t[2][t[2] >= 0]] *= 0.3
    a["ks"][t[2][t[2] >= 0]] *= 0.7
    a["ks"][t[3][t[3] >= 0]] = 0.0                # all scores equal
    check_attention(a)
    a["vs"][t[3][t[3] >= 0]] = 2.0 ** -90
    a["vs"][t[1][t[1] >= 0]] *= 2.0 ** 90
    check_attention(a)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_many_rows_bad_blocks(d):
    a = attention_inputs(4, 32, 2, d, [200, 60, 14, 40], CHAIN(5), 5, seed=64)
    a["table"][0, 3] = 10 ** 6
    a["table"][1, :] = -1                         # nothing left: 0 and -inf
    out, lse = check_attention(a, expect=ssd.FLAG_BAD_BLOCK)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    a["ks"][a["table"][0, 5], 1], a["vs"][a["table"][2, 0], 0] = -1.0, math.inf
    check_attention(a, expect=ssd.FLAG_BAD_BLOCK | ssd.FLAG_BAD_VALUE)
    a["prefix"][2], a["prefix"][3] = 16 * a["table"].shape[1] - 1, -7
    a["parent"][0, 1] = 1
    check_attention(a, expect=ssd.FLAG_BAD_BLOCK | ssd.FLAG_BAD_VALUE | ssd.FLAG_BAD_PREFIX | ssd.FLAG_BAD_TREE)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_many_rows_nan(d):
    parent = [-1, 0, 0, 1, 2]                     # 1 and 2 are siblings
    for length in (5, 126, 300, 1500):
        a = attention_inputs(2, 32, 2, d, [length, 40], parent, 5, seed=65 + length)

        def at(b, pos, h):
            return a["table"][b, pos // 16], h, pos % 16
        a["vc"][at(0, length + 1, 0)][3] = 0xFF   # a tree node: seen by itself and node 3, 16 heads each
        a["kc"][at(0, length + 2, 1)][5] = 0x7F   # a tree node: seen by itself and node 4
        a["vc"][at(1, 7, 1)][d - 1] = 0x7F        # the prefix: seen by all
        out, _ = check_attention(a)
        assert np.isnan(out).sum() == 2 * 16 + 2 * 16 * d + 5 * 16
        a["q"][0, 3, 1, 0] = math.inf
        o, l, st = gpu_attention(a, 0.1)
        assert np.isnan(o[0, 3, 1]).all() and np.isnan(l[0, 3, 1]) and not np.isnan(o[0, 3, 0, :3]).any()


def test_attention_two_streams_and_graph():
    """Two calls at once with workspaces of their own, and a captured call replayed on new inputs."""
    sets = [attention_inputs(3, 8, 2, 128, [4000, 50, 900], CHAIN(4), 4, seed=50 + i) for i in range(3)]
    B, Nq, Hq, d = sets[0]["q"].shape
    base = [gpu_attention(a, 0.1) for a in sets]
    g = [{k: dev(v) for k, v in a.items()} for a in sets[:2]]
    for x in g:
        x["qb"], x["out"] = x["q"].to(torch.bfloat16), torch.empty(B, Nq, Hq, d, dtype=torch.bfloat16, device="cuda")
        x["lse"], x["st"] = torch.empty(B, Nq, Hq, device="cuda"), new_status()
        x["ws"] = torch.empty(max(256, ssd.ssd_attention_q8_workspace_size(B, Nq, Hq, 2, d)), dtype=torch.uint8,
                              device="cuda")
        x["s"] = torch.cuda.Stream()
    torch.cuda.synchronize()

    def launch(x, stream=None):
        ssd.ssd_branch_attention_q8(x["qb"], x["kc"], x["vc"], x["ks"], x["vs"], x["table"], x["prefix"], x["parent"],
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
    nb = min(len(sets[0]["kc"]), len(sets[2]["kc"]))
    assert nb == len(sets[0]["kc"]) == len(sets[2]["kc"])
    for k in ("kc", "vc", "ks", "vs", "table", "prefix", "parent"):
        x[k].copy_(dev(sets[2][k]))
    x["qb"].copy_(dev(sets[2]["q"]))
    graph.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(x["out"].float().cpu().numpy(), base[2][0])
    np.testing.assert_array_equal(x["lse"].cpu().numpy(), base[2][1])


def test_attention_without_lse_and_repeated():
    """The same call twice gives the same bits; without the log-sum-exp too."""
    a = attention_inputs(2, 8, 2, 64, [1500, 700], CHAIN(6), 6, seed=60)
    o1, l1, _ = gpu_attention(a, 0.125)
    o2, l2, _ = gpu_attention(a, 0.125)
    o3, _, _ = gpu_attention(a, 0.125, want_lse=False)
    np.testing.assert_array_equal(o1, o2)
    np.testing.assert_array_equal(l1, l2)
    np.testing.assert_array_equal(o1, o3)


# ---------------------------------------------------------------------------
# one decode step after the other
# ---------------------------------------------------------------------------
def test_decode_steps_together():
    """Blocks for the tree, then per step rotary positions, the append and the attention over what it wrote;
    then the accepted tokens alone.  Every stage against its plain form on what the GPU had before it."""
    rng = np.random.default_rng(70)
    B, Hq, Hkv, d, K, F, steps = 3, 8, 2, 64, 3, (3, 2, 1, 1), 3
    S = sum(F)
    N = K + steps * S
    maxb, nb = 12, 40
    lengths = np.array([20, 0, 95], np.int32)
    st = table_state(rng, B, maxb, nb, nb)
    kc, ks = cache(rng, nb, Hkv, d)
    vc, vs = cache(rng, nb, Hkv, d)
    g = {k: dev(v) for k, v in st.items()}
    gk, gv, gks, gvs = dev(kc), dev(vc), dev(ks), dev(vs)
    status = new_status()
    prefix = dev(lengths)
    turns, _ = ssd.ssd_rope_frequencies(d)
    theta = turns.numpy().astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    gt = turns.cuda()
    ssd.ssd_block_table_update(prefix, N, g["table"], g["pages"], g["ring"], g["pool"], status=status)
    ref.block_table_update(lengths, N, st["table"], st["pages"], st["ring"], st["pool"], 0)
    # the prompts (a padded batch), then the spine, then the branches' steps
    feeds = [(np.zeros(B, np.int32), 0, int(lengths.max()), lengths, None)]
    feeds.append((lengths, 0, K, None, w.chain_tree(K)))
    feeds += [(lengths, K + t * S, S, None, w.fill_tree(K, F, t + 1)) for t in range(steps)]
    for base, node0, n, count, parent in feeds:
        x = bf16(rng.standard_normal((B, n, Hq + 2 * Hkv, d))).cuda()
        q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
        before = x.float().cpu().numpy()
        gp = None if parent is None else dev(np.broadcast_to(parent, (B, len(parent))))
        gb = dev(base)
        ssd.ssd_tree_rope(q, k, gt, d, gb, q, k, parent=gp, node0=node0, status=status)
        ssd.ssd_kv_append_q8(k, v, gk, gv, gks, gvs, g["table"], gb, node0,
                             count=None if count is None else dev(count), status=status)
        after = x.float().cpu().numpy()
        pos = base[:, None].astype(np.int64) + (np.arange(n) if parent is None else ref.depths(parent, node0, n))
        rope_close(after[:, :, :Hq + Hkv], before[:, :, :Hq + Hkv],
                   ref.rope(before, theta, d, pos, False, 1.0)[:, :, :Hq + Hkv], d, 1.0, True)
        for y, c, s, gc, gs in ((after[:, :, Hq:Hq + Hkv], kc, ks, gk, gks), (after[:, :, Hq + Hkv:], vc, vs, gv, gvs)):
            assert ref.kv_append(y.astype(np.float64), c, s, st["table"], base, node0, count) == 0
            np.testing.assert_array_equal(gc.cpu().numpy(), c)
            np.testing.assert_array_equal(gs.cpu().numpy(), s)
        if parent is not None:
            a = dict(q=after[:, :, :Hq], kc=kc, vc=vc, ks=ks, vs=vs, table=st["table"], prefix=lengths,
                     parent=np.broadcast_to(parent, (B, len(parent))).copy())
            check_attention(a)
            out = torch.empty(B, n, Hq, d, dtype=torch.bfloat16, device="cuda")
            ssd.ssd_branch_attention_q8(q.contiguous(), gk, gv, gks, gvs, g["table"], prefix, gp, out, status=status)
            np.testing.assert_array_equal(out.float().cpu().numpy(), gpu_attention(a, d ** -0.5, use_ws=False)[0])
    accepted = lengths + np.array([2, 4, 1], np.int32)
    ssd.ssd_block_table_update(dev(accepted), 0, g["table"], g["pages"], g["ring"], g["pool"], status=status)
    ref.block_table_update(accepted, 0, st["table"], st["pages"], st["ring"], st["pool"], 0)
    for key in st:
        np.testing.assert_array_equal(g[key].cpu().numpy(), st[key])
    assert int(status.item()) == 0

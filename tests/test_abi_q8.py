"""CPU-side checks of the 8-bit cache calls: host validation that returns
before any launch, the frequency table, and the binding's refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

from speculative_decoding_vocab_gb300 import binding as ssd
from speculative_decoding_vocab_gb300 import build

INV, UNS, OK = ssd.SSD_ERR_INVALID_ARG, ssd.SSD_ERR_UNSUPPORTED, ssd.SSD_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ssd.load()


P = ctypes.c_void_p(0x100000)   # never dereferenced: each call returns before a launch
ODD = ctypes.c_void_p(0x100004)
BYTE = ctypes.c_void_p(0x100001)


def call(fn, good, expect, **change):
    args = dict(good)
    args.update(change)
    assert fn(*args.values()) == expect, change


def test_block_table_refusals(lib):
    good = dict(len=P, reserve=6, B=2, table=P, maxb=4, pages=P, ring=P, n=8, pool=P, slots=P, S=6, status=P, s=None)
    f = lib.ssd_block_table_update
    for k in ("len", "table", "pages", "ring", "pool", "slots", "status"):
        call(f, good, INV, **{k: None})
    for k, v in (("reserve", -1), ("B", -1), ("maxb", 0), ("n", 0), ("S", -1)):
        call(f, good, INV, **{k: v})
    call(f, good, UNS, n=(1 << 27) + 1)
    call(f, good, UNS, B=65537)
    call(f, good, OK, B=0, len=None, table=None)


def test_rope_refusals(lib):
    good = dict(q=P, qs=512, qt=64, qo=P, qos=512, qot=64, k=P, ks=512, kt=64, ko=P, kos=512, kot=64, dt=ssd.SSD_BF16,
                turns=P, rot=64, inter=0, m=1.0, prefix=P, parent=P, N=8, node0=0, B=2, S=8, Hq=1, Hkv=1, d=64,
                status=P, s=None)
    f = lib.ssd_tree_rope
    for k in ("q", "qo", "k", "ko", "turns", "prefix", "status"):
        call(f, good, INV, **{k: None})
    for k, v in (("rot", 63), ("rot", 0), ("rot", 66), ("d", 0), ("node0", -1), ("node0", 1), ("B", -1), ("S", -1),
                 ("S", 9), ("Hq", -1), ("Hkv", -1), ("N", -1), ("dt", 7), ("m", math.nan), ("m", math.inf)):
        call(f, good, INV, **{k: v})
    call(f, good, UNS, N=129)
    call(f, good, UNS, d=520)
    call(f, good, UNS, q=BYTE)              # not a multiple of the element
    call(f, good, UNS, parent=None, S=1 << 30, B=4)
    call(f, good, OK, B=0, q=None)
    call(f, good, OK, S=0)


def test_append_refusals(lib):
    good = dict(k=P, kss=1024, kts=128, v=P, vss=1024, vts=128, kc=P, vc=P, ks=P, vs=P, table=P, maxb=4, n=8,
                prefix=P, count=None, node0=0, B=2, S=8, Hkv=2, d=64, status=P, s=None)
    f = lib.ssd_kv_append_q8
    for k in ("k", "v", "kc", "vc", "ks", "vs", "table", "prefix", "status"):
        call(f, good, INV, **{k: None})
    for k, v in (("B", -1), ("S", -1), ("Hkv", 0), ("d", 0), ("node0", -1), ("maxb", 0), ("n", 0)):
        call(f, good, INV, **{k: v})
    for k, v in (("d", 96), ("d", 256), ("k", ODD), ("v", ODD), ("kc", ODD), ("vc", ODD), ("kts", 124), ("vss", 1)):
        call(f, good, UNS, **{k: v})
    call(f, good, OK, B=0, k=None)
    call(f, good, OK, S=0)


def test_attention_refusals(lib):
    good = dict(q=P, kc=P, vc=P, ks=P, vs=P, table=P, maxb=4, n=100, prefix=P, parent=P, B=2, N=4, Nq=4, Hq=8, Hkv=2,
                d=64, scale=0.1, out=P, lse=None, status=P, ws=None, wsb=0, s=None)
    f = lib.ssd_branch_attention_q8
    for k in ("q", "kc", "vc", "ks", "vs", "table", "prefix", "parent", "out", "status"):
        call(f, good, INV, **{k: None})
    for k, v in (("B", -1), ("Hq", 0), ("Hkv", 0), ("Hq", 7), ("maxb", 0), ("n", 0), ("scale", 0.0),
                 ("scale", -1.0), ("scale", math.nan), ("scale", math.inf)):
        call(f, good, INV, **{k: v})
    for k, v in (("d", 96), ("Hq", 34), ("N", 129), ("N", 0), ("Nq", 5), ("Nq", 0), ("q", ODD), ("kc", ODD),
                 ("vc", ODD), ("out", ODD)):
        call(f, good, UNS, **{k: v})
    call(f, good, OK, B=0, q=None)
    size = lib.ssd_attention_q8_workspace_size
    assert size(0, 1, 8, 2, 64) == 0 and size(2, 1, 7, 2, 64) == 0 and size(2, 1, 8, 2, 96) == 0


def test_sizes_beyond_the_counters(lib):
    """Calls whose counts would leave 32 bits are refused before anything is launched."""
    good = dict(q=P, kc=P, vc=P, ks=P, vs=P, table=P, maxb=1 << 30, n=100, prefix=P, parent=P, B=1 << 20, N=4, Nq=4,
                Hq=256, Hkv=32, d=64, scale=0.1, out=P, lse=None, status=P, ws=None, wsb=0, s=None)
    call(lib.ssd_branch_attention_q8, good, UNS)
    call(lib.ssd_branch_attention_q8, good, UNS, B=1 << 26)
    call(lib.ssd_branch_attention_q8, good, UNS, n=1 << 31)
    good = dict(length=P, reserve=0, B=2, table=P, maxb=4, pages=P, ring=P, n=8, pool=P, slots=P, S=3, status=P, s=None)
    for k, v in (("S", (1 << 24) + 1), ("B", 65537), ("n", (1 << 27) + 1), ("maxb", (1 << 27) + 1)):
        call(lib.ssd_block_table_update, good, UNS, **{k: v})


@pytest.mark.parametrize("rot,base,factor,original,fast,slow", [
    (64, 10000.0, 1.0, 0.0, 32.0, 1.0), (128, 500000.0, 8.0, 0.0, 32.0, 1.0), (128, 10000.0, 16.0, 4096.0, 32.0, 1.0),
    (2, 10000.0, 2.0, 2048.0, 32.0, 1.0), (24, 1000.0, 40.0, 4096.0, 16.0, 2.0)])
def test_rope_frequencies(lib, rot, base, factor, original, fast, slow):
    turns, m = ssd.ssd_rope_frequencies(rot, base, factor, original, fast, slow)
    i = np.arange(rot // 2)
    theta = base ** (-2.0 * i / rot)
    if original and factor > 1:
        def pair(r):
            return rot * math.log(original / (r * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        theta = theta / factor * ramp + theta * (1 - ramp)
        want = 0.1 * math.log(factor) + 1
    else:
        theta, want = theta / factor, 1.0
    got = turns.numpy().astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    # pow, log and three products in 64 bits, then half a step of 2^-64 turns (2^-65 * 2 pi = 1.71e-19)
    np.testing.assert_allclose(got, theta, rtol=1e-14, atol=1.72e-19)
    assert abs(m - want) <= 2.0 ** -24 * want


def test_rope_frequency_refusals(lib):
    t, m = (ctypes.c_uint64 * 1024)(), ctypes.c_float()
    f = lib.ssd_rope_frequencies
    good = dict(rot=64, base=1e4, factor=4.0, original=4096.0, fast=32.0, slow=1.0, t=t, m=ctypes.byref(m))
    call(f, good, OK)
    for k, v in (("rot", 63), ("rot", 0), ("base", 1.0), ("base", math.inf), ("factor", 0.5), ("factor", math.nan),
                 ("original", -1.0), ("slow", 0.0), ("fast", 1.0), ("fast", math.inf), ("t", None), ("m", None)):
        call(f, good, INV, **{k: v})
    call(f, good, UNS, rot=1026)


def test_binding_refuses_wrong_tensors(lib):
    x = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)
    codes = torch.zeros(8, 2, 16, 64, dtype=torch.uint8)
    scale = torch.zeros(8, 2)
    i32 = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 3, dtype=torch.int32)
    good = [x, x, codes, codes, scale, scale, table, i32, 0]
    with pytest.raises(ValueError, match="CUDA device"):
        ssd.ssd_kv_append_q8(*good)
    for at, bad, word in ((0, x.float(), "bfloat16"), (1, x[:, :3], "shape"), (0, x.transpose(2, 3).contiguous().transpose(2, 3), "contiguous"),
                          (2, codes.float(), "e4m3"), (3, codes[:, :, :8], "shape")):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError, match=word):
            ssd.ssd_kv_append_q8(*args)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ssd.ssd_tree_rope(x.half(), None, torch.zeros(32, dtype=torch.int64), 64, i32, x.half(), None)
    with pytest.raises(ValueError, match="CUDA device"):
        ssd.ssd_block_table_update(i32, 0, table, i32, torch.zeros(8, dtype=torch.int32),
                                   torch.zeros(4, dtype=torch.int32), status=torch.zeros(1, dtype=torch.int32))


def _bad(x):
    """The same tensor with a wrong dtype, a wrong shape, and strides that are not dense."""
    yield x.to(torch.float64)
    yield x.reshape(-1)[:-1] if x.numel() > 1 else x.expand(2)
    if x.dim() > 1 and x.shape[-2] > 1 and x.shape[-1] > 1:
        yield x.transpose(-1, -2).contiguous().transpose(-1, -2)


def test_every_tensor_is_checked():
    """A tensor that is not as the call wants it is refused by its name, whichever it is."""
    B, S, Hq, Hkv, d, nb, maxb = 2, 3, 4, 2, 64, 5, 3
    z = torch.zeros
    i32, bf = torch.int32, torch.bfloat16
    cache = {k: z(nb, Hkv, 16, d, dtype=torch.uint8) for k in ("k_cache", "v_cache")}
    cache.update({k: z(nb, Hkv) for k in ("k_scale", "v_scale")})
    table = dict(block_table=z(B, maxb, dtype=i32), prefix_len=z(B, dtype=i32))
    calls = [
        (ssd.ssd_branch_attention_q8, dict(q=z(B, S, Hq, d, dtype=bf), **cache, **table, parent=z(B, S, dtype=i32),
                                           out=z(B, S, Hq, d, dtype=bf), lse=z(B, S, Hq), status=z(1, dtype=i32),
                                           ws=z(512, dtype=torch.uint8))),
        (ssd.ssd_kv_append_q8, dict(k_new=z(B, S, Hkv, d, dtype=bf), v_new=z(B, S, Hkv, d, dtype=bf), **cache, **table,
                                    node0=0, count=z(B, dtype=i32), status=z(1, dtype=i32))),
        (ssd.ssd_tree_rope, dict(q=z(B, S, Hq, d, dtype=bf), k=z(B, S, Hkv, d, dtype=bf), turns=z(d // 2, dtype=torch.int64),
                                 rot=d, prefix_len=z(B, dtype=i32), q_out=z(B, S, Hq, d, dtype=bf),
                                 k_out=z(B, S, Hkv, d, dtype=bf), parent=z(B, S, dtype=i32), status=z(1, dtype=i32))),
        (ssd.ssd_block_table_update, dict(length=z(B, dtype=i32), reserve=0, block_table=z(B, maxb, dtype=i32),
                                          pages=z(B, dtype=i32), ring=z(nb, dtype=i32), pool=z(4, dtype=i32),
                                          slots=z(B, 2, dtype=i32), status=z(1, dtype=i32))),
    ]
    for fn, good in calls:
        with pytest.raises(ValueError, match="CUDA device"):
            fn(**good)
        for name, x in good.items():
            if not torch.is_tensor(x):
                continue
            for k, bad in enumerate(_bad(x)):
                if name == "ws" and k == 1 or name == "ring" and k == 1:  # any length will do
                    continue
                with pytest.raises((ValueError, IndexError)) as e:
                    fn(**{**good, name: bad})
                assert "CUDA device" not in str(e.value), (fn.__name__, name, k)

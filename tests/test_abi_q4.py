"""CPU-side checks of the 4-bit cache calls and the token log probabilities:
host validation that returns before any launch, and the binding's refusals."""
import ctypes
import math

import pytest
import torch

from speculative_decoding_vocab_gb300 import binding as ssd
from speculative_decoding_vocab_gb300 import build

INV, UNS, OK = ssd.SSD_ERR_INVALID_ARG, ssd.SSD_ERR_UNSUPPORTED, ssd.SSD_OK
P = ctypes.c_void_p(0x100000)   # never dereferenced: each call returns before a launch
ODD = ctypes.c_void_p(0x100004)
HALF = ctypes.c_void_p(0x100010)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ssd.load()


def call(fn, good, expect, **change):
    args = dict(good)
    args.update(change)
    assert fn(*args.values()) == expect, change


def test_append_refusals(lib):
    good = dict(k=P, kss=1024, kts=128, v=P, vss=1024, vts=128, kc=P, vc=P, ks=P, vs=P, table=P, maxb=4, n=8,
                prefix=P, count=None, node0=0, B=2, S=8, Hkv=2, d=64, status=P, s=None)
    f = lib.ssd_kv_append_q4
    for k in ("k", "v", "kc", "vc", "ks", "vs", "table", "prefix", "status"):
        call(f, good, INV, **{k: None})
    for k, v in (("B", -1), ("S", -1), ("Hkv", 0), ("d", 0), ("node0", -1), ("maxb", 0), ("n", 0)):
        call(f, good, INV, **{k: v})
    for k, v in (("d", 96), ("d", 256), ("k", ODD), ("v", ODD), ("kc", ODD), ("vc", ODD), ("ks", ODD), ("vs", ODD),
                 ("kts", 124), ("vss", 1)):
        call(f, good, UNS, **{k: v})
    call(f, good, UNS, S=1 << 30, B=8)
    call(f, good, OK, B=0, k=None)
    call(f, good, OK, S=0)


def test_read_refusals(lib):
    good = dict(kc=P, vc=P, ks=P, vs=P, table=P, maxb=4, n=8, prefix=P, count=None, node0=0, ko=P, kss=1024, kts=128,
                vo=P, vss=1024, vts=128, dt=ssd.SSD_BF16, B=2, S=8, Hkv=2, d=64, status=P, s=None)
    f = lib.ssd_kv_read_q4
    for k in ("kc", "vc", "ks", "vs", "table", "prefix", "status"):
        call(f, good, INV, **{k: None})
    for k, v in (("B", -1), ("S", -1), ("Hkv", 0), ("d", 0), ("node0", -1), ("maxb", 0), ("n", 0), ("dt", 5)):
        call(f, good, INV, **{k: v})
    for k, v in (("d", 96), ("kc", ODD), ("vc", ODD), ("ks", ODD), ("vs", ODD), ("ko", ODD), ("vo", ODD), ("kts", 124),
                 ("vss", 1)):
        call(f, good, UNS, **{k: v})
    call(f, good, UNS, dt=ssd.SSD_F32, kts=130)
    call(f, good, OK, ko=None, vo=None)
    call(f, good, OK, B=0, kc=None)
    call(f, good, OK, S=0)


def test_attention_refusals(lib):
    good = dict(q=P, kc=P, vc=P, ks=P, vs=P, table=P, maxb=4, n=100, prefix=P, parent=P, B=2, N=4, Nq=4, Hq=8, Hkv=2,
                d=64, scale=0.1, out=P, lse=None, status=P, ws=None, wsb=0, s=None)
    f = lib.ssd_branch_attention_q4
    for k in ("q", "kc", "vc", "ks", "vs", "table", "prefix", "parent", "out", "status"):
        call(f, good, INV, **{k: None})
    for k, v in (("B", -1), ("Hq", 0), ("Hkv", 0), ("Hq", 7), ("maxb", 0), ("n", 0), ("scale", 0.0),
                 ("scale", -1.0), ("scale", math.nan), ("scale", math.inf)):
        call(f, good, INV, **{k: v})
    for k, v in (("d", 96), ("Hq", 34), ("N", 129), ("N", 0), ("Nq", 5), ("Nq", 0), ("q", ODD), ("kc", HALF),
                 ("vc", HALF), ("ks", ODD), ("vs", ODD), ("out", ODD)):
        call(f, good, UNS, **{k: v})
    call(f, good, OK, B=0, q=None)
    size = lib.ssd_attention_q4_workspace_size
    assert size(0, 1, 8, 2, 64) == 0 and size(2, 1, 7, 2, 64) == 0 and size(2, 1, 8, 2, 96) == 0
    good.update(maxb=1 << 30, B=1 << 20, Hq=256, Hkv=32)
    call(f, good, UNS)
    call(f, good, UNS, B=1 << 26)
    call(f, good, UNS, n=1 << 31)


def test_logprob_refusals(lib):
    good = dict(z=P, dt=ssd.SSD_BF16, ss=8192, rs=1024, B=2, R=8, V=1000, T=1.0, tokens=P, lp=P, rank=P, ent=P, n=5,
                ids=P, top=P, status=P, s=None)
    f = lib.ssd_token_logprobs
    for k, v in (("z", None), ("status", None), ("tokens", None), ("B", -1), ("R", -1), ("V", 0), ("n", -1),
                 ("T", -0.5), ("T", math.nan), ("T", math.inf), ("dt", 3)):
        call(f, good, INV, **{k: v})
    for k, v in (("z", ODD), ("ss", 8193), ("rs", 1004), ("n", 65), ("V", (1 << 21) + 1), ("T", 1e-30), ("B", 1 << 25)):
        call(f, good, UNS, **{k: v})
    call(f, good, UNS, V=4, n=5)
    call(f, good, UNS, dt=ssd.SSD_F32, V=(1 << 20) + 1)
    call(f, good, OK, B=0, z=None)
    call(f, good, OK, R=0)


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
u8, i32, bf, f32 = torch.uint8, torch.int32, torch.bfloat16, torch.float32
B, S, H, D, NB = 2, 3, 2, 64, 5


def cache():
    return dict(zip(("k_cache", "v_cache", "k_scale", "v_scale"), ssd.q4_cache(NB, H, D, device="cpu")))


def place():
    return dict(block_table=torch.zeros(B, 4, dtype=i32), prefix_len=torch.zeros(B, dtype=i32),
                status=torch.zeros(1, dtype=i32))


def spoil(fn, good, names, **kw):
    """Each tensor alone of another dtype, shape or layout is refused by name."""
    for k in names:
        x = good[k]
        wrong = [x.to(torch.float64), torch.zeros(x.numel() + 1, dtype=x.dtype).view(*([1] * (x.dim() - 1)), -1)]
        if x.numel() > 1:
            wrong.append(torch.zeros(*x.shape[:-1], x.shape[-1] * 2, dtype=x.dtype)[..., ::2])
        for w in wrong:
            with pytest.raises(ValueError):
                fn(**{**good, k: w}, **kw)
    with pytest.raises(ValueError, match="CUDA device"):
        fn(**good, **kw)


def test_binding_append():
    rows = dict(k_new=torch.zeros(B, S, H, D, dtype=bf), v_new=torch.zeros(B, S, H, D, dtype=bf))
    good = {**rows, **cache(), **place(), "count": torch.zeros(B, dtype=i32)}
    spoil(ssd.ssd_kv_append_q4, good, list(cache()) + ["k_new", "v_new", "prefix_len", "count", "status"], node0=0)
    with pytest.raises(ValueError, match="heads"):
        ssd.ssd_kv_append_q4(**{**good, "k_new": torch.zeros(B, S, D, H, dtype=bf).transpose(2, 3)}, node0=0)


def test_binding_read():
    rows = dict(k_out=torch.zeros(B, S, H, D, dtype=f32), v_out=torch.zeros(B, S, H, D, dtype=f32))
    good = {**rows, **cache(), **place(), "count": torch.zeros(B, dtype=i32)}
    spoil(ssd.ssd_kv_read_q4, good, list(cache()) + ["prefix_len", "count", "status"], node0=0)
    for k in rows:
        for bad in (torch.zeros(B, S, H, D, dtype=torch.float16), torch.zeros(B, S + 1, H, D),
                    torch.zeros(B, 1, H, D).expand(B, S, H, D), torch.zeros(B, S, D, H).transpose(2, 3)):
            with pytest.raises(ValueError):
                ssd.ssd_kv_read_q4(**{**good, k: bad}, node0=0)


def test_binding_attention():
    q = torch.zeros(B, S, 4, D, dtype=bf)
    good = {**cache(), **place(), "q": q, "out": q.clone(), "lse": torch.zeros(B, S, 4),
            "parent": torch.zeros(B, S, dtype=i32), "ws": torch.zeros(512, dtype=u8)}
    spoil(ssd.ssd_branch_attention_q4, good, list(cache()) + ["q", "out", "lse", "prefix_len", "status"])


def test_binding_logprobs():
    z = torch.zeros(B, S, 16)
    good = dict(logits=z, tokens=torch.zeros(B, S, dtype=i32), logprob=torch.zeros(B, S),
                rank=torch.zeros(B, S, dtype=i32), entropy=torch.zeros(B, S), top_ids=torch.zeros(B, S, 3, dtype=i32),
                top_logprob=torch.zeros(B, S, 3), status=torch.zeros(1, dtype=i32))
    spoil(ssd.ssd_token_logprobs, good, [k for k in good if k != "logits"], V=16, T=1.0)
    for bad in (z.half(), z[0], torch.zeros(B, S, 32)[..., ::2]):
        with pytest.raises(ValueError):
            ssd.ssd_token_logprobs(**{**good, "logits": bad}, V=16, T=1.0)
    with pytest.raises(ValueError, match="V is"):
        ssd.ssd_token_logprobs(**good, V=17, T=1.0)

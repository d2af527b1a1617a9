"""Attention over the 8-bit cache where one key takes most of a row (an attention
sink with a value near 0): what the many other keys bring has to reach the output
as it does with probabilities rounded to bf16, however long the context and
whether or not its items are cut."""
import math

import pytest
import torch

from speculative_decoding_vocab_gb300 import binding as ssd

pytestmark = pytest.mark.gpu

PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_vocab_gb300 import build
    build.build()
    ssd.load()


def codes_of(x):
    """[L, H, d] values -> codes [blocks, H, 16, d] and power-of-two block scales [blocks, H]."""
    n, H, d = x.shape
    pad = -n % PAGE
    x = torch.cat((x, torch.zeros(pad, H, d, device="cuda"))).reshape(-1, PAGE, H, d).transpose(1, 2)
    s = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)).clamp(min=2.0 ** -20) / 448)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s.float()


def make(d, Hq, Hkv, Nq, keys, weight, at, seed):
    """One sequence of `keys` prefix keys and a chain of Nq nodes.  Element 0 of a query meets only the key at
    position `at`, whose score is set so that it takes about `weight` of every row, and whose value is 0."""
    g = torch.Generator("cuda").manual_seed(seed)
    n, scale = keys + Nq, d ** -0.5
    q = torch.randn(1, Nq, Hq, d, generator=g, device="cuda")
    k, v = (torch.randn(n, Hkv, d, generator=g, device="cuda") for _ in range(2))
    k[:, :, 0] = 0
    k[at] = 0
    k[at, :, 0] = 4.0
    v[at] = 0
    q[..., 0] = (math.log(n) + 0.5 + math.log(weight / (1 - weight))) / (scale * 4.0)
    kc, ks = codes_of(k)
    vc, vs = codes_of(v)
    nb = kc.shape[0]
    order = torch.randperm(nb, generator=g, device="cuda")
    inv = torch.argsort(order)
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(q=q.to(torch.bfloat16), kc=kc.view(torch.uint8)[inv].contiguous(), ks=ks[inv].contiguous(),
                vc=vc.view(torch.uint8)[inv].contiguous(), vs=vs[inv].contiguous(), table=order.int()[None].contiguous(),
                prefix=torch.tensor([keys], **i32), parent=torch.arange(-1, Nq - 1, **i32)[None].contiguous(), scale=scale)


def reference(a):
    """(out, out with the probabilities and the output rounded to bf16, lse) in 64 bits."""
    _, Nq, Hq, d = a["q"].shape
    Hkv, keys = a["ks"].shape[1], int(a["prefix"])
    n, blk = keys + Nq, a["table"][0].long()

    def values(c, s):
        x = c[blk].view(torch.float8_e4m3fn).double() * s[blk].double()[:, :, None, None]
        return x.transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
    k, v = values(a["kc"], a["ks"]), values(a["vc"], a["vs"])
    q = a["q"][0].double().reshape(Nq, Hkv, Hq // Hkv, d)
    x = torch.einsum("nhgd,htd->nhgt", q, k) * a["scale"]
    hidden = torch.arange(n, device="cuda") > keys + torch.arange(Nq, device="cuda")[:, None]
    x = x.masked_fill(hidden[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    pb = p.to(torch.bfloat16).double()
    o, ob = (torch.einsum("nhgt,htd->nhgd", w, v) / w.sum(-1, keepdim=True) for w in (p, pb))
    return (o.reshape(1, Nq, Hq, d), ob.to(torch.bfloat16).double().reshape(1, Nq, Hq, d),
            torch.logsumexp(x, -1).reshape(1, Nq, Hq))


def run(a, use_ws):
    q = a["q"]
    _, Nq, Hq, d = q.shape
    out, lse = torch.full_like(q, 7.0), torch.empty(1, Nq, Hq, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = None
    if use_ws:
        ws = torch.empty(ssd.ssd_attention_q8_workspace_size(1, Nq, Hq, a["ks"].shape[1], d), dtype=torch.uint8,
                         device="cuda")
    ssd.ssd_branch_attention_q8(q, a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["prefix"], a["parent"], out,
                                lse=lse, scale=a["scale"], status=status, ws=ws)
    assert int(status.item()) == 0
    return out.double(), lse.double()


def row_error(x, o):
    return (x - o).norm(dim=-1) / o.norm(dim=-1)


@pytest.mark.parametrize("use_ws", [True, False], ids=["split", "unsplit"])
@pytest.mark.parametrize("weight", [0.5, 0.9, 0.99])
@pytest.mark.parametrize("keys,at", [(8192, 0), (32768, 0), (32768, 20000), (100003, 0)])
@pytest.mark.parametrize("d,Hq,Hkv,Nq", [(64, 8, 2, 3), (128, 8, 1, 4), (128, 8, 1, 6), (64, 16, 1, 4), (64, 16, 1, 8),
                                         (128, 32, 2, 9)], ids=["12", "32", "48", "64", "128", "144"])
def test_sink(d, Hq, Hkv, Nq, keys, at, weight, use_ws):
    """The relative error of a row is that of bf16 probabilities: both round the output by up to 2^-8 of each
    element, and a probability by no more than bf16 does (2^-8 of it).  Over the d >= 64 elements of a row two such
    sums of independent roundings stay within a factor of two."""
    a = make(d, Hq, Hkv, Nq, keys, weight, at, seed=keys + Nq)
    o, ob, l = reference(a)
    out, lse = run(a, use_ws)
    err, base = row_error(out, o), row_error(ob, o)
    assert (err <= 2 * base).all(), f"relative error up to {err.max():.2g}, with bf16 probabilities {base.max():.2g}"
    # a score: q's elements are off by up to 2^-17 of the largest, so 2^-17 * scale max|q| (below 4.4) * sum|k| (below
    # 2^7) < 2^-7.8; the fp32 sum of products 2^-20 of their magnitudes' sum (below 2^6); the sum of p 2^-20
    assert ((lse - l).abs() <= 2.0 ** -7 + 2.0 ** -22 * l.abs()).all()


@pytest.mark.parametrize("d,Hq,Hkv,Nq", [(128, 8, 1, 8), (64, 16, 1, 8)], ids=["64", "128"])
def test_sink_in_a_large_batch(d, Hq, Hkv, Nq):
    """More items than the GPU has SMs, with a workspace: most items are whole, and give what a call alone gives."""
    a = make(d, Hq, Hkv, Nq, 9000, 0.95, 0, seed=1)
    B = 200
    b = dict(a)
    for k in ("q", "table", "prefix", "parent"):
        b[k] = a[k].expand(B, *a[k].shape[1:]).contiguous()
    o, ob, _ = reference(a)
    out, status = torch.empty_like(b["q"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(ssd.ssd_attention_q8_workspace_size(B, Nq, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    ssd.ssd_branch_attention_q8(b["q"], b["kc"], b["vc"], b["ks"], b["vs"], b["table"], b["prefix"], b["parent"], out,
                                scale=b["scale"], status=status, ws=ws)
    assert int(status.item()) == 0
    assert (row_error(out.double(), o) <= 2 * row_error(ob, o)).all()

"""The 4-bit cache in use: the target's verification pass from block tables to
the log probabilities of the emitted tokens, a prefix moved into the bf16
cache, caches beyond 2^31 bytes, and rows of which one key takes most."""
import math

import numpy as np
import pytest
import torch

import q4_ref as ref
import q8_ref
from speculative_decoding_vocab_gb300 import binding as ssd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_vocab_gb300 import build
    build.build()
    ssd.load()


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32), device="cuda")


def new_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def plain_attention(q, cache, table, prefix, parent, scale):
    """softmax(scale q k^T + mask) v in 64 bits over values read back from the cache; q [B, Nq, Hq, d]."""
    B, Nq, Hq, d = q.shape
    N, H = parent.shape[1], cache[0].shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(prefix[b]) + N
        k, v = (torch.empty(1, n, H, d, device="cuda") for _ in range(2))
        ssd.ssd_kv_read_q4(*cache, table[b:b + 1].contiguous(), i32([0]), 0, k, v, status=new_status())
        seen, _ = q8_ref.paths(parent[b].cpu().numpy(), Nq)
        vis = torch.as_tensor(np.concatenate([np.ones((Nq, n - N), bool), seen], axis=1), device="cuda")
        x = torch.einsum("nhgd,thd->nhgt", q[b].double().reshape(Nq, H, Hq // H, d), k[0].double()) * scale
        p = torch.softmax(x.masked_fill(~vis[:, None, None], -math.inf), -1)
        out[b] = torch.einsum("nhgt,thd->nhgd", p, v[0].double()).reshape(Nq, Hq, d)
    return out


class Pass:
    """One verification pass of a batch: everything that its calls need, allocated once (also for capture)."""

    def __init__(self, B, K, Hq, Hkv, d, V, lengths, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        self.B, self.K, self.V, self.d, self.Hq, self.Hkv = B, K, V, d, Hq, Hkv
        n, maxb = K + 1, 40
        nb = B * maxb
        f32 = dict(dtype=torch.float32, device="cuda")
        self.x = torch.randn(B, n, Hq + 2 * Hkv, d, generator=g, device="cuda").to(torch.bfloat16)
        self.proj = (torch.randn(Hq * d, V, generator=g, device="cuda") * 0.3).to(torch.bfloat16)
        self.draft = torch.randn(B, n, V, generator=g, device="cuda").to(torch.bfloat16)
        self.d_tok = torch.randint(0, V, (B, K), generator=g, device="cuda").int()
        self.u_acc, self.u_bonus = torch.rand(B, K, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
        self.prefix, self.grown = i32(lengths), i32(lengths)
        self.parent = i32([list(range(-1, K))] * B)
        self.turns = ssd.ssd_rope_frequencies(d)[0].cuda()
        self.table = torch.full((B, maxb), -1, dtype=torch.int32, device="cuda")
        self.pages, self.ring, self.pool = i32([0] * B), i32(np.arange(nb)), i32([0, nb, 0, 0])
        self.cache = ssd.q4_cache(nb, Hkv, d)
        self.out = torch.empty(B, n, Hq, d, dtype=torch.bfloat16, device="cuda")
        self.ws = torch.empty(max(256, ssd.ssd_attention_q4_workspace_size(B, n, Hq, Hkv, d)), dtype=torch.uint8,
                              device="cuda")
        self.F = (1,) * n
        self.vws = ssd.workspace(B, K, V, "bf16", self.F)
        self.logits = torch.empty(B, n, V, dtype=torch.bfloat16, device="cuda")
        self.accept, self.bonus = i32([0] * B), i32([0] * B)
        self.tokens = i32(np.zeros((B, n)))
        self.lp, self.ent, self.rank = torch.zeros(B, n, **f32), torch.zeros(B, n, **f32), i32(np.zeros((B, n)))
        self.ids, self.top = i32(np.zeros((B, n, 5))), torch.zeros(B, n, 5, **f32)
        self.status = new_status()
        # the prompts
        ssd.ssd_block_table_update(self.prefix, n, self.table, self.pages, self.ring, self.pool, status=self.status)
        L = max(lengths)
        p = torch.randn(B, L, 2 * Hkv, d, generator=g, device="cuda").to(torch.bfloat16)
        ssd.ssd_kv_append_q4(p[:, :, :Hkv], p[:, :, Hkv:], *self.cache, self.table, i32([0] * B), 0, count=self.prefix,
                             status=self.status)

    def run(self):
        Hq, Hkv, n = self.Hq, self.Hkv, self.K + 1
        q, k, v = self.x[:, :, :Hq], self.x[:, :, Hq:Hq + Hkv], self.x[:, :, Hq + Hkv:]
        self.qr, kr = torch.empty(self.B, n, Hq, self.d, dtype=q.dtype, device="cuda"), torch.empty_like(k).contiguous()
        ssd.ssd_tree_rope(q, k, self.turns, self.d, self.prefix, self.qr, kr, parent=self.parent, status=self.status)
        ssd.ssd_kv_append_q4(kr, v, *self.cache, self.table, self.prefix, 0, status=self.status)
        ssd.ssd_branch_attention_q4(self.qr, *self.cache, self.table, self.prefix, self.parent, self.out,
                                    status=self.status, ws=self.ws)
        torch.matmul(self.out.reshape(self.B, n, -1), self.proj, out=self.logits)
        ssd.ssd_verify(self.logits, self.draft, self.V, self.F, 1.0, 1.0, self.d_tok, self.u_acc, self.u_bonus,
                       self.accept, self.tokens, self.bonus, status=self.status, ws=self.vws)
        ssd.ssd_token_logprobs(self.logits, self.V, 1.0, tokens=self.tokens, logprob=self.lp, rank=self.rank,
                               entropy=self.ent, top_ids=self.ids, top_logprob=self.top, status=self.status)
        torch.add(self.prefix, self.accept, out=self.grown)
        self.grown.add_(1)
        ssd.ssd_block_table_update(self.grown, 0, self.table, self.pages, self.ring, self.pool, status=self.status)


@pytest.mark.parametrize("d,Hq,Hkv,K", [(128, 16, 2, 5), (64, 8, 2, 3)])
def test_verification_pass(d, Hq, Hkv, K):
    B, V = 5, 3001
    V8 = -(-V // 8) * 8
    lengths = [300, 17, 64, 2, 511]
    s = Pass(B, K, Hq, Hkv, d, V8, lengths, seed=d)
    table = s.table.clone()
    s.run()
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    # attention over what the cache holds: fp16 probabilities, fp32 sums, two-term queries, and bf16's rounding of
    # the output; values are below 2^3 and scores below 2^6 here, so 2^-8 |o| + (2^-11 + 2 * 2^-17 * 2^6) * 2^3
    want = plain_attention(s.qr, s.cache, table, np.array(lengths), s.parent, d ** -0.5)
    assert ((s.out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -10) * 2 ** 3).all()
    # the emitted tokens' log probabilities, and nothing behind them
    tokens = s.tokens.cpu().numpy()
    accept = s.accept.cpu().numpy()
    for b in range(B):
        assert (tokens[b, :accept[b] + 1] >= 0).all() and (tokens[b, accept[b] + 1:] == -1).all()
    o, flags = ref.token_logprobs(s.logits.double().cpu().numpy(), 1.0, tokens, 5)
    live = o["wanted"]
    assert flags == 0 and (s.lp.cpu().numpy()[~live] == 0).all()
    np.testing.assert_array_equal(s.rank.cpu().numpy()[live], o["rank"][live])
    np.testing.assert_array_equal(s.ids.cpu().numpy()[live], o["top_ids"][live])
    for got, k in ((s.lp, "logprob"), (s.ent, "entropy"), (s.top, "top_logprob")):
        x = o[k][live]
        assert (np.abs(got.cpu().numpy()[live] - x) <= 2.0 ** -22 * np.abs(x) + 2.0 ** -15).all(), k
    # the accepted tokens alone keep their blocks
    assert (s.pages.cpu().numpy() == -(-(np.array(lengths) + accept + 1) // 16)).all()


def test_verification_pass_captured():
    """A captured pass replayed gives the bits of the eager one."""
    args = (3, 5, 16, 2, 128, 2000, [300, 17, 64])
    a, b = Pass(*args, seed=1), Pass(*args, seed=1)
    a.run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    state = [x.clone() for x in (b.table, b.pages, b.ring, b.pool)]
    with torch.cuda.graph(graph):
        b.run()
    for x, y in zip((b.table, b.pages, b.ring, b.pool), state):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    for k in ("out", "logits", "tokens", "lp", "rank", "ent", "ids", "top", "table", "pages", "ring"):
        assert torch.equal(getattr(a, k), getattr(b, k)), k
    assert all(torch.equal(x, y) for x, y in zip(a.cache, b.cache))
    assert int(a.status.item()) == int(b.status.item()) == 0


def test_prefix_into_the_bf16_cache():
    """Rows read back in pages of 16 tokens are the bf16 cache's blocks; attention over both agrees."""
    g = torch.Generator("cuda").manual_seed(2)
    H, d, n, Hq = 2, 64, 80, 8
    cache = ssd.q4_cache(8, H, d)
    table, start, st = i32([[5, 2, 7, 0, 3, 1]]), i32([0]), new_status()
    kv = torch.randn(1, n, 2 * H, d, generator=g, device="cuda").to(torch.bfloat16)
    ssd.ssd_kv_append_q4(kv[:, :, :H], kv[:, :, H:], *cache, table, start, 0, status=st)
    k, v = (torch.empty(1, n, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ssd.ssd_kv_read_q4(*cache, table, start, 0, k, v, status=st)
    kb, vb = (torch.zeros(8, H, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ssd.ssd_kv_append(k, v, kb, vb, table, start, 0, status=st)
    q = torch.randn(1, 3, Hq, d, generator=g, device="cuda").to(torch.bfloat16)
    parent, prefix = i32([[-1, 0, 1]]), i32([n - 3])
    o4, o16 = torch.empty_like(q), torch.empty_like(q)
    ssd.ssd_branch_attention_q4(q, *cache, table, prefix, parent, o4, status=st)
    ssd.ssd_branch_attention(q, kb, vb, table, prefix, parent, o16, status=st)
    # the same values: probabilities in halves and in bf16 (2^-11 + 2^-8 of weighted |v| <= 2^2), two roundings to bf16
    assert ((o4.float() - o16.float()).abs() <= 2.0 ** -7 * o16.float().abs() + (2.0 ** -11 + 2.0 ** -8) * 4).all()
    assert int(st.item()) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_cache_beyond_32_bits(d):
    """Blocks whose codes lie past 2^31 (and, with the head, 2^32) bytes give what the same rows give in a small cache."""
    H, Hq, n = 8, 16, 600
    nb = (1 << 31) // (H * 16 * d // 2) + 5000
    g = torch.Generator("cuda").manual_seed(d)
    kv = torch.randn(1, n, 2 * H, d, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(1, 2, Hq, d, generator=g, device="cuda").to(torch.bfloat16)
    pages = -(-n // 16)
    got = []
    for blocks, ids in ((pages, np.arange(pages)), (nb, nb - 1 - 100 * np.arange(pages))):
        cache = ssd.q4_cache(blocks, H, d)
        table, st = i32([ids]), new_status()
        ssd.ssd_kv_append_q4(kv[:, :, :H], kv[:, :, H:], *cache, table, i32([0]), 0, status=st)
        k, v = (torch.empty(1, n, H, d, device="cuda") for _ in range(2))
        ssd.ssd_kv_read_q4(*cache, table, i32([0]), 0, k, v, status=st)
        out = torch.empty_like(q)
        ssd.ssd_branch_attention_q4(q, *cache, table, i32([n - 2]), i32([[-1, 0]]), out, status=st)
        assert int(st.item()) == 0
        got.append((k, v, out))
        del cache
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert got[0][0].abs().max() > 1


@pytest.mark.parametrize("use_ws", [True, False], ids=["split", "unsplit"])
@pytest.mark.parametrize("weight", [0.5, 0.99])
@pytest.mark.parametrize("keys,at", [(8192, 0), (32768, 20000)])
@pytest.mark.parametrize("d,Hq,Hkv,Nq", [(64, 8, 2, 3), (128, 8, 1, 6), (64, 16, 1, 4), (128, 32, 2, 9)],
                         ids=["12", "48", "64", "144"])
def test_sink(d, Hq, Hkv, Nq, keys, at, weight, use_ws):
    """One key, its value 0, takes `weight` of every row: what the many others bring reaches the output as it does with
    probabilities rounded to bf16 (the relative error of a row stays within twice theirs: both round the output by up to
    2^-8 of each element, and a probability by no more than bf16 does)."""
    g = torch.Generator("cuda").manual_seed(keys + Nq)
    n, scale = keys + Nq, d ** -0.5
    q = torch.randn(1, Nq, Hq, d, generator=g, device="cuda")
    k, v = (torch.randn(1, n, Hkv, d, generator=g, device="cuda") for _ in range(2))
    k[:, :, :, 0] = 0
    k[:, at] = 0
    k[:, at, :, 0] = 4.0
    v[:, at] = 0
    q[..., 0] = (math.log(n) + 0.5 + math.log(weight / (1 - weight))) / (scale * 4.0)
    q = q.to(torch.bfloat16)
    pages = -(-n // 16)
    cache, st = ssd.q4_cache(pages, Hkv, d), new_status()
    table = torch.randperm(pages, generator=g, device="cuda").int()[None].contiguous()
    ssd.ssd_kv_append_q4(k.to(torch.bfloat16), v.to(torch.bfloat16), *cache, table, i32([0]), 0, status=st)
    ssd.ssd_kv_read_q4(*cache, table, i32([0]), 0, k, v, status=st)
    out, lse = torch.empty_like(q), torch.empty(1, Nq, Hq, device="cuda")
    ws = torch.empty(max(256, ssd.ssd_attention_q4_workspace_size(1, Nq, Hq, Hkv, d)), dtype=torch.uint8, device="cuda")
    ssd.ssd_branch_attention_q4(q, *cache, table, i32([keys]), i32([list(range(-1, Nq - 1))]), out, lse=lse, scale=scale,
                                status=st, ws=ws if use_ws else None)
    assert int(st.item()) == 0
    x = torch.einsum("nhgd,thd->nhgt", q[0].double().reshape(Nq, Hkv, Hq // Hkv, d), k[0].double()) * scale
    hidden = torch.arange(n, device="cuda") > keys + torch.arange(Nq, device="cuda")[:, None]
    x = x.masked_fill(hidden[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    pb = p.to(torch.bfloat16).double()
    o, ob = (torch.einsum("nhgt,thd->nhgd", w, v[0].double()) / w.sum(-1, keepdim=True) for w in (p, pb))
    o, ob = o.reshape(1, Nq, Hq, d), ob.to(torch.bfloat16).double().reshape(1, Nq, Hq, d)
    err, base = ((y - o).norm(dim=-1) / o.norm(dim=-1) for y in (out.double(), ob))
    assert (err <= 2 * base).all(), f"relative error up to {err.max():.2g}, with bf16 probabilities {base.max():.2g}"
    # scale max|q| below 4.4, sum|k| below 2^7 (as for the 8-bit cache), the fp32 sum of products below 2^6
    assert ((lse.double() - torch.logsumexp(x, -1).reshape(1, Nq, Hq)).abs() <= 2.0 ** -7 + 2.0 ** -22 * 16).all()

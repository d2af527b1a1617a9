"""Workloads of the verification pass over a 4-bit paged K/V cache: the
quantising append and its rows read back, the tree-masked attention over the
codes, and the log probabilities of the tokens that the pass emits.

A cache holds e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) with
a power-of-two scale byte (2^(byte - 127), 255 for NaN) per 32 elements of a
token and head.  Key codes are packed along the head dimension (even element
in the low four bits), value codes along the positions (even position in the
low four bits).

``run`` computes an operator in elementary torch operations, or, where ``own``
is true, by the library's calls.
"""
import math

import torch

own = False

PAGE = 16    # positions per cache block
GROUP = 32   # elements per scale
MIN_EXP, MAX_EXP = -100, 125


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # The target verifying a chain of drafted tokens over long contexts: the bandwidth-bound call.
        dict(name="attention verify", op="attention", B=64, Hq=64, Hkv=8, d=128, lo=8192, hi=8192, spine=6,
             chains=0, chain=0),
        # The draft decoding every branch of a speculation tree in one pass: 4 spine nodes, 16 chains of 4.
        dict(name="attention draft tree", op="attention", B=16, Hq=32, Hkv=8, d=64, lo=2048, hi=2048, spine=4,
             chains=16, chain=4),
        # One request, one token, a very long context: few rows, the keys have to be split.
        dict(name="attention one token", op="attention", B=1, Hq=32, Hkv=8, d=128, lo=100003, hi=100003, spine=1,
             chains=0, chain=0),
        # A serving batch of unequal lengths verifying a small tree, group of 8 query heads per KV head.
        dict(name="attention ragged", op="attention", B=48, Hq=32, Hkv=4, d=128, lo=1, hi=16384, spine=5,
             chains=4, chain=2),
        # The start of a conversation: latency counts.
        dict(name="attention short", op="attention", B=2, Hq=8, Hkv=2, d=64, lo=37, hi=100, spine=4, chains=9,
             chain=1),
        # One decode step's new tokens, in the middle of a page, and what the cache holds of them.
        dict(name="append step", op="append", B=16, Hkv=8, d=64, S=16, lo=2048, hi=2048, node0=4, ragged=False),
        # The prompts of a padded batch: unequal token counts, whole pages.
        dict(name="append prompts", op="append", B=8, Hkv=8, d=128, S=8191, lo=0, hi=0, node0=0, ragged=True),
        # A cached prefix brought back for a request whose layers run in bf16.
        dict(name="read prefix", op="read", B=4, Hkv=8, d=128, S=16384, start=0, ragged=False, dtype="bf16"),
        # The last positions of a ragged batch in fp32, for a check of the cache.
        dict(name="read window", op="read", B=24, Hkv=4, d=64, S=99, start=1001, ragged=True, dtype="f32"),
        # The emitted tokens of a verified batch: accepted prefix and bonus, five alternatives each.
        dict(name="logprobs emitted", op="logprobs", B=64, R=6, V=128256, dtype="bf16", n=5, T=1.0, tail=True),
        # A prompt's tokens, twenty alternatives each, at a sampling temperature.
        dict(name="logprobs prompt", op="logprobs", B=1, R=2048, V=151936, dtype="bf16", n=20, T=0.7, tail=False),
        # One request's step, logits in 32 bits: latency counts.
        dict(name="logprobs step", op="logprobs", B=1, R=5, V=128256, dtype="f32", n=20, T=1.0, tail=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "read", "logprobs", "logprobs"])
    if op == "attention":
        Hkv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 3, 4, 7, 8, 16])
        d = rng.choice([64, 128])
        spine, chains, chain = rng.randint(1, 8), rng.choice([0, 0, 3, 9, 16]), rng.randint(1, 4)
        rows = group * (chains * chain if chains else spine)
        keys = int(1.0e11 / (Hkv * max(rows, 64) * d * 4))  # the cost of the largest listed case
        hi = _log(rng, 1, min(60000, keys - 128))
        lo = rng.choice([hi, hi // 7])
        B = max(1, min(_log(rng, 1, 64), keys // (hi + 128)))
        return dict(op=op, B=B, Hq=Hkv * group, Hkv=Hkv, d=d, lo=lo, hi=hi, spine=spine, chains=chains, chain=chain)
    if op == "append":
        S = _log(rng, 1, 8000)
        hi = _log(rng, 1, 9000)
        B = max(1, min(_log(rng, 1, 64), 60000 // S))
        return dict(op=op, B=B, Hkv=rng.choice([1, 2, 3, 8]), d=rng.choice([64, 128]), S=S,
                    lo=rng.choice([hi, hi // 3]), hi=hi, node0=rng.choice([0, 4, 5, 20]), ragged=rng.random() < 0.5)
    if op == "read":
        S = _log(rng, 1, 16000)
        return dict(op=op, B=max(1, min(_log(rng, 1, 64), 60000 // S)), Hkv=rng.choice([1, 2, 3, 8]),
                    d=rng.choice([64, 128]), S=S, start=rng.choice([0, 16, 7, 1001]), ragged=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "f32"]))
    V = _log(rng, 500, 160000)
    rows = _log(rng, 1, min(4000, 200000000 // V))
    R = min(rows, rng.choice([1, 3, 5, 6, 17, 4000]))
    return dict(op=op, B=max(1, rows // R), R=R, V=V, dtype=rng.choice(["bf16", "bf16", "f32"]),
                n=rng.choice([0, 1, 5, 8, 20]), T=rng.choice([0.6, 1.0, 1.3]), tail=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# what a user's program has in hand
# ---------------------------------------------------------------------------
def _lengths(case):
    """The batch's prefix lengths, evenly spread over [lo, hi] (their order is drawn by the seed)."""
    n = case["B"]
    return [case["lo"] + (case["hi"] - case["lo"]) * i // max(1, n - 1) for i in range(n)]


def _counts(case):
    """Tokens of each sequence of a padded batch."""
    B, S = case["B"], case["S"]
    return [S - (S // 2) * i // max(1, B - 1) if case["ragged"] else S for i in range(B)]


def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(int(seed))
    return g


def _shuffled(values, g, dtype=torch.int32):
    x = torch.tensor(values, dtype=dtype, device="cuda")
    return x[torch.randperm(len(values), generator=g, device="cuda")].contiguous()


def _tree(case):
    """Parent indices: a spine of ``spine`` nodes, then ``chains`` chains of ``chain`` nodes, chain c hung off
    spine node c % (spine + 1) - 1 (-1: the prefix end)."""
    spine = case["spine"]
    parent = list(range(-1, spine - 1))
    for c in range(case["chains"]):
        for t in range(case["chain"]):
            parent.append(c % (spine + 1) - 1 if t == 0 else len(parent) - 1)
    return parent


def _randn(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _quantised(x):
    """Codes (uint8, one per element) and scale bytes (one per 32) of fp32 rows [..., d]: the smallest power of two
    in [2^-100, 2^125] with max|x| <= 6 scale, nearest code, ties to the even one; a group with a value that is not
    finite gets the byte 255 and codes 0."""
    y = x.reshape(*x.shape[:-1], -1, GROUP)
    bad = ~y.isfinite().all(-1, keepdim=True)
    amax = torch.where(bad, torch.zeros_like(y), y).abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.75, e - 3, e - 2)
    e = torch.where(amax == 0, torch.full_like(e, MIN_EXP), e).clamp(MIN_EXP, MAX_EXP)
    a = torch.ldexp(y.abs(), -e)
    c = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
         + (a >= 3.5).byte() + (a > 5.0).byte() + torch.signbit(y).byte() * 8)
    c = torch.where(bad, torch.zeros_like(c), c)
    byte = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return c.reshape(x.shape), byte.squeeze(-1)


def _values(codes, byte):
    """fp32 values [..., d] of codes [..., d] and scale bytes [..., d / 32]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    mag = table[(codes & 7).long()]
    v = torch.where(codes > 7, -mag, mag).reshape(*byte.shape, GROUP)
    e = byte.int()[..., None] - 127
    v = torch.ldexp(torch.ldexp(v, e // 2), e - e // 2)  # each power of two a normal number
    return torch.where(byte[..., None] == 255, torch.full_like(v, math.nan), v).reshape(codes.shape)


def _pack(codes, dim):
    """Neighbours along `dim` in a byte, the even one in its low four bits."""
    pairs = codes.unflatten(dim, (-1, 2))
    at = dim if dim < 0 else dim + 1
    return pairs.select(at, 0) | (pairs.select(at, 1) << 4)


def _unpack(bytes_, dim):
    at = dim if dim < 0 else dim + 1
    pair = torch.stack((bytes_ & 15, bytes_ >> 4), dim=at)
    return pair.flatten(at - 1, at)


def _filled_cache(nb, Hkv, d, along, g):
    """Codes and scales of normal values (each head's channels of unequal size), packed along dimension `along`."""
    shape = (nb, Hkv, PAGE, d // 2) if along == -1 else (nb, Hkv, PAGE // 2, d)
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    scale = torch.empty(nb, Hkv, PAGE, d // GROUP, dtype=torch.uint8, device="cuda")
    channel = torch.exp(0.5 * _randn((1, Hkv, 1, d), g, torch.float32))
    step = max(1, (1 << 25) // (Hkv * PAGE * d))
    for o in range(0, nb, step):
        n = min(step, nb - o)
        c, s = _quantised(_randn((n, Hkv, PAGE, d), g).float() * channel)
        codes[o:o + n], scale[o:o + n] = _pack(c, along), s
    return codes, scale


def _paged(lengths, maxb, g, spare=0):
    """Block tables over a shuffled pool: [B, maxb] int32 (-1 past the end), and the number of blocks."""
    need = (lengths.long() + PAGE - 1) // PAGE
    nb = int(need.sum()) + spare
    order = torch.randperm(nb - spare, generator=g, device="cuda").int()
    first = need.cumsum(0) - need
    p = torch.arange(maxb, device="cuda")
    at = (first[:, None] + p).clamp(max=max(nb - spare - 1, 0))
    return torch.where(p < need[:, None], order[at], torch.full_like(at, -1, dtype=torch.int32)).contiguous(), nb


def prepare(case, seed):
    return {"attention": _prepare_attention, "append": _prepare_append, "read": _prepare_read,
            "logprobs": _prepare_logprobs}[case["op"]](case, seed)


def _prepare_attention(c, seed):
    g = _gen(seed)
    parent = _tree(c)
    N = len(parent)
    Nq = c["chains"] * c["chain"] or N
    prefix = _shuffled(_lengths(c), g)
    maxb = (c["hi"] + N + PAGE - 1) // PAGE
    table, nb = _paged(prefix + N, maxb, g)
    kc, ks = _filled_cache(nb, c["Hkv"], c["d"], -1, g)
    vc, vs = _filled_cache(nb, c["Hkv"], c["d"], -2, g)
    q = _randn((c["B"], Nq, c["Hq"], c["d"]), g)
    return dict(op=c["op"], q=q, kc=kc, ks=ks, vc=vc, vs=vs, table=table, prefix=prefix,
                parent=torch.tensor([parent] * c["B"], dtype=torch.int32, device="cuda"),
                out=torch.empty_like(q), lse=torch.empty(q.shape[:3], dtype=torch.float32, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"), scale=c["d"] ** -0.5,
                ws=torch.empty(128 << 20, dtype=torch.uint8, device="cuda"))


def _prepare_append(c, seed):
    g = _gen(seed)
    B, S, Hkv, d = c["B"], c["S"], c["Hkv"], c["d"]
    prefix = _shuffled(_lengths(c), g)
    count = _shuffled(_counts(c), g) if c["ragged"] else None
    maxb = (c["hi"] + c["node0"] + S + PAGE - 1) // PAGE
    table, nb = _paged(prefix + c["node0"] + S, maxb, g, spare=1)
    kc, ks = _filled_cache(nb, Hkv, d, -1, g)
    vc, vs = _filled_cache(nb, Hkv, d, -2, g)
    for x in (kc, ks, vc, vs):  # the spare block: where the plain form puts what is not written
        x[-1] = 0
    qkv = _randn((B, S, 2, Hkv, d), g)  # the projections' rows: a token's key heads, then its value heads
    out = torch.zeros(2, B, S, Hkv, d, dtype=torch.bfloat16, device="cuda")
    return dict(op=c["op"], kn=qkv[:, :, 0], vn=qkv[:, :, 1], kc=kc, ks=ks, vc=vc, vs=vs, table=table, prefix=prefix,
                count=count, node0=c["node0"], ko=out[0], vo=out[1],
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_read(c, seed):
    g = _gen(seed)
    B, S, Hkv, d = c["B"], c["S"], c["Hkv"], c["d"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    start = torch.full((B,), c["start"], dtype=torch.int32, device="cuda")
    count = _shuffled(_counts(c), g) if c["ragged"] else None
    maxb = (c["start"] + S + PAGE - 1) // PAGE
    table, nb = _paged(start + S, maxb, g)
    kc, ks = _filled_cache(nb, Hkv, d, -1, g)
    vc, vs = _filled_cache(nb, Hkv, d, -2, g)
    out = torch.zeros(2, B, S, Hkv, d, dtype=dt, device="cuda")
    return dict(op=c["op"], kc=kc, ks=ks, vc=vc, vs=vs, table=table, prefix=start, count=count, node0=0, ko=out[0],
                vo=out[1], status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_logprobs(c, seed):
    g = _gen(seed)
    B, R, V, n = c["B"], c["R"], c["V"], c["n"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    z = torch.empty(B, R, -(-V // 8) * 8, dtype=dt, device="cuda")  # rows of a multiple of 16 bytes
    z.normal_(0.0, 2.5, generator=g)
    banned = torch.rand(z.shape[2], generator=g, device="cuda") < 0.01  # tokens that a grammar forbids in some rows
    z[:, 3::4].masked_fill_(banned, -math.inf)
    # half of the tokens are their row's likeliest
    likely = z[:, :, :V].argmax(-1)
    other = torch.randint(0, V, (B, R), generator=g, device="cuda")
    tokens = torch.where(torch.rand(B, R, generator=g, device="cuda") < 0.5, likely, other).int()
    if c["tail"]:  # behind the accepted tokens and the bonus
        emitted = 1 + torch.arange(B, device="cuda")[torch.randperm(B, generator=g, device="cuda")] % R
        tokens[torch.arange(R, device="cuda") >= emitted[:, None]] = -1
    f32 = dict(dtype=torch.float32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(op=c["op"], z=z, V=V, T=c["T"], n=n, tokens=tokens, logprob=torch.zeros(B, R, **f32),
                rank=torch.zeros(B, R, **i32), entropy=torch.zeros(B, R, **f32), ids=torch.zeros(B, R, n, **i32),
                top=torch.zeros(B, R, n, **f32), status=torch.zeros(1, **i32))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"attention": _plain_attention, "append": _plain_append, "read": _plain_read,
            "logprobs": _plain_logprobs}[s["op"]](s)


def _run_own(s):
    from speculative_decoding_vocab_gb300 import binding as ssd
    if s["op"] == "attention":
        ssd.ssd_branch_attention_q4(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["prefix"], s["parent"],
                                    s["out"], lse=s["lse"], scale=s["scale"], status=s["status"], ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "append":
        ssd.ssd_kv_append_q4(s["kn"], s["vn"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["prefix"], s["node0"],
                             count=s["count"], status=s["status"])
    if s["op"] in ("append", "read"):
        ssd.ssd_kv_read_q4(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["prefix"], s["node0"], s["ko"], s["vo"],
                           count=s["count"], status=s["status"])
        return _rows_and_cache(s)
    ssd.ssd_token_logprobs(s["z"], s["V"], s["T"], tokens=s["tokens"], logprob=s["logprob"], rank=s["rank"],
                           entropy=s["entropy"], top_ids=s["ids"] if s["n"] else None,
                           top_logprob=s["top"] if s["n"] else None, status=s["status"])
    return {"logprob": s["logprob"], "rank": s["rank"], "entropy": s["entropy"], "ids": s["ids"], "top": s["top"]}


def _rows_and_cache(s):
    out = {"k": s["ko"], "v": s["vo"]}
    if s["op"] == "append":  # the updated cache; its new codes are k and v as values
        out |= {"k_cache": s["kc"], "v_cache": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
    return out


def _ancestors(parent):
    """[B, N, N]: node n is m or one of its ancestors (the closure of the parent relation, by squaring)."""
    N = parent.shape[1]
    n = torch.arange(N, device=parent.device)
    a = ((parent[:, :, None] == n) | (n[:, None] == n)).float()
    a = (a @ a).clamp(max=1.0)
    a = (a @ a).clamp(max=1.0)
    a = (a @ a).clamp(max=1.0)
    a = (a @ a).clamp(max=1.0)
    a = (a @ a).clamp(max=1.0)
    a = (a @ a).clamp(max=1.0)
    return (a @ a).clamp(max=1.0)  # paths of up to 128 nodes


def _plain_attention(s):
    q, table, prefix, parent = s["q"], s["table"], s["prefix"].long(), s["parent"]
    B, Nq, Hq, d = q.shape
    Hkv, N = s["kc"].shape[1], parent.shape[1]
    G = Hq // Hkv
    blk = table.clamp(min=0).long()

    def gather(codes, scale, along):
        x = _values(_unpack(codes[blk], along), scale[blk])
        return x.transpose(1, 2).reshape(B, Hkv, -1, d)
    k, v = gather(s["kc"], s["ks"], -1), gather(s["vc"], s["vs"], -2)
    keys = k.shape[2]
    node = torch.arange(keys, device=q.device) - prefix[:, None]  # [B, keys]: the tree node there
    seen = _ancestors(parent)[:, N - Nq:] > 0
    tree = seen.gather(2, node.clamp(0, N - 1)[:, None].expand(B, Nq, keys))
    visible = (node < 0)[:, None] | (tree & ((node >= 0) & (node < N))[:, None])  # [B, Nq, keys]
    rows = q.float().reshape(B, Nq, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Nq * G, d)
    x = (rows @ k.transpose(2, 3)) * s["scale"]
    x = x.reshape(B, Hkv, Nq, G, keys).masked_fill(~visible[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, Hkv, Nq * G, keys) @ v).reshape(B, Hkv, Nq, G, d) / total
    lse = (top + total.log()).squeeze(-1)
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(B, Nq, Hq, d).to(torch.bfloat16),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, Nq, Hq)}


def _plain_append(s):
    """Windows of whole blocks around the new rows: their codes and scales replaced, the others as they were."""
    B, S = s["kn"].shape[:2]
    dev = s["kn"].device
    table = s["table"]
    first = s["prefix"].long() + s["node0"]
    count = s["count"].long() if s["count"] is not None else torch.full((B,), S, device=dev)
    page = first[:, None] // PAGE + torch.arange((S + PAGE - 2) // PAGE + 1, device=dev)  # [B, P]
    rel = page[..., None] * PAGE + torch.arange(PAGE, device=dev) - first[:, None, None]   # [B, P, 16]
    new = (rel >= 0) & (rel < count[:, None, None])
    touched = new.any(-1)
    nb = s["kc"].shape[0]
    blk = torch.where(touched, table.gather(1, page.clamp(max=table.shape[1] - 1)).long(),
                      torch.full_like(page, nb - 1))
    src = rel.clamp(0, S - 1)
    b = torch.arange(B, device=dev)[:, None, None]

    def write(x, codes, scale, along):
        c, e = _quantised(x.float())
        n = new[:, :, None, :, None]
        c = torch.where(n, c[b, src].transpose(2, 3), _unpack(codes[blk], along))  # [B, P, Hkv, 16, d]
        codes[blk] = _pack(c, along)
        scale[blk] = torch.where(n, e[b, src].transpose(2, 3), scale[blk])
    write(s["kn"], s["kc"], s["ks"], -1)
    write(s["vn"], s["vc"], s["vs"], -2)
    return _plain_read(s)


def _plain_read(s):
    B, S = s["ko"].shape[:2]
    dev = s["ko"].device
    i = torch.arange(S, device=dev)
    pos = s["prefix"].long()[:, None] + s["node0"] + i
    blk = s["table"].gather(1, pos // PAGE).clamp(min=0).long()
    count = s["count"].long() if s["count"] is not None else torch.full((B,), S, device=dev)
    wanted = (i < count[:, None])[..., None, None]
    at = pos % PAGE
    k = _values(_unpack(s["kc"][blk, :, at], -1), s["ks"][blk, :, at])  # [B, S, Hkv, d]
    byte = s["vc"][blk, :, at // 2]
    odd = (at % 2 == 1)[..., None, None]
    v = _values(torch.where(odd, byte >> 4, byte & 15), s["vs"][blk, :, at])
    s["ko"].copy_(torch.where(wanted, k, s["ko"].float()))
    s["vo"].copy_(torch.where(wanted, v, s["vo"].float()))
    return _rows_and_cache(s)


def _plain_logprobs(s):
    z, V, n, tokens = s["z"][:, :, :s["V"]].float(), s["V"], s["n"], s["tokens"].long()
    index = torch.arange(V, device=z.device)
    x = z / s["T"]
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp()
    total = p.sum(-1, keepdim=True)
    t = tokens.clamp(min=0)[..., None]
    zt = z.gather(2, t)
    wanted = tokens >= 0
    out = {"logprob": ((x.gather(2, t) - m) - total.log())[..., 0],
           "rank": ((z > zt).sum(-1) + ((z == zt) & (index < t)).sum(-1)).int(),
           "entropy": (total.log() - torch.where(p > 0, (x - m) * p, torch.zeros_like(p)).sum(-1, keepdim=True)
                       / total)[..., 0]}
    # the order (value descending, index ascending) as one integer per entry
    bits = (z + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) * (1 << 32) + (0xFFFFFFFF - index)
    ids = 0xFFFFFFFF - (order.topk(n, dim=-1).values & 0xFFFFFFFF)
    out["ids"] = ids.int()
    out["top"] = (x.gather(2, ids) - m) - total.log()
    keep = {"logprob": s["logprob"], "rank": s["rank"], "entropy": s["entropy"], "ids": s["ids"], "top": s["top"]}
    return {k: torch.where(wanted if v.dim() == 2 else wanted[..., None], v, keep[k]) for k, v in out.items()}


# ---------------------------------------------------------------------------
# the work of a pass
# ---------------------------------------------------------------------------
def work(c):
    if c["op"] == "attention":
        N = c["spine"] + c["chains"] * c["chain"]
        Nq = c["chains"] * c["chain"] or N
        keys = sum(n + N for n in _lengths(c))
        pages = sum((n + N + PAGE - 1) // PAGE for n in _lengths(c))
        rows = Nq * c["Hq"]
        cache = keys * c["Hkv"] * 2 * (c["d"] // 2 + c["d"] // GROUP) + pages * 4
        return {"bytes": cache + c["B"] * rows * (4 * c["d"] + 4) + c["B"] * 4 * (N + 1),
                "flops": 4 * keys * rows * c["d"]}
    if c["op"] in ("append", "read"):
        tokens = sum(_counts(c))
        values = tokens * c["Hkv"] * 2 * c["d"]
        held = values // 2 + values // GROUP
        tables = tokens // PAGE * 4 + c["B"] * 8
        if c["op"] == "read":
            return {"bytes": held + values * (2 if c["dtype"] == "bf16" else 4) + tables, "flops": values}
        return {"bytes": 2 * held + values * 4 + tables, "flops": values * 4}  # written, and read back
    rows = c["B"] * c["R"]
    if c["tail"]:
        rows = sum(1 + b % c["R"] for b in range(c["B"]))
    return {"bytes": rows * (c["V"] * (2 if c["dtype"] == "bf16" else 4) + 16 + 8 * c["n"]), "flops": rows * c["V"] * 6}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "read": _exact_read,
            "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_values(nibbles, byte):
    """e2m1: bit 3 the sign, bits 2 and 1 the exponent, bit 0 the fraction; times 2^(byte - 127)."""
    c = nibbles.long()
    e, f = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e == 0, 0.5 * f, (1.0 + 0.5 * f) * torch.exp2(e.double() - 1.0))
    sign = 1.0 - 2.0 * (c >> 3).double()
    scale = torch.exp2(byte.double() - 127.0)
    scale = torch.where(byte == 255, torch.full_like(scale, math.nan), scale)
    return sign * mag * scale.repeat_interleave(GROUP, dim=-1)


def _exact_rows(s, ids, h, n):
    """The first n positions of the blocks `ids`, head h: (k, v) [n, d]."""
    kb, vb = s["kc"][ids, h], s["vc"][ids, h]  # [P, 16, d / 2], [P, 8, d]
    P, d = kb.shape[0], vb.shape[2]
    kn = torch.empty(P, PAGE, d, dtype=torch.uint8, device=kb.device)
    vn = torch.empty_like(kn)
    kn[..., 0::2], kn[..., 1::2] = kb % 16, kb // 16
    vn[:, 0::2], vn[:, 1::2] = vb % 16, vb // 16
    return tuple(_exact_values(x.reshape(-1, d)[:n], sc[ids, h].reshape(P * PAGE, -1)[:n])
                 for x, sc in ((kn, s["ks"]), (vn, s["vs"])))


def _exact_attention(s):
    q, parent = s["q"], s["parent"].tolist()
    B, Nq, Hq, d = q.shape
    Hkv, N = s["kc"].shape[1], len(parent[0])
    paths = []
    for m in range(N - Nq, N):
        path, x = [False] * N, m
        while x >= 0:
            path[x] = True
            x = parent[0][x]
        paths.append(path)
    paths = torch.tensor(paths, device=q.device)
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.empty(q.shape[:3], dtype=torch.float64, device=q.device)
    for b, L in enumerate(s["prefix"].tolist()):
        ids = s["table"][b, :(L + N + PAGE - 1) // PAGE].long()
        hidden = torch.cat((torch.zeros(Nq, L, dtype=torch.bool, device=q.device), ~paths), dim=1)
        for h in range(Hkv):
            k, v = _exact_rows(s, ids, h, L + N)
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = torch.einsum("ngd,td->ngt", q[b, :, heads].double(), k) * s["scale"]
            x = x.masked_fill(hidden[:, None], -math.inf)
            lse[b, :, heads] = torch.logsumexp(x, -1)
            out[b, :, heads] = torch.einsum("ngt,td->ngd", torch.softmax(x, -1), v)
    return {"out": out, "lse": lse}


def _exact_append(s):
    """Each new value rounded to its group's grid: steps of 1/2 below 2, 1 below 4, 2 up to 6, times the scale."""
    def rounded(x):
        y = x.double().reshape(*x.shape[:-1], -1, GROUP)
        amax = y.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(amax / 6.0))
        e = torch.where(amax > 6.0 * torch.exp2(e), e + 1, e)
        e = torch.where(amax <= 6.0 * torch.exp2(e - 1), e - 1, e)
        unit = torch.exp2(torch.where(amax == 0, torch.full_like(e, MIN_EXP), e).clamp(MIN_EXP, MAX_EXP))
        a = (y / unit).abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        a = (torch.round(a / step) * step).clamp(max=6.0)
        return (torch.sign(y) * a * unit).reshape(x.shape)
    B, S = s["kn"].shape[:2]
    count = [S] * B if s["count"] is None else s["count"].tolist()
    out = {"k": rounded(s["kn"]), "v": rounded(s["vn"])}
    for b, n in enumerate(count):
        out["k"][b, n:], out["v"][b, n:] = 0, 0
    return out | {"k_cache": None, "v_cache": None, "k_scale": None, "v_scale": None}


def _exact_read(s):
    B, S, Hkv, d = s["ko"].shape
    out = {"k": torch.zeros(B, S, Hkv, d, dtype=torch.float64, device="cuda")}
    out["v"] = torch.zeros_like(out["k"])
    for b, start in enumerate(s["prefix"].tolist()):
        n = S if s["count"] is None else int(s["count"][b])
        ids = s["table"][b, :(start + n + PAGE - 1) // PAGE].long()
        for h in range(Hkv):
            k, v = _exact_rows(s, ids, h, start + n)
            out["k"][b, :n, h], out["v"][b, :n, h] = k[start:], v[start:]
    return out


def _exact_logprobs(s):
    B, R = s["tokens"].shape
    V, n = s["V"], s["n"]
    out = {k: torch.zeros(v.shape, dtype=torch.float64, device="cuda")
           for k, v in (("logprob", s["logprob"]), ("entropy", s["entropy"]), ("top", s["top"]))}
    for b in range(B):
        for o in range(0, R, 128):
            t = s["tokens"][b, o:o + 128].long()
            logp = torch.log_softmax(s["z"][b, o:o + 128, :V].double() / s["T"], -1)
            h = -(logp.exp() * logp.clamp(min=-1e6)).sum(-1)
            best = logp.sort(-1, descending=True).values[:, :n]
            live = t >= 0
            zero = torch.zeros_like(h)
            out["logprob"][b, o:o + 128] = torch.where(live, logp.gather(1, t.clamp(min=0)[:, None])[:, 0], zero)
            out["entropy"][b, o:o + 128] = torch.where(live, h, zero)
            out["top"][b, o:o + 128] = torch.where(live[:, None], best, torch.zeros_like(best))
    return {"logprob": out["logprob"], "rank": None, "entropy": out["entropy"], "ids": None, "top": out["top"]}

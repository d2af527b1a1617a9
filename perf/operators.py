"""Workloads of the 8-bit paged K/V cache path of the branch decode: rotary
positions of tree nodes, the quantising append, the tree-masked attention that
reads the 8-bit cache, and the block tables kept on the GPU.

``run`` computes an operator in elementary torch operations, or, where ``own``
is true, by the library's calls.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16          # positions per cache block
E4M3_MAX = 448.0
MIN_SCALE_EXP = -100


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # The draft decoding every branch of a speculation tree in one pass: 4 spine nodes, 16 chains of 4.
        dict(name="attention draft tree", op="attention", B=16, Hq=32, Hkv=8, d=64, lo=2048, hi=2048, spine=4,
             chains=16, chain=4),
        # The target verifying a chain of drafted tokens over long contexts: the bandwidth-bound call.
        dict(name="attention verify", op="attention", B=64, Hq=64, Hkv=8, d=128, lo=8192, hi=8192, spine=6,
             chains=0, chain=0),
        # One request, one token, a very long context: few rows, the keys have to be split.
        dict(name="attention one token", op="attention", B=1, Hq=32, Hkv=8, d=128, lo=100003, hi=100003, spine=1,
             chains=0, chain=0),
        # A serving batch of unequal lengths verifying a small tree, group of 8 query heads per KV head.
        dict(name="attention ragged", op="attention", B=48, Hq=32, Hkv=4, d=128, lo=1, hi=16384, spine=5,
             chains=4, chain=2),
        # The start of a conversation: latency counts.
        dict(name="attention short", op="attention", B=2, Hq=8, Hkv=2, d=64, lo=37, hi=100, spine=4, chains=9,
             chain=1),
        # One decode step of the cache fill: 16 fed branch tokens per sequence, in the middle of a page.
        dict(name="append step", op="append", B=16, Hkv=8, d=64, S=16, lo=2048, hi=2048, node0=4, ragged=False),
        # The prompts of a padded batch: unequal token counts, whole pages.
        dict(name="append prompts", op="append", B=8, Hkv=8, d=128, S=8191, lo=0, hi=0, node0=0, ragged=True),
        # The fed branch tokens of a decode step at their depths in the tree.
        dict(name="rope step", op="rope", B=16, Hq=32, Hkv=8, d=64, S=16, rot=64, interleaved=False, dtype="bf16",
             lo=2048, hi=2048, chain=4, chains=16, factor=1.0),
        # A long prompt's queries and keys: half of the head rotated, frequencies scaled for long contexts.
        dict(name="rope prompts", op="rope", B=4, Hq=64, Hkv=8, d=128, S=4099, rot=64, interleaved=True,
             dtype="bf16", lo=0, hi=100000, chain=0, chains=0, factor=16.0),
        # The same in 32 bits, the whole head, an odd batch.
        dict(name="rope fp32", op="rope", B=3, Hq=32, Hkv=8, d=128, S=1025, rot=128, interleaved=False, dtype="f32",
             lo=5, hi=30001, chain=0, chains=0, factor=4.0),
        # The verification batch's tables over one round: room for the tree before it, the accepted tokens after it.
        dict(name="tables round", op="tables", B=64, lo=8192, hi=8192, nodes=6, maxb=544),
        # A large batch of unequal lengths with a wide tree.
        dict(name="tables wide", op="tables", B=1024, lo=1, hi=32768, nodes=68, maxb=2053),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "rope", "tables"])
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
    if op == "rope":
        d = rng.choice([64, 128])
        tree = rng.random() < 0.5
        chains, chain = rng.choice([3, 9, 16]), rng.randint(1, 4)
        S = chains if tree else _log(rng, 1, 4000)
        hi = _log(rng, 1, 1000000)
        return dict(op=op, B=max(1, min(_log(rng, 1, 64), 16000 // S)), Hq=rng.choice([4, 12, 32, 64]),
                    Hkv=rng.choice([1, 4, 8]), d=d, S=S, rot=rng.choice([d, d // 2, 24]),
                    interleaved=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]), lo=hi // 3, hi=hi,
                    chain=chain if tree else 0, chains=chains if tree else 0, factor=rng.choice([1.0, 8.0, 40.0]))
    hi = _log(rng, 1, 32000)
    nodes = rng.choice([1, 6, 27, 68, 128])
    return dict(op=op, B=_log(rng, 1, 1024), lo=rng.choice([hi, hi // 5]), hi=hi, nodes=nodes,
                maxb=(hi + nodes + PAGE) // PAGE + rng.choice([0, 3, 64]))


# ---------------------------------------------------------------------------
# what a user's program has in hand
# ---------------------------------------------------------------------------
def _lengths(case):
    """The batch's prefix lengths, evenly spread over [lo, hi] (their order is drawn by the seed)."""
    n = case["B"]
    return [case["lo"] + (case["hi"] - case["lo"]) * i // max(1, n - 1) for i in range(n)]


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


def _pow2_scale(amax):
    """The smallest power of two s (not below 2^-100) with amax / s <= 448."""
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(amax == 0, torch.full_like(k, MIN_SCALE_EXP), k).clamp(min=MIN_SCALE_EXP)
    return torch.ldexp(torch.ones_like(amax), k)


def _filled_cache(nb, Hkv, d, gain, g):
    """A cache of normal values (each head's channels of unequal size), quantised block by block."""
    codes = torch.empty(nb, Hkv, PAGE, d, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(nb, Hkv, dtype=torch.float32, device="cuda")
    channel = torch.exp(gain * _randn((1, Hkv, 1, d), g, torch.float32))
    step = max(1, (1 << 25) // (Hkv * PAGE * d))
    for o in range(0, nb, step):
        n = min(step, nb - o)
        x = _randn((n, Hkv, PAGE, d), g).float() * channel
        s = _pow2_scale(x.abs().amax(dim=(2, 3)))
        scale[o:o + n] = s
        codes[o:o + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
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


def _frequencies(rot, base, factor, original=4096, fast=32.0, slow=1.0):
    """Angle per position of each rotated pair (64 bits), scaled by parts for a ``factor`` times longer context:
    pairs that turn often in the original length keep their frequency, slow ones are divided by the factor,
    a linear ramp between; and the magnitude 0.1 ln(factor) + 1."""
    i = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2.0 * i / rot)
    if factor > 1.0:
        def pair(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        f = f / factor * ramp + f * (1.0 - ramp)
    return f, (0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0)


def prepare(case, seed):
    return {"attention": _prepare_attention, "append": _prepare_append, "rope": _prepare_rope,
            "tables": _prepare_tables}[case["op"]](case, seed)


def _prepare_attention(c, seed):
    g = _gen(seed)
    parent = _tree(c)
    N = len(parent)
    Nq = c["chains"] * c["chain"] or N
    prefix = _shuffled(_lengths(c), g)
    maxb = (c["hi"] + N + PAGE - 1) // PAGE
    table, nb = _paged(prefix + N, maxb, g)
    kc, ks = _filled_cache(nb, c["Hkv"], c["d"], 0.5, g)
    vc, vs = _filled_cache(nb, c["Hkv"], c["d"], 0.5, g)
    q = _randn((c["B"], Nq, c["Hq"], c["d"]), g)
    s = dict(op=c["op"], q=q, kc=kc, ks=ks, vc=vc, vs=vs, table=table, prefix=prefix,
             parent=torch.tensor([parent] * c["B"], dtype=torch.int32, device="cuda"),
             out=torch.empty_like(q), lse=torch.empty(q.shape[:3], dtype=torch.float32, device="cuda"),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"), scale=c["d"] ** -0.5)
    s["ws"] = torch.empty(128 << 20, dtype=torch.uint8, device="cuda")
    return s


def _prepare_append(c, seed):
    g = _gen(seed)
    B, S, Hkv, d = c["B"], c["S"], c["Hkv"], c["d"]
    prefix = _shuffled(_lengths(c), g)
    count = _shuffled([S - (S // 2) * i // max(1, B - 1) for i in range(B)], g) if c["ragged"] else None
    maxb = (c["hi"] + c["node0"] + S + PAGE - 1) // PAGE
    table, nb = _paged(prefix + c["node0"] + S, maxb, g, spare=1)
    kc, ks = _filled_cache(nb, Hkv, d, 0.5, g)
    vc, vs = _filled_cache(nb, Hkv, d, 0.5, g)
    for codes, scale in ((kc, ks), (vc, vs)):  # the spare block: where the plain form puts what is not written
        codes[-1] = torch.zeros(Hkv, PAGE, d, device="cuda").to(codes.dtype)
        scale[-1] = 0
    qkv = _randn((B, S, 2, Hkv, d), g)  # the projections' rows: a token's key heads, then its value heads
    return dict(op=c["op"], kn=qkv[:, :, 0], vn=qkv[:, :, 1], kc=kc, ks=ks, vc=vc, vs=vs, table=table, prefix=prefix,
                count=count, node0=c["node0"], status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_rope(c, seed):
    g = _gen(seed)
    B, S, d = c["B"], c["S"], c["d"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    freq, mscale = _frequencies(c["rot"], 500000.0 if c["d"] == 64 else 10000.0, c["factor"])
    turns = torch.tensor([round(f / (2 * math.pi) * 2.0 ** 64) for f in freq], dtype=torch.int64, device="cuda")
    parent, node0 = None, 0
    if c["chains"]:  # the last decode step's fed nodes, numbered step by step
        n = c["chains"]
        p = list(range(-1, 3)) + [i % 5 - 1 if t == 0 else 4 + (t - 1) * n + i for t in range(c["chain"])
                                  for i in range(n)]
        parent = torch.tensor([p] * B, dtype=torch.int32, device="cuda")
        node0 = len(p) - n
    H = c["Hq"] + c["Hkv"]
    x = _randn((B, S, H + c["Hkv"], d), g, dt)  # the fused projections: query, key and value heads of a token
    return dict(op=c["op"], q=x[:, :, :c["Hq"]], k=x[:, :, c["Hq"]:H], freq=torch.tensor(freq, device="cuda"),
                turns=turns, mscale=mscale, rot=c["rot"], interleaved=c["interleaved"], parent=parent, node0=node0,
                prefix=_shuffled(_lengths(c), g), qo=torch.empty(B, S, c["Hq"], d, dtype=dt, device="cuda"),
                ko=torch.empty(B, S, c["Hkv"], d, dtype=dt, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_tables(c, seed):
    g = _gen(seed)
    B, maxb, nodes = c["B"], c["maxb"], c["nodes"]
    before = _shuffled(_lengths(c), g)
    accepted = torch.randint(1, nodes + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    done = torch.rand(B, generator=g, device="cuda") < 0.02  # requests that end with this round
    after = torch.where(done, torch.full_like(before, -1), before + accepted)
    table, nb = _paged(before, maxb, g)
    pages = ((before + PAGE - 1) // PAGE).int()
    free = B * ((nodes + PAGE - 1) // PAGE + 1) + 7
    spare = (nb + torch.randperm(free, generator=g, device="cuda")).int()
    total = nb + free
    head = int(torch.randint(0, total, (1,), generator=g, device="cuda"))
    ring = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(free, device="cuda")) % total] = spare
    return dict(op=c["op"], before=before, after=after, table=table, pages=pages, ring=ring, nodes=nodes,
                pool=torch.tensor([head, free, 0, 0], dtype=torch.int32, device="cuda"),
                slots=torch.empty(B, nodes, dtype=torch.int32, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"attention": _plain_attention, "append": _plain_append, "rope": _plain_rope,
            "tables": _plain_tables}[s["op"]](s)


def _run_own(s):
    from speculative_decoding_vocab_gb300 import binding as ssd
    if s["op"] == "attention":
        ssd.ssd_branch_attention_q8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["prefix"], s["parent"],
                                    s["out"], lse=s["lse"], scale=s["scale"], status=s["status"], ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "append":
        ssd.ssd_kv_append_q8(s["kn"], s["vn"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["prefix"], s["node0"],
                             count=s["count"], status=s["status"])
        return {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
    if s["op"] == "rope":
        ssd.ssd_tree_rope(s["q"], s["k"], s["turns"], s["rot"], s["prefix"], s["qo"], s["ko"], parent=s["parent"],
                          node0=s["node0"], interleaved=s["interleaved"], mscale=s["mscale"], status=s["status"])
        return {"q": s["qo"], "k": s["ko"]}
    # a round: room for the tree's nodes, then the accepted tokens alone
    ssd.ssd_block_table_update(s["before"], s["nodes"], s["table"], s["pages"], s["ring"], s["pool"],
                               slots=s["slots"], status=s["status"])
    ssd.ssd_block_table_update(s["after"], 0, s["table"], s["pages"], s["ring"], s["pool"], status=s["status"])
    return {"table": s["table"], "pages": s["pages"], "ring": s["ring"], "pool": s["pool"], "slots": s["slots"]}


def _ancestors(parent):
    """[B, N, N]: node n is m or one of its ancestors (the closure of the parent relation, by squaring)."""
    N = parent.shape[1]
    n = torch.arange(N, device=parent.device)
    a = ((parent[:, :, None] == n) | (n[:, None] == n)).float()
    for _ in range(max(1, math.ceil(math.log2(max(N, 2))))):
        a = (a @ a).clamp(max=1.0)
    return a


def _plain_attention(s):
    q, table, prefix, parent = s["q"], s["table"], s["prefix"].long(), s["parent"]
    B, Nq, Hq, d = q.shape
    Hkv, N = s["kc"].shape[1], parent.shape[1]
    G = Hq // Hkv
    blk = table.clamp(min=0).long()

    def gather(codes, scale):
        x = codes.view(torch.uint8)[blk].view(torch.float8_e4m3fn).float() * scale[blk][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, -1, d)
    k, v = gather(s["kc"], s["ks"]), gather(s["vc"], s["vs"])
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
    """Block windows around the new rows: a block's scale grows to what its new rows need, rows that it already
    held are rewritten at the new scale, rows behind the new ones stay as they are."""
    B, S = s["kn"].shape[:2]
    dev = s["kn"].device
    table = s["table"]
    first = s["prefix"].long() + s["node0"]
    count = s["count"].long() if s["count"] is not None else torch.full((B,), S, device=dev)
    page = first[:, None] // PAGE + torch.arange((S + PAGE - 2) // PAGE + 1, device=dev)  # [B, P]
    rel = page[..., None] * PAGE + torch.arange(PAGE, device=dev) - first[:, None, None]   # [B, P, 16]
    new, kept = (rel >= 0) & (rel < count[:, None, None]), rel < 0
    touched = new.any(-1)
    nb = s["kc"].shape[0]
    blk = torch.where(touched, table.gather(1, page.clamp(max=table.shape[1] - 1)).long(),
                      torch.full_like(page, nb - 1))
    src = rel.clamp(0, S - 1)
    b = torch.arange(B, device=dev)[:, None, None]

    def write(x, codes, scale):
        rows = x[b, src].float().transpose(2, 3)                        # [B, P, Hkv, 16, d]
        n, kp = new[:, :, None, :, None], kept[:, :, None, :, None]
        finite = torch.where(n & rows.isfinite(), rows, torch.zeros_like(rows))
        need = _pow2_scale(finite.abs().amax(dim=(3, 4)))
        old = scale[blk]
        at = torch.where(kept.any(-1)[:, :, None], torch.maximum(old, need), need)
        held = codes.view(torch.uint8)[blk].view(torch.float8_e4m3fn).float()
        held = torch.where(kp, held * old[..., None, None] / at[..., None, None], held)
        out = torch.where(n, rows / at[..., None, None], held)
        out = torch.where(touched[:, :, None, None, None], out, torch.zeros_like(out)).to(torch.float8_e4m3fn)
        codes.view(torch.uint8)[blk] = out.view(torch.uint8)
        scale[blk] = torch.where(touched[:, :, None], at, torch.zeros_like(at))
    write(s["kn"], s["kc"], s["ks"])
    write(s["vn"], s["vc"], s["vs"])
    return {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}


def _plain_rope(s):
    B, S = s["q"].shape[:2]
    dev, rot = s["q"].device, s["rot"]
    if s["parent"] is None:
        pos = s["prefix"].long()[:, None] + s["node0"] + torch.arange(S, device=dev)
    else:
        depth = _ancestors(s["parent"]).sum(-1).long() - 1
        pos = s["prefix"].long()[:, None] + depth[:, s["node0"]:s["node0"] + S]
    angle = pos[:, :, None].double() * s["freq"]
    cos, sin = ((f(angle) * s["mscale"]).float()[:, :, None] for f in (torch.cos, torch.sin))

    def turn(x):
        y = x.float()
        r = y[..., :rot]
        if s["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
        return torch.cat((r, y[..., rot:]), dim=-1).to(x.dtype)
    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _plain_tables(s):
    def update(length, reserve, slots):
        table, pages, ring, pool = s["table"], s["pages"], s["ring"], s["pool"]
        B, maxb = table.shape
        n = ring.shape[0]
        head, free = pool[0].long(), pool[1].long()
        want = torch.where(length < 0, torch.zeros_like(length), (length + reserve + PAGE - 1) // PAGE).long()
        have = pages.long()
        grow = (want - have).clamp(min=0)
        ends = grow.cumsum(0)
        fits = ends <= free
        want = torch.where(fits, want, torch.minimum(want, have))
        p = torch.arange(maxb, device=table.device)
        at = (head + (ends - grow)[:, None] + p - have[:, None]) % n
        given = ring[at]
        taken = torch.where(fits, grow, torch.zeros_like(grow)).sum()
        released = (p >= want[:, None]) & (p < have[:, None])
        order = released.flatten().cumsum(0) - 1
        to = torch.where(released.flatten(), (head + free + order) % n, torch.full_like(order, n))
        ring.copy_(torch.cat((ring, ring[:1])).scatter(0, to, table.flatten())[:n])
        new = torch.where(p < have[:, None], table, given)
        table.copy_(torch.where(p < want[:, None], new, torch.full_like(table, -1)))
        pages.copy_(want)
        pool[0], pool[1] = (head + taken) % n, free - taken + released.sum()
        if slots:
            at = length.clamp(min=0).long()[:, None] + torch.arange(slots, device=table.device)
            blk = table.gather(1, (at // PAGE).clamp(max=maxb - 1))
            ok = (at // PAGE < want[:, None]) & (length >= 0)[:, None]
            s["slots"].copy_(torch.where(ok, blk * PAGE + at % PAGE, torch.full_like(at, -1)))
    update(s["before"], s["nodes"], s["nodes"])
    update(s["after"], 0, 0)
    return {"table": s["table"], "pages": s["pages"], "ring": s["ring"], "pool": s["pool"], "slots": s["slots"]}


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
        cache = keys * c["Hkv"] * 2 * c["d"] + pages * (c["Hkv"] * 8 + 4)
        return {"bytes": cache + c["B"] * rows * (4 * c["d"] + 4) + c["B"] * 4 * (N + 1),
                "flops": 4 * keys * rows * c["d"]}
    if c["op"] == "append":
        B, S = c["B"], c["S"]
        tokens = sum(S - (S // 2) * i // max(1, B - 1) for i in range(B)) if c["ragged"] else B * S
        return {"bytes": tokens * c["Hkv"] * 2 * c["d"] * 3 + tokens // PAGE * (c["Hkv"] * 8 + 4) + B * 4,
                "flops": tokens * c["Hkv"] * 2 * c["d"] * 2}
    if c["op"] == "rope":
        n = c["B"] * c["S"] * (c["Hq"] + c["Hkv"])
        return {"bytes": n * c["d"] * (2 if c["dtype"] == "bf16" else 4) * 2 + c["rot"] * 4 + c["B"] * 4,
                "flops": n * c["rot"] * 3}
    # read: lengths, page counts, the entries behind the accepted tokens' pages; written: the new entries, the
    # freed ids, the slots
    grown = c["B"] * ((c["nodes"] + PAGE - 1) // PAGE)
    return {"bytes": c["B"] * 4 * 6 + grown * 4 * 6 + c["B"] * c["nodes"] * 4, "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "rope": _exact_rope,
            "tables": lambda _: None}[case["op"]](s)


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
        blk = s["table"][b, :(L + N + PAGE - 1) // PAGE].long()
        hidden = torch.cat((torch.zeros(Nq, L, dtype=torch.bool, device=q.device), ~paths), dim=1)
        for h in range(Hkv):
            k, v = (codes.view(torch.uint8)[blk, h].view(torch.float8_e4m3fn).double() * scale[blk, h].double()[:, None, None]
                    for codes, scale in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            k, v = k.reshape(-1, d)[:L + N], v.reshape(-1, d)[:L + N]
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = torch.einsum("ngd,td->ngt", q[b, :, heads].double(), k) * s["scale"]
            x = x.masked_fill(hidden[:, None], -math.inf)
            lse[b, :, heads] = torch.logsumexp(x, -1)
            out[b, :, heads] = torch.einsum("ngt,td->ngd", torch.softmax(x, -1), v)
    return {"out": out, "lse": lse}


def _exact_append(s):
    """Sequence by sequence, in logical order: read the sequence's blocks as values, place the rows, quantise."""
    B, S = s["kn"].shape[:2]
    for b in range(B):
        first = int(s["prefix"][b]) + s["node0"]
        n = S if s["count"] is None else int(s["count"][b])
        if n == 0:
            continue
        p0, p1 = first // PAGE, (first + n - 1) // PAGE
        ids = s["table"][b, p0:p1 + 1].long()
        for x, codes, scale in ((s["kn"], s["kc"], s["ks"]), (s["vn"], s["vc"], s["vs"])):
            Hkv, d = x.shape[2:]
            held = codes.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()      # [P, Hkv, 16, d]
            flat = held.transpose(1, 2).reshape(-1, Hkv, d)
            lead = first - p0 * PAGE
            fresh = torch.zeros_like(flat)
            fresh[lead:lead + n] = x[b, :n].double()
            amax = fresh.reshape(-1, PAGE, Hkv, d).abs().amax(dim=(1, 3))               # [P, Hkv]
            e = torch.ceil(torch.log2(amax / E4M3_MAX))
            e = torch.where(amax > E4M3_MAX * torch.exp2(e), e + 1, e)
            e = torch.where(amax <= E4M3_MAX * torch.exp2(e - 1), e - 1, e).clamp(min=MIN_SCALE_EXP)
            at = torch.exp2(e)
            if lead:
                at[0] = torch.maximum(at[0], scale[ids[0]].double())
                flat[:lead] = flat[:lead] * (scale[ids[0]].double() / at[0])[:, None]
            wide = at.repeat_interleave(PAGE, 0)[:, :, None]
            flat[lead:lead + n] = x[b, :n].double() / wide[lead:lead + n]
            done = flat.reshape(-1, PAGE, Hkv, d).transpose(1, 2).float().to(torch.float8_e4m3fn)
            codes.view(torch.uint8)[ids] = done.view(torch.uint8)
            scale[ids] = at.float()
    return {"k": s["kc"].double(), "v": s["vc"].double(), "k_scale": s["ks"].double(), "v_scale": s["vs"].double()}


def _exact_rope(s):
    B, S = s["q"].shape[:2]
    dev, rot = s["q"].device, s["rot"]
    if s["parent"] is None:
        steps = list(range(s["node0"], s["node0"] + S))
    else:
        parent, steps = s["parent"][0].tolist(), []
        for m in range(s["node0"], s["node0"] + S):
            depth = 0
            while parent[m] >= 0:
                m, depth = parent[m], depth + 1
            steps.append(depth)
    pos = s["prefix"].double()[:, None] + torch.tensor(steps, dtype=torch.float64, device=dev)
    unit = torch.polar(torch.full((1,), s["mscale"], dtype=torch.float64, device=dev),
                       torch.zeros(1, dtype=torch.float64, device=dev))
    z = torch.exp(1j * (pos[..., None] * s["freq"])) * unit

    def turn(x):
        y = x.double().clone()
        even, odd = (slice(0, rot, 2), slice(1, rot, 2)) if s["interleaved"] else (slice(0, rot // 2),
                                                                                  slice(rot // 2, rot))
        w = torch.complex(y[..., even], y[..., odd]) * z[:, :, None]
        y[..., even], y[..., odd] = w.real, w.imag
        return y
    return {"q": turn(s["q"]), "k": turn(s["k"])}

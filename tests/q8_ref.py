"""Plain 64-bit forms of the 8-bit cache calls (block tables, rotary tree
positions, quantising append, tree attention), sequence by sequence, written
from the definitions in include/ssd.h; nothing of the library is used."""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE = 16
BAD_TREE, BAD_BLOCK, BAD_PREFIX, BAD_VALUE, NO_BLOCKS = 16, 32, 64, 512, 1024
MIN_SCALE = 2.0 ** -100


def e4m3_values():
    """The value of each of the 256 codes (NaN for 0x7F and 0xFF)."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        v[c] = -x if c & 128 else x
    v[0x7F] = v[0xFF] = np.nan
    return v


VALUES = e4m3_values()
_POS = VALUES[:127]  # 0 .. 448, increasing


def e4m3_round(x):
    """Codes of the nearest e4m3 values (ties to the even code), clamped to +-448; 0x7F for NaN."""
    a = np.minimum(np.abs(x), 448.0)
    nan = np.isnan(x)
    a = np.where(nan, 0, a)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.signbit(x), c | 128, c)
    return np.where(nan, 0x7F, c).astype(np.uint8)


def pow2_scale(amax):
    if amax == 0:
        return MIN_SCALE
    e = math.ceil(math.log2(amax / 448.0))
    while 448.0 * 2.0 ** e < amax:
        e += 1
    while 448.0 * 2.0 ** (e - 1) >= amax:
        e -= 1
    return max(2.0 ** e, MIN_SCALE)


def block_table_update(length, reserve, table, pages, ring, pool, S):
    """In place on numpy arrays; returns (slots, flags)."""
    B, maxb = table.shape
    n = len(ring)
    flags = 0
    head, free = int(pool[0]), int(pool[1])
    if not (0 <= head < n and 0 <= free <= n):
        head = free = 0
        flags |= BAD_PREFIX
    old = table.copy()
    total, taken, back = 0, 0, []
    for b in range(B):
        have = min(max(int(pages[b]), 0), maxb)
        if have != pages[b]:
            flags |= BAD_PREFIX
        want = 0 if length[b] < 0 else -(-(int(length[b]) + reserve) // PAGE)
        if want > maxb:
            flags |= BAD_PREFIX
            want = have
        if want > have:
            start = total
            total += want - have
            if total > free:
                flags |= NO_BLOCKS
                want = have
            else:
                taken = total
                for p in range(have, want):
                    table[b, p] = ring[(head + start + p - have) % n]
        for p in range(want, have):
            back.append(old[b, p])
            table[b, p] = -1
        pages[b] = want
    for i, blk in enumerate(back):
        ring[(head + free + i) % n] = blk
    pool[0], pool[1] = (head + taken) % n, free - taken + len(back)
    slots = np.full((B, S), -1, np.int64)
    for b in range(B):
        for i in range(S):
            pos = int(length[b]) + i
            if length[b] >= 0 and pos // PAGE < pages[b]:
                slots[b, i] = int(table[b, pos // PAGE]) * PAGE + pos % PAGE
    return slots, flags


def depths(parent, node0, S):
    out = []
    for m in range(node0, node0 + S):
        n, x = 0, m
        while -1 < parent[x] < x:
            x = parent[x]
            n += 1
        out.append(n)
    return out


def rope(x, theta, rot, pos, interleaved, mscale):
    """x [B, S, H, d], pos [B, S] integers, theta [rot/2]: fp64."""
    y = x.astype(np.float64).copy()
    ang = pos[:, :, None].astype(np.float64) * theta
    c, s = np.cos(ang)[:, :, None] * mscale, np.sin(ang)[:, :, None] * mscale
    i0, i1 = ((np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved
              else (np.arange(rot // 2), np.arange(rot // 2, rot)))
    a, b = y[..., i0].copy(), y[..., i1].copy()
    y[..., i0], y[..., i1] = a * c - b * s, a * s + b * c
    return y


def kv_append(x, codes, scale, table, prefix, node0, count):
    """One operand, in place: x [B, S, H, d] fp64, codes uint8, scale fp64-valued fp32; returns flags."""
    B, S, H, d = x.shape
    nb, maxb = codes.shape[0], table.shape[1]
    flags = 0
    for b in range(B):
        n = S if count is None else int(count[b])
        if n != min(max(n, 0), S):
            flags |= BAD_PREFIX
            n = min(max(n, 0), S)
        if prefix[b] < 0:
            flags |= BAD_PREFIX
            continue
        first = int(prefix[b]) + node0
        for page in range(first // PAGE, (first + n - 1) // PAGE + 1 if n else first // PAGE):
            if page >= maxb:
                flags |= BAD_PREFIX
                continue
            blk = int(table[b, page])
            if not 0 <= blk < nb:
                flags |= BAD_BLOCK
                continue
            rows = [(r, page * PAGE + r - first) for r in range(PAGE)]
            new = [(r, i) for r, i in rows if 0 <= i < n]
            held = [r for r, i in rows if i < 0]
            for h in range(H):
                vals = np.stack([x[b, i, h] for _, i in new])
                ok = np.isfinite(vals)
                if not ok.all():
                    flags |= BAD_VALUE
                at = pow2_scale(np.abs(np.where(ok, vals, 0)).max())
                if held:
                    old = float(scale[blk, h])
                    if not (0 <= old < math.inf):
                        flags |= BAD_VALUE
                        old = 0.0
                    if at > old:
                        f = VALUES[codes[blk, h][held]]
                        q = (np.float32(f) * np.float32(old)) / np.float32(at)
                        codes[blk, h][held] = e4m3_round(q.astype(np.float64))
                    else:
                        at = old
                f32 = np.where(ok, vals, np.nan).astype(np.float32) / np.float32(at)
                for (r, _), q in zip(new, f32):
                    codes[blk, h, r] = e4m3_round(q.astype(np.float64))
                scale[blk, h] = at
    return flags


def paths(parent, Nq):
    """[Nq, N]: the nodes that each query node sees; and whether a parent is bad."""
    N = len(parent)
    seen, bad = np.zeros((Nq, N), bool), False
    for i in range(Nq):
        m = N - Nq + i
        while True:
            seen[i, m] = True
            up = int(parent[m])
            if up < -1 or up >= m:
                bad = True
                break
            if up < 0:
                break
            m = up
    return seen, bad


def attention(q, kc, vc, ks, vs, table, prefix, parent, scale, device="cpu"):
    """q [B, Nq, Hq, d] (any float), codes uint8, scales fp32.  Returns fp64
    (out, lse, weight, (xabs, xcut), share) and the flags: weight =
    softmax-weighted |v| per element, xabs = the largest sum of |scale q k| of a
    row, xcut = scale max|q| times the largest sum of |k| of a key, share =
    max p v_scale * sum of |code| over the visible keys / sum of p, p = exp(x -
    max): what errors in p v_scale, relative to the row's largest, may move."""
    B, Nq, Hq, d = q.shape
    nb, Hkv = ks.shape
    maxb, N, G = table.shape[1], parent.shape[1], Hq // Hkv
    out = np.zeros((B, Nq, Hq, d))
    lse, xabs, xcut = np.full((B, Nq, Hq), -np.inf), np.zeros((B, Nq, Hq)), np.zeros((B, Nq, Hq))
    weight, share = np.zeros((B, Nq, Hq, d)), np.zeros((B, Nq, Hq, d))
    flags = 0
    val = torch.tensor(VALUES, device=device)
    for b in range(B):
        seen, bad = paths(parent[b], Nq)
        flags |= BAD_TREE if bad else 0
        L = max(int(prefix[b]), 0)
        nk = L + N
        if prefix[b] < 0 or nk > maxb * PAGE:
            flags |= BAD_PREFIX
        nk = min(nk, maxb * PAGE)
        ids = table[b, :-(-nk // PAGE)].astype(np.int64)
        in_pool = (ids >= 0) & (ids < nb)
        flags |= 0 if in_pool.all() else BAD_BLOCK
        safe = torch.tensor(np.where(in_pool, ids, 0), device=device)
        vis = np.concatenate([np.ones((Nq, min(L, nk)), bool), seen[:, :max(nk - L, 0)]], axis=1)
        for h in range(Hkv):
            sk, sv = ks[np.where(in_pool, ids, 0), h], vs[np.where(in_pool, ids, 0), h]
            good = np.isfinite(sk) & np.isfinite(sv) & (sk >= 0) & (sv >= 0)
            flags |= 0 if good[in_pool].all() else BAD_VALUE
            usable = np.repeat(in_pool & good, PAGE)[:nk]
            mask = torch.tensor(vis & usable, device=device)
            svf = np.where(sv < MIN_SCALE, 0, sv)

            def rows(codes, sc):
                c = torch.as_tensor(codes, device=device)[safe, h].long()
                f = torch.tensor(np.where(good, sc, 0).astype(np.float64), device=device)
                return (val[c] * f[:, None, None]).reshape(-1, d)[:nk]
            k, v = rows(kc, sk), rows(vc, svf)
            qq = torch.as_tensor(q[b][:, h * G:(h + 1) * G].astype(np.float64), device=device)
            kz = torch.where(mask.any(0)[:, None], k, torch.zeros_like(k))
            x = torch.einsum("ngd,td->ngt", qq, kz) * scale
            xa = torch.einsum("ngd,td->ngt", qq.abs(), kz.abs().nan_to_num(0)) * scale
            x = torch.where(mask[:, None], x, torch.full_like(x, -math.inf))
            top = x.nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf).amax(-1, keepdim=True)
            top = torch.where(top == -math.inf, torch.zeros_like(top), top)
            p = torch.exp(x - top)
            tot = p.sum(-1, keepdim=True)
            # hidden keys take no part, whatever they hold: only a row that sees a NaN in v gets it
            vz, vn = v.nan_to_num(0.0), v.isnan().double()
            sees = mask[:, None].expand(Nq, G, nk).double()
            o = torch.einsum("ngt,td->ngd", p, vz)
            hit = torch.einsum("ngt,td->ngd", sees, vn) > 0
            den = torch.where(tot == 0, torch.ones_like(tot), tot)
            o = torch.where(hit, torch.full_like(o, math.nan), o / den)
            hs = slice(h * G, (h + 1) * G)
            out[b][:, hs] = o.cpu().numpy()
            lse[b][:, hs] = (top + tot.log()).squeeze(-1).cpu().numpy()
            weight[b][:, hs] = (torch.einsum("ngt,td->ngd", p, vz.abs()) / den).cpu().numpy()
            codes = rows(vc, np.ones_like(sv)).nan_to_num(0).abs()
            sc = torch.tensor(np.repeat(np.where(good, svf, 0).astype(np.float64), PAGE)[:nk], device=device)
            big = (p.nan_to_num(0) * sc).amax(-1, keepdim=True)
            share[b][:, hs] = (big * torch.einsum("ngt,td->ngd", sees, codes) / den).cpu().numpy()
            xabs[b][:, hs] = torch.where(mask[:, None], xa, torch.zeros_like(xa)).amax(-1).cpu().numpy()
            ksum = torch.where(mask, kz.abs().nan_to_num(0).sum(-1), torch.zeros_like(kz[:, 0])).amax(-1)
            xcut[b][:, hs] = (scale * qq.abs().amax(-1) * ksum[:, None]).cpu().numpy()
    return out, lse, weight, (xabs, xcut), share, flags

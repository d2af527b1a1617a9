"""Plain 64-bit forms of the 4-bit cache calls (quantising append, rows read
back, tree attention) and of the token log probabilities, written from the
definitions in include/ssd.h; nothing of the library is used."""
from __future__ import annotations

import math

import numpy as np
import torch

from q8_ref import BAD_BLOCK, BAD_PREFIX, BAD_TREE, BAD_VALUE, PAGE, paths

BAD_TOKEN = 1
GROUP = 32
MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
VALUES = np.concatenate([MAGNITUDES, -MAGNITUDES])


def e2m1_round(x):
    """Codes of the nearest e2m1 values (ties to the even code), clamped to +-6; the sign of zeros is kept."""
    a = np.minimum(np.abs(x), 6.0)
    d = np.abs(a[..., None] - MAGNITUDES)
    near = d == d.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    c = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    return np.where(np.signbit(x), c | 8, c).astype(np.uint8)


def scale_exp(amax):
    """The smallest e in [-100, 125] with amax <= 6 * 2^e (125 where there is none)."""
    for e in range(-100, 125):
        if amax <= 6.0 * 2.0 ** e:
            return e
    return 125


def quantise(row):
    """(codes, bytes, bad) of one row [d]."""
    d = len(row)
    codes, bytes_, bad = np.zeros(d, np.uint8), np.zeros(d // GROUP, np.uint8), False
    for g in range(d // GROUP):
        x = row[g * GROUP:(g + 1) * GROUP]
        if not np.isfinite(x).all():
            bytes_[g], bad = 255, True
            continue
        e = scale_exp(np.abs(x).max())
        codes[g * GROUP:(g + 1) * GROUP] = e2m1_round(x * 2.0 ** -e)
        bytes_[g] = e + 127
    return codes, bytes_, bad


def scale_values(b):
    return np.where(b == 255, np.nan, 2.0 ** (b.astype(np.float64) - 127))


class Cache:
    """One operand's codes [nb, H, 16, d] (a code each) and scale bytes [nb, H, 16, d / 32]."""

    def __init__(self, codes, scale):
        self.codes, self.scale = codes, scale

    def packed(self, which):
        c = self.codes
        if which == "k":
            return c[..., 0::2] | (c[..., 1::2] << 4)
        return c[:, :, 0::2] | (c[:, :, 1::2] << 4)

    def values(self):
        return VALUES[self.codes] * np.repeat(scale_values(self.scale), GROUP, axis=-1)


def rows_of(table, nb, prefix, node0, S, count):
    """(flags, [(b, i, block, slot)]) of the rows that a call reaches."""
    flags, rows = 0, []
    maxb = table.shape[1]
    for b in range(len(prefix)):
        if prefix[b] == -1:
            continue
        n = S if count is None else int(count[b])
        if n != min(max(n, 0), S):
            flags |= BAD_PREFIX
            n = min(max(n, 0), S)
        if prefix[b] < 0:
            flags |= BAD_PREFIX
            continue
        for i in range(n):
            pos = int(prefix[b]) + node0 + i
            if pos // PAGE >= maxb:
                flags |= BAD_PREFIX
                continue
            blk = int(table[b, pos // PAGE])
            if not 0 <= blk < nb:
                flags |= BAD_BLOCK
                continue
            rows.append((b, i, blk, pos % PAGE))
    return flags, rows


def kv_append(x, cache, table, prefix, node0, count):
    """One operand, in place: x [B, S, H, d] fp64; returns flags."""
    flags, rows = rows_of(table, len(cache.codes), prefix, node0, x.shape[1], count)
    for b, i, blk, r in rows:
        for h in range(x.shape[2]):
            c, e, bad = quantise(x[b, i, h])
            cache.codes[blk, h, r], cache.scale[blk, h, r] = c, e
            flags |= BAD_VALUE if bad else 0
    return flags


def kv_read(cache, table, prefix, node0, count, out):
    """In place on out [B, S, H, d]; returns flags."""
    flags, rows = rows_of(table, len(cache.codes), prefix, node0, out.shape[1], count)
    v = cache.values()
    for b, i, blk, r in rows:
        out[b, i] = v[blk, :, r]
    return flags


def attention(q, kc, vc, table, prefix, parent, scale, device="cpu"):
    """q [B, Nq, Hq, d] (any float), Caches.  Returns fp64 (out, lse, weight,
    (xabs, xcut), (share, cut)) and the flags: weight = softmax-weighted |v| per
    element, xabs = the largest sum of |scale q k| of a row, xcut = scale max|q|
    times the largest sum of |k| of a key; with t the largest v scale of a key
    and p = exp(x - max): share = max(p t) * sum of |v| / t over the visible
    keys / sum of p (what errors in p t, relative to the row's largest, may
    move), cut = sum of p t / sum of p (what errors in v / t may)."""
    B, Nq, Hq, d = q.shape
    nb, Hkv = kc.codes.shape[:2]
    maxb, N, G = table.shape[1], parent.shape[1], Hq // Hkv
    out = np.zeros((B, Nq, Hq, d))
    lse, xabs, xcut = np.full((B, Nq, Hq), -np.inf), np.zeros((B, Nq, Hq)), np.zeros((B, Nq, Hq))
    weight, share, cut = np.zeros((B, Nq, Hq, d)), np.zeros((B, Nq, Hq, d)), np.zeros((B, Nq, Hq))
    flags = 0
    kval = torch.tensor(kc.values(), device=device)
    vbytes = np.where(vc.scale < 27, 0, vc.scale)
    vval = torch.tensor(VALUES[vc.codes] * np.repeat(np.where(vc.scale < 27, 0, scale_values(vbytes)), GROUP, axis=-1),
                        device=device)
    top_scale = np.where(vc.scale == 255, 0, scale_values(np.where(vc.scale == 255, 0, vc.scale))).max(-1)
    top_scale = torch.tensor(np.maximum(top_scale, 2.0 ** -100), device=device)
    for b in range(B):
        if prefix[b] == -1:
            continue
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
        mask = torch.tensor(vis & np.repeat(in_pool, PAGE)[:nk], device=device)
        for h in range(Hkv):
            k, v = kval[safe, h].reshape(-1, d)[:nk], vval[safe, h].reshape(-1, d)[:nk]
            t = top_scale[safe, h].reshape(-1)[:nk]
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
            pt = p.nan_to_num(0) * t
            share[b][:, hs] = (pt.amax(-1, keepdim=True) * torch.einsum("ngt,td->ngd", sees, vz.abs() / t[:, None])
                               / den).cpu().numpy()
            cut[b][:, hs] = (pt.sum(-1) / den[..., 0]).cpu().numpy()
            xabs[b][:, hs] = torch.where(mask[:, None], xa, torch.zeros_like(xa)).amax(-1).cpu().numpy()
            ksum = torch.where(mask, kz.abs().nan_to_num(0).sum(-1), torch.zeros_like(kz[:, 0])).amax(-1)
            xcut[b][:, hs] = (scale * qq.abs().amax(-1) * ksum[:, None]).cpu().numpy()
    return out, lse, weight, (xabs, xcut), (share, cut), flags


def token_logprobs(z, T, tokens, n):
    """z [B, R, V] fp64, tokens [B, R] or None.  Returns a dict of fp64 / int arrays (rows that are not wanted:
    None in `wanted`) and the flags."""
    B, R, V = z.shape
    o = dict(logprob=np.zeros((B, R)), rank=np.zeros((B, R), np.int64), entropy=np.zeros((B, R)),
             top_ids=np.zeros((B, R, n), np.int64), top_logprob=np.zeros((B, R, n)),
             wanted=np.ones((B, R), bool))
    flags = 0
    for b in range(B):
        for r in range(R):
            t = 0 if tokens is None else int(tokens[b, r])
            if t == -1:
                o["wanted"][b, r] = False
                continue
            row = z[b, r]
            good = 0 <= t < V
            flags |= 0 if good else BAD_TOKEN
            if np.isnan(row).any() or (row == np.inf).any() or not np.isfinite(row).any():
                flags |= BAD_VALUE
                o["logprob"][b, r], o["rank"][b, r], o["entropy"][b, r] = np.nan, -1, np.nan
                o["top_ids"][b, r], o["top_logprob"][b, r] = -1, np.nan
                continue
            order = np.lexsort((np.arange(V), -row))
            if T == 0:
                lp = np.full(V, -np.inf)
                lp[order[0]] = 0.0
                h = 0.0
            else:
                x = row / T
                m = x.max()
                ls = math.log(np.exp(x - m).sum())
                lp = x - m - ls
                p = np.exp(lp)
                h = -(p[p > 0] * lp[p > 0]).sum()
            o["entropy"][b, r] = h
            o["logprob"][b, r] = lp[t] if good else np.nan
            o["rank"][b, r] = int(np.flatnonzero(order == t)[0]) if good else -1
            o["top_ids"][b, r] = order[:n]
            o["top_logprob"][b, r] = lp[order[:n]]
    return o, flags

"""Plain definitions of the operators around the indexer, in 64 bits.

Written from the formulas of include/idx.h for one request (or one token) at
a time, with no code of the CUDA path: slot maps and tree masks as Python
integers, rotary positions and attention in float64, the drafted tokens'
verification with the residual row kept and normalised at each refusal.
"""

from __future__ import annotations

import math

import numpy as np


def build_slots(ctx_lens, new_lens, owned, table, free_blocks, cursor, num_blocks, page, num_tokens, parents=None):
    """Returns a dict of the outputs of idx_build_slots and the status bits."""
    reqs, max_blocks = table.shape
    table = np.array(table, dtype=np.int64)
    cursor = min(max(int(cursor), 0), len(free_blocks))
    cu, seq, pages, pos, slots, mask = [0], [], [], [], [], []
    status = 0
    taken = 0
    for r in range(reqs):
        ctx, new = max(0, int(ctx_lens[r])), max(0, int(new_lens[r]))
        own = min(max(0, int(owned[r])), max_blocks)
        need = min(-(-(ctx + new) // page), max_blocks)
        got = own
        for j in range(own, need):
            at = cursor + taken
            taken += 1
            if at < len(free_blocks):
                table[r, j] = free_blocks[at]
                got += 1
            else:
                table[r, j] = -1
                status |= 16
        if ctx + new > max_blocks * page:
            status |= 2
        seq.append(min(ctx + new, 2**31 - 1))
        pages.append(got)
        par = None if parents is None else [int(x) for x in parents[cu[-1] : cu[-1] + new]]
        for i in range(new):
            if cu[-1] + i >= num_tokens:
                break
            place = ctx + i
            b = int(table[r, place // page]) if place // page < max(own, need) else -1
            if b < -1 or b >= num_blocks:
                status |= 1
                b = -1
            slots.append(b * page + place % page if b >= 0 else -1)
            depth, bits = i, 0
            if par is not None:
                if i < 64:
                    depth, j = -1, i
                    while j >= 0:
                        bits |= 1 << j
                        depth += 1
                        up = par[j]
                        if not -1 <= up < j:
                            status |= 32
                            up = -1
                        j = up
                else:
                    status |= 32
            pos.append(min(ctx + depth, 2**31 - 1))
            mask.append(bits)
        cu.append(cu[-1] + new)
    if cu[-1] > num_tokens:
        status |= 2
    fill = num_tokens - len(slots)
    return dict(block_table=table, cu_tokens=np.minimum(cu, num_tokens), seq_lens=np.array(seq), pages_out=np.array(pages),
                cursor_out=min(cursor + taken, len(free_blocks)), positions=np.array(pos + [0] * fill),
                slots=np.array(slots + [-1] * fill), tree_mask=np.array(mask + [0] * fill, dtype=np.uint64), status=status)


def rotate(x, positions, inv_freq, mscale, interleaved):
    """x [T, heads, D] float64 -> rotated; each pair turned by position * inv_freq."""
    x = np.asarray(x, dtype=np.float64)
    half = len(inv_freq)
    a = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq)[None]
    c, s = (np.cos(a) * mscale)[:, None], (np.sin(a) * mscale)[:, None]
    y = x.copy()
    one = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
    two = one + 1 if interleaved else one + half
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def rope_frequencies(rotary_dim, base, kind, factor=1.0, orig_len=0.0, beta_fast=32.0, beta_slow=1.0):
    """inv_freq and mscale of idx_rope_frequencies (kind 0 plain, 1 linear, 2 ramp)."""
    f = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if kind == 0:
        return np.array(f), 1.0
    if kind == 1:
        return np.array(f) / factor, 1.0
    e = lambda b: rotary_dim * math.log(orig_len / (2 * math.pi * b)) / (2 * math.log(base))
    lo, hi = max(0, math.floor(e(beta_fast))), min(rotary_dim - 1, math.ceil(e(beta_slow)))
    out = []
    for i, x in enumerate(f):
        w = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
        out.append(x * (1 - w) + x / factor * w)
    return np.array(out), 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def visible_places(seq_len, n, i, mask, pages, page, max_blocks, block_row, num_blocks):
    """Places that token i of a request's n sees, ascending."""
    ctx = seq_len - n
    used = min(-(-seq_len // page), max_blocks)
    out = []
    for pg in range(used) if pages is None else sorted({int(p) for p in pages if 0 <= p < used}):
        if not 0 <= int(block_row[pg]) < num_blocks:
            continue
        for place in range(pg * page, min((pg + 1) * page, seq_len)):
            j = place - ctx
            if j < 0 or (j <= i if mask is None else j < 64 and (int(mask) >> j) & 1):
                out.append(place)
    return np.array(out, dtype=np.int64)


def tree_attention(q, k_cache, v_cache, block_table, seq_lens, cu, scale, tree_mask=None, pages=None):
    """q [T,Hq,D], caches [nb,P,Hk,D] (float64) -> out, lse, and per element the mean magnitude sum p |v| and per row
    the largest sum |q k| scale (for error bounds)."""
    tokens, hq, d = q.shape
    nb, page, hk = k_cache.shape[:3]
    g = hq // hk
    out, lse = np.zeros((tokens, hq, d)), np.full((tokens, hq), -np.inf)
    mag, big, count = np.zeros((tokens, hq, d)), np.zeros((tokens, hq)), np.zeros(tokens, dtype=np.int64)
    for r in range(len(seq_lens)):
        n = int(cu[r + 1] - cu[r])
        for i in range(n):
            t = int(cu[r]) + i
            mask = None if tree_mask is None else int(np.uint64(tree_mask[t]))
            seen = {}
            for h in range(hk):
                which = -1 if pages is None else h // (hk // pages.shape[1])
                if which not in seen:
                    seen[which] = visible_places(int(seq_lens[r]), n, i, mask, None if pages is None else pages[t, which], page,
                                                 block_table.shape[1], block_table[r], nb)
                at = seen[which]
                count[t] = max(count[t], len(at))
                if len(at) == 0:
                    continue
                b = block_table[r][at // page].astype(np.int64)
                k, v = k_cache[b, at % page, h], v_cache[b, at % page, h]
                x = q[t, h * g : (h + 1) * g] @ k.T * scale
                big[t, h * g : (h + 1) * g] = (np.abs(q[t, h * g : (h + 1) * g]) @ np.abs(k).T).max(1) * abs(scale)
                top = x.max(1, keepdims=True)
                e = np.exp(x - top)
                mass = e.sum(1, keepdims=True)
                out[t, h * g : (h + 1) * g] = e @ v / mass
                mag[t, h * g : (h + 1) * g] = e @ np.abs(v) / mass
                lse[t, h * g : (h + 1) * g] = (top + np.log(mass))[:, 0]
    return out, lse, mag, big, count


def _rows(target, draft, t):
    p = np.maximum(np.nan_to_num(target[t].astype(np.float64), nan=0.0), 0.0)
    q = None if draft is None else np.maximum(np.nan_to_num(draft[t].astype(np.float64), nan=0.0), 0.0)
    return p, q


def verify(target, draft, tokens, parents, cu, accept_u, sample_u, max_out):
    """Returns num_accepted [R], out_tokens and out_nodes [R, max_out]; the residual is kept whole and normalised."""
    vocab = target.shape[1]
    reqs = len(cu) - 1
    acc = np.zeros(reqs, dtype=np.int64)
    out_t, out_n = np.full((reqs, max_out), -1, dtype=np.int64), np.full((reqs, max_out), -1, dtype=np.int64)
    for r in range(reqs):
        t0, n = int(cu[r]), int(cu[r + 1] - cu[r])
        if n == 0:
            continue
        at, k = 0, 0
        while True:
            p, q = _rows(target, draft, t0 + at)
            rest, gone_mass, gone, stood = p.copy(), 0.0, set(), False
            for i in range(at + 1, n) if k < max_out - 1 else ():
                par = i - 1 if parents is None else int(parents[t0 + i])
                x = int(tokens[t0 + i])
                if par != at or not 0 <= x < vocab:
                    continue
                u = float(accept_u[t0 + i])
                if draft is not None:
                    if u * q[x] < rest[x]:
                        stood = True
                    else:
                        rest = np.maximum(rest - q, 0.0)
                        mass = float(rest.sum())
                        rest = rest / mass if mass > 0 else rest
                else:
                    if u * (1.0 - gone_mass) < (0.0 if x in gone else p[x]):
                        stood = True
                    elif x not in gone:
                        gone.add(x)
                        gone_mass += p[x]
                        rest[x] = 0.0
                if stood:
                    out_t[r, k], out_n[r, k] = x, i
                    k, at = k + 1, i
                    break
            if not stood:
                break
        if not rest.sum() > 0:
            rest = p
        cum = np.cumsum(rest)
        above = np.nonzero(cum > float(sample_u[r]) * cum[-1])[0]
        out_t[r, k] = above[0] if len(above) and cum[-1] > 0 else vocab - 1
        acc[r] = k
    return acc, out_t, out_n

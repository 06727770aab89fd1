"""The calls between those of a decoding step, written from their definitions in numpy, 64 bits.

norm_rotate      norms of heads, then the rotation (idx_norm_rope_append)
index_rows       E4M3 queries with scales, NVFP4 keys (idx_index_append)
logit_probs      penalties, biases, masks, softmax (idx_logit_probs)
settle           rows of the drafts that stand moved together (idx_settle_drafts)
fork, release    pages shared and given back (idx_fork_pages, idx_release_pages)
"""

import numpy as np

from . import formats, step


def norm_rotate(x, weight, eps, offset, positions, inv_freq, mscale, interleaved):
    """x [T, H, D] -> (offset + w) x / sqrt(mean x^2 + eps), turned; weight None: turned only."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x * (offset + weight.astype(np.float64)) / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return step.rotate(x, positions, inv_freq, mscale, interleaved)


# values of the codes 0, 1, ... (E4M3 without its NaN)
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([formats.e4m3_value(b) for b in range(127)])


def nearest_code(x, values):
    """Code of the nearest value to |x|, halves to the even code, the sign above the magnitude's bits."""
    a = np.minimum(np.abs(x), values[-1])
    middle = (values[1:] + values[:-1]) / 2
    low, high = np.searchsorted(middle, a, "left"), np.searchsorted(middle, a, "right")
    code = np.where(low == high, low, low + low % 2)
    sign = 8 if len(values) == 8 else 128
    return (code + sign * (x < 0)).astype(np.uint8)


def _unnormed(x, weight, offset, positions, inv_freq, mscale, interleaved):
    x = x.astype(np.float64)
    w = 1.0 if weight is None else offset + weight.astype(np.float64)
    return step.rotate(x * w, positions, inv_freq, mscale, interleaved)


def _inverse_rms(x, weight, eps):
    x = x.astype(np.float64)
    return np.ones(x.shape[:-1]) if weight is None else 1.0 / np.sqrt(np.mean(x * x, axis=-1) + eps)


def index_queries(q, weight, eps, offset, positions, inv_freq, mscale, interleaved, scale, head_weights):
    """q [T, H, 128] -> codes [T, H, 128] uint8, scales [T, H] float64."""
    u = _unnormed(q, weight, offset, positions, inv_freq, mscale, interleaved)
    top = np.abs(u).max(-1)
    with np.errstate(invalid="ignore", divide="ignore"):
        codes = nearest_code(np.where(top[..., None] > 0, 448.0 * u / top[..., None], 0.0), E4M3)
    s = scale * top * _inverse_rms(q, weight, eps) / 448.0
    bad = ~np.isfinite(q.astype(np.float64)).all(-1)
    codes[bad], s[bad] = 0x7F, np.nan
    return codes, s if head_weights is None else s * head_weights.astype(np.float64)


def index_keys(k, weight, eps, offset, positions, inv_freq, mscale, interleaved):
    """k [T, 128] -> code bytes [T, 64], scale bytes [T, 8]."""
    y = _unnormed(k[:, None], weight, offset, positions, inv_freq, mscale, interleaved)[:, 0] * _inverse_rms(k, weight, eps)[:, None]
    y = y.reshape(-1, 8, 16)
    scales = nearest_code(np.abs(y).max(-1) / 6.0, E4M3)
    s = E4M3[np.minimum(scales, 126)][..., None]
    codes = np.where(s > 0, nearest_code(np.where(s > 0, y / np.where(s > 0, s, 1.0), 0.0), E2M1), 0).reshape(-1, 64, 2)
    bad = ~np.isfinite(k.astype(np.float64)).all(-1)
    codes[bad], scales[bad] = 0, 0x7F
    return (codes[..., 0] + 16 * codes[..., 1]).astype(np.uint8), scales


def logit_probs(logits, cu, temperature=None, repetition=None, presence=None, frequency=None, counts=None, tokens=None, tree_mask=None,
                biases=None, allowed=None):
    """logits [T, V] -> p [T, V], L [T] in float64; biases: a list of (token, value) for each request."""
    rows, vocab = logits.shape
    p, lse = np.zeros((rows, vocab)), np.full(rows, -np.inf)
    pick = lambda a, r, default: default if a is None else float(a[r])
    penal = not (repetition is None and presence is None and frequency is None)
    for r in range(len(cu) - 1):
        for t in range(cu[r], cu[r + 1]):
            i, n = t - cu[r], cu[r + 1] - cu[r]
            x = logits[t].astype(np.float64)
            if penal:
                c, prompt = np.zeros(vocab, dtype=np.int64), np.zeros(vocab, dtype=bool)
                if counts is not None:
                    c, prompt = counts[r].astype(np.int64) & 0x7FFFFFFF, counts[r] < 0
                if tokens is not None:
                    on = range(1, i + 1) if tree_mask is None else [j for j in range(1, min(n, 64)) if int(tree_mask[t]) >> j & 1]
                    for j in on:
                        if 0 <= tokens[cu[r] + j] < vocab:
                            c[tokens[cu[r] + j]] += 1
                rep = pick(repetition, r, 1.0)
                x = np.where(prompt | (c > 0), np.where(x > 0, x / rep, x * rep), x)
                x = np.where(c > 0, x - (pick(frequency, r, 0.0) * c + pick(presence, r, 0.0)), x)
            for v, b in biases[r] if biases is not None else ():
                if 0 <= v < vocab:
                    x[v] += b
            if allowed is not None:
                v = np.arange(vocab)
                x = np.where((allowed[t].astype(np.int64)[v >> 5] >> (v & 31)) & 1, x, -np.inf)
            if np.isnan(x).any() or (x == np.inf).any():
                p[t], lse[t] = np.nan, np.nan
                continue
            if not (x > -np.inf).any():
                continue
            heat = pick(temperature, r, 1.0)
            if not heat > 2.0**-60:
                p[t, np.argmax(x)], lse[t] = 1.0, x.max()
                continue
            x[x > -np.inf] /= heat  # (an infinite T leaves out what is left out)
            e = np.exp(x - x.max())
            p[t], lse[t] = e / e.sum(), np.log(e.sum()) + x.max()
    return p, lse


def settle(caches, slots, cu, out_tokens, out_nodes, accepted, ctx, counts):
    """caches: arrays [planes, blocks, page, ...]; new caches, contexts and counts."""
    caches, out, counts = [c.copy() for c in caches], np.array(ctx), None if counts is None else counts.copy()
    for r in range(len(cu) - 1):
        n = cu[r + 1] - cu[r]
        if n <= 0:
            continue
        a = max(0, min(accepted[r], min(n, out_nodes.shape[1]) - 1))
        out[r] += 1 + a
        for i in range(a):
            node = out_nodes[r, i]
            if not i + 1 <= node < n:
                continue
            src, dst = slots[cu[r] + node], slots[cu[r] + 1 + i]
            for c in caches:
                places, page = c.shape[1] * c.shape[2], c.shape[2]
                if 0 <= src < places and 0 <= dst < places:
                    c[:, dst // page, dst % page] = c[:, src // page, src % page]
        if counts is not None:
            for x in out_tokens[r, : a + 1]:
                if 0 <= x < counts.shape[1]:
                    counts[r, x] += 1
    return caches, out, counts


def fork(caches, parents, children, ctx, owned, table, refs, free, cursor, page, num_blocks):
    """New caches, ctx, owned, table, refs, cursor and the status bits."""
    caches, ctx, owned, table, refs = [c.copy() for c in caches], ctx.copy(), owned.copy(), table.copy(), refs.copy()
    reqs, width = table.shape
    status, taken = 0, 0
    old = (ctx.copy(), owned.copy(), table.copy())
    parents_of = [p for p, c in zip(parents, children) if c != -1]
    for f in range(len(parents)):
        p, c = parents[f], children[f]
        if c == -1:
            continue
        if not (0 <= p < reqs and 0 <= c < reqs) or c in parents_of or list(children).count(c) > 1:
            status |= 64
            continue
        own = min(max(old[1][p], 0), width)
        length = max(old[0][p], 0)
        if length > own * page:
            length, status = own * page, status | 2
        full, rest = divmod(int(length), page)
        if rest:
            at = cursor + taken
            taken += 1
            if at >= len(free):
                status |= 16
                ctx[c], owned[c] = 0, 0
                continue
        for i in range(full):
            b = table[c, i] = old[2][p, i]
            if 0 <= b < num_blocks:
                refs[b] += 1
            else:
                status |= 1
        if rest:
            table[c, full] = free[at]
            src = old[2][p, full]
            if 0 <= src < num_blocks:
                for k in caches:
                    k[:, free[at], :rest] = k[:, src, :rest]
            else:
                status |= 1
        ctx[c], owned[c] = length, full + (rest > 0)
    return caches, ctx, owned, table, refs, min(cursor + taken, len(free)), status


def release(keep, owned, table, refs, free, cursor, page):
    """New refs, free list, cursor, pages and the status bits."""
    refs, free = refs.copy(), free.copy()
    status, kept = 0, np.zeros_like(owned)
    left = refs.astype(np.int64)
    for r in range(len(keep)):
        own = min(max(owned[r], 0), table.shape[1])
        kept[r] = min(own, -(-max(int(keep[r]), 0) // page))
        for b in table[r, kept[r] : own]:
            if 0 <= b < len(refs):
                left[b] -= 1
            elif b != -1:
                status |= 1
    gone = np.nonzero(left < 0)[0]
    begin = cursor - len(gone)
    if begin < 0:
        status |= 4
    for i, b in enumerate(gone):
        if begin + i >= 0:
            free[begin + i] = b
    return np.maximum(left, 0).astype(np.int32), free, max(begin, 0), kept, status

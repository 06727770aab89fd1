"""What is timed of the operators around the indexer: one step of decoding with drafted tokens.

Four operators, in the order in which a serving step calls them:

* slots   block tables, slot maps, positions and tree masks from the requests' lengths
* rope    rotary positions of queries and keys, keys and values appended to the paged cache
* tree    attention of a tree of drafted tokens over the paged cache, over all pages or over those the indexer chose
* verify  which drafted tokens stand, from the target's (and the drafter's) probabilities and given random numbers

`run` computes them in elementary torch operations, or, with `own` true, by the
calls of sparse_attention_indexer_nvfp4_gb300.  Lengths and trees belong to a
case; values, block ids and random numbers come from the seed.
"""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # 64 requests with drafted trees of 8 tokens: the start of a decoding step, all latency
        dict(name="slots_drafts", op="slots", reqs=64, new_lo=8, new_hi=8, ctx_lo=8192, ctx_hi=172032, page=128, tree=True),
        # a batch of prompt chunks of all lengths entering the cache at once, small pages
        dict(name="slots_prompts", op="slots", reqs=1021, new_lo=1, new_hi=2048, ctx_lo=0, ctx_hi=8192, page=16, tree=False),
        # one token of one request, part of the head rotated
        dict(name="rope_token", op="rope", tokens=1, q_heads=64, kv_heads=4, dim=128, rotary=64, interleaved=False,
             scaled=False, dtype="bf16", page=128, pos_hi=172032),
        # 64 requests with 8 drafted tokens each, whole head, frequencies scaled for long contexts
        dict(name="rope_drafts", op="rope", tokens=512, q_heads=64, kv_heads=4, dim=128, rotary=128, interleaved=True,
             scaled=True, dtype="fp16", page=128, pos_hi=500000),
        # a prompt chunk of odd length
        dict(name="rope_prompt", op="rope", tokens=30011, q_heads=64, kv_heads=4, dim=128, rotary=64, interleaved=False,
             scaled=False, dtype="bf16", page=128, pos_hi=172032),
        # one request, one token, short context: the single-token form where latency counts
        dict(name="tree_token", op="tree", reqs=1, new=1, ragged=False, ctx_lo=1000, ctx_hi=1000, q_heads=64, kv_heads=4,
             dim=128, page=128, dtype="bf16", pages=0),
        # the ordinary batch: 64 requests, trees of 8 tokens, every cached key read
        dict(name="tree_drafts", op="tree", reqs=64, new=8, ragged=False, ctx_lo=1024, ctx_hi=16384, q_heads=64, kv_heads=4,
             dim=128, page=128, dtype="bf16", pages=0),
        # few requests with wide trees of different sizes over long contexts, small pages, 4 query heads a KV head
        dict(name="tree_wide", op="tree", reqs=5, new=61, ragged=True, ctx_lo=20000, ctx_hi=40000, q_heads=32, kv_heads=8,
             dim=128, page=16, dtype="fp16", pages=0),
        # the pages that the indexer chose: 16 per drafted token and index head
        dict(name="tree_pages", op="tree", reqs=64, new=8, ragged=False, ctx_lo=8192, ctx_hi=65536, q_heads=64, kv_heads=4,
             dim=128, page=128, dtype="bf16", pages=16),
        # one request, a chain of drafts with the drafter's probabilities
        dict(name="verify_one", op="verify", reqs=1, new=4, vocab=32000, tree=False, draft=True),
        # the batch of 64 with chains of 8, large vocabulary
        dict(name="verify_chains", op="verify", reqs=64, new=8, vocab=200003, tree=False, draft=True),
        # trees whose siblings were drawn from one draft row: several residuals of one node
        dict(name="verify_trees", op="verify", reqs=48, new=24, vocab=128000, tree=True, draft=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["slots", "rope", "tree", "tree", "verify"])
    if op == "slots":
        reqs = _log_int(rng, 1, 1021)
        tree = rng.random() < 0.5
        hi = _log_int(rng, 1, 64 if tree else min(2048, max(2, 1000000 // reqs)))
        return dict(op=op, reqs=reqs, new_lo=rng.randint(0, hi), new_hi=hi, ctx_lo=0, ctx_hi=_log_int(rng, 100, 172032 if reqs < 400 else 8192),
                    page=rng.choice([16, 32, 64, 128, 256]), tree=tree)
    if op == "rope":
        heads = rng.choice([(64, 4), (32, 8), (40, 10), (8, 8), (16, 1)])
        dim = rng.choice([64, 96, 128])
        return dict(op=op, tokens=_log_int(rng, 1, 30000), q_heads=heads[0], kv_heads=heads[1], dim=dim,
                    rotary=rng.choice([dim, dim // 2, 32]), interleaved=rng.random() < 0.5, scaled=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]) if dim < 128 or heads[0] < 64 else rng.choice(["bf16", "fp16"]),
                    page=rng.choice([16, 64, 128, 256]), pos_hi=_log_int(rng, 1000, 500000))
    if op == "tree":
        heads = rng.choice([(64, 4), (32, 8), (40, 10), (8, 8), (12, 1)])
        if rng.random() < 0.3:  # over chosen pages
            return dict(op=op, reqs=_log_int(rng, 1, 64), new=rng.randint(1, 8), ragged=False, ctx_lo=8192, ctx_hi=_log_int(rng, 9000, 65536),
                        q_heads=64, kv_heads=4, dim=128, page=128, dtype=rng.choice(["bf16", "fp16"]), pages=16)
        reqs = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, 64)
        keys = min(2200000 // heads[1], 270000000 // (new * heads[0]))  # as much to read, as much to compute as tree_drafts
        hi = _log_int(rng, 50, max(60, min(40000, keys // reqs)))
        return dict(op=op, reqs=reqs, new=new, ragged=rng.random() < 0.5, ctx_lo=rng.randint(0, hi), ctx_hi=hi, q_heads=heads[0],
                    kv_heads=heads[1], dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128, 256]),
                    dtype=rng.choice(["bf16", "fp16"]), pages=0)
    tree, draft = rng.random() < 0.4, rng.random() < 0.7
    return dict(op=op, reqs=_log_int(rng, 1, 48), new=rng.randint(1, 24 if tree else 8), vocab=_log_int(rng, 1000, 128000 if tree else 200003),
                tree=tree, draft=draft)


# ---------------------------------------------------------------- what belongs to a case: lengths and trees


def _rng_of(case):
    return random.Random("|".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))


def _parents(r, n):
    """A drafted tree: node 0 is the last certain token; siblings follow one another in order of their numbers."""
    if n <= 1:
        return [-1] * n
    return [-1] + [max(0, i - 1 - int(r.random() * min(i, 4))) for i in range(1, n)]


def _lengths(case):
    r = _rng_of(case)
    reqs = case["reqs"]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(reqs)]
    if case["op"] == "slots":
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(reqs)]
    else:
        new = [r.randint(1, case["new"]) if case["ragged"] else case["new"] for _ in range(reqs)]
    return ctx, new, r


def _ancestors(parents):
    """Bit j of entry i: token j of the same request is i itself or an ancestor of i (as signed 64-bit numbers)."""
    bits = []
    for i, p in enumerate(parents):
        m = (1 << i) | (bits[p] if p >= 0 else 0)
        bits.append(m)
    return [m - (1 << 64) if m >= 1 << 63 else m for m in bits]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _cu(new):
    return np.concatenate([[0], np.cumsum(np.asarray(new, dtype=np.int64))]).astype(np.int64)


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    s = {"slots": _prepare_slots, "rope": _prepare_rope, "tree": _prepare_tree, "verify": _prepare_verify}[case["op"]](case, g)
    s["op"] = case["op"]
    return s


def _prepare_slots(case, g):
    """Requests that own the pages of their contexts (some one more, left from refused drafts) and a list of free blocks."""
    ctx, new, r = _lengths(case)
    p = case["page"]
    need = [-(-(c + n) // p) for c, n in zip(ctx, new)]
    have = [min(nd, -(-c // p) + (1 if r.random() < 0.2 else 0)) for c, nd in zip(ctx, need)]
    width = max(max(need), 1) + 3
    num_blocks = sum(need) + 64
    perm = torch.randperm(num_blocks, device="cuda", generator=g).to(torch.int32)
    table = torch.full((case["reqs"], width), -1, dtype=torch.int32)
    owned = sum(have)
    col = torch.arange(width)[None]
    held = col < torch.tensor(have)[:, None]
    table = table.cuda()
    table[held.cuda()] = perm[:owned]
    tokens = sum(new)
    parents = None
    if case["tree"]:
        parents = _i32([q for n in new for q in _parents(r, n)])
    cap = tokens + 5  # room for a padded batch
    if parents is not None:
        parents = torch.cat([parents, torch.full((5,), -1, dtype=torch.int32, device="cuda")])
    out = dict(cu=torch.empty(case["reqs"] + 1, dtype=torch.int32, device="cuda"),
               seq=torch.empty(case["reqs"], dtype=torch.int32, device="cuda"),
               pages=torch.empty(case["reqs"], dtype=torch.int32, device="cuda"),
               cursor=torch.empty(1, dtype=torch.int32, device="cuda"),
               pos=torch.empty(cap, dtype=torch.int32, device="cuda"), slots=torch.empty(cap, dtype=torch.int64, device="cuda"),
               mask=torch.empty(cap, dtype=torch.int64, device="cuda") if case["tree"] else None)
    return dict(ctx=_i32(ctx), new=_i32(new), have=_i32(have), table=table, free=perm[owned:].contiguous(), cursor=_i32([3]),
                num_blocks=num_blocks, page=p, parents=parents, depth=case.get("new_hi", 0), out=out,
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _inv_freq(case):
    """Rotary frequencies; scaled: high frequencies kept, low ones divided by 8, a ramp between, and the matching magnitude."""
    rd = case["rotary"]
    i = np.arange(0, rd, 2, dtype=np.float64)
    f = 500000.0 ** (-i / rd)
    if not case["scaled"]:
        return f, 1.0
    factor, length = 8.0, 32768.0
    edge = lambda turns: rd * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(500000.0))
    lo, hi = max(0.0, math.floor(edge(32.0))), min(rd - 1.0, math.ceil(edge(1.0)))
    ramp = np.clip((np.arange(rd // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0


def _prepare_rope(case, g):
    """One projection's output with queries, keys and values side by side, and a cache with places in any order."""
    t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    dt = DTYPES[case["dtype"]]
    qkv = torch.randn(t, (hq + 2 * hk) * d, device="cuda", generator=g, dtype=torch.float32).to(dt)
    q = qkv[:, : hq * d].view(t, hq, d)
    k = qkv[:, hq * d : (hq + hk) * d].view(t, hk, d)
    v = qkv[:, (hq + hk) * d :].view(t, hk, d)
    blocks = -(-t // case["page"]) + 7
    cache = torch.randn(2, blocks, case["page"], hk, d, device="cuda", generator=g, dtype=torch.float32).to(dt)
    # tokens of a request lie one after another in a page, pages anywhere
    perm = torch.randperm(blocks, device="cuda", generator=g)
    place = torch.arange(t, device="cuda")
    slots = perm[place // case["page"]] * case["page"] + place % case["page"]
    start = int(torch.randint(0, max(1, case["pos_hi"] - t), (1,), device="cuda", generator=g))
    f, m = _inv_freq(case)
    return dict(q=q, k=k, v=v, k_cache=cache[0], v_cache=cache[1], slots=slots, pos=(start + place).to(torch.int32),
                inv_freq=torch.from_numpy(f).cuda(), mscale=m, interleaved=case["interleaved"],
                q_out=torch.empty(t, hq, d, dtype=dt, device="cuda"))


def _prepare_tree(case, g):
    ctx, new, r = _lengths(case)
    p, hk, d, dt = case["page"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    need = [-(-(c + n) // p) for c, n in zip(ctx, new)]
    blocks, width = sum(need) + 3, max(need)
    cache = torch.empty(2, blocks, p, hk, d, device="cuda", dtype=dt).normal_(generator=g)
    table = torch.full((case["reqs"], width), -1, dtype=torch.int32, device="cuda")
    held = (torch.arange(width)[None] < torch.tensor(need)[:, None]).cuda()
    table[held] = torch.randperm(blocks, device="cuda", generator=g)[: sum(need)].to(torch.int32)
    mask = []
    for n in new:
        mask += _ancestors(_parents(r, n))
    tokens = sum(new)
    q = torch.empty(tokens, case["q_heads"], d, device="cuda", dtype=dt).normal_(generator=g)
    s = dict(q=q, k_cache=cache[0], v_cache=cache[1], table=table, seq=_i32([c + n for c, n in zip(ctx, new)]),
             cu=torch.from_numpy(_cu(new)).to(torch.int32).cuda(), mask=torch.tensor(mask, dtype=torch.int64).cuda(),
             scale=d**-0.5, new=max(new), out=torch.empty_like(q), pages=None,
             lse=torch.empty(tokens, case["q_heads"], dtype=torch.float32, device="cuda"),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["pages"]:
        s["pages"] = _page_lists(case, ctx, new[0], g)
    return s


def _page_lists(case, ctx, n, g):
    """Lists as the indexer gives them: ranked pages below the token's own page, then the own page.  The drafted tokens
    of a request look at much the same pages: of the 15, 12 are those of the first token, 3 are its own."""
    reqs, h, p, per = case["reqs"], case["kv_heads"], case["page"], case["pages"]
    c = torch.tensor(ctx, device="cuda")[:, None, None]
    below = torch.div(c, p, rounding_mode="floor")  # pages below the first token's own one
    rank = torch.rand(reqs, h, -(-case["ctx_hi"] // p) + 1, device="cuda", generator=g)
    rank = rank.masked_fill(torch.arange(rank.shape[-1], device="cuda") >= below, -1.0)
    common, each = per - 4, 3
    best = rank.topk(min(common + each * n, rank.shape[-1]), -1).indices.to(torch.int32)
    lists = torch.empty(reqs, n, h, per, dtype=torch.int32, device="cuda")
    lists[..., :common] = best[:, None, :, :common]
    lists[..., common : common + each] = best[:, :, common:].reshape(reqs, h, n, each).transpose(1, 2)
    own_page = torch.div(c + torch.arange(n, device="cuda")[None, :, None], p, rounding_mode="floor")
    lists[..., -1] = own_page.expand(reqs, n, h).to(torch.int32)
    return lists.reshape(reqs * n, h, per)


def _prepare_verify(case, g):
    """Target rows, draft rows near them, and tokens drawn from the draft rows."""
    r = _rng_of(case)
    reqs, n, v = case["reqs"], case["new"], case["vocab"]
    t = reqs * n
    parents = [_parents(r, n) if case["tree"] else list(range(-1, n - 1)) for _ in range(reqs)]
    logits = torch.randn(t, v, device="cuda", generator=g) * 3.0
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits + 0.8 * torch.randn(t, v, device="cuda", generator=g), -1)
    del logits
    par = torch.tensor(parents, device="cuda")
    rows = (torch.arange(reqs, device="cuda")[:, None] * n + par.clamp(min=0)).reshape(-1)
    # a draw by the largest of logarithm plus Gumbel noise (from the target itself where the drafter has no probabilities)
    src = draft if case["draft"] else target
    noise = torch.empty(v, device="cuda")
    tokens = torch.stack([(src[i].log() - noise.exponential_(generator=g).log()).argmax() for i in rows.tolist()])
    return dict(target=target, draft=draft if case["draft"] else None, tokens=tokens.to(torch.int32),
                parents=par.reshape(-1).to(torch.int32) if case["tree"] else None,
                cu=torch.arange(0, t + 1, n, device="cuda", dtype=torch.int32), new=n,
                accept_u=torch.rand(t, device="cuda", generator=g), sample_u=torch.rand(reqs, device="cuda", generator=g),
                out_tokens=torch.empty(reqs, n, dtype=torch.int32, device="cuda"),
                out_nodes=torch.empty(reqs, n, dtype=torch.int32, device="cuda"),
                accepted=torch.empty(reqs, dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------- one pass


def run(state):
    if own:
        return {"slots": _own_slots, "rope": _own_rope, "tree": _own_tree, "verify": _own_verify}[state["op"]](state)
    return {"slots": _plain_slots, "rope": _plain_rope, "tree": _plain_tree, "verify": _plain_verify}[state["op"]](state)


def _own_slots(s):
    import sparse_attention_indexer_nvfp4_gb300 as idx

    o = s["out"]
    idx.idx_build_slots(s["ctx"], s["new"], s["have"], s["table"], s["free"], s["cursor"], s["num_blocks"], s["page"], o["cu"], o["seq"],
                        o["pages"], o["cursor"], o["pos"], o["slots"], parents=s["parents"], tree_mask=o["mask"], status=s["status"])
    return s["table"], o


def _own_rope(s):
    import sparse_attention_indexer_nvfp4_gb300 as idx

    idx.idx_rope_append(s["q"], s["k"], s["v"], s["pos"], s["inv_freq"], s["q_out"], s["k_cache"], s["v_cache"], s["slots"],
                        mscale=s["mscale"], interleaved=s["interleaved"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_tree(s):
    import sparse_attention_indexer_nvfp4_gb300 as idx

    if "workspace" not in s:  # kept by the program from its first step on
        lists, per = (0, 0) if s["pages"] is None else s["pages"].shape[1:]
        size = idx.idx_tree_attention_workspace_bytes(s["seq"].shape[0], s["q"].shape[0], s["q"].shape[1], s["k_cache"].shape[2],
                                                      s["q"].shape[2], lists, per)
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    idx.idx_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq"], s["cu"], s["out"], s["scale"], tree_mask=s["mask"],
                           pages=s["pages"], lse=s["lse"], workspace=s["workspace"], status=s["status"])
    return s["out"], s["lse"]


def _own_verify(s):
    import sparse_attention_indexer_nvfp4_gb300 as idx

    idx.idx_verify_drafts(s["target"], s["draft"], s["tokens"], s["cu"], s["accept_u"], s["sample_u"], s["out_tokens"], s["out_nodes"],
                          s["accepted"], parents=s["parents"])
    return s["accepted"], s["out_tokens"], s["out_nodes"]


def _plain_slots(s):
    ctx, new, have, table, free, p = (s[k] for k in ("ctx", "new", "have", "table", "free", "page"))
    ctx, new, have = ctx.long(), new.long(), have.long()
    width, cap = table.shape[1], s["out"]["pos"].shape[0]
    need = torch.div(ctx + new + p - 1, p, rounding_mode="floor").clamp(max=width)
    take = (need - have).clamp(min=0)
    first = s["cursor"].long() + take.cumsum(0) - take
    col = torch.arange(width, device="cuda")[None]
    src = first[:, None] + col - have[:, None]
    fresh = torch.where(src < free.shape[0], free[src.clamp(0, free.shape[0] - 1)], -1)
    table = torch.where((col >= have[:, None]) & (col < need[:, None]), fresh, table)
    end = new.cumsum(0)
    tok = torch.arange(cap, device="cuda")
    r = torch.searchsorted(end, tok, right=True)
    live = r < ctx.shape[0]
    r = r.clamp(max=ctx.shape[0] - 1)
    i = tok - (end - new)[r]
    place = ctx[r] + i
    block = table[r, torch.div(place, p, rounding_mode="floor").clamp(max=width - 1)].long()
    slots = torch.where(live & (block >= 0), block * p + place % p, -1)
    depth, mask = i, None
    if s["parents"] is not None:
        # nodes above each token, one level further in each of `depth` steps
        up = torch.where(live, s["parents"].long(), -1)
        base = tok - i
        at, mask, depth = tok, torch.zeros_like(tok), torch.full_like(tok, -1)
        on = live
        for _ in range(s["depth"]):
            mask = mask | torch.where(on, torch.ones_like(tok) << (at - base), 0)
            depth = depth + on
            nxt = torch.where(on, up[at], -1)
            on = nxt >= 0
            at = torch.where(on, base + nxt, at)
        mask = torch.where(live, mask, 0)
    pos = torch.where(live, ctx[r] + depth, 0)
    i32 = lambda x: x.to(torch.int32)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), end])
    return table, dict(cu=i32(cu), seq=i32(ctx + new), pages=i32(torch.maximum(have, need)), cursor=i32(s["cursor"] + take.sum()),
                       pos=i32(pos), slots=slots, mask=mask)


def _plain_rope(s):
    a = s["pos"].double()[:, None] * s["inv_freq"][None]
    cos, sin = (a.cos() * s["mscale"]).float()[:, None], (a.sin() * s["mscale"]).float()[:, None]
    rd = 2 * s["inv_freq"].shape[0]

    def turn(x):
        y = x.float()
        if s["interleaved"]:
            a, b = y[..., 0:rd:2], y[..., 1:rd:2]
            z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., : rd // 2], y[..., rd // 2 : rd]
            z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([z, y[..., rd:]], -1).to(x.dtype)

    page = s["k_cache"].shape[1]
    b, o = torch.div(s["slots"], page, rounding_mode="floor"), s["slots"] % page
    s["k_cache"][b, o] = turn(s["k"])
    s["v_cache"][b, o] = s["v"]
    return turn(s["q"]), s["k_cache"], s["v_cache"]


def _plain_tree(s):
    q, cu, table = s["q"], s["cu"].long(), s["table"].long()
    hq, d = q.shape[1:]
    page, hk = s["k_cache"].shape[1:3]
    seq = s["seq"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(s["new"], device="cuda")
    inside = i[None] < n[:, None]
    tok = (cu[:-1, None] + i[None]).clamp(max=q.shape[0] - 1)
    if s["pages"] is None:
        # [request, key, head, dim], a query's keys those of its request
        k = s["k_cache"][table.clamp(min=0)].flatten(1, 2).float()
        v = s["v_cache"][table.clamp(min=0)].flatten(1, 2).float()
        place = torch.arange(k.shape[1], device="cuda").expand(k.shape[0], -1)
        rows = q[tok].float().view(*tok.shape, hk, hq // hk, d)
        scores = torch.einsum("rihgd,rkhd->rhigk", rows, k) * s["scale"]
        seen = _seen(s["mask"][tok], place[:, None], (seq - n)[:, None, None], n[:, None, None])[:, None, :, None]
        v = torch.where((place < seq[:, None])[..., None, None], v, 0.0)
        o, lse = _softmax_times(scores, seen, v, "rhigk,rkhd->rhigd")
        o, lse = o.permute(0, 2, 1, 3, 4).reshape(*tok.shape, hq, d), lse.permute(0, 2, 1, 3).reshape(*tok.shape, hq)
        return o[inside].to(q.dtype), lse[inside]
    # [token, head, key, dim], a query's keys those of its list
    r = torch.repeat_interleave(torch.arange(n.shape[0], device="cuda"), n)
    lists = s["pages"].long()
    block = table[r[:, None, None], lists.clamp(min=0)]
    head = torch.arange(hk, device="cuda")[None, :, None]
    k = s["k_cache"][block, :, head].flatten(2, 3).float()
    v = s["v_cache"][block, :, head].flatten(2, 3).float()
    place = (lists[..., None] * page + torch.arange(page, device="cuda")).flatten(2)
    scores = torch.einsum("thgd,thkd->thgk", q.float().view(-1, hk, hq // hk, d), k) * s["scale"]
    seen = _seen(s["mask"], place, (seq - n)[r][:, None, None], n[r][:, None, None]) & (lists >= 0).repeat_interleave(page, -1)
    v = torch.where((place < seq[r][:, None, None])[..., None], v, 0.0)
    o, lse = _softmax_times(scores, seen[:, :, None], v, "thgk,thkd->thgd")
    return o.reshape(-1, hq, d).to(q.dtype), lse.reshape(-1, hq)


def _seen(mask, place, ctx, n):
    """Which keys a token sees: every one of the context, and of the drafted ones those of its mask."""
    j = place - ctx
    drafted = (mask[..., None].expand(*mask.shape, place.shape[-1]) if mask.dim() == 2 else mask[:, None, None]) >> j.clamp(0, 63)
    return (j < 0) | ((j < n) & (j < 64) & ((drafted & 1) != 0))


def _softmax_times(scores, seen, v, product):
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = (scores - top).exp()
    mass = e.sum(-1)
    o = torch.einsum(product, e, v) / torch.where(mass == 0, 1.0, mass)[..., None]
    return o, mass.log() + top[..., 0]


def _plain_verify(s):
    """All requests at once, one step for each drafted token: a node's children follow it in order of their numbers, so a
    token is tried exactly when its parent is the node that its request stands at."""
    n = s["new"]
    reqs = s["cu"].shape[0] - 1
    base = s["cu"][:-1].long()
    every = torch.arange(reqs, device="cuda")
    at = torch.zeros(reqs, dtype=torch.int64, device="cuda")
    taken = torch.zeros_like(at)
    mass = torch.ones(reqs, dtype=torch.float64, device="cuda")  # of the residual
    c = torch.zeros_like(mass)
    gone = torch.zeros(reqs, n, dtype=torch.bool, device="cuda")  # siblings refused at this node
    out_tokens = torch.full((reqs, n), -1, dtype=torch.int64, device="cuda")
    out_nodes = out_tokens.clone()
    parents = s["parents"].view(reqs, n).long() if s["parents"] is not None else torch.arange(-1, n - 1, device="cuda").expand(reqs, n)
    tokens = s["tokens"].view(reqs, n).long()
    for i in range(1, n):
        row, x = base + at, tokens[:, i]
        p, u = s["target"][row, x].double(), s["accept_u"][base + i].double()
        tried = parents[:, i] == at
        if s["draft"] is not None:
            q = s["draft"][row, x].double()
            ok = u * q * mass < (p - c * q).clamp(min=0)
        else:
            p = torch.where((gone & (tokens == x[:, None])).any(1), 0.0, p)
            ok = u * mass < p
        ok, no = tried & ok, tried & ~ok
        if s["draft"] is not None:
            hit = no.nonzero()[:, 0]  # what is left of the rows of those that refused
            c[hit] += mass[hit]
            left = (s["target"][row[hit]].double() - c[hit, None] * s["draft"][row[hit]].double()).clamp_(min=0).sum(1)
            mass[hit] = left
        else:
            mass = torch.where(no, mass - p, mass)
        gone[:, i] = no
        gone = gone & ~ok[:, None]
        out_tokens[every, taken] = torch.where(ok, x, out_tokens[every, taken])
        out_nodes[every, taken] = torch.where(ok, i, out_nodes[every, taken])
        taken = taken + ok
        at = torch.where(ok, i, at)
        mass, c = torch.where(ok, 1.0, mass), torch.where(ok, 0.0, c)
    left = s["target"][base + at].double()
    if s["draft"] is not None:
        rest = (left - c[:, None] * s["draft"][base + at].double()).clamp_(min=0)
    else:
        r, i = gone.nonzero(as_tuple=True)
        rest = left.clone()
        rest[r, tokens[r, i]] = 0.0
    left = torch.where(rest.sum(1, keepdim=True) > 0, rest, left)
    left = left.cumsum(1)
    drawn = (left > s["sample_u"].double()[:, None] * left[:, -1:]).to(torch.uint8).argmax(1)
    out_tokens[every, taken] = drawn
    return taken.to(torch.int32), out_tokens.to(torch.int32), out_nodes.to(torch.int32)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "slots":
        ctx, new, _ = _lengths(case)
        fresh = sum(max(0, -(-(c + n) // case["page"]) - (-(-c // case["page"]))) for c, n in zip(ctx, new))
        per_token = 24 if case["tree"] else 12
        return {"bytes": 24 * case["reqs"] + 8 * fresh + per_token * sum(new), "flops": 0}
    if case["op"] == "rope":
        size = 4 if case["dtype"] == "fp32" else 2
        t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        return {"bytes": t * (2 * size * d * (hq + 2 * hk) + 12) + 4 * case["rotary"], "flops": 3 * t * (hq + hk) * case["rotary"]}
    if case["op"] == "tree":
        ctx, new, _ = _lengths(case)
        hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
        io = sum(new) * hq * (4 * d + 4)
        if case["pages"]:
            # a request's tokens share 12 ranked pages and the own page (whose part in use is counted), 3 are each token's own
            keys = sum((12 + 3 * n) * case["page"] + (c + n) % case["page"] for c, n in zip(ctx, new))
            pairs = sum(n * ((case["pages"] - 1) * case["page"] + (c % case["page"])) for c, n in zip(ctx, new))
        else:
            keys = sum(c + n for c, n in zip(ctx, new))
            pairs = sum(n * c for c, n in zip(ctx, new))
        return {"bytes": keys * hk * d * 4 + io, "flops": pairs * hq * d * 4}
    # the row of the target where the walk ends, and that of the drafter, for nearly every walk ends at a refused token
    rows = 2 if case["draft"] and case["new"] > 1 else 1
    return {"bytes": case["reqs"] * case["vocab"] * 4 * rows, "flops": case["reqs"] * case["vocab"] * rows}


# ---------------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"slots": lambda c, s: None, "rope": _exact_rope, "tree": _exact_tree, "verify": _exact_verify}[case["op"]](case, s)


def _exact_rope(case, s):
    """Each pair as a complex number, turned by the angle."""
    w = torch.polar(torch.tensor(s["mscale"], dtype=torch.float64, device="cuda").expand(s["pos"].shape[0], s["inv_freq"].shape[0]).contiguous(),
                    torch.outer(s["pos"].double(), s["inv_freq"]))
    half = s["inv_freq"].shape[0]
    order = torch.arange(2 * half, device="cuda")
    re, im = (order[0::2], order[1::2]) if case["interleaved"] else (order[:half], order[half:])

    def turn(x):
        y = x.double().clone()
        z = torch.complex(y[..., re], y[..., im]) * w[:, None]
        y[..., re], y[..., im] = z.real, z.imag
        return y

    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kc.view(-1, *kc.shape[2:]).index_copy_(0, s["slots"], turn(s["k"]))
    vc.view(-1, *vc.shape[2:]).index_copy_(0, s["slots"], s["v"].double())
    return turn(s["q"]), kc, vc


def _exact_tree(case, s):
    """Request by request and head by head, the keys in blocks, each token's keys by their places."""
    cu, seq, table = s["cu"].tolist(), s["seq"].tolist(), s["table"].tolist()
    page, hk = s["k_cache"].shape[1:3]
    tokens, hq, d = s["q"].shape
    g = hq // hk
    out = torch.zeros(tokens, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((tokens, hq), -math.inf, dtype=torch.float64, device="cuda")
    bits = torch.arange(64, device="cuda")
    anc = (s["mask"][:, None] >> bits[None]) & 1 == 1
    for r in range(len(seq)):
        a, b = cu[r], cu[r + 1]
        n, ctx = b - a, seq[r] - (b - a)
        blocks = torch.tensor(table[r][: -(-seq[r] // page)], device="cuda")
        for h in range(hk):
            kr = s["k_cache"][blocks, :, h].reshape(-1, d)[: seq[r]].double()
            vr = s["v_cache"][blocks, :, h].reshape(-1, d)[: seq[r]].double()
            see = torch.ones(n, seq[r], dtype=torch.bool, device="cuda")
            if case["pages"]:
                ks = torch.arange(seq[r], device="cuda") // page
                see = (ks[None, :, None] == s["pages"][a:b, h][:, None, :]).any(-1)
            see[:, ctx:] &= anc[a:b, :n]
            x = s["q"][a:b, h * g : (h + 1) * g].double().reshape(n * g, d) @ kr.T * s["scale"]
            x = x.view(n, g, -1).masked_fill(~see[:, None], -math.inf)
            lse[a:b, h * g : (h + 1) * g] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1).nan_to_num(0.0)
            out[a:b, h * g : (h + 1) * g] = (p.reshape(n * g, -1) @ vr).view(n, g, d)
    return out, lse


def _exact_verify(case, s):
    """The walk of each request down its tree, a residual row kept and made smaller at each refusal."""
    n = case["new"]
    toks, us = s["tokens"].tolist(), s["accept_u"].tolist()
    par = s["parents"].tolist() if s["parents"] is not None else None
    taken, out_t, out_n = [], [], []
    for r in range(case["reqs"]):
        at, path, going = 0, [], True
        while going:
            rest = s["target"][r * n + at].double()
            whole = 1.0
            going = False
            for i in range(at + 1, n):
                if (par[r * n + i] if par is not None else i - 1) != at:
                    continue
                x, u = toks[r * n + i], us[r * n + i]
                if s["draft"] is not None:
                    q = s["draft"][r * n + at].double()
                    going = u * float(q[x]) < float(rest[x])
                else:
                    going = u * whole < float(rest[x])
                if going:
                    path.append(i)
                    at = i
                    break
                if s["draft"] is not None:  # normalised again after each refusal
                    rest = (rest - q).clamp(min=0)
                    rest = rest / rest.sum()
                else:
                    whole -= float(rest[x])
                    rest = rest.index_fill(0, torch.tensor([x], device="cuda"), 0.0)
        cum = rest.cumsum(0)
        drawn = int((cum > s["sample_u"][r].double() * cum[-1]).to(torch.uint8).argmax())
        taken.append(len(path))
        out_t.append([toks[r * n + i] for i in path] + [drawn] + [-1] * (n - 1 - len(path)))
        out_n.append(path + [-1] * (n - len(path)))
    return _i32(taken), _i32(out_t), _i32(out_n)

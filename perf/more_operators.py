"""What is timed of the operators between the calls of a decoding step with drafted tokens.

Six operators, in the order in which a serving step calls them:

* norm     norms of each head of queries and keys, rotary positions, keys and values appended to the paged cache
* index    the indexer's inputs: E4M3 queries with a scale a head, NVFP4 keys appended to the index-K pages
* probs    probabilities from logits: penalties for repeated tokens, biases, grammar masks, temperature
* settle   after the verification of drafts: rows of the tokens that stand moved together in every cache, lengths, token counts
* fork     a request's pages shared with new requests, the last page copied
* release  pages of finished and shortened requests given back to the free list

`run` computes them in elementary torch operations, or, with `own` true, by the
calls of sparse_attention_indexer_nvfp4_gb300.  Lengths, trees and sharing
belong to a case; values, block ids and tokens come from the seed.
"""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token of one request: the single-token form, all latency
        dict(name="norm_token", op="norm", tokens=1, q_heads=64, kv_heads=4, dim=128, rotary=64, interleaved=False, dtype="bf16", page=128,
             pos_hi=172032),
        # a prompt chunk of odd length
        dict(name="norm_prompt", op="norm", tokens=30011, q_heads=64, kv_heads=4, dim=128, rotary=64, interleaved=False, dtype="bf16", page=128,
             pos_hi=172032),
        # 64 requests with 8 drafted tokens each, four index heads: the inputs of a decode step
        dict(name="index_drafts", op="index", reqs=64, new=8, heads=4, rotary=64, interleaved=False, dtype="bf16", pos_hi=172032, slots=True,
             weighted=False),
        # a prompt chunk of odd length with 64 index heads and weights: the inputs of the prefill chain
        dict(name="index_prompt", op="index", reqs=1, new=8191, heads=64, rotary=64, interleaved=False, dtype="bf16", pos_hi=172032, slots=False,
             weighted=True),
        # one row, as a request without drafts has it
        dict(name="probs_one", op="probs", reqs=1, new=1, vocab=32000, tree=False, dtype="fp32", penalties=True, biases=4, grammar=False),
        # 64 requests with trees of 8 drafted tokens, large odd vocabulary, penalties, some biases, a grammar's mask a row
        dict(name="probs_drafts", op="probs", reqs=64, new=8, vocab=200003, tree=True, dtype="bf16", penalties=True, biases=16, grammar=True),
        # 64 requests with trees of 8, keys and values of one layer and the index-K pages
        dict(name="settle_drafts", op="settle", reqs=64, new=8, planes=2, heads=4, dim=128, page=128, dtype="bf16", index=True, vocab=32000,
             ctx_lo=1, ctx_hi=250),
        # wider trees, keys and values of 48 layers at once
        dict(name="settle_layers", op="settle", reqs=64, new=24, planes=96, heads=4, dim=128, page=128, dtype="bf16", index=True, vocab=128000,
             ctx_lo=1, ctx_hi=120),
        # one request forked into three, one layer
        dict(name="fork_one", op="fork", reqs=1, forks=3, ctx_lo=1000, ctx_hi=1000, width=1347, planes=2, heads=4, dim=128, page=128, dtype="bf16",
             index=True),
        # 64 forks of 16 requests with long contexts, keys and values of 48 layers at once
        dict(name="fork_layers", op="fork", reqs=16, forks=64, ctx_lo=8192, ctx_hi=172032, width=1347, planes=96, heads=4, dim=128, page=128,
             dtype="bf16", index=True),
        # one long request ends
        dict(name="release_one", op="release", reqs=1, group=1, ctx_lo=172032, ctx_hi=172032, page=128),
        # a batch of forked requests, most of which end, small pages
        dict(name="release_batch", op="release", reqs=1021, group=5, ctx_lo=0, ctx_hi=8192, page=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "index", "probs", "probs", "settle", "fork", "release"])
    if op == "norm":
        heads = rng.choice([(64, 4), (32, 8), (40, 10), (8, 8), (16, 1)])
        dim = rng.choice([64, 80, 96, 128])
        wide = dim == 128 and heads[0] == 64
        return dict(op=op, tokens=_log_int(rng, 1, 30000), q_heads=heads[0], kv_heads=heads[1], dim=dim, rotary=rng.choice([dim, dim // 2, 32]),
                    interleaved=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16"] if wide else ["bf16", "fp16", "fp32"]),
                    page=rng.choice([16, 64, 128, 256]), pos_hi=_log_int(rng, 40000, 500000))
    if op == "index":
        slots = rng.random() < 0.5
        return dict(op=op, reqs=_log_int(rng, 1, 64) if slots else rng.randint(1, 7), new=rng.randint(1, 8) if slots else _log_int(rng, 1, 1170),
                    heads=4 if slots else rng.choice([4, 8, 64]), rotary=rng.choice([32, 64, 128]), interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "fp16", "fp32"] if slots else ["bf16", "fp16"]),
                    pos_hi=_log_int(rng, 10000, 500000), slots=slots, weighted=not slots and rng.random() < 0.5)
    if op == "probs":
        tree = rng.random() < 0.5
        reqs, new = _log_int(rng, 1, 64), rng.randint(1, 24 if tree else 8)
        return dict(op=op, reqs=reqs, new=new, vocab=_log_int(rng, 1000, max(1001, min(200003, 60000000 // (reqs * new)))), tree=tree,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), penalties=rng.random() < 0.8, biases=rng.choice([0, 3, 100]), grammar=rng.random() < 0.5)
    if op == "settle":
        heads, dim = rng.choice([(4, 128), (8, 64), (1, 576), (5, 40)])
        return dict(op=op, reqs=_log_int(rng, 1, 64), new=rng.randint(2, 24), planes=_log_int(rng, 1, 96), heads=heads, dim=dim, page=128,
                    dtype=rng.choice(["bf16", "fp32"]) if heads * dim < 300 else "bf16", index=rng.random() < 0.5, vocab=_log_int(rng, 1000, 128000),
                    ctx_lo=0, ctx_hi=rng.randint(1, 120))
    if op == "fork":
        heads, dim = rng.choice([(4, 128), (8, 64), (1, 576), (5, 40)])
        reqs = rng.randint(1, 16)
        return dict(op=op, reqs=reqs, forks=_log_int(rng, 1, 64), ctx_lo=0, ctx_hi=_log_int(rng, 100, 172032), width=1400, planes=_log_int(rng, 1, 80),
                    heads=heads, dim=dim, page=128, dtype="bf16", index=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    reqs = _log_int(rng, 1, 1000)
    return dict(op=op, reqs=reqs, group=rng.choice([1, 2, 5, 16]), ctx_lo=0, ctx_hi=_log_int(rng, 100, min(172032, 8000000 * page // 16 // reqs)), page=page)


# ---------------------------------------------------------------- what belongs to a case: lengths, trees, sharing


def _rng_of(case):
    return random.Random("|".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))


def _parents(r, n):
    """A drafted tree: node 0 is the last certain token; siblings follow one another in order of their numbers."""
    return [-1] + [max(0, i - 1 - int(r.random() * min(i, 4))) for i in range(1, n)]


def _ancestors(parents):
    """Bit j of entry i: token j of the same request is i itself or an ancestor of i (as signed 64-bit numbers)."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((1 << i) | (bits[p] if p >= 0 else 0))
    return [m - (1 << 64) if m >= 1 << 63 else m for m in bits]


def _settled(case):
    """Contexts, and for each request the path of the nodes that stand."""
    r = _rng_of(case)
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["reqs"])]
    paths = []
    for _ in ctx:
        parents, at, path = _parents(r, case["new"]), 0, []
        while r.random() < 0.85:
            below = [i for i, p in enumerate(parents) if p == at]
            if not below:
                break
            at = r.choice(below)
            path.append(at)
        paths.append(path)
    return ctx, paths


def _forked(case):
    r = _rng_of(case)
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["reqs"])]
    return ctx, [r.randrange(case["reqs"]) for _ in range(case["forks"])]


def _shared(case):
    """Contexts, tokens that are kept, and pages at the begin of each request that its group shares."""
    r = _rng_of(case)
    n, g, p = case["reqs"], case["group"], case["page"]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
    keep = []
    for c in ctx:
        x = r.random()
        keep.append(0 if x < 0.6 or n == 1 else r.randint(0, c) if x < 0.8 else c)
    prefix = []
    for i in range(0, n, g):
        members = ctx[i : i + g]
        prefix += [int(min(members) * r.random()) // p if len(members) > 1 else 0] * len(members)
    return ctx, keep, prefix


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    s = {"norm": _prepare_norm, "index": _prepare_index, "probs": _prepare_probs, "settle": _prepare_settle, "fork": _prepare_fork,
         "release": _prepare_release}[case["op"]](case, g)
    s["op"] = case["op"]
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def _inv_freq(rotary):
    return torch.from_numpy(500000.0 ** (-np.arange(0, rotary, 2, dtype=np.float64) / rotary)).cuda()


def _places(tokens, page, g, blocks):
    """Tokens of a request lie one after another in a page, pages anywhere."""
    perm = torch.randperm(blocks, device="cuda", generator=g)
    at = torch.arange(tokens, device="cuda")
    return perm[torch.div(at, page, rounding_mode="floor")] * page + at % page


def _prepare_norm(case, g):
    """One projection's output with queries, keys and values side by side, and a cache with places in any order."""
    t, hq, hk, d, dt = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    qkv = (2.0 * torch.randn(t, (hq + 2 * hk) * d, device="cuda", generator=g)).to(dt)
    blocks = -(-t // case["page"]) + 7
    cache = torch.randn(2, blocks, case["page"], hk, d, device="cuda", generator=g).to(dt)
    start = int(torch.randint(0, case["pos_hi"] - t, (1,), device="cuda", generator=g))
    weights = (1.0 + 0.2 * torch.randn(2, d, device="cuda", generator=g)).to(dt)
    return dict(q=qkv[:, : hq * d].view(t, hq, d), k=qkv[:, hq * d : (hq + hk) * d].view(t, hk, d), v=qkv[:, (hq + hk) * d :].view(t, hk, d),
                q_weight=weights[0], k_weight=weights[1], eps=1e-6, k_cache=cache[0], v_cache=cache[1], slots=_places(t, case["page"], g, blocks),
                pos=(start + torch.arange(t, device="cuda")).to(torch.int32), inv_freq=_inv_freq(case["rotary"]), interleaved=case["interleaved"],
                q_out=torch.empty(t, hq, d, dtype=dt, device="cuda"))


def _prepare_index(case, g):
    """One projection's output with index queries and the index key side by side, and pages of random codes."""
    reqs, n, h, p, dt = case["reqs"], case["new"], case["heads"], 128, DTYPES[case["dtype"]]
    t = reqs * n
    x = (2.0 * torch.randn(t, (h + 1) * 128, device="cuda", generator=g)).to(dt)
    blocks = -(-t // p) + 7
    index_k = torch.randint(0, 256, (blocks, p * 72), device="cuda", generator=g, dtype=torch.uint8)
    index_k[:, 64 * p :] = torch.randint(0x28, 0x50, (blocks, 8 * p), device="cuda", generator=g, dtype=torch.uint8)
    slots = _places(t, p, g, blocks)
    start = torch.randint(0, case["pos_hi"] - n, (reqs, 1), device="cuda", generator=g)
    weights = (1.0 + 0.2 * torch.randn(2, 128, device="cuda", generator=g)).to(dt)
    shape = (reqs, 8, h) if case["slots"] else (t, h)
    pages = -(-t // p)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    return dict(table=torch.div(slots[::p], p, rounding_mode="floor").to(torch.int32)[None], num_pages=zero + pages, first_page=zero,
                read=torch.empty(pages, p, 128, dtype=torch.uint8, device="cuda"), q=x[:, : h * 128].view(t, h, 128), k=x[:, h * 128 :], q_weight=weights[0], k_weight=weights[1], eps=1e-6,
                pos=(start + torch.arange(n, device="cuda")).flatten().to(torch.int32), inv_freq=_inv_freq(case["rotary"]),
                interleaved=case["interleaved"], slots=slots, index_k=index_k.view(blocks, p, 72),
                cu=torch.arange(0, t + 1, n, device="cuda", dtype=torch.int32) if case["slots"] else None, new=n,
                q_out=torch.zeros(*shape, 128, dtype=torch.uint8, device="cuda"), q_scale=torch.zeros(shape, dtype=torch.float32, device="cuda"),
                head_weights=torch.rand(t, h, device="cuda", generator=g) if case["weighted"] else None, scale=128**-0.5)


def _prepare_probs(case, g):
    """Logits, the requests' settings and counts of their tokens, the drafted tokens (likely ones) and their trees."""
    r = _rng_of(case)
    reqs, n, v = case["reqs"], case["new"], case["vocab"]
    t = reqs * n
    logits = torch.randn(t, v, device="cuda", generator=g).mul_(3.0).to(DTYPES[case["dtype"]])
    rand = lambda *shape: torch.rand(*shape, device="cuda", generator=g)
    integers = lambda hi, *shape: torch.randint(0, hi, shape, device="cuda", generator=g)
    temperature = 0.5 + rand(reqs)
    temperature[7::8] = 0.0  # a request that takes the largest
    s = dict(logits=logits, temperature=temperature, cu=torch.arange(0, t + 1, n, device="cuda", dtype=torch.int32), new=n,
             repetition=None, presence=None, frequency=None, counts=None, tokens=None, mask=None, bias_cu=None, bias_tokens=None, bias_values=None,
             allowed=None, probs=torch.empty(t, v, dtype=torch.float32, device="cuda"), lse=torch.empty(t, dtype=torch.float32, device="cuda"))
    if case["penalties"]:
        s["repetition"], s["presence"], s["frequency"] = 1.0 + 0.3 * rand(reqs), rand(reqs), 0.5 * rand(reqs)
        # about 500 tokens of the answer and 2,000 of the prompt in each request
        counts = torch.zeros(reqs, v, dtype=torch.int32, device="cuda")
        counts.scatter_add_(1, (rand(reqs, 500).square() * v).long().clamp_(max=v - 1), torch.ones(reqs, 500, dtype=torch.int32, device="cuda"))
        prompt = torch.zeros(reqs, v, dtype=torch.bool, device="cuda").scatter_(1, integers(v, reqs, 2000), True)
        s["counts"] = torch.where(prompt, counts | -(1 << 31), counts)
        s["tokens"] = (rand(t).square() * v).to(torch.int32).clamp_(max=v - 1)
        if case["tree"]:
            s["mask"] = torch.tensor([m for _ in range(reqs) for m in _ancestors(_parents(r, n))], dtype=torch.int64).cuda()
    if case["biases"]:
        each = min(case["biases"], v)
        s["bias_cu"] = torch.arange(0, reqs * each + 1, each, device="cuda", dtype=torch.int32)
        s["bias_tokens"] = rand(reqs, v).topk(each, 1).indices.flatten().to(torch.int32)
        s["bias_values"] = 4.0 * torch.randn(reqs * each, device="cuda", generator=g)
    if case["grammar"]:
        s["allowed"] = integers(1 << 32, t, -(-v // 32)).to(torch.int32)
    return s


def _caches(case, blocks, g):
    """Keys and values of all layers, [planes, blocks, page, row], and the two parts of the index-K pages."""
    cache = torch.empty(case["planes"], blocks, case["page"], case["heads"], case["dim"], device="cuda", dtype=DTYPES[case["dtype"]]).normal_(generator=g)
    if not case["index"]:
        return [cache]
    index_k = torch.randint(0, 256, (1, blocks, 128 * 72), device="cuda", generator=g, dtype=torch.uint8)
    return [cache, index_k[:, :, : 128 * 64].view(1, blocks, 128, 64), index_k[:, :, 128 * 64 :].view(1, blocks, 128, 8)]


def _prepare_settle(case, g):
    ctx, paths = _settled(case)
    reqs, n, p, v = case["reqs"], case["new"], case["page"], case["vocab"]
    need = [-(-(c + n) // p) for c in ctx]
    blocks = sum(need) + 3
    table = torch.full((reqs, max(need)), -1, dtype=torch.int64)
    table = table.cuda()
    held = (torch.arange(max(need))[None] < torch.tensor(need)[:, None]).cuda()
    table[held] = torch.randperm(blocks, device="cuda", generator=g)[: sum(need)]
    place = _i32(ctx).long()[:, None] + torch.arange(n, device="cuda")
    slots = table.gather(1, torch.div(place, p, rounding_mode="floor")) * p + place % p
    nodes = torch.full((reqs, n), -1, dtype=torch.int32)
    for r, path in enumerate(paths):
        nodes[r, : len(path)] = torch.tensor(path, dtype=torch.int32)
    accepted = _i32([len(path) for path in paths])
    tokens = torch.randint(0, v, (reqs, n), device="cuda", generator=g, dtype=torch.int32)
    tokens = torch.where(torch.arange(n, device="cuda") <= accepted[:, None], tokens, -1)
    return dict(caches=_caches(case, blocks, g), slots=slots.flatten(), cu=torch.arange(0, reqs * n + 1, n, device="cuda", dtype=torch.int32),
                out_tokens=tokens, out_nodes=nodes.cuda(), accepted=accepted, ctx=_i32(ctx), ctx_out=torch.empty(reqs, dtype=torch.int32, device="cuda"),
                counts=torch.randint(0, 9, (reqs, v), device="cuda", generator=g, dtype=torch.int32))


def _prepare_fork(case, g):
    """Requests with their pages in the first rows of the tables, rows for their forks after them."""
    ctx, parents = _forked(case)
    reqs, forks, p = case["reqs"], case["forks"], case["page"]
    need = [-(-c // p) for c in ctx]
    # a block table of long contexts over caches of some hundred pages: pages but the last of a request lie anywhere in them
    blocks = reqs + forks + 200
    perm = torch.randperm(blocks, device="cuda", generator=g).to(torch.int32)
    table = torch.randint(0, 200, (reqs + forks, case["width"]), device="cuda", generator=g, dtype=torch.int32)
    last = _i32([max(0, x - 1) for x in need]).long()
    table = perm[table.long()]
    table[torch.arange(reqs, device="cuda"), last] = perm[200 : 200 + reqs]
    total = reqs + forks
    return dict(caches=_caches(case, blocks, g), parents=_i32(parents), children=_i32(list(range(reqs, total))),
                ctx=_i32(ctx + [0] * forks), owned=_i32(need + [0] * forks), table=table, refs=torch.zeros(blocks, dtype=torch.int32, device="cuda"),
                free=perm[200 + reqs :].contiguous(), cursor=_i32([0]), cursor_out=_i32([0]), page=p)


def _prepare_release(case, g):
    ctx, keep, prefix = _shared(case)
    n, group, p = case["reqs"], case["group"], case["page"]
    need = np.array([-(-c // p) for c in ctx])
    first = np.array([i // group * group for i in range(n)])
    blocks_most = int(need.sum()) + 64
    perm = torch.randperm(blocks_most, device="cuda", generator=g).to(torch.int32)
    width = max(1, int(need.max()))
    col = torch.arange(width, device="cuda")
    have, lead, pre = (torch.tensor(x, device="cuda") for x in (need, first, np.array(prefix)))
    begin = have.cumsum(0) - have
    # a page of the shared begin is that of the group's first request
    src = torch.where(col[None] < pre[:, None], begin[lead][:, None], begin[:, None]) + col
    table = torch.where(col[None] < have[:, None], perm[src.clamp(max=blocks_most - 1)], -1)
    held = torch.bincount(table[table >= 0].long(), minlength=blocks_most)
    used = int(have.sum())
    free = torch.cat([table[table >= 0].unique(), perm[used:]])  # taken ones (their entries are to be written over), then free ones
    return dict(keep=_i32(keep), owned=_i32(need.tolist()), table=table.contiguous(), refs=(held - 1).clamp(min=0).to(torch.int32),
                free=free.contiguous(), cursor=_i32([free.shape[0] - 64]), cursor_out=_i32([0]), pages_out=torch.empty(n, dtype=torch.int32, device="cuda"),
                page=p)


# ---------------------------------------------------------------- one pass


def run(state):
    if own:
        return {"norm": _own_norm, "index": _own_index, "probs": _own_probs, "settle": _own_settle, "fork": _own_fork,
                "release": _own_release}[state["op"]](state)
    return {"norm": _plain_norm, "index": _plain_index, "probs": _plain_probs, "settle": _plain_settle, "fork": _plain_fork,
            "release": _plain_release}[state["op"]](state)


def _own_norm(s):
    import sparse_attention_indexer_nvfp4_gb300 as idx

    idx.idx_norm_rope_append(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["eps"], s["pos"], s["inv_freq"], s["q_out"], s["k_cache"],
                             s["v_cache"], slots=s["slots"], interleaved=s["interleaved"], status=s["status"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_index(s):
    import sparse_attention_indexer_nvfp4_gb300 as idx

    idx.idx_index_append(s["q"], s["k"], s["q_weight"], s["k_weight"], s["eps"], s["pos"], s["inv_freq"], s["q_out"], s["q_scale"], s["index_k"],
                         slots=s["slots"], cu_tokens=s["cu"], head_weights=s["head_weights"], scale=s["scale"], interleaved=s["interleaved"],
                         status=s["status"])
    # the keys' values, as the indexer reads them
    idx.idx_dequant_nvfp4_pages(s["index_k"], s["table"], s["num_pages"], s["first_page"], s["read"].shape[0], s["read"], s["status"])
    return s["q_out"].view(torch.float8_e4m3fn), s["q_scale"], s["read"].view(torch.float8_e4m3fn)


def _own_probs(s):
    import sparse_attention_indexer_nvfp4_gb300 as idx

    idx.idx_logit_probs(s["logits"], s["probs"], s["cu"], temperature=s["temperature"], repetition=s["repetition"], presence=s["presence"],
                        frequency=s["frequency"], counts=s["counts"], tokens=s["tokens"], tree_mask=s["mask"], bias_cu=s["bias_cu"],
                        bias_tokens=s["bias_tokens"], bias_values=s["bias_values"], allowed=s["allowed"], lse=s["lse"], status=s["status"])
    return s["probs"], s["lse"]


def _own_settle(s):
    import sparse_attention_indexer_nvfp4_gb300 as idx

    idx.idx_settle_drafts(s["caches"], s["slots"], s["cu"], s["out_tokens"], s["out_nodes"], s["accepted"], s["ctx"], s["ctx_out"], counts=s["counts"],
                          status=s["status"])
    return s["caches"], s["ctx_out"], s["counts"]


def _own_fork(s):
    import sparse_attention_indexer_nvfp4_gb300 as idx

    idx.idx_fork_pages(s["caches"], s["parents"], s["children"], s["ctx"], s["owned"], s["table"], s["refs"], s["free"], s["cursor"], s["cursor_out"],
                       status=s["status"])
    return s["caches"], s["ctx"], s["owned"], s["table"], s["refs"], s["cursor_out"]


def _own_release(s):
    import sparse_attention_indexer_nvfp4_gb300 as idx

    idx.idx_release_pages(s["keep"], s["owned"], s["table"], s["refs"], s["free"], s["cursor"], s["cursor_out"], s["pages_out"], s["page"],
                          status=s["status"])
    return s["refs"], s["free"], s["cursor_out"], s["pages_out"]


def _turned(y, pos, inv_freq, interleaved):
    """The first elements of each head turned, in y's type; angles in 64 bits."""
    a = pos.double()[:, None] * inv_freq[None]
    a = a.view(a.shape[0], *([1] * (y.dim() - 2)), a.shape[1])
    cos, sin = a.cos().to(y.dtype), a.sin().to(y.dtype)
    rd = 2 * inv_freq.shape[0]
    if interleaved:
        one, two = y[..., 0:rd:2], y[..., 1:rd:2]
        z = torch.stack([one * cos - two * sin, two * cos + one * sin], -1).flatten(-2)
    else:
        one, two = y[..., : rd // 2], y[..., rd // 2 : rd]
        z = torch.cat([one * cos - two * sin, two * cos + one * sin], -1)
    return torch.cat([z, y[..., rd:]], -1)


def _plain_norm(s):
    page = s["k_cache"].shape[1]
    b, o = torch.div(s["slots"], page, rounding_mode="floor"), s["slots"] % page
    normed = lambda x, w: x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + s["eps"]) * w.float()
    turn = lambda x, w: _turned(normed(x, w), s["pos"], s["inv_freq"], s["interleaved"]).to(x.dtype)
    s["k_cache"][b, o] = turn(s["k"], s["k_weight"])
    s["v_cache"][b, o] = s["v"]
    return turn(s["q"], s["q_weight"]), s["k_cache"], s["v_cache"]


def _to_e4m3(x):
    """To the nearest E4M3 value, halves to even, in 64 bits."""
    a = x.abs()
    e = torch.frexp(a)[1].long().clamp(min=-5) - 1
    step = ((e - 3 + 1023) << 52).view(torch.float64)  # 2^(e - 3) by its bits
    return (torch.round(a / step) * step).clamp(max=448.0).copysign(x)


def _plain_index(s):
    """In 64 bits: values lie next to borders of the codes, and on them (the quotient of two elements that are not turned)."""
    turn = lambda x, w: _turned(x.double() * w.double(), s["pos"], s["inv_freq"], s["interleaved"])
    rms = lambda x: torch.rsqrt(x.double().square().mean(-1) + s["eps"])
    u = turn(s["q"], s["q_weight"])  # without the norm, which an element's share of the largest does not need
    top = u.abs().amax(-1, keepdim=True)
    codes = _to_e4m3(torch.where(top > 0, 448.0 * u / top, 0.0)).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = top[..., 0] * rms(s["q"]) / 448.0 * s["scale"]
    if s["head_weights"] is not None:
        scale = scale * s["head_weights"]
    if s["cu"] is not None:  # the trailing slots of each request
        s["q_out"][:, 8 - s["new"] :] = codes.view(-1, s["new"], *codes.shape[1:])
        s["q_scale"][:, 8 - s["new"] :] = scale.float().view(-1, s["new"], scale.shape[1])
    else:
        s["q_out"].copy_(codes)
        s["q_scale"].copy_(scale)
    y = (turn(s["k"], s["k_weight"]) * rms(s["k"])[:, None]).view(-1, 8, 16)
    scale = _to_e4m3(y.abs().amax(-1) / 6.0)
    z = torch.where(scale[..., None] > 0, y / scale[..., None], 0.0)
    a = z.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    code = (2.0 * a - (a - 2.0).clamp(min=0.0) - 0.5 * (a - 4.0).clamp(min=0.0)).to(torch.uint8) + 8 * torch.signbit(z).to(torch.uint8)
    code = code.view(-1, 64, 2)
    b, o = torch.div(s["slots"], 128, rounding_mode="floor"), s["slots"] % 128
    pages = s["index_k"].flatten(1)
    pages[:, : 64 * 128].view(-1, 128, 64)[b, o] = code[..., 0] + 16 * code[..., 1]
    pages[:, 64 * 128 :].view(-1, 128, 8)[b, o] = scale.to(torch.float8_e4m3fn).view(torch.uint8)
    # the pages' values, as the indexer reads them: code times scale, to the nearest E4M3 value
    here = pages[s["table"][0].long()]
    code = here[:, : 64 * 128].view(-1, 128, 64, 1)
    code = torch.cat([code & 15, code >> 4], -1).flatten(2)
    a = (code & 7).double()
    a = a * 0.5 + (a - 4.0).clamp(min=0.0) * 0.5 + (a - 6.0).clamp(min=0.0)
    value = torch.where(code > 7, -a, a) * here[:, 64 * 128 :].view(-1, 128, 8).view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    return s["q_out"].view(torch.float8_e4m3fn), s["q_scale"], _to_e4m3(value).to(torch.float8_e4m3fn)


def _plain_probs(s):
    reqs, n = s["cu"].shape[0] - 1, s["new"]
    x = s["logits"].float()
    t, v = x.shape
    r = torch.arange(reqs, device="cuda").repeat_interleave(n)
    i = torch.arange(n, device="cuda")
    per_row = lambda p: p[r][:, None]
    if s["counts"] is not None:
        c = s["counts"][r]
        prompt = c < 0
        c &= 0x7FFFFFFF
        # the drafted tokens on each node's path, node 0's left out: it is counted already
        path = (s["mask"][:, None] >> i) & 1 if s["mask"] is not None else (i[None] <= i[:, None]).repeat(reqs, 1)
        c.scatter_add_(1, s["tokens"].view(reqs, n)[r].long(), (path * (i > 0)).to(torch.int32))
        rep = per_row(s["repetition"])
        x = torch.where(prompt | (c > 0), torch.where(x > 0, x / rep, x * rep), x)
        x = torch.where(c > 0, x - (per_row(s["frequency"]) * c + per_row(s["presence"])), x)
    if s["bias_cu"] is not None:
        x.scatter_add_(1, s["bias_tokens"].view(reqs, -1)[r].long(), s["bias_values"].view(reqs, -1)[r])
    if s["allowed"] is not None:
        at = torch.arange(v, device="cuda")
        x = x.masked_fill((s["allowed"][:, at >> 5] >> (at & 31)) & 1 == 0, -math.inf)
    heat = per_row(s["temperature"])
    top = x.amax(1, keepdim=True)
    first = torch.where(x == top, torch.arange(v, dtype=torch.int32, device="cuda"), v).amin(1, keepdim=True)
    best = top > -math.inf
    one = torch.zeros_like(x).scatter_(1, first.clamp(max=v - 1).long(), best.float())
    x = x / torch.where(heat > 0, heat, 1.0)
    peak = torch.where(best, x.amax(1, keepdim=True), 0.0)
    e = (x - peak).exp()
    mass = e.sum(1, keepdim=True)
    p = torch.where(heat > 0, e / torch.where(best, mass, 1.0), one)
    return p, torch.where(heat > 0, mass.log() + peak, top)[:, 0]


def _plain_settle(s):
    reqs, n = s["out_nodes"].shape
    i = torch.arange(n, device="cuda")
    first = s["cu"][:-1].long()[:, None]
    stands = i[None] < s["accepted"][:, None]
    src = s["slots"][(first + s["out_nodes"].clamp(min=0))[stands]]
    dst = s["slots"][(first + 1 + i).clamp(max=s["slots"].shape[0] - 1)[stands]]
    for cache in s["caches"]:
        page = cache.shape[2]
        cache[:, torch.div(dst, page, rounding_mode="floor"), dst % page] = cache[:, torch.div(src, page, rounding_mode="floor"), src % page]
    counted = i[None] <= s["accepted"][:, None]
    s["counts"].scatter_add_(1, s["out_tokens"].clamp(min=0).long(), counted.to(torch.int32))
    return s["caches"], s["ctx"] + 1 + s["accepted"], s["counts"]


def _plain_fork(s):
    page, table = s["page"], s["table"]
    par, child = s["parents"].long(), s["children"].long()
    ctx = s["ctx"][par]
    full, rest = torch.div(ctx, page, rounding_mode="floor"), ctx % page
    part = rest > 0
    taken = s["cursor"] + part.cumsum(0) - part.long()
    block = s["free"][taken.clamp(max=s["free"].shape[0] - 1)]
    col = torch.arange(table.shape[1], device="cuda")[None]
    rows, shared = table[par], col < full[:, None]
    s["refs"].scatter_add_(0, torch.where(shared, rows, 0).flatten().long(), shared.flatten().to(torch.int32))
    table[child] = torch.where(shared, rows, torch.where((col == full[:, None]) & part[:, None], block[:, None], table[child]))
    # the last page's tokens
    fork, tok = (torch.arange(page, device="cuda")[None] < rest[:, None]).nonzero(as_tuple=True)
    src, dst = rows.gather(1, full[:, None].clamp(max=table.shape[1] - 1).long())[fork, 0].long(), block[fork].long()
    for cache in s["caches"]:
        cache[:, dst, tok] = cache[:, src, tok]
    s["ctx"][child] = ctx
    s["owned"][child] = full + part.to(torch.int32)
    return s["caches"], s["ctx"], s["owned"], table, s["refs"], s["cursor"] + part.sum().to(torch.int32)


def _plain_release(s):
    kept = torch.minimum(torch.div(s["keep"] + s["page"] - 1, s["page"], rounding_mode="floor"), s["owned"])
    col = torch.arange(s["table"].shape[1], device="cuda")[None]
    gone = (col >= kept[:, None]) & (col < s["owned"][:, None])
    times = torch.zeros_like(s["refs"]).scatter_add_(0, s["table"].clamp(min=0).flatten().long(), gone.flatten().to(torch.int32))
    left = s["refs"] - times
    ids = ((times > 0) & (left < 0)).nonzero()[:, 0]
    begin = s["cursor"] - ids.shape[0]
    s["free"][begin + torch.arange(ids.shape[0], device="cuda")] = ids.to(torch.int32)
    s["refs"].copy_(left.clamp(min=0))
    return s["refs"], s["free"], begin.to(torch.int32), kept


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op, size = case["op"], {"bf16": 2, "fp16": 2, "fp32": 4}.get(case.get("dtype"), 4)
    if op == "norm":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        return {"bytes": t * (2 * size * d * (hq + 2 * hk) + 12) + 4 * case["rotary"], "flops": t * (hq + hk) * (4 * d + 3 * case["rotary"])}
    if op == "index":
        t, h = case["reqs"] * case["new"], case["heads"]
        # rows read; codes, scales and key rows written; the pages' values read and written
        return {"bytes": t * ((h + 1) * 128 * size + h * (132 + (4 if case["weighted"] else 0)) + 72 + 12 + 72 + 128), "flops": t * (h + 1) * 128 * 10}
    if op == "probs":
        t, v = case["reqs"] * case["new"], case["vocab"]
        per = size + 4 + (0.125 if case["grammar"] else 0)
        return {"bytes": int(t * v * per) + (4 * case["reqs"] * v if case["penalties"] else 0), "flops": 6 * t * v}
    if op == "settle":
        _, paths = _settled(case)
        moved = sum(1 for path in paths for i, node in enumerate(path) if node != i + 1)
        row = case["planes"] * case["heads"] * case["dim"] * size + (72 if case["index"] else 0)
        return {"bytes": 2 * moved * row + 20 * sum(len(p) + 1 for p in paths) + 8 * case["reqs"], "flops": 0}
    if op == "fork":
        ctx, parents = _forked(case)
        row = case["planes"] * case["heads"] * case["dim"] * size + (72 if case["index"] else 0)
        return {"bytes": sum(16 * (ctx[p] // case["page"]) + 2 * (ctx[p] % case["page"]) * row + 16 for p in parents), "flops": 0}
    ctx, keep, _ = _shared(case)
    gone = sum(-(-c // case["page"]) - -(-k // case["page"]) for c, k in zip(ctx, keep))
    return {"bytes": 16 * gone + 16 * case["reqs"], "flops": 0}


# ---------------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    if case["op"] not in ("norm", "index", "probs"):
        return None  # nothing is computed: rows, ids and counts, which have to be equal
    s = prepare(case, seed)
    with torch.no_grad():
        return {"norm": _exact_norm, "index": _exact_index, "probs": _exact_probs}[case["op"]](s)


def _exact_root(s, x):
    return (x.double().pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt()


def _exact_turn(s, x):
    """Each pair as a complex number turned by its angle."""
    rd = 2 * s["inv_freq"].shape[0]
    a = torch.outer(s["pos"].double(), s["inv_freq"])
    turn = torch.polar(torch.ones_like(a), a)
    turn = turn.reshape(turn.shape[0], *([1] * (x.dim() - 2)), rd // 2)
    head = x[..., :rd]
    if s["interleaved"]:
        z = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (rd // 2, 2)).contiguous()) * turn).flatten(-2)
    else:
        z = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (2, rd // 2)).transpose(-1, -2).contiguous()) * turn).transpose(-1, -2).flatten(-2)
    return torch.cat([z, x[..., rd:]], -1)


def _exact_norm(s):
    rows = lambda x, w: _exact_turn(s, x.double() * w.double() / _exact_root(s, x))
    caches = []
    for cache, new in ((s["k_cache"], rows(s["k"], s["k_weight"])), (s["v_cache"], s["v"].double())):
        flat = cache.double().flatten(0, 1)
        flat[s["slots"]] = new
        caches.append(flat.view(cache.shape))
    return rows(s["q"], s["q_weight"]), *caches


def _nearest(x, values):
    """Indices of the nearest of the ascending values (from 0 on; halves to the even index), and the values with x's sign."""
    a = x.abs().contiguous()
    middle = (values[1:] + values[:-1]) / 2
    low, high = torch.searchsorted(middle, a), torch.searchsorted(middle, a, right=True)
    at = torch.where(low == high, low, low + low % 2)
    return at, torch.where(x < 0, -values[at], values[at])


def _exact_index(s):
    bytes_ = torch.arange(127, dtype=torch.uint8, device="cuda")
    e4m3 = bytes_.view(torch.float8_e4m3fn).double()
    e2m1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    y = _exact_turn(s, s["q"].double() * s["q_weight"].double())
    top = y.abs().amax(-1, keepdim=True)
    q = _nearest(y * 448.0 / top, e4m3)[1]
    scale = (top / _exact_root(s, s["q"]))[..., 0] * s["scale"] / 448.0 * (1.0 if s["head_weights"] is None else s["head_weights"].double())
    q_out, q_scale = s["q_out"].view(torch.float8_e4m3fn).double(), s["q_scale"].double()
    if s["cu"] is None:
        q_out, q_scale = q, scale
    else:
        for i in range(s["new"]):
            q_out[:, 8 - s["new"] + i], q_scale[:, 8 - s["new"] + i] = q[i :: s["new"]], scale[i :: s["new"]]
    # the pages as they were, with the new rows in their places
    pages = s["index_k"].flatten(1)[s["table"][0].long()]
    old = pages[:, : 64 * 128].view(-1, 128, 64)
    old = torch.stack([old & 15, old >> 4], -1).flatten(2).long()
    old_scale = pages[:, 64 * 128 :].view(-1, 128, 8).view(torch.float8_e4m3fn).double()
    code = torch.where(old > 7, -e2m1[old % 8], e2m1[old % 8])
    y = (_exact_turn(s, s["k"].double() * s["k_weight"].double()) / _exact_root(s, s["k"])).view(-1, 8, 16)
    k_scale = _nearest(y.abs().amax(-1) / 6.0, e4m3)[1]
    k = _nearest(y / k_scale[..., None], e2m1)[1]
    n = k.shape[0]
    code.view(-1, 128)[:n], old_scale.view(-1, 8)[:n] = k.view(-1, 128), k_scale
    return q_out, q_scale, _nearest(code * old_scale.repeat_interleave(16, -1), e4m3)[1]


def _exact_probs(s):
    n, v = s["new"], s["logits"].shape[1]
    probs, lses = [], []
    for r in range(s["cu"].shape[0] - 1):
        rows = slice(r * n, r * n + n)
        x = s["logits"][rows].double()
        if s["counts"] is not None:
            known = s["counts"][r].long()
            for i in range(n):
                on = [j for j in range(1, n) if (j <= i if s["mask"] is None else int(s["mask"][r * n + i]) >> j & 1)]
                drafted = s["tokens"][rows].long()[on]
                c = (known & 0x7FFFFFFF) + torch.bincount(drafted, minlength=v)
                seen = (known < 0) | (c > 0)
                factor = torch.where(x[i] > 0, 1.0 / s["repetition"][r].double(), s["repetition"][r].double())
                x[i] *= torch.where(seen, factor, 1.0)
                x[i] -= torch.where(c > 0, s["frequency"][r].double() * c + s["presence"][r].double(), 0.0)
        if s["bias_cu"] is not None:
            mine = slice(int(s["bias_cu"][r]), int(s["bias_cu"][r + 1]))
            x[:, s["bias_tokens"][mine].long()] += s["bias_values"][mine].double()
        if s["allowed"] is not None:
            bits = (s["allowed"][rows].long()[:, :, None] >> torch.arange(32, device="cuda")) & 1
            x = torch.where(bits.flatten(1)[:, :v] > 0, x, -math.inf)
        if float(s["temperature"][r]) > 0:
            x = x / s["temperature"][r].double()
            lses.append(torch.logsumexp(x, 1))
            probs.append((x - lses[-1][:, None]).exp())
        else:
            lses.append(x.max(1).values)
            probs.append(torch.stack([torch.zeros_like(row).index_fill_(0, (row == row.max()).nonzero()[0], 1.0) for row in x]))
    return torch.cat(probs), torch.cat(lses)

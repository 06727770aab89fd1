"""Requests served with drafted tokens, forked on their way and released at the end.

A step of `Server` runs, with no host synchronisation,

    idx_build_slots       pages taken from the free list; slots, positions, masks
    idx_norm_rope_append  norms of each head of q and k, both turned; k and v into the paged cache
    idx_index_append      the indexer's queries (E4M3), and its keys into the index-K pages (NVFP4)
    idx_decode_step       the 16 pages that each drafted token looks at
    idx_tree_attention    attention over those pages
    idx_logit_probs       the target's probabilities: penalties for tokens that a request has already, a grammar's mask
    idx_verify_drafts     which drafted tokens stand, and the token after them
    idx_settle_drafts     rows of those that stand moved together in all caches, contexts and token counts

so it can be captured into a CUDA graph.  Between steps idx_fork_pages lets new
requests share the pages of old ones, and idx_release_pages gives pages back.
Where a model would form q, k, v, the index rows and the logits, this example
draws them at random.

    python examples/serve_steps.py [--reqs 48] [--forks 16] [--context 8000] [--steps 20]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_nvfp4_gb300 as idx  # noqa: E402

PAGE, DRAFTS, LISTS, PICKED = 128, 8, 4, 16  # the decode step's geometry
# node 0 is the last certain token; three children, two of which go on
PARENTS = [-1, 0, 0, 0, 1, 1, 2, 4]


class Server:
    """Caches, tables and buffers of up to `rows` requests, the first `active` of which are served."""

    def __init__(self, rows, max_len, q_heads=64, kv_heads=4, dim=128, vocab=32000, dtype=torch.bfloat16, device="cuda", seed=0):
        self.rows, self.active, self.vocab, self.scale = rows, 0, vocab, dim**-0.5
        self.gen = torch.Generator(device=device)
        self.gen.manual_seed(seed)
        tokens, width = rows * DRAFTS, -(-max_len // PAGE)
        blocks = rows * width
        i32 = dict(dtype=torch.int32, device=device)
        new = lambda *shape, **kind: torch.empty(shape, device=device, **kind)
        f32 = lambda *shape: new(*shape, dtype=torch.float32)

        # lengths, tables, the free list and the pages' further holders
        self.ctx, self.new, self.keep = torch.zeros(rows, **i32), torch.full((rows,), DRAFTS, **i32), torch.zeros(rows, **i32)
        self.owned, self.pages_out = torch.zeros(rows, **i32), torch.zeros(rows, **i32)
        self.cursor, self.cursor_out = torch.zeros(1, **i32), torch.zeros(1, **i32)
        self.table = torch.full((rows, width), -1, **i32)
        self.free = torch.randperm(blocks, device=device, generator=self.gen).to(torch.int32)
        self.refs, self.blocks = torch.zeros(blocks, **i32), blocks
        self.parents = torch.tensor(PARENTS * rows, **i32)
        self.cu, self.seq = new(rows + 1, dtype=torch.int32), new(rows, dtype=torch.int32)
        self.positions, self.slots = new(tokens, dtype=torch.int32), new(tokens, dtype=torch.int64)
        self.mask = new(tokens, dtype=torch.int64)

        # caches: keys and values [2, blocks, page, heads, dim], index-K pages
        self.cache = torch.randn(2, blocks, PAGE, kv_heads, dim, device=device, generator=self.gen, dtype=torch.float32).to(dtype)
        self.index_k = torch.randint(0, 256, (blocks, PAGE, 72), device=device, generator=self.gen, dtype=torch.uint8)
        self.index_k.view(blocks, -1)[:, 64 * PAGE :] = 0x38  # block scales of 1
        self.caches = [self.cache, *idx.index_caches(self.index_k)]

        # a step's inputs and outputs
        freq, self.mscale = idx.idx_rope_frequencies(64, 500000.0)
        self.freq, self.eps = freq.to(device), 1e-6
        weight = lambda n: (1.0 + 0.1 * torch.randn(n, device=device, generator=self.gen)).to(dtype)
        self.q_weight, self.k_weight, self.iq_weight, self.ik_weight = weight(dim), weight(dim), weight(128), weight(128)
        self.qkv = new(tokens, q_heads + 2 * kv_heads, dim, dtype=dtype)
        self.q, self.k, self.v = self.qkv.split([q_heads, kv_heads, kv_heads], dim=1)
        self.index_rows = new(tokens, LISTS + 1, 128, dtype=dtype)
        self.q_turned, self.out = new(tokens, q_heads, dim, dtype=dtype), new(tokens, q_heads, dim, dtype=dtype)
        self.index_q, self.index_scale = new(rows, DRAFTS, LISTS, 128, dtype=torch.uint8), f32(rows, DRAFTS, LISTS)
        self.scores, self.pages = f32(rows, DRAFTS * LISTS, width), new(rows, DRAFTS, LISTS, PICKED, dtype=torch.int32)
        self.logits, self.target, self.draft = new(tokens, vocab, dtype=dtype), f32(tokens, vocab), f32(tokens, vocab)
        self.drafted = new(tokens, dtype=torch.int32)
        self.temperature, self.repetition = torch.full((rows,), 0.8, device=device), torch.full((rows,), 1.1, device=device)
        self.presence, self.frequency = torch.full((rows,), 0.2, device=device), torch.full((rows,), 0.1, device=device)
        self.counts = torch.zeros(rows, vocab, **i32)
        self.allowed = torch.full((tokens, (vocab + 31) // 32), -1, **i32)
        self.accept_u, self.sample_u = f32(tokens), f32(rows)
        self.out_tokens, self.out_nodes = new(rows, DRAFTS, dtype=torch.int32), new(rows, DRAFTS, dtype=torch.int32)
        self.accepted = new(rows, dtype=torch.int32)
        self.status = torch.zeros(1, **i32)
        bytes_of = lambda n: new(max(n, 8), dtype=torch.uint8)
        self.select_ws = bytes_of(idx.idx_decode_workspace_bytes(rows, DRAFTS, width))
        self.attention_ws = bytes_of(idx.idx_tree_attention_workspace_bytes(rows, tokens, q_heads, kv_heads, dim, LISTS, PICKED))

    def admit(self, reqs, context):
        """Requests with random prompts; their pages are taken from the free list in the first step."""
        self.active = reqs
        self.ctx[:reqs] = context
        prompt = torch.randint(0, self.vocab, (reqs, 200), device=self.counts.device, generator=self.gen)
        self.counts[:reqs].scatter_(1, prompt, -(2**31))

    def draw(self):
        """What the model, the drafter and the grammar would have formed."""
        g, n, t = self.gen, self.active, self.active * DRAFTS
        self.qkv[:t].normal_(generator=g)
        self.index_rows[:t].normal_(generator=g)
        logits = 3.0 * torch.randn(t, self.vocab, device=self.logits.device, generator=g)
        self.logits[:t] = logits
        idx.idx_logit_probs(logits.add_(0.3 * torch.randn(logits.shape, device=logits.device, generator=g)), self.draft[:t], self.first(t),
                            temperature=self.temperature[:n], status=self.status)
        # a node's token was drawn from its parent's row
        rows = (torch.arange(n, device=logits.device)[:, None] * DRAFTS + torch.tensor(PARENTS, device=logits.device).clamp(min=0)).flatten()
        own = torch.multinomial(self.draft[:t], DRAFTS, replacement=True, generator=g)
        self.drafted[:t] = own[rows, torch.arange(DRAFTS, device=logits.device).repeat(n)]
        self.allowed[:t] = torch.randint(-(2**31), 2**31, self.allowed[:t].shape, device=logits.device, generator=g) | 0x55555555
        self.accept_u[:t].uniform_(generator=g)
        self.sample_u[:n].uniform_(generator=g)

    def first(self, t):
        return torch.arange(0, t + 1, DRAFTS, dtype=torch.int32, device=self.cu.device)

    def attend(self):
        """Slots, rows in the caches, pages and attention of the step's drafted tokens."""
        n, t = self.active, self.active * DRAFTS
        self.seq_, self.cu_ = self.seq[:n], self.cu[: n + 1]
        idx.idx_build_slots(self.ctx[:n], self.new[:n], self.owned[:n], self.table[:n], self.free, self.cursor, self.blocks, PAGE, self.cu_, self.seq_,
                            self.pages_out[:n], self.cursor_out, self.positions[:t], self.slots[:t], parents=self.parents[:t], tree_mask=self.mask[:t],
                            status=self.status)
        idx.idx_norm_rope_append(self.q[:t], self.k[:t], self.v[:t], self.q_weight, self.k_weight, self.eps, self.positions[:t], self.freq,
                                 self.q_turned[:t], self.cache[0], self.cache[1], slots=self.slots[:t], mscale=self.mscale, status=self.status)
        idx.idx_index_append(self.index_rows[:t, :LISTS], self.index_rows[:t, LISTS], self.iq_weight, self.ik_weight, self.eps, self.positions[:t],
                             self.freq, self.index_q[:n], self.index_scale[:n], self.index_k, slots=self.slots[:t], cu_tokens=self.cu_,
                             scale=128**-0.5, mscale=self.mscale, status=self.status)
        idx.idx_decode_step(self.index_q[:n], self.index_scale[:n], self.index_k, self.table[:n], self.seq_, DRAFTS, self.scores[:n], self.pages[:n],
                            self.select_ws, self.status)
        idx.idx_tree_attention(self.q_turned[:t], self.cache[0], self.cache[1], self.table[:n], self.seq_, self.cu_, self.out[:t], self.scale,
                               tree_mask=self.mask[:t], pages=self.pages[:n], workspace=self.attention_ws, status=self.status)

    def judge(self):
        """The target's probabilities, and which of the drafts stand."""
        n, t = self.active, self.active * DRAFTS
        idx.idx_logit_probs(self.logits[:t], self.target[:t], self.cu_, temperature=self.temperature[:n], repetition=self.repetition[:n],
                            presence=self.presence[:n], frequency=self.frequency[:n], counts=self.counts[:n], tokens=self.drafted[:t],
                            tree_mask=self.mask[:t], allowed=self.allowed[:t], status=self.status)
        idx.idx_verify_drafts(self.target[:t], self.draft[:t], self.drafted[:t], self.cu_, self.accept_u[:t], self.sample_u[:n], self.out_tokens[:n],
                              self.out_nodes[:n], self.accepted[:n], parents=self.parents[:t], status=self.status)

    def settle(self):
        """The caches, lengths and counts made ready for the next step."""
        n, t = self.active, self.active * DRAFTS
        idx.idx_settle_drafts(self.caches, self.slots[:t], self.cu_, self.out_tokens[:n], self.out_nodes[:n], self.accepted[:n], self.ctx[:n],
                              self.ctx[:n], counts=self.counts[:n], status=self.status)
        self.owned[:n].copy_(self.pages_out[:n])
        self.cursor.copy_(self.cursor_out)

    def step(self):
        self.attend()
        self.judge()
        self.settle()

    def fork(self, parents):
        """New requests behind the active ones, each with the context of its parent."""
        n, m = self.active, len(parents)
        parents = torch.tensor(parents, dtype=torch.int32, device=self.cu.device)
        children = torch.arange(n, n + m, dtype=torch.int32, device=self.cu.device)
        idx.idx_fork_pages(self.caches, parents, children, self.ctx, self.owned, self.table, self.refs, self.free, self.cursor, self.cursor_out,
                           status=self.status)
        self.cursor.copy_(self.cursor_out)
        self.counts[n : n + m] = self.counts[parents.long()]
        self.active = n + m

    def release(self, keep):
        """Pages past the kept lengths (one for each active request) go back; requests that keep nothing end, from the last on.

        A request cut back into a page that others hold too would write over their tokens in its next step.  It is forked at
        its kept length into the row behind the active ones, which copies that page, and its child takes its place.
        """
        n, spare = self.active, max((i + 1 for i, k in enumerate(keep) if k > 0), default=0)
        lens = torch.tensor(keep + [0] * (self.rows - n), dtype=torch.int32, device=self.cu.device)
        shared = self.inside_shared(torch.minimum(self.ctx, lens))
        if shared and spare == self.rows:
            raise ValueError(f"requests {shared} end inside pages that others hold, and no row is free to copy them into")
        self.give_back(lens)
        self.active = spare
        for r in self.inside_shared(self.ctx):
            self.fork([r])
            self.active = spare
            lens = self.ctx.clone()
            lens[r] = 0
            self.give_back(lens)
            for a in (self.ctx, self.owned, self.table):
                a[r] = a[spare]
            self.ctx[spare], self.owned[spare] = 0, 0

    def inside_shared(self, lens):
        """Requests whose next token would have its place in a page that others hold too."""
        page = (lens // PAGE).clamp(max=self.table.shape[1] - 1).long()
        block = self.table.gather(1, page[:, None])[:, 0].clamp(0, self.blocks - 1).long()
        return ((lens % PAGE > 0) & (self.refs[block] > 0)).nonzero()[:, 0].tolist()

    def give_back(self, lens):
        self.keep.copy_(lens)
        idx.idx_release_pages(self.keep, self.owned, self.table, self.refs, self.free, self.cursor, self.cursor_out, self.pages_out, PAGE, status=self.status)
        self.owned.copy_(self.pages_out)
        self.cursor.copy_(self.cursor_out)
        self.ctx.copy_(torch.minimum(self.ctx, self.keep))


def timed(server, steps):
    for _ in range(3):
        server.draw()
        server.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # nothing runs in here
        server.step()
    took, stood = [], 0
    for _ in range(steps):
        server.draw()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        graph.replay()
        end.record()
        end.synchronize()
        took.append(begin.elapsed_time(end) * 1e3)
        stood += int(server.accepted[: server.active].sum())
    took.sort()
    print(f"{server.active} requests, {DRAFTS} nodes each: {took[len(took) // 2]:.1f} us a step, "
          f"{1 + stood / steps / server.active:.2f} tokens a request and step")


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--reqs", type=int, default=48)
    p.add_argument("--forks", type=int, default=16)
    p.add_argument("--context", type=int, default=8000)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    s = Server(a.reqs + a.forks, a.context + 2 * DRAFTS * (a.steps + 5))
    s.admit(a.reqs, a.context)
    timed(s, a.steps)
    s.fork([i % a.reqs for i in range(a.forks)])
    timed(s, a.steps)
    s.release([0] * s.active)
    assert int(s.status.item()) == 0, f"status {int(s.status.item())}"
    assert int(s.cursor.item()) == 0 and not s.refs.any(), "pages were lost"
    print(f"all {s.blocks} blocks are free again")


if __name__ == "__main__":
    main()

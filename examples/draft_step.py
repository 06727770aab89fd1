"""Steps of decoding with drafted tokens, every call of the library in its place.

Each step of `Decoder` is one request-packed batch of small trees of drafted
tokens and runs, with no host synchronisation,

    idx_build_slots     pages taken from the free list; slots, positions, masks
    idx_rope_append     q and k turned, k and v into the paged cache
    idx_decode_step     the 16 pages that each drafted token looks at
    idx_tree_attention  attention over those pages
    idx_verify_drafts   which drafted tokens stand, and the token after them
    idx_rope_append     (with nothing to turn) keys and values of those that
                        stand moved together, so that the next step's context
                        is without gaps

so a step can be captured into a CUDA graph and replayed: lengths, tables and
the free list's cursor stay on the GPU.  Where a model would form q, k, v, the
index queries and the two distributions, this example draws them at random;
the index-K pages hold random codes.

    python examples/draft_step.py [--reqs 64] [--context 16384] [--steps 20]
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


class Decoder:
    """A batch's caches, tables and buffers, and the step over them."""

    def __init__(self, reqs, context, max_len, q_heads=64, kv_heads=4, dim=128, vocab=32000, dtype=torch.bfloat16, device="cuda", seed=0):
        self.reqs, self.vocab, self.dim, self.scale = reqs, vocab, dim, dim**-0.5
        self.gen = torch.Generator(device=device)
        self.gen.manual_seed(seed)
        tokens, width = reqs * DRAFTS, -(-max_len // PAGE)
        blocks = reqs * width
        i32 = dict(dtype=torch.int32, device=device)
        new = lambda *shape, **kind: torch.empty(shape, device=device, **kind)

        # lengths and tables: the contexts' pages come from the free list in the first step
        self.ctx = torch.full((reqs,), context, **i32)
        self.new = torch.full((reqs,), DRAFTS, **i32)
        self.owned, self.pages_out = torch.zeros(reqs, **i32), torch.zeros(reqs, **i32)
        self.cursor, self.cursor_out = torch.zeros(1, **i32), torch.zeros(1, **i32)
        self.table = torch.full((reqs, width), -1, **i32)
        self.free = torch.randperm(blocks, device=device, generator=self.gen).to(torch.int32)
        self.parents = torch.tensor(PARENTS * reqs, **i32)
        self.blocks = blocks
        self.cu, self.seq = new(reqs + 1, dtype=torch.int32), new(reqs, dtype=torch.int32)
        self.positions, self.slots = new(tokens, dtype=torch.int32), new(tokens, dtype=torch.int64)
        self.mask = new(tokens, dtype=torch.int64)

        # caches
        self.cache = torch.randn(2, blocks, PAGE, kv_heads, dim, device=device, generator=self.gen, dtype=torch.float32).to(dtype)
        self.index_k = torch.randint(0, 256, (blocks, PAGE, 72), device=device, generator=self.gen, dtype=torch.uint8)
        self.index_k.view(blocks, -1)[:, 64 * PAGE :] = 0x38  # block scales of 1

        # a step's inputs and outputs
        freq, self.mscale = idx.idx_rope_frequencies(dim)
        self.freq, self.no_freq = freq.to(device), torch.zeros(0, dtype=torch.float64, device=device)
        self.qkv = new(tokens, q_heads + 2 * kv_heads, dim, dtype=dtype)
        self.q, self.k, self.v = self.qkv.split([q_heads, kv_heads, kv_heads], dim=1)
        self.q_turned, self.out = new(tokens, q_heads, dim, dtype=dtype), new(tokens, q_heads, dim, dtype=dtype)
        self.index_q, self.index_scale = new(reqs, DRAFTS, LISTS, 128, dtype=torch.uint8), new(reqs, DRAFTS, LISTS, dtype=torch.float32)
        self.scores = new(reqs, DRAFTS * LISTS, width, dtype=torch.float32)
        self.pages = new(reqs, DRAFTS, LISTS, PICKED, dtype=torch.int32)
        self.target, self.draft = new(tokens, vocab, dtype=torch.float32), new(tokens, vocab, dtype=torch.float32)
        self.drafted = new(tokens, dtype=torch.int32)
        self.accept_u, self.sample_u = new(tokens, dtype=torch.float32), new(reqs, dtype=torch.float32)
        self.out_tokens, self.out_nodes = new(reqs, DRAFTS, dtype=torch.int32), new(reqs, DRAFTS, dtype=torch.int32)
        self.accepted = new(reqs, dtype=torch.int32)
        self.status = torch.zeros(1, **i32)
        bytes_of = lambda n: new(max(n, 8), dtype=torch.uint8)
        self.select_ws = bytes_of(idx.idx_decode_workspace_bytes(reqs, DRAFTS, width))
        self.attention_ws = bytes_of(idx.idx_tree_attention_workspace_bytes(reqs, tokens, q_heads, kv_heads, dim, LISTS, PICKED))
        # first token of each request, and the node's number within it
        self.first = torch.arange(reqs, device=device)[:, None] * DRAFTS
        self.number = torch.arange(DRAFTS - 1, device=device)[None, :]

    def draw(self):
        """What the model and the drafter would have formed."""
        g = self.gen
        self.qkv.normal_(generator=g)
        self.index_q.copy_(torch.randint(0, 0x78, self.index_q.shape, device=self.index_q.device, generator=g))
        self.index_scale.uniform_(0.5, 2.0, generator=g)
        logits = 3.0 * torch.randn(self.target.shape, device=self.target.device, generator=g)
        self.target.copy_(torch.softmax(logits, 1))
        self.draft.copy_(torch.softmax(logits + 0.5 * torch.randn(logits.shape, device=logits.device, generator=g), 1))
        # a node's token was drawn from its parent's row
        parents = (self.first + torch.clamp(self.parents.view(self.reqs, DRAFTS), min=0)).flatten()
        self.drafted.copy_(torch.multinomial(self.draft, DRAFTS, replacement=True, generator=g)[parents, torch.arange(DRAFTS, device=logits.device).repeat(self.reqs)])
        self.accept_u.uniform_(generator=g)
        self.sample_u.uniform_(generator=g)

    def attend(self):
        """Slots, positions, pages and attention of the step's drafted tokens."""
        idx.idx_build_slots(self.ctx, self.new, self.owned, self.table, self.free, self.cursor, self.blocks, PAGE, self.cu, self.seq,
                            self.pages_out, self.cursor_out, self.positions, self.slots, parents=self.parents, tree_mask=self.mask,
                            status=self.status)
        idx.idx_rope_append(self.q, self.k, self.v, self.positions, self.freq, self.q_turned, self.cache[0], self.cache[1],
                            slots=self.slots, mscale=self.mscale, status=self.status)
        idx.idx_decode_step(self.index_q, self.index_scale, self.index_k, self.table, self.seq, DRAFTS, self.scores, self.pages,
                            self.select_ws, self.status)
        idx.idx_tree_attention(self.q_turned, self.cache[0], self.cache[1], self.table, self.seq, self.cu, self.out, self.scale,
                               tree_mask=self.mask, pages=self.pages, workspace=self.attention_ws, status=self.status)

    def settle(self):
        """Verification; the cache and the lengths made ready for the next step."""
        idx.idx_verify_drafts(self.target, self.draft, self.drafted, self.cu, self.accept_u, self.sample_u, self.out_tokens,
                              self.out_nodes, self.accepted, parents=self.parents, status=self.status)
        # the i-th node that stands goes to place ctx + 1 + i: read first, then written
        nodes = self.out_nodes[:, : DRAFTS - 1]
        source = self.slots[(self.first + nodes.clamp(min=0)).flatten()].clamp(min=0)
        target = torch.where(nodes >= 0, self.slots[(self.first + 1 + self.number)], -1).flatten()
        rows = self.cache.flatten(1, 2)
        idx.idx_rope_append(None, rows[0][source], rows[1][source], self.positions[: len(source)], self.no_freq, None, self.cache[0],
                            self.cache[1], slots=target, status=self.status)
        self.ctx.add_(self.accepted).add_(1)
        self.owned.copy_(self.pages_out)
        self.cursor.copy_(self.cursor_out)

    def step(self):
        self.attend()
        self.settle()


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--reqs", type=int, default=64)
    p.add_argument("--context", type=int, default=16384)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    d = Decoder(a.reqs, a.context, a.context + DRAFTS * (a.steps + 5))
    for _ in range(3):
        d.draw()
        d.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # nothing runs in here
        d.step()
    took, stood = [], 0
    for _ in range(a.steps):
        d.draw()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        graph.replay()
        end.record()
        end.synchronize()
        took.append(begin.elapsed_time(end) * 1e3)
        stood += int(d.accepted.sum())
    assert int(d.status.item()) == 0, f"status {int(d.status.item())}"
    took.sort()
    print(f"{a.reqs} requests of {a.context} tokens, {DRAFTS} nodes each: {took[len(took) // 2]:.1f} us a step, "
          f"{1 + stood / a.steps / a.reqs:.2f} tokens a request and step")


if __name__ == "__main__":
    main()

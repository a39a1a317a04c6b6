"""Beam search over a paged KV cache: the beams of a request share the pages of what they have in
common, and a step, one CUDA graph replay, is all on the device.

    python examples/beam_search.py [--steps 24] [--beams 4] [--cache fp16|bf16|q8_0]

The model is the small random-weight decoder of examples/paged_decode.py.  Prompts are fed a
token at a time, one row for each request; then every request's row is forked into its beams.
A step:

    kv_page_plan        a page for every beam that runs out, positions and slots
    per layer           gemm_bf16 (QKV) -> rope_kv_write -> attn_paged_prefix -> gemm_bf16 (O):
                        the prompt's keys and values are read once for all beams of a request
    gemm_bf16           the lm_head
    beam_select         each request's next beams, and the candidates that end
    kv_page_fork        their block table rows: shared pages, and copies to make
    kv_page_copy        the copies of partly filled last pages, in every layer
    kv_page_compact     pages that no beam lists any more back to the free list
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for p in (ROOT, os.path.join(ROOT, "examples")):
    if p not in sys.path:
        sys.path.insert(0, p)

import torch  # noqa: E402

import weight_streaming_warp_gb300 as wsw  # noqa: E402
from paged_decode import CACHES, Decoder, Server  # noqa: E402


class Beams:
    """The beams of several requests: pages, block table, lengths, scores, and a step's buffers."""

    def __init__(self, model, prompts, beams=4, end_token=0, page_size=16, max_new=64, cache="fp16", share=False):
        self.model, self.beams, self.end, self.share = model, beams, end_token, share
        requests, n = len(prompts), len(prompts) * beams
        self.n, self.page_size = n, page_size
        longest = max(len(p) for p in prompts)
        per = -(-(longest + max_new) // page_size)
        # the prompts' pages, and of each beam two full lineages' worth at the worst
        self.pages = requests * per + 2 * n * (-(-max_new // page_size) + 2)
        server = Server(model, requests, self.pages, page_size, per, cache)
        for t in range(longest - 1):  # all but each prompt's last token; shorter prompts wait
            feed = [p[t] if t < len(p) - 1 else 0 for p in prompts]
            server.new.copy_(torch.tensor([int(t < len(p) - 1) for p in prompts], dtype=torch.int32))
            server.tokens.copy_(torch.tensor(feed, dtype=torch.int32))
            server.step()
        self.caches = server.caches
        i32 = dict(dtype=torch.int32, device="cuda")
        f32 = dict(dtype=torch.float32, device="cuda")
        # every beam continues its request's row
        start = torch.arange(requests, **i32).repeat_interleave(beams).contiguous()
        first = wsw.kv_page_fork(start, server.lens, server.free, server.first_free, server.table, page_size,
                                 err_flag=server.err)
        wsw.kv_page_copy(first.copies, self.caches, err_flag=server.err)
        self.err = server.err
        self.table, self.lens = first.table, first.seq_len
        self.free, self.head = torch.full((self.pages,), -1, **i32), torch.zeros(1, **i32)
        self.compact_ws = torch.zeros(wsw.kv_page_compact_workspace_bytes(self.pages), dtype=torch.uint8, device="cuda")
        none = torch.empty(0, **i32)
        self.freed = wsw.KvCompact(self.table, self.free, self.head, wsw.PageCopies(none, none, None, torch.zeros(1, **i32)))
        self._free_pages()
        # what the beams of a request share for good: the prompt but its last token
        self.groups = (torch.arange(requests + 1, device="cuda") * beams).to(torch.int32)
        self.prefix = server.lens.clone()
        self.fork = wsw.KvFork(self.table, self.lens, self.head, wsw.PageCopies(
            torch.empty(n, **i32), torch.empty(n, **i32), torch.empty(n, **i32), torch.empty(1, **i32)))
        self.new = torch.ones(n, **i32)
        self.plan = wsw.KvPlan(torch.empty(n, **i32), torch.empty(n, dtype=torch.int64, device="cuda"),
                               torch.empty(n + 1, **i32), self.lens, self.head)
        self.tokens = torch.tensor([p[-1] for p in prompts], **i32).repeat_interleave(beams).contiguous()
        self.scores = torch.full((requests, beams), float("-inf"), **f32)
        self.scores[:, 0] = 0  # one beam at first: the others are copies of it
        self.chosen = wsw.beam_select_out(requests, beams)
        self.select_ws = torch.zeros(wsw.beam_select_workspace_bytes(requests, beams, model.vocab, 1), dtype=torch.uint8,
                                     device="cuda")
        m = model
        self.q = [torch.empty(n, m.q_heads, m.head_dim, device="cuda") for _ in m.layers]
        self.attn = [torch.empty_like(x) for x in self.q]
        self.attn_ws = torch.zeros(wsw.attn_paged_prefix_workspace_bytes(n, requests, m.q_heads, m.kv_heads, m.head_dim),
                                   dtype=torch.uint8, device="cuda")
        self.graph = None

    def _free_pages(self):
        wsw.kv_page_compact(self.lens, self.table, self.page_size, self.pages, out=self.freed, err_flag=self.err,
                            ws=self.compact_ws)

    def _step(self):
        m, n = self.model, self.n
        wsw.kv_page_plan(self.lens, self.new, self.free, self.head, self.table, self.page_size, n, out=self.plan,
                         err_flag=self.err)
        x = m.embed[self.tokens.long().clamp(min=0)]
        for i, (w_qkv, w_out) in enumerate(m.layers):
            normed = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
            qkv = wsw.gemm_bf16(w_qkv, normed.to(torch.bfloat16)).view(n, -1, m.head_dim)
            q, k, v = qkv.split([m.q_heads, m.kv_heads, m.kv_heads], 1)
            wsw.rope_kv_write(q, k, v, m.rope, self.plan.positions, self.plan.slots, self.caches[i], out=self.q[i],
                              err_flag=self.err)
            wsw.attn_paged_prefix(self.q[i], self.caches[i], self.table, self.lens, self.groups, self.prefix,
                                  out=self.attn[i], ws=self.attn_ws, err_flag=self.err, share=self.share)
            x = x + wsw.gemm_bf16(w_out, self.attn[i].view(n, -1).to(torch.bfloat16))
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        self.logits = wsw.gemm_bf16(m.head, x.to(torch.bfloat16))
        wsw.beam_select(self.logits, self.scores, [self.end], out=self.chosen, ws=self.select_ws)
        wsw.kv_page_fork(self.chosen.parent.view(-1), self.lens, self.free, self.head, self.table, self.page_size,
                         out=self.fork, err_flag=self.err)
        wsw.kv_page_copy(self.fork.copies, self.caches, err_flag=self.err)
        self._free_pages()
        self.tokens.copy_(self.chosen.token.view(-1))
        self.scores.copy_(self.chosen.score)

    def step(self):
        """One token for every beam.  The first call runs the step as it is (it loads the kernels), the
        second captures it, later ones replay."""
        if self.graph is None:
            self._step()
            self.graph = False
        elif self.graph is False:
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self._step()
            self.graph.replay()  # a capture only records
        else:
            self.graph.replay()


def search(model, prompts, steps, beams=4, end_token=0, **kw):
    """The hypotheses of every prompt, best first by log probability per token: [(tokens, score)], those
    that ended and the beams of the last step."""
    b = Beams(model, prompts, beams, end_token, max_new=steps + 1, **kw)
    found = [[] for _ in prompts]
    history = [[] for _ in range(b.n)]
    for _ in range(steps):
        b.step()
        c = b.chosen
        for r in range(len(prompts)):
            for p, s in zip(c.end_parent[r].tolist(), c.end_score[r].tolist()):
                if p >= 0:
                    found[r].append((history[p] + [end_token], s))
        history = [history[p] + [t] if p >= 0 else [] for p, t in
                   zip(c.parent.view(-1).tolist(), c.token.view(-1).tolist())]
    if int(b.err):
        raise RuntimeError("the step reported error bits %d" % int(b.err))
    for r in range(len(prompts)):
        found[r] += [(history[r * beams + i], s) for i, s in enumerate(b.scores[r].tolist()) if history[r * beams + i]]
        found[r].sort(key=lambda h: -h[1] / len(h[0]))
    return found, b


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--cache", choices=sorted(CACHES), default="fp16")
    a = ap.parse_args()
    from weight_streaming_warp_gb300 import build
    build.build()
    found, _ = search(Decoder(), [[1], [5, 6, 7], list(range(40)), [9] * 17], a.steps, a.beams, cache=a.cache)
    for hypotheses in found:
        print("\n".join("%8.3f  %s" % (s, t) for t, s in hypotheses[:2]))


if __name__ == "__main__":
    main()

"""A decode loop around the paged KV cache: several requests of different lengths generate
tokens together from one pool of pages, one CUDA graph replay per step.

    python examples/paged_decode.py [--steps 32] [--cache fp16|bf16|q8_0]

The model is a small random-weight decoder (one fused QKV product, attention and an output
product per layer, a tied width throughout; no training, so the text means nothing).  A
step is, all on the device:

    kv_page_plan        a page for every request that runs out, positions and slots
    per layer           gemm_bf16 (QKV) -> rope_kv_write -> attn_paged_decode -> gemm_bf16 (O)
    gemm_bf16           the lm_head
    token_logprobs      each request's most likely next tokens and their log probabilities

Lengths, block table and free list stay on the device and advance in place, so the captured
step is replayed as it is.
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import weight_streaming_warp_gb300 as wsw  # noqa: E402

CACHES = {"fp16": torch.float16, "bf16": torch.bfloat16, "q8_0": torch.int8}


class Decoder:
    """Random weights of `layers` attention layers over `vocab` tokens."""

    def __init__(self, layers=2, q_heads=8, kv_heads=2, head_dim=128, vocab=2048, context=32768, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.vocab = q_heads, kv_heads, head_dim, vocab
        self.width = q_heads * head_dim

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g, device="cuda") / cols ** 0.5).to(torch.bfloat16)

        self.embed = torch.randn(vocab, self.width, generator=g, device="cuda")
        self.layers = [(weight((q_heads + 2 * kv_heads) * head_dim, self.width), weight(self.width, self.width))
                       for _ in range(layers)]
        self.head = weight(vocab, self.width)
        self.rope = wsw.rope_table(head_dim, scaling="by_parts", factor=4.0, original=context)


class Server:
    """The requests' shared state: pages, block table, lengths, and the buffers of a step."""

    def __init__(self, model, requests, pages, page_size=16, max_pages=64, cache="fp16"):
        dev = "cuda"
        self.model, self.n, self.page_size = model, requests, page_size
        m, shape = model, (pages, page_size, model.kv_heads)
        dtype = CACHES[cache]

        def layer_cache():
            kv = [torch.zeros(*shape, m.head_dim, dtype=dtype, device=dev) for _ in range(2)]
            scales = [torch.zeros(*shape, m.head_dim // 32, dtype=torch.float16, device=dev) if cache == "q8_0" else None
                      for _ in range(2)]
            return wsw.PagedKV(*kv, *scales)

        self.caches = [layer_cache() for _ in m.layers]
        i32 = dict(dtype=torch.int32, device=dev)
        self.table = torch.full((requests, max_pages), -1, **i32)
        self.lens, self.new = torch.zeros(requests, **i32), torch.ones(requests, **i32)
        self.free, self.first_free = torch.arange(pages, **i32), torch.zeros(1, **i32)
        self.err = torch.zeros(1, **i32)
        self.plan = wsw.KvPlan(torch.empty(requests, **i32), torch.empty(requests, dtype=torch.int64, device=dev),
                               torch.empty(requests + 1, **i32), self.lens, self.first_free)
        self.tokens = torch.zeros(requests, **i32)    # what the step feeds
        self.report = wsw.token_logprobs_out(requests, 4, tokens=False)
        self.q = [torch.empty(requests, m.q_heads, m.head_dim, device=dev) for _ in m.layers]
        self.attn = [torch.empty_like(x) for x in self.q]
        self.attn_ws = torch.zeros(wsw.attn_paged_decode_workspace_bytes(requests, m.q_heads, m.kv_heads, m.head_dim),
                                   dtype=torch.uint8, device=dev)
        need = wsw.token_logprobs_workspace_bytes(requests, m.vocab, 4)
        self.lp_ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=dev)
        self.graph = None

    def _step(self):
        m, n = self.model, self.n
        wsw.kv_page_plan(self.lens, self.new, self.free, self.first_free, self.table, self.page_size, n,
                         out=self.plan, err_flag=self.err)
        x = m.embed[self.tokens.long()]
        for i, (w_qkv, w_out) in enumerate(m.layers):
            normed = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
            self.qkv = wsw.gemm_bf16(w_qkv, normed.to(torch.bfloat16)).view(n, -1, m.head_dim)
            q, k, v = self.qkv.split([m.q_heads, m.kv_heads, m.kv_heads], 1)
            wsw.rope_kv_write(q, k, v, m.rope, self.plan.positions, self.plan.slots, self.caches[i], out=self.q[i],
                              err_flag=self.err)
            wsw.attn_paged_decode(self.q[i], self.caches[i], self.table, self.lens, out=self.attn[i], ws=self.attn_ws,
                                  err_flag=self.err)
            x = x + wsw.gemm_bf16(w_out, self.attn[i].view(n, m.width).to(torch.bfloat16))
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        self.logits = wsw.gemm_bf16(m.head, x.to(torch.bfloat16))
        wsw.token_logprobs(self.logits, top=4, out=self.report, ws=self.lp_ws)

    def step(self):
        """Feed self.tokens; self.report then tells about the next ones.  The first call runs the
        step as it is (it loads the kernels), the second captures it, later ones replay."""
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


def generate(model, prompts, steps, cache="fp16", page_size=16):
    """Greedy tokens of every prompt (lists of token ids), `steps` of them, and their log
    probabilities.  Prompts are fed a token at a time; a shorter one starts to generate
    earlier."""
    n = len(prompts)
    longest = max(len(p) for p in prompts) + steps
    per = -(-longest // page_size)
    server = Server(model, n, pages=n * per, page_size=page_size, max_pages=per, cache=cache)
    out, logprob = [list(p) for p in prompts], [[] for _ in prompts]
    for t in range(longest - 1):
        server.tokens.copy_(torch.tensor([o[t] if t < len(o) else 0 for o in out], dtype=torch.int32))
        server.step()
        best, lp = server.report.top_id[:, 0].tolist(), server.report.top_logprob[:, 0].tolist()
        for r in range(n):
            if len(out[r]) == t + 1 and len(logprob[r]) < steps:
                out[r].append(best[r])
                logprob[r].append(lp[r])
    if int(server.err):
        raise RuntimeError("the step reported error bits %d" % int(server.err))
    return out, logprob, server


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--cache", choices=sorted(CACHES), default="fp16")
    a = ap.parse_args()
    from weight_streaming_warp_gb300 import build
    build.build()
    model = Decoder()
    prompts = [[1], [5, 6, 7], list(range(40)), [9] * 17]
    out, logprob, _ = generate(model, prompts, a.steps, a.cache)
    for p, o, lp in zip(prompts, out, logprob):
        print("prompt of %d: %s  mean log probability %.4f" % (len(p), o[len(p): len(p) + a.steps], sum(lp) / len(lp)))


if __name__ == "__main__":
    main()

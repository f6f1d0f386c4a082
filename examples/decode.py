"""A small decoder on the library's operators: prompts and sampled tokens for a batch.

Every projection is a Q4_0 matmul; keys and values live in the paged 8-bit
cache; prompts of different lengths go through one packed batch, and then each
step (one token a sequence) is one replay of a CUDA graph: the cache's lengths,
the positions and the last tokens are device tensors that the graph itself
moves on.  Weights are random: the text is noise, the work is that of a real
decoder.

    python examples/decode.py [--steps 32] [--layers 4] [--batch 4]
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_weight_q4_gb300 as q4  # noqa: E402


def q4_weight(K, N, gen):
    """Random K x N weights as Q4_0 blocks."""
    W = torch.randn(K, N, generator=gen, device="cuda") * K ** -0.5
    B = torch.empty(K, (N + 31) // 32 * 18, dtype=torch.uint8, device="cuda")
    q4.q4_quantize(B, W, K, N)
    return B


def rms(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Decoder:
    def __init__(self, layers=4, hidden=1024, heads=8, kv_heads=2, dim=128, inner=2816, vocab=32000, seqs=4,
                 max_tokens=1024, page_tokens=64, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, dim
        self.inner, self.vocab, self.seqs, self.max_tokens = inner, vocab, seqs, max_tokens
        self.qkv_width = (heads + 2 * kv_heads) * dim
        self.layers = [dict(qkv=q4_weight(hidden, self.qkv_width, gen), out=q4_weight(heads * dim, hidden, gen),
                            gate=q4_weight(hidden, inner, gen), up=q4_weight(hidden, inner, gen),
                            down=q4_weight(inner, hidden, gen),
                            q_norm=torch.ones(dim, device="cuda"), k_norm=torch.ones(dim, device="cuda"),
                            cache=q4.KVCache.empty(seqs * -(-max_tokens // page_tokens), kv_heads, dim, page_tokens))
                       for _ in range(layers)]
        self.embed = (torch.randn(vocab, hidden, generator=gen, device="cuda")).to(torch.bfloat16)
        self.head = q4_weight(hidden, vocab, gen)
        # every sequence has its pages from the start; a server would hand them out as sequences grow
        pages = -(-max_tokens // page_tokens)
        self.table = torch.randperm(seqs * pages, generator=gen, device="cuda").to(torch.int32).view(seqs, pages)
        half = dim // 2
        turn = torch.arange(max_tokens)[:, None] * 10000.0 ** (-torch.arange(half) / half)
        self.cos, self.sin = turn.cos().float().cuda(), turn.sin().float().cuda()
        self.kv_len = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        # workspaces that captured calls use: the projections of a step, and attention
        self.mm_ws = torch.zeros(max(q4.q4_matmul_workspace_size(seqs, n, k) for k, n in self.shapes()) or 16,
                                 dtype=torch.uint8, device="cuda")
        self.attn_ws = torch.zeros(q4.q4_kv_attention_workspace_size(self.layers[0]["cache"], heads, seqs, seqs, 1,
                                                                     max_tokens), dtype=torch.uint8, device="cuda")

    def shapes(self):
        h = self.hidden
        return [(h, self.qkv_width), (self.heads * self.dim, h), (h, self.inner), (self.inner, h), (h, self.vocab)]

    def project(self, x, B, N, dtype=torch.bfloat16, workspace=None):
        y = torch.empty(x.shape[0], N, dtype=dtype, device="cuda")
        q4.q4_matmul_ex(y, x, B, x.shape[0], N, x.shape[1], workspace=workspace)
        return y

    def forward(self, tokens, cu, max_q, mm_ws=None, attn_ws=None):
        """Hidden states of the new tokens [T]; kv_len already counts them."""
        T, h, hk, d = tokens.shape[0], self.heads, self.kv_heads, self.dim
        x = self.embed[tokens.long()]
        for w in self.layers:
            qkv = self.project(rms(x), w["qkv"], self.qkv_width, workspace=mm_ws)
            q = qkv[:, :h * d].unflatten(1, (h, d))
            k = qkv[:, h * d:(h + hk) * d].unflatten(1, (hk, d))
            v = qkv[:, (h + hk) * d:].unflatten(1, (hk, d))
            turned = torch.empty(T, h, d, dtype=torch.bfloat16, device="cuda")
            q4.q4_kv_append(w["cache"], turned, q, k, v, self.table, self.kv_len, cu, cos=self.cos, sin=self.sin,
                            q_norm=w["q_norm"], k_norm=w["k_norm"])
            seen = torch.empty_like(turned)
            q4.q4_kv_attention(seen, turned, w["cache"], self.table, self.kv_len, cu, max_q=max_q,
                               max_kv=self.max_tokens, workspace=attn_ws)
            x = x + self.project(seen.view(T, h * d), w["out"], self.hidden, workspace=mm_ws)
            y = rms(x)
            g = self.project(y, w["gate"], self.inner, workspace=mm_ws)
            u = self.project(y, w["up"], self.inner, workspace=mm_ws)
            x = x + self.project(torch.nn.functional.silu(g) * u, w["down"], self.hidden, workspace=mm_ws)
        return x

    def choose(self, x, u, settings, out, workspace=None, penalties=None):
        logits = self.project(rms(x), self.head, self.vocab, dtype=torch.float32, workspace=workspace)
        if penalties is not None:       # in place: a history on the device, and how much of it there is
            q4.q4_adjust_logits(logits, logits, **penalties)
        q4.q4_sample(out, logits, u, **settings)
        return logits

    def prompts(self, prompts, u, settings):
        """Fills the cache from the prompts (one tensor of tokens each); their first sampled tokens."""
        lens = torch.tensor([p.numel() for p in prompts], dtype=torch.int32)
        cu = torch.zeros(self.seqs + 1, dtype=torch.int32)
        cu[1:] = lens.cumsum(0)
        self.kv_len.copy_(lens)
        x = self.forward(torch.cat(prompts), cu.cuda(), int(lens.max()))
        tokens = torch.empty(self.seqs, dtype=torch.int32, device="cuda")
        logits = self.choose(x[(cu[1:] - 1).cuda().long()], u, settings, tokens)
        return tokens, logits

    def capture_step(self, tokens, u, settings, penalties=None):
        """A graph of one step for the whole batch: reads `tokens` and `u`, writes the next ones into `tokens`.
        penalties: arguments of q4_adjust_logits; the chosen tokens are put behind the history that they name."""
        self.step_cu = cu = torch.arange(self.seqs + 1, dtype=torch.int32, device="cuda")   # the graph reads it

        def step():
            self.kv_len += 1
            x = self.forward(tokens, cu, 1, self.mm_ws, self.attn_ws)
            logits = self.choose(x, u, settings, tokens, self.mm_ws, penalties)
            if penalties is not None:
                history, length = penalties["history"], penalties["history_len"]
                # a full history keeps its last place for the newest token
                history.scatter_(1, length.clamp(max=history.shape[1] - 1).long()[:, None], tokens[:, None])
                length += 1
            return logits

        stream = torch.cuda.Stream()
        keep = self.kv_len.clone(), tokens.clone()
        if penalties is not None:
            keep += penalties["history_len"].clone(),
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):     # once outside the capture, on positions that are written again
            step()
        torch.cuda.current_stream().wait_stream(stream)
        self.kv_len.copy_(keep[0])
        tokens.copy_(keep[1])
        if penalties is not None:
            penalties["history_len"].copy_(keep[2])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            logits = step()
        return graph, logits


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--repetition", type=float, default=1.0, help="penalty of tokens that a sequence has already")
    a = ap.parse_args()
    lens, most = [37 + 61 * i for i in range(a.batch)], 1024
    if a.batch < 1 or a.steps < 1 or lens[-1] + a.steps > most:
        ap.error(f"{a.batch} prompts, the longest of {lens[-1] if lens else 0} tokens, and {a.steps} steps: the cache has "
                 f"room for {most} tokens a sequence")
    gen = torch.Generator("cuda").manual_seed(1)
    m = Decoder(layers=a.layers, seqs=a.batch, max_tokens=most)
    settings = dict(temperature=torch.full((a.batch,), 0.8, device="cuda"),
                    top_k=torch.full((a.batch,), 50, dtype=torch.int32, device="cuda"),
                    top_p=torch.full((a.batch,), 0.95, device="cuda"))
    prompts = [torch.randint(0, m.vocab, (n,), generator=gen, device="cuda", dtype=torch.int32) for n in lens]
    u = torch.rand(a.batch, generator=gen, device="cuda")
    tokens, _ = m.prompts(prompts, u, settings)
    penalties = None
    if a.repetition != 1:
        # the cached tokens, and the newest one, which is not cached yet
        history = torch.full((a.batch, m.max_tokens + 1), -1, dtype=torch.int32, device="cuda")
        for row, p in zip(history, prompts):
            row[:p.numel()] = p
        prompt_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        history.scatter_(1, prompt_len.long()[:, None], tokens[:, None])
        penalties = dict(history=history, history_len=prompt_len + 1, prompt_len=prompt_len,
                         repetition=torch.full((a.batch,), a.repetition, device="cuda"))
    graph, _ = m.capture_step(tokens, u, settings, penalties)
    out = [tokens.clone()]
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        u.uniform_(generator=gen)
        graph.replay()
        out.append(tokens.clone())
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    assert q4.q4_get_device_status() == q4.Q4_OK
    for i, row in enumerate(torch.stack(out, 1).tolist()):
        print(f"sequence {i}: {prompts[i].numel()} prompt tokens, then {row[:8]} ...")
    print(f"{a.steps} steps of {a.batch} sequences: {t / a.steps * 1e6:.0f} us each")


if __name__ == "__main__":
    main()

"""The operators together, as the decoding example runs them: a ragged batch of
prompts, then captured steps, against the same decoder in 64 bits (the weights
dequantised, no cache)."""

import os
import sys

import numpy as np
import pytest

from gpu_util import device, torch

import quantized_weight_q4_gb300 as q4

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def plain(m, tokens):
    """Logits of the last token of one sequence, in 64 bits."""
    def weight(B, K, N):
        W = torch.empty(K, N, device=device())
        q4.q4_dequant(W, B, K, N)
        return W.double()

    def norm(x):
        return x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()

    def turn(x):
        n, half = x.shape[0], m.dim // 2
        c, s = m.cos[:n].double()[:, None], m.sin[:n].double()[:, None]
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    h, hk, d = m.heads, m.kv_heads, m.dim
    x = m.embed[tokens.long()].double()
    n = x.shape[0]
    mask = torch.ones(n, n, device=device()).tril().bool()
    for w in m.layers:
        qkv = norm(x) @ weight(w["qkv"], m.hidden, m.qkv_width)
        q = turn(norm(qkv[:, :h * d].unflatten(1, (h, d))))
        k = turn(norm(qkv[:, h * d:(h + hk) * d].unflatten(1, (hk, d))))
        v = qkv[:, (h + hk) * d:].unflatten(1, (hk, d))
        k, v = k.repeat_interleave(h // hk, 1), v.repeat_interleave(h // hk, 1)
        p = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
        p = torch.softmax(p.masked_fill(~mask, -torch.inf), -1)
        x = x + torch.einsum("hij,jhd->ihd", p, v).flatten(1) @ weight(w["out"], h * d, m.hidden)
        y = norm(x)
        g, u = y @ weight(w["gate"], m.hidden, m.inner), y @ weight(w["up"], m.hidden, m.inner)
        x = x + (torch.nn.functional.silu(g) * u) @ weight(w["down"], m.inner, m.hidden)
    return norm(x[-1:]) @ weight(m.head, m.hidden, m.vocab)


def test_prompts_then_steps():
    import decode
    m = decode.Decoder(layers=2, hidden=512, heads=4, kv_heads=2, dim=64, inner=1024, vocab=2048, seqs=3,
                       max_tokens=320, page_tokens=32, seed=3)
    gen = torch.Generator("cuda").manual_seed(4)
    prompts = [torch.randint(0, m.vocab, (n,), generator=gen, device=device(), dtype=torch.int32)
               for n in (1, 150, 47)]
    settings = dict(temperature=torch.tensor([0.0, 0.7, 1.0], device=device()),
                    top_k=torch.tensor([0, 20, 0], dtype=torch.int32, device=device()),
                    top_p=torch.tensor([1.0, 1.0, 0.9], device=device()))
    u = torch.rand(3, generator=gen, device=device())
    tokens, logits = m.prompts(prompts, u, settings)
    texts = list(prompts)

    def check(logits, tokens):
        for b in range(3):
            want = plain(m, texts[b])[0]
            # bf16 activations (2^-9 at each of some ten roundings a layer) and 8-bit keys and values (steps
            # of 1/127 of a block's largest, half a step at most): a few percent
            rel = float((logits[b].double() - want).norm() / want.norm())
            assert rel < 0.05, (b, rel)
        assert int(tokens[0]) == int(logits[0].argmax())
        for b in range(3):
            texts[b] = torch.cat([texts[b], tokens[b:b + 1]])

    check(logits, tokens)
    graph, step_logits = m.capture_step(tokens, u, settings)
    for _ in range(3):
        u.uniform_(generator=gen)
        graph.replay()
        torch.cuda.synchronize()
        check(step_logits, tokens)
    assert m.kv_len.tolist() == [4, 153, 50]
    assert q4.q4_get_device_status() == q4.Q4_OK

"""The decoding example's room: steps that its cache and history do not hold."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("args", [["--steps", "900"], ["--batch", "17"], ["--batch", "0"], ["--steps", "0"],
                                  ["--repetition", "1.2", "--steps", "805"]])
def test_the_command_refuses(args):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decode.py"), *args], capture_output=True, text=True)
    assert r.returncode == 2 and "room for 1024 tokens" in r.stderr


@pytest.mark.gpu
def test_a_full_history():
    """Steps past the history's end store their tokens in its last place, and nowhere else."""
    import decode
    from gpu_util import device, torch

    import quantized_weight_q4_gb300 as q4
    m = decode.Decoder(layers=1, hidden=512, heads=4, kv_heads=2, dim=64, inner=1024, vocab=2048, seqs=2, max_tokens=64,
                       page_tokens=32, seed=3)
    settings = dict(temperature=torch.zeros(2, device=device()))
    u = torch.rand(2, device=device())
    prompts = [torch.arange(n, device=device(), dtype=torch.int32) for n in (5, 3)]
    tokens, _ = m.prompts(prompts, u, settings)
    around = torch.full((4, 8), -1, dtype=torch.int32, device=device())
    history = around[1:3]
    length = torch.tensor([5, 3], dtype=torch.int32, device=device())
    graph, _ = m.capture_step(tokens, u, settings, dict(history=history, history_len=length,
                                                        repetition=torch.full((2,), 1.1, device=device())))
    said = []
    for _ in range(9):
        graph.replay()
        said.append(tokens.clone())
    said = torch.stack(said, 1).tolist()
    assert length.tolist() == [14, 12]
    for row, n, got in zip(history.tolist(), (5, 3), said):
        assert row[n:7] == got[:7 - n] and row[7] == got[-1]
    assert (around[0] == -1).all() and (around[3] == -1).all()
    assert q4.q4_get_device_status() == q4.Q4_OK

"""Calls of a new process that are recorded into a graph before any of them has run: every kernel is met for the first
time inside the capture."""
import subprocess
import sys
from pathlib import Path

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SCRIPT = """
import torch
from kv_cache_attention_ff_gb300 import ff
dev = torch.device("cuda:0")
gen = torch.Generator(device=dev).manual_seed(3)
draw = lambda *s: torch.randn(*s, device=dev, generator=gen).to(torch.bfloat16)
B, H, KV, D, CAP = 2, 4, 2, {d}, 700
inputs = [draw(B, 600, KV, D), draw(B, 600, KV, D)] + [draw(B, n, H, D) for n in (1, 6, 14, 40, 300)]

def state():
    return (ff.KV8Cache(n_layers=2, batch=B, capacity=CAP, heads=H, kv_heads=KV, head_dim=D, max_tokens=300),
            [torch.zeros_like(q) for q in inputs[2:]], torch.zeros(B, KV, CAP, device=dev), torch.zeros(B, KV, CAP, device=dev),
            torch.zeros(B, KV, 200, dtype=torch.int32, device=dev), torch.zeros(B, 200, KV, D, dtype=torch.bfloat16, device=dev),
            torch.zeros(B, 200, KV, D, dtype=torch.bfloat16, device=dev))

def calls(cache, outs, w, w2, kept, k, v):
    cache.append(0, inputs[0], inputs[1])
    for q, out in zip(inputs[2:], outs):
        cache.attn(0, q, out, causal=True, weights=w)
    cache.evict(0, cache, 1, 200, 20, w, w2, kept)
    cache.load(1, k, v)

a, b = state(), state()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls(*a)
graph.replay()
calls(*b)
torch.cuda.synchronize()
assert a[0].error_poll() == 0 and b[0].error_poll() == 0
flat = lambda s: [*s[1], *s[2:], *s[0].layer(1)[2:]]
assert a[0].lengths(1).tolist() == [200, 200] and float(a[2].sum()) > 0
for x, y in zip(flat(a), flat(b)):
    assert torch.equal(x, y)
print("same")
"""


@pytest.mark.parametrize("d", [64, 128])
def test_the_first_calls_are_captured(d):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_attention_ff_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(d=d)], cwd=Path(__file__).resolve().parent.parent,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr

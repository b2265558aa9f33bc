"""A process whose first call of the library is captured into a graph: nothing that a first call sets up may spoil the capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import sys
import torch
from rotation_int4_w4a4_b200 import pq

which, dev = sys.argv[1], "cuda"


def attention(q, n, hq=8, hkv=2, hd=128, page=16):
    pages = -(-n // page) + 1
    tensors = []
    for _ in "kv":
        tensors += [torch.randint(0, 256, (pages, hkv, page, hd // 2), device=dev, dtype=torch.uint8),
                    torch.rand(pages, hkv, page, device=dev) * 0.1 + 0.2]
    cache, Q = pq.KV4Cache(*tensors), torch.randn(q, hq, hd, device=dev).to(torch.bfloat16)
    O, table = torch.zeros_like(Q), torch.randperm(pages, device=dev)[None].to(torch.int32)
    starts, lens = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([0, q], [n]))
    return O, lambda: pq.pq_kv4_attention(cache, Q, O, starts, lens, table, q, n)


def append(T=20, hkv=2, hd=128):
    cache = pq.KV4Cache.empty(4, hkv, 16, hd)
    Q, K = (torch.randn(T, h * hd, device=dev).to(torch.bfloat16) for h in (4 * hkv, hkv))
    out, slots = torch.zeros_like(Q), torch.arange(T, device=dev)
    return out, lambda: pq.pq_kv4_append(cache, Q, K, K, out, None, slots)


def linear(T, N, D=512):
    X = torch.randn(T, D, device=dev).to(torch.bfloat16)
    W, sw = torch.randint(-127, 128, (N, D), dtype=torch.int8, device=dev), torch.rand(N, device=dev)
    codes, sc, Y = torch.empty(T, D, dtype=torch.int8, device=dev), torch.empty(T, device=dev), torch.zeros(T, N, device=dev)
    return Y, lambda: pq.pq_w8a8_linear(X, codes, sc, W, sw, Y, g=128)


out, call = {"one token": lambda: attention(1, 3000), "a chunk": lambda: attention(200, 900), "append": append,
             "linear 1": lambda: linear(1, 100), "linear 600": lambda: linear(600, 9000)}[which]()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
replayed = out.clone()
out.zero_()
call()
assert replayed.abs().sum() > 0 and torch.equal(replayed, out)
pq.pq_check_status()
print("done")
"""


@pytest.mark.parametrize("which", ["one token", "a chunk", "append", "linear 1", "linear 600"])
def test_the_first_call_is_captured(which):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE, which], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stdout + r.stderr

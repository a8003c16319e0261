"""One workspace for calls of different sizes, shapes and kernels: what one call leaves in it must not reach
the next."""
import pytest
import torch

import paged_kv_cache_462_b200 as pkv

pytestmark = pytest.mark.gpu


def decode(ws, S, Hq, Hkv, D, L, block, dtype, seed=0):
    """A dense decode; returns its output (rows it does not write stay 7)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = -(-L // block)
    k, v = (torch.randn(S * nb, Hkv, block, D, generator=g, device="cuda").to(dtype) for _ in range(2))
    t = torch.randperm(S * nb, generator=g, device="cuda").to(torch.int32).reshape(S, nb)
    sl = torch.full((S,), L, dtype=torch.int32, device="cuda")
    q = torch.randn(S, Hq, D, generator=g, device="cuda").to(dtype)
    out = torch.full_like(q, 7.0)
    pkv.paged_attention_decode(out, q, k, v, t, sl, 0.1, workspace=ws)
    return out


F, B = torch.float32, torch.bfloat16
CALLS = [                                  # S, Hq, Hkv, D, L, block, dtype
    (1, 8, 2, 128, 60000, 16, B),          # tensor cores: stamps behind 64 counters, many partials
    (96, 8, 8, 64, 700, 16, F),            # CUDA cores: 768 counters, where those stamps lie
    (700, 8, 8, 64, 41, 16, F),            # 5600 counters, reaching into the partials of few pairs
    (3, 8, 2, 64, 9000, 16, F),
    (96, 16, 8, 128, 300, 8, B),           # CUDA cores, blocks of 8
    (700, 8, 8, 64, 41, 16, F),
    (2, 64, 8, 128, 30000, 16, B),
    (96, 8, 8, 64, 700, 16, F),
]


def test_calls_of_other_sizes_between():
    n = max(pkv.workspace_size(S, Hq, Hkv, D) for S, Hq, Hkv, D, *_ in CALLS)
    want = [decode(torch.zeros(n, dtype=torch.uint8, device="cuda"), *c, seed=i) for i, c in enumerate(CALLS)]
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for i, c in enumerate(CALLS):
            assert torch.equal(decode(ws, *c, seed=i), want[i]), c
    assert pkv.read_device_error(ws) == 0


def test_calls_of_other_sizes_captured():
    """The same in one graph: counters are cleared inside it."""
    S, Hq, Hkv, D, L = 96, 8, 8, 64, 700
    ws = torch.zeros(max(pkv.workspace_size(S, Hq, Hkv, D), pkv.workspace_size(1, 8, 2, 128)), dtype=torch.uint8, device="cuda")
    nb = -(-L // 16)
    k, v = (torch.randn(S * nb, Hkv, 16, D, device="cuda") for _ in range(2))
    t = torch.arange(S * nb, dtype=torch.int32, device="cuda").reshape(S, nb)
    sl = torch.full((S,), L, dtype=torch.int32, device="cuda")
    q = torch.randn(S, Hq, D, device="cuda")
    want, out = torch.empty_like(q), torch.full_like(q, 7.0)
    pkv.paged_attention_decode(want, q, k, v, t, sl, 0.1, workspace=torch.zeros_like(ws))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_attention_decode(out, q, k, v, t, sl, 0.1, workspace=ws)
    for _ in range(3):
        decode(ws, 1, 8, 2, 128, 60000, 16, torch.bfloat16)
        out.fill_(7.0)
        graph.replay()
        assert torch.equal(out, want)

"""Decodes recorded into a CUDA graph: every replay merges its own pieces. (A chunk's completion stamp
is a kernel parameter, so a replay would find the stamps of the replay before; recorded calls must
not go by them.) Sequences are long enough that every stream is split."""
import pytest
import torch

import paged_kv_cache_462_b200 as pkv

pytestmark = pytest.mark.gpu


def batch(kv, seed=0, S=3, Hq=8, Hkv=2, L=6000):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    nb = -(-L // 16)
    shape = (S * nb, Hkv, 16, 128)
    k = torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)
    v = torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)
    if kv == "e4m3":
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
    t = torch.randperm(S * nb, generator=gen, device="cuda").to(torch.int32).reshape(S, nb)
    sl = torch.full((S,), L, dtype=torch.int32, device="cuda")
    qs = [torch.randn(S, Hq, 128, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(12)]
    return k, v, t, sl, qs


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("form", ["plain", "static", "step"])
def test_replays_equal_eager_calls(kv, form):
    k, v, t, sl, qs = batch(kv)
    ws = pkv.new_workspace(3, 8, 2, 128)
    new = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.full((3,), -1, dtype=torch.int64, device="cuda")

    def run(out, q):
        if form == "plain":
            pkv.paged_attention_decode(out, q, k, v, t, sl, 0.4, workspace=ws)
        elif form == "step":
            pkv.paged_decode_step(out, q, k, v, t, sl, new, new, slots, 0.4, workspace=ws)
        else:
            st = pkv.load_library().paged_attention_decode_static(
                out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), t.data_ptr(), sl.data_ptr(), 3, 8, 2, 128, 16,
                0.4, t.shape[1], k.shape[0], pkv.BF16, pkv.BF16 if kv == "bf16" else pkv.FP8_E4M3, 1.0, 1.0, 0,
                torch.cuda.current_stream().cuda_stream)
            assert st == 0

    if form == "static":
        import ctypes
        P, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        pkv.load_library().paged_attention_decode_static.argtypes = [P] * 6 + [i32] * 5 + [f32] + [i32] * 4 + [f32, f32, i32, P]
    want = []
    for q in qs:
        o = torch.empty_like(q)
        run(o, q)
        want.append(o)
    torch.cuda.synchronize()
    q, out = torch.zeros_like(qs[0]), torch.zeros_like(qs[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(out, q)
    for _ in range(4):
        for x, w in zip(qs, want):
            q.copy_(x)
            g.replay()
            assert torch.equal(out, w)

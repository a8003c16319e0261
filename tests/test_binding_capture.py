"""Which workspace a call gets while a stream is being captured: one of the graph's own where the captured stream is
the current one and the call's, and no call otherwise. CPU: a stand-in for the library says which
streams are captured."""
import pytest
import torch

import paged_kv_cache_462_b200 as pkv
from test_binding_threads import SlowLib, Stream, calls, slow  # noqa: F401 (fixture)

OPERATORS = ("select", "sparse", "block_scales")


@pytest.fixture
def lib(slow, monkeypatch):  # noqa: F811
    captured = set()
    monkeypatch.setattr(SlowLib, "pkv_stream_recorded", lambda self, s: int((getattr(s, "value", s) or 0) in captured),
                        raising=False)
    slow.captured = captured
    return slow


def streamed(name, monkeypatch, handle):
    """The call with stream=handle."""
    entry = {"select": "select_blocks", "sparse": "paged_attention_decode_sparse",
             "block_scales": "paged_attention_decode_block_scales", "decode": "paged_attention_decode",
             "step": "paged_decode_step", "mq": "paged_attention_decode_mq",
             "head_scales": "paged_attention_decode_head_scales"}[name]
    real = getattr(pkv, entry)
    monkeypatch.setattr(pkv, entry, lambda *a, **k: real(*a, **k, stream=Stream(handle)))
    return calls()[name]


def launched(lib):
    return [c for c in lib.calls if c[0] in lib.WORKSPACE or c[0] == "pkv_workspace_init"]


@pytest.mark.parametrize("name", OPERATORS)
@pytest.mark.parametrize("captured", [{7}, {0}, {0, 7}])
def test_another_stream_than_the_current_one(lib, monkeypatch, name, captured):
    call = streamed(name, monkeypatch, 7)
    lib.captured |= captured
    with pytest.raises(ValueError, match="pass a workspace"):
        call()
    assert not launched(lib) and not pkv._op_ws


@pytest.mark.parametrize("name", OPERATORS)
def test_the_current_stream(lib, name):
    call = calls()[name]
    lib.captured.add(0)
    call(), call()
    assert not pkv._op_ws                                    # each had its own, and neither is kept
    assert len([c for c in lib.calls if c[0] == "pkv_workspace_init"]) == 2
    lib.captured.clear()
    call(), call()
    assert len(pkv._op_ws) == 1
    assert len([c for c in lib.calls if c[0] == "pkv_workspace_init"]) == 3


@pytest.mark.gpu
def test_a_captured_stream_given_by_argument():
    q = torch.randn(1, 8, 128, device="cuda").to(torch.bfloat16)
    kb = torch.randn(9, 2, 2, 128, device="cuda").to(torch.bfloat16)
    t = torch.arange(9, dtype=torch.int32, device="cuda").reshape(1, 9)
    sl = torch.full((1,), 140, dtype=torch.int32, device="cuda")
    sel, want = (torch.zeros(1, 2, 4, dtype=torch.int32, device="cuda") for _ in range(2))
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    pkv.select_blocks(want, q, kb, t, sl, 16)
    ws = pkv.new_select_workspace(1, 2, 9)
    with torch.cuda.stream(side):                            # a kept workspace for that stream
        pkv.select_blocks(sel, q, kb, t, sl, 16)
    torch.cuda.synchronize()
    sel.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(other):
            with pytest.raises(ValueError, match="pass a workspace"):
                pkv.select_blocks(sel, q, kb, t, sl, 16, stream=side)
            pkv.select_blocks(sel, q, kb, t, sl, 16, workspace=ws, stream=side)
    graph.replay()
    assert torch.equal(sel, want)


DENSE = ("decode", "step", "mq", "head_scales")


@pytest.mark.parametrize("name", DENSE)
@pytest.mark.parametrize("captured", [{7}, {0}])
def test_dense_calls_on_another_stream(lib, monkeypatch, name, captured):
    call = streamed(name, monkeypatch, 7)
    lib.captured |= captured
    with pytest.raises(ValueError, match="pass a workspace"):
        call()
    assert not launched(lib) and not pkv._ws_cache


@pytest.mark.parametrize("name", DENSE)
def test_dense_calls_on_the_current_stream(lib, name):
    call = calls()[name]
    lib.captured.add(0)
    call(), call()
    assert not pkv._ws_cache
    assert len([c for c in lib.calls if c[0] == "pkv_workspace_init"]) == 2
    lib.captured.clear()
    call()
    assert len(pkv._ws_cache) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,Hkv", [(torch.bfloat16, 2), (torch.float32, 16)])
def test_a_dense_decode_captured_without_a_workspace(dtype, Hkv):
    """The first call on the stream is a captured one; then larger eager calls; then replays with other queries."""
    S, Hq, D, L = 6, 16, 128 if dtype == torch.bfloat16 else 64, 2000
    n = -(-L // 16)
    t = torch.randperm(S * n, device="cuda").to(torch.int32).reshape(S, n)
    k, v = (torch.randn(S * n, Hkv, 16, D, device="cuda").to(dtype) for _ in range(2))
    sl = torch.full((S,), L, dtype=torch.int32, device="cuda")
    q = torch.randn(S, Hq, D, device="cuda").to(dtype)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.paged_attention_decode(out, q, k, v, t, sl, 0.1)
    big = [x.repeat(8, *[1] * (x.dim() - 1)) for x in (q, t, sl)]
    for i in range(3):
        q.normal_()
        want, wide = torch.empty_like(q), torch.empty_like(big[0])
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            pkv.paged_attention_decode(wide, big[0], k, v, big[1], big[2], 0.1)
            pkv.paged_attention_decode(want, q, k, v, t, sl, 0.1)
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)

"""Workspaces that the binding makes are ready on the stream that uses them, whichever stream is current. CPU: with
stand-ins for the library and for torch's stream calls, in the order in which they are made."""
import pytest
import torch

import paged_kv_cache_462_b200 as pkv
from test_binding_cpu import Stream, cuda, decode_inputs
from test_binding_threads import run_threads, slow  # noqa: F401 (fixture)


def plan(S=3, MB=4):
    p = pkv.DevicePrefixPlan.__new__(pkv.DevicePrefixPlan)
    z = lambda *s: cuda(torch.zeros(*s, dtype=torch.int32))
    p.num_groups, p.max_group = 1, 2
    p.members, p.offsets, p.tables, p.lens, p.shared = z(2), z(2), z(1, MB), z(1), z(S)
    return p


@pytest.fixture
def order(slow, monkeypatch):  # noqa: F811
    """What is done, in order: C calls by name, torch's stream calls."""
    done, real_empty = [], torch.empty
    slow.done = done
    slow.WORKSPACE = {**slow.WORKSPACE, "paged_attention_decode_shared_prefix": 25, "paged_decode_step_shared_prefix": 25}

    class Using:
        def __init__(self, handle):
            self.handle = handle

        def __enter__(self):
            done.append(("current", self.handle))

        def __exit__(self, *_):
            done.append(("current", 0))

    def empty(n, dtype=None, device=None):
        done.append(("empty",))
        return cuda(real_empty(n, dtype=dtype))
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: h)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: Using(getattr(s, "cuda_stream", s)))
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda dev=None: done.append(("synchronize",)))
    real = type(slow).__getattr__

    def named(self, name):
        f = real(self, name)
        if name == "paged_attention_shared_prefix_workspace_size":
            return lambda *a: 1 << 16

        def call(*a):
            if name == "pkv_workspace_init":
                done.append(("clear", getattr(a[2], "value", a[2]) or 0))
            return f(*a)
        return call
    monkeypatch.setattr(type(slow), "__getattr__", named)
    return slow


def test_shared_prefix_workspaces(order):
    x = decode_inputs(D=128)
    row = cuda(torch.zeros(3, 2, 128, dtype=torch.bfloat16))
    slots = cuda(torch.zeros(3, dtype=torch.int64))
    calls = [lambda **k: pkv.paged_attention_decode_shared_prefix(**x, plan=plan(), scale=0.1, **k),
             lambda **k: pkv.paged_decode_step_shared_prefix(**x, plan=plan(), new_k=row, new_v=row, slot_mapping=slots,
                                                             scale=0.1, **k)]
    for f in calls * 2:
        f(stream=Stream(7))
    assert order.done == [("current", 7), ("empty",), ("current", 0), ("clear", 7)]    # one, kept
    for f in calls:
        f()
    assert [d for d in order.done[4:] if d[0] == "clear"] == [("clear", 0)]
    run_threads(calls * 2, 3)
    assert order.overlaps == 0


@pytest.mark.parametrize("handle", [0, 7])
def test_dense_workspaces(order, handle):
    x = decode_inputs()
    for _ in range(2):
        pkv.paged_attention_decode(**x, scale=0.1, stream=Stream(handle))
    want = [("empty",), ("clear", handle)]
    if handle:                                # memory that the current stream may still be using
        want.insert(1, ("synchronize",))
    assert order.done == want


@pytest.mark.gpu
def test_shared_prefix_on_a_stream_given_by_argument():
    import oracle
    import workloads as W
    from gpu_harness import TOL, GpuStep, max_err
    from paged_kv_cache_462_b200 import blocks
    b = W.config_batch(3, num_seqs=16)
    ref, _, _ = oracle.run_step(b)
    g = GpuStep(b)
    g.append()
    dplan = pkv.DevicePrefixPlan(blocks.prefix_plan(b.block_tables, b.seq_lens, b.spec.block_size, 8), 8)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream, side, None):
        out = torch.full_like(g.q, float("nan"))
        torch.cuda.synchronize()
        pkv.paged_attention_decode_shared_prefix(out, g.q, g.kc, g.vc, g.bt, g.sl, dplan, float(b.scale), stream=stream)
        torch.cuda.synchronize()
        assert max_err(out, ref) <= TOL["bf16"]


@pytest.mark.parametrize("where", ["pkv_workspace_init", "paged_attention_decode_sparse"])
def test_an_interrupted_call_frees_the_workspace(order, monkeypatch, where):
    """Ctrl-C in the library's calls: another thread can use the workspace after it."""
    from test_binding_threads import calls
    real = type(order).__getattr__

    def interrupted(self, name):
        def stop(*a):
            raise KeyboardInterrupt
        return stop if name == where else real(self, name)
    with monkeypatch.context() as m:
        m.setattr(type(order), "__getattr__", interrupted)
        with pytest.raises(KeyboardInterrupt):
            calls()["sparse"]()
    run_threads([calls()["sparse"]] * 2, 2)
    assert len([c for c in order.calls if c[0] == "paged_attention_decode_sparse"]) == 4

"""Two threads on one stream share the workspaces that the binding keeps. A call's two launches hand over
through its workspace, so no other call may be issued between them: on the CPU, with a stand-in for
the library whose calls take a while and see who else is in their workspace."""
import threading
import time

import pytest
import torch

import paged_kv_cache_462_b200 as pkv
from test_binding_cpu import FakeLib, Stream, cuda, decode_inputs


class SlowLib(FakeLib):
    """Calls on the same workspace that overlap in time are counted."""
    WORKSPACE = {"paged_attention_decode": 19, "paged_decode_step": 19, "paged_attention_decode_mq": 20,
                 "paged_attention_decode_head_scales": 19, "select_blocks": 15, "paged_attention_decode_sparse": 23,
                 "paged_attention_decode_block_scales": 19}

    def __init__(self):
        super().__init__()
        self.inside, self.overlaps, self.mutex = {}, 0, threading.Lock()

    def __getattr__(self, name):
        plain = super().__getattr__(name)
        if name not in self.WORKSPACE:
            return (lambda *a: 1 << 16) if name == "pkv_select_workspace_size" else plain

        def call(*args):
            at = args[self.WORKSPACE[name]]
            at = getattr(at, "value", at)
            with self.mutex:
                self.overlaps += self.inside.get(at, 0) > 0
                self.inside[at] = self.inside.get(at, 0) + 1
            time.sleep(0.01)
            with self.mutex:
                self.inside[at] -= 1
            return plain(*args)
        return call


@pytest.fixture
def slow(monkeypatch):
    lib = SlowLib()
    real_empty = torch.empty
    monkeypatch.setattr(pkv, "load_library", lambda: lib)
    monkeypatch.setattr(pkv, "_fast", None)
    monkeypatch.setattr(pkv, "_ws_cache", {})
    monkeypatch.setattr(pkv, "_op_ws", {})
    monkeypatch.setattr(pkv, "_sizes", {})
    monkeypatch.setattr(pkv, "_current_raw_stream", lambda dev: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a, **k: Stream(0))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: threading.Lock())     # any context manager
    monkeypatch.setattr(torch, "empty", lambda n, dtype=None, device=None: cuda(real_empty(n, dtype=dtype)))
    return lib


def calls():
    x = decode_inputs(D=128, kv=torch.uint8)
    S, Hkv = 3, 2
    sel = cuda(torch.zeros(S, Hkv, 2, dtype=torch.int32))
    ones, bs = cuda(torch.ones(Hkv)), cuda(torch.ones(10, Hkv))
    kb = cuda(torch.zeros(10, Hkv, 2, 128, dtype=torch.bfloat16))
    row = cuda(torch.zeros(S, Hkv, 128, dtype=torch.bfloat16))
    slots = cuda(torch.zeros(S, dtype=torch.int64))
    q4 = cuda(torch.zeros(S, 2, 8, 128, dtype=torch.bfloat16))
    rest = {n: x[n] for n in ("k_cache", "v_cache", "block_tables", "seq_lens")}
    return {
        "decode": lambda: pkv.paged_attention_decode(**x, scale=0.1),
        "step": lambda: pkv.paged_decode_step(**x, new_k=row, new_v=row, slot_mapping=slots, scale=0.1),
        "mq": lambda: pkv.paged_attention_decode_mq(q4, q4, **rest, scale=0.1),
        "head_scales": lambda: pkv.paged_attention_decode_head_scales(**x, scale=0.1, k_head_scales=ones, v_head_scales=ones),
        "select": lambda: pkv.select_blocks(sel, x["q"], kb, x["block_tables"], x["seq_lens"], 16),
        "sparse": lambda: pkv.paged_attention_decode_sparse(**x, selected=sel, scale=0.1),
        "block_scales": lambda: pkv.paged_attention_decode_block_scales(**x, scale=0.1, k_block_scales=bs, v_block_scales=bs),
    }


def run_threads(fns, times):
    errors = []

    def body(fn):
        try:
            for _ in range(times):
                fn()
        except BaseException as e:      # noqa: B902 - reported by the test
            errors.append(e)
    threads = [threading.Thread(target=body, args=(f,)) for f in fns]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("name", sorted(calls()))
def test_calls_that_share_a_workspace_are_issued_one_by_one(slow, name):
    run_threads([calls()[name]] * 3, 4)
    assert len([c for c in slow.calls if c[0] in slow.WORKSPACE]) == 12
    assert slow.overlaps == 0


def test_a_call_that_fails_frees_the_workspace(slow):
    slow.status = 5
    for f in calls().values():
        with pytest.raises(pkv.PkvError):
            f()
    slow.status = 0
    run_threads(list(calls().values()), 1)
    assert slow.overlaps == 0


@pytest.mark.gpu
def test_two_threads_on_one_stream():
    """Selection, sparse decode, block-scaled decode and the dense decode without workspaces of their own, from two
    threads on the default stream: each thread finds its own answers."""
    gen = torch.Generator().manual_seed(71)
    S, n = 6, 190
    table = torch.randperm(S * n, generator=gen).to(torch.int32).reshape(S, n).cuda()
    sl = torch.tensor([3000, 700, 1999, 40, 2500, 16], dtype=torch.int32).cuda()
    k, v = (torch.randn(S * n, 2, 16, 128, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    k8, v8 = (torch.randn(S * n, 2, 16, 128, generator=gen).to(torch.float8_e4m3fn).cuda() for _ in range(2))
    scales = torch.ones(S * n, 2, device="cuda")
    kb = torch.stack([k.amax(2), k.amin(2)], 2).contiguous()
    qs = [torch.randn(S, 8, 128, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    torch.cuda.synchronize()

    def run(q):
        sel = torch.empty(S, 2, 24, dtype=torch.int32, device="cuda")
        outs = [torch.empty_like(q) for _ in range(3)]
        pkv.select_blocks(sel, q, kb, table, sl, 16)
        pkv.paged_attention_decode_sparse(outs[0], q, k, v, table, sl, sel, 0.1)
        pkv.paged_attention_decode_block_scales(outs[1], q, k8, v8, table, sl, 0.1, scales, scales)
        pkv.paged_attention_decode(outs[2], q, k, v, table, sl, 0.1)
        return [sel, *outs]

    want = [run(q) for q in qs]
    torch.cuda.synchronize()
    got = [[], []]

    def loop(i):
        return lambda: got[i].append(run(qs[i]))
    run_threads([loop(0), loop(1)], 200)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for x in g:
            assert all(torch.equal(a, b) for a, b in zip(w, x))

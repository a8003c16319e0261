"""Tensors that have no storage of their own or no sizes in numbers (vmap's wrappers, symbolic shapes, fake
tensors) reach the binding's hot path: it declines them, and the checks behind it raise. On the CPU,
with fake tensors that claim a CUDA device, each in a process of its own: an exception that left the C
function would end the process."""
import subprocess
import sys
import textwrap

import pytest

PRELUDE = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import paged_kv_cache_462_b200 as pkv
from paged_kv_cache_462_b200 import build
build.build()
pkv.load_library()
assert pkv._fast is not None
torch.cuda.current_device = lambda: 0
bf = torch.bfloat16

def rest(S):
    t = lambda *s, d=bf: torch.empty(*s, dtype=d, device="cuda")
    return t(S, 2, 128), t(S, 8, 128), t(128), t(128), t(10, 128, d=torch.float32), t(S, d=torch.int64), t(S, 2, 128)

def refused(q, k, qo, qw, kw, cs, pos, ko):
    assert pkv._match("norm", q, k, qo, qw, kw, cs, pos, ko) is None
    try:
        pkv.qk_norm_rope(qo, ko, q, k, qw, kw, 1e-6, cs, pos, stream=0)
    except Exception as e:
        print("raised", type(e).__name__)
    else:
        raise SystemExit("not refused")
"""
CASES = {
    "vmap": """
        with FakeTensorMode():
            other = rest(3)
            def f(x):
                refused(x, *other)
                return x
            torch.vmap(f)(torch.empty(5, 3, 8, 128, dtype=bf, device="cuda"))
    """,
    "symbolic": """
        from torch.fx.experimental.symbolic_shapes import ShapeEnv
        mode = FakeTensorMode(shape_env=ShapeEnv())
        q = mode.from_tensor(torch.empty(3, 8, 128, dtype=bf))
        with mode:
            q = q.cuda()
            assert isinstance(q.shape[0], torch.SymInt)
            refused(q, *rest(3))
    """,
    "fake": """
        with FakeTensorMode():
            refused(torch.empty(3, 8, 128, dtype=bf, device="cuda"), *rest(3))
    """,
}


@pytest.mark.parametrize("case", sorted(CASES))
def test_declined_not_aborted(case):
    r = subprocess.run([sys.executable, "-c", PRELUDE + textwrap.dedent(CASES[case])], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout[-500:], r.stderr[-1500:])
    assert "raised" in r.stdout

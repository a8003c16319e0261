"""The error words of the workspaces that the binding keeps can be read and cleared."""
import pytest
import torch

import paged_kv_cache_462_b200 as pkv
from test_binding_cpu import Stream
from test_binding_threads import SlowLib, calls, slow  # noqa: F401 (fixture)


@pytest.fixture
def lib(slow, monkeypatch):  # noqa: F811
    slow.words, slow.inits = {}, []

    def read(self, ws, n, out, clear, stream):
        out._obj.value = self.words.get(ws.value, 0)
        if clear:
            self.words[ws.value] = 0
        return 0

    def init(self, ws, n, stream):
        self.inits.append((getattr(ws, "value", ws), n))
        return 0
    monkeypatch.setattr(SlowLib, "pkv_read_device_error", read, raising=False)
    monkeypatch.setattr(SlowLib, "pkv_workspace_init", init, raising=False)
    return slow


def test_words_of_the_kept_workspaces(lib, monkeypatch):
    assert pkv.read_device_error() == 0
    for name in ("select", "sparse", "decode"):
        calls()[name]()
    kept = {kind: pkv._op_ws[(kind, 0, 0)].tensor for kind in ("select", "decode")}
    dense = next(iter(pkv._ws_cache.values())).tensor
    lib.words = {kept["select"].data_ptr(): pkv.DEVERR_BLOCK_ID, kept["decode"].data_ptr(): pkv.DEVERR_SELECTION,
                 dense.data_ptr(): pkv.DEVERR_SEQ_LEN}
    want = pkv.DEVERR_BLOCK_ID | pkv.DEVERR_SELECTION | pkv.DEVERR_SEQ_LEN
    assert pkv.read_device_error() == want
    assert pkv.read_device_error(stream=Stream(9)) == 0           # another stream's
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert pkv.read_device_error() == 0
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert pkv.read_device_error(clear=True) == want
    assert pkv.read_device_error() == 0


def test_a_timeout_initialises_the_workspace(lib):
    calls()["sparse"]()
    ws = pkv._op_ws[("decode", 0, 0)].tensor
    lib.words[ws.data_ptr()] = pkv.DEVERR_TIMEOUT
    lib.inits.clear()
    assert pkv.read_device_error() == pkv.DEVERR_TIMEOUT and not lib.inits
    assert pkv.read_device_error(clear=True) == pkv.DEVERR_TIMEOUT
    assert lib.inits == [(ws.data_ptr(), ws.numel())]


@pytest.mark.gpu
def test_errors_of_calls_without_a_workspace():
    q = torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16)
    k = torch.randn(20, 2, 16, 128, device="cuda").to(torch.bfloat16)
    kb = torch.stack([k.amax(2), k.amin(2)], 2).contiguous()
    t = torch.arange(18, dtype=torch.int32, device="cuda").reshape(2, 9)
    t[1, 4] = 99
    sl = torch.tensor([140, 144], dtype=torch.int32, device="cuda")
    sel = torch.zeros(2, 2, 4, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert pkv.read_device_error(clear=True) == 0
        pkv.select_blocks(sel, q, kb, t, sl, 16)
        assert pkv.read_device_error(clear=True) == pkv.DEVERR_BLOCK_ID
        sel.fill_(9)
        pkv.paged_attention_decode_sparse(out, q, k, k, t, sl, sel, 0.1)
        assert pkv.read_device_error(clear=True) == pkv.DEVERR_SELECTION
        pkv.paged_attention_decode(out, q, k, k, t, sl, 0.1)
        assert pkv.read_device_error() == pkv.DEVERR_BLOCK_ID
        sel.fill_(0)
        pkv.paged_attention_decode_sparse(out, q, k, k, t, sl, sel, 0.1)
        assert pkv.read_device_error(clear=True) == pkv.DEVERR_BLOCK_ID     # still the decode's
        assert pkv.read_device_error() == 0
    torch.cuda.synchronize()

"""Host checks of the operators around the cache, on the CPU: the C ABI refuses bad arguments before
any device access, and the binding refuses tensors it cannot pass on."""
import ctypes

import pytest
import torch

import paged_kv_cache_462_b200 as pkv
from test_binding_cpu import FakeLib, cuda

P = 0x100000        # never dereferenced: the calls below fail a host check first, or have nothing to do
FAR = 0x40000000
NULL, SHAPE, DTYPE, WS, DEVICE = 1, 2, 3, 4, 6


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_462_b200 import build
    build.build()
    return pkv.load_library()


def norm_rope(lib, cached, **kw):
    a = dict(qo=FAR, ko=2 * FAR, q=P, k=3 * FAR, v=4 * FAR, qw=P, kw=P, eps=1e-6, cs=P, pos=P, kc=P, vc=P, sl=P, T=4,
             Hq=8, Hkv=2, D=128, R=128, NP=64, BS=16, NB=8, il=0, qs=1024, ks=256, vs=256, dt=1, kv=1, sk=1.0, sv=1.0)
    a.update(kw)
    if cached:
        return lib.qk_norm_rope_and_cache(a["qo"], a["q"], a["k"], a["v"], a["qw"], a["kw"], a["eps"], a["cs"],
                                          a["pos"], a["kc"], a["vc"], a["sl"], a["T"], a["Hq"], a["Hkv"], a["D"],
                                          a["R"], a["NP"], a["BS"], a["NB"], a["il"], a["qs"], a["ks"], a["vs"],
                                          a["dt"], a["kv"], a["sk"], a["sv"], None, None)
    return lib.qk_norm_rope(a["qo"], a["ko"], a["q"], a["k"], a["qw"], a["kw"], a["eps"], a["cs"], a["pos"], a["T"],
                            a["Hq"], a["Hkv"], a["D"], a["R"], a["NP"], a["il"], a["qs"], a["ks"], a["dt"], None, None)


@pytest.mark.parametrize("cached", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), SHAPE), (dict(Hq=0), SHAPE), (dict(D=96), SHAPE), (dict(R=4), SHAPE), (dict(R=136), SHAPE),
    (dict(R=-8), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(dt=2, kv=2), DTYPE),
    (dict(q=None), NULL), (dict(cs=None), NULL), (dict(qw=None), NULL), (dict(q=P + 8), SHAPE), (dict(qs=1020), SHAPE),
    (dict(ks=250), SHAPE), (dict(ks=128), SHAPE), (dict(T=0, q=None), 0),
    # q_out on top of q's rows, but not row by row the same
    (dict(qo=P + 2048), SHAPE), (dict(qo=P, qs=2048), SHAPE), (dict(qo=3 * FAR), SHAPE)])
def test_norm_rope_refusals(lib, cached, kw, want):
    assert norm_rope(lib, cached, **kw) == want


def test_norm_rope_refusals_of_one_form(lib):
    assert norm_rope(lib, False, ko=None) == NULL
    assert norm_rope(lib, False, ko=FAR) == SHAPE            # both outputs in one place
    assert norm_rope(lib, False, ko=P) == SHAPE              # k_out over q
    assert norm_rope(lib, True, v=None) == NULL
    assert norm_rope(lib, True, sl=None) == NULL
    assert norm_rope(lib, True, BS=12) == SHAPE
    assert norm_rope(lib, True, NB=0) == SHAPE
    assert norm_rope(lib, True, kv=0) == DTYPE               # bf16 rows, f32 cache
    assert norm_rope(lib, True, kv=2, sk=0.0) == SHAPE
    assert norm_rope(lib, True, kv=4, sv=-1.0) == SHAPE
    assert norm_rope(lib, True, vs=100) == SHAPE
    assert norm_rope(lib, True, qo=4 * FAR) == SHAPE         # over v


def append(lib, **kw):
    a = dict(k=P, v=P, kc=P, vc=P, ks=P, vs=P, bt=P, sl=P, ro=P, T=4, S=2, Hkv=2, D=128, BS=16, MB=4, NB=8, st=256,
             sv=256, dt=1, kv=2)
    a.update(kw)
    return lib.reshape_and_cache_block_scales(a["k"], a["v"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["sl"],
                                              a["ro"], a["T"], a["S"], a["Hkv"], a["D"], a["BS"], a["MB"], a["NB"],
                                              a["st"], a["sv"], a["dt"], a["kv"], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), SHAPE), (dict(S=-1), SHAPE), (dict(S=20000), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=80), SHAPE),
    (dict(BS=4), SHAPE), (dict(MB=0), SHAPE), (dict(NB=0), SHAPE), (dict(kv=1), DTYPE), (dict(kv=0, dt=0), DTYPE),
    (dict(dt=2), DTYPE), (dict(k=None), NULL), (dict(ks=None), NULL), (dict(ro=None), NULL), (dict(k=P + 4), SHAPE),
    (dict(st=100), SHAPE), (dict(sv=257), SHAPE), (dict(MB=1 << 28), SHAPE), (dict(T=0, k=None), 0),
    (dict(S=0, ro=None), 0)])
def test_append_refusals(lib, kw, want):
    assert append(lib, **kw) == want


def decode(lib, sparse, **kw):
    a = dict(o=P, q=P, kc=P, vc=P, bt=P, sl=P, sel=P, S=2, Hq=8, Hkv=2, D=128, BS=16, MB=4, NB=8, W=3, qd=1, kv=2,
             ks=1.0, vs=1.0, kb=P, vb=P, parts=8, ws=P, wsb=1 << 30)
    a.update(kw)
    if sparse:
        return lib.paged_attention_decode_sparse(a["o"], a["q"], a["kc"], a["vc"], a["bt"], a["sl"], a["sel"], a["S"],
                                                 a["Hq"], a["Hkv"], a["D"], a["BS"], 0.1, a["MB"], a["NB"], a["W"],
                                                 a["qd"], a["kv"], a["ks"], a["vs"], a["kb"], a["vb"], a["parts"],
                                                 a["ws"], a["wsb"], None)
    return lib.paged_attention_decode_block_scales(a["o"], a["q"], a["kc"], a["vc"], a["bt"], a["sl"], a["S"], a["Hq"],
                                                   a["Hkv"], a["D"], a["BS"], 0.1, a["MB"], a["NB"], a["qd"], a["kv"],
                                                   a["kb"], a["vb"], a["parts"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(S=-1), SHAPE), (dict(Hq=6, Hkv=2), SHAPE), (dict(Hq=7), SHAPE), (dict(D=64), SHAPE), (dict(BS=8), SHAPE),
    (dict(qd=0), DTYPE), (dict(kv=0), DTYPE), (dict(parts=-1), SHAPE), (dict(o=None), NULL), (dict(sl=None), NULL),
    (dict(kc=P + 8), SHAPE), (dict(q=P + 8), SHAPE), (dict(ws=None), WS), (dict(wsb=1024), WS), (dict(MB=0), SHAPE), (dict(NB=0), SHAPE),
    (dict(vb=None), NULL), (dict(S=0, o=None), 0)])
def test_decode_refusals(lib, sparse, kw, want):
    assert decode(lib, sparse, **kw) == want


def test_decode_refusals_of_one_form(lib):
    assert decode(lib, False, kv=1) == DTYPE                       # block scales need an 8-bit cache
    assert decode(lib, True, kv=1) == DTYPE
    assert decode(lib, False, kb=None) == NULL
    assert decode(lib, True, W=0) == SHAPE
    assert decode(lib, True, sel=None) == NULL
    assert decode(lib, True, W=1 << 30) == SHAPE
    assert decode(lib, True, kb=None, vb=None, ks=0.0) == SHAPE    # per-tensor scales must be positive


def bounds(lib, **kw):
    a = dict(b=P, kc=P, bt=P, sl=P, ro=P, T=4, S=2, Hkv=2, D=128, BS=16, MB=4, NB=8, kv=1, ks=1.0, kb=None)
    a.update(kw)
    return lib.update_key_bounds(a["b"], a["kc"], a["bt"], a["sl"], a["ro"], a["T"], a["S"], a["Hkv"], a["D"],
                                 a["BS"], a["MB"], a["NB"], a["kv"], a["ks"], a["kb"], None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=32), SHAPE), (dict(BS=64), SHAPE), (dict(kv=0), DTYPE),
    (dict(kv=1, kb=P), DTYPE), (dict(kv=2, ks=0.0), SHAPE), (dict(b=None), NULL), (dict(ro=None), NULL),
    (dict(b=P + 2), SHAPE), (dict(kc=P + 2), SHAPE), (dict(T=0, b=None), 0)])
def test_bounds_refusals(lib, kw, want):
    assert bounds(lib, **kw) == want


def select(lib, **kw):
    a = dict(o=P, q=P, b=P, bt=P, sl=P, S=2, Hq=8, Hkv=2, D=128, BS=16, MB=9, NB=8, W=4, sink=1, rec=1, ws=P,
             wsb=1 << 30)
    a.update(kw)
    return lib.select_blocks(a["o"], a["q"], a["b"], a["bt"], a["sl"], a["S"], a["Hq"], a["Hkv"], a["D"], a["BS"],
                             a["MB"], a["NB"], a["W"], a["sink"], a["rec"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(S=-1), SHAPE), (dict(Hq=6), SHAPE), (dict(Hq=9), SHAPE), (dict(D=256), SHAPE), (dict(BS=5), SHAPE),
    (dict(MB=0), SHAPE), (dict(NB=0), SHAPE), (dict(W=0), SHAPE), (dict(sink=-1), SHAPE), (dict(rec=-1), SHAPE),
    (dict(sink=3, rec=2), SHAPE), (dict(S=16385), SHAPE), (dict(NB=1 << 30), SHAPE), (dict(o=None), NULL), (dict(b=None), NULL),
    (dict(ws=None), WS), (dict(wsb=512), WS), (dict(q=P + 2), SHAPE), (dict(S=0, o=None), 0)])
def test_select_refusals(lib, kw, want):
    assert select(lib, **kw) == want


def test_select_workspace_size(lib):
    one = lib.pkv_select_workspace_size(1, 1, 1)
    assert one >= 256
    assert lib.pkv_select_workspace_size(64, 8, 2048) >= one + 64 * 8 * 2048 * 16
    for bad in ((-1, 8, 4), (4, 0, 4), (4, 8, 0), (20000, 1, 4), (16384, 16, 1 << 20)):
        assert lib.pkv_select_workspace_size(*bad) == 0
    with pytest.raises(pkv.PkvError):
        pkv.select_workspace_size(4, 0, 4)


# ------------------------------------------------------------------ the binding

@pytest.fixture
def fake(monkeypatch):
    f = FakeLib()
    monkeypatch.setattr(pkv, "load_library", lambda: f)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(pkv, "_current_raw_stream", lambda dev: 7)
    return f


def bf(*shape):
    return cuda(torch.zeros(*shape, dtype=torch.bfloat16))


def rope_inputs():
    return dict(q_out=bf(3, 8, 64), q=bf(3, 8, 64), k=bf(3, 2, 64), v=bf(3, 2, 64), q_weight=bf(64), k_weight=bf(64),
                eps=1e-6, cos_sin=cuda(torch.zeros(10, 32)), positions=cuda(torch.zeros(3, dtype=torch.int64)),
                k_cache=bf(4, 2, 16, 64), v_cache=bf(4, 2, 16, 64),
                slot_mapping=cuda(torch.zeros(3, dtype=torch.int64)))


def test_norm_rope_argument_order(fake):
    x = rope_inputs()
    qkv = torch.zeros(3, 12 * 64, dtype=torch.bfloat16)
    x["q"], x["k"], x["v"] = (cuda(t.unflatten(1, (-1, 64))) for t in qkv.split([512, 128, 128], 1))
    pkv.qk_norm_rope_and_cache(**x, interleaved=True, k_scale=2.0, v_scale=3.0)
    name, a = fake.calls[-1]
    assert name == "qk_norm_rope_and_cache"
    assert a[1] == x["q"].data_ptr() and a[3] == x["v"].data_ptr() and a[-1] == 7
    assert a[12:21] == (3, 8, 2, 64, 32, 10, 16, 4, 1)
    assert a[21:24] == (768, 768, 768)                    # the projection's row, in elements
    assert a[24:28] == (pkv.BF16, pkv.BF16, 2.0, 3.0)


@pytest.mark.parametrize("name,bad,err", [
    ("q", torch.zeros(3, 8, 64, dtype=torch.bfloat16), ValueError),           # on the host
    ("q_out", bf(3, 4, 64), ValueError), ("k", bf(4, 2, 64), ValueError), ("k", bf(3, 2, 128), ValueError),
    ("v", bf(3, 1, 64), ValueError), ("q_weight", bf(128), ValueError),
    ("k_weight", cuda(torch.zeros(64)), TypeError), ("cos_sin", bf(10, 32), TypeError),
    ("positions", cuda(torch.zeros(3, dtype=torch.int32)), TypeError),
    ("slot_mapping", cuda(torch.zeros(2, dtype=torch.int64)), TypeError), ("k_cache", bf(4, 2, 16, 128), ValueError),
    ("v_cache", cuda(torch.zeros(4, 2, 16, 64)), TypeError), ("v_cache", bf(5, 2, 16, 64), ValueError),
    ("k", cuda(torch.zeros(3, 2, 128, dtype=torch.bfloat16)[:, :, ::2]), ValueError),
    ("v", cuda(torch.zeros(3, 64, 2, dtype=torch.bfloat16).transpose(1, 2)), ValueError),
    ("k", cuda(torch.zeros(1, 2, 64, dtype=torch.bfloat16).expand(3, 2, 64)), ValueError)])
def test_norm_rope_binding_refusals(fake, name, bad, err):
    x = rope_inputs()
    x[name] = bad
    with pytest.raises(err):
        pkv.qk_norm_rope_and_cache(**x)
    assert not fake.calls


def i32(*shape):
    return cuda(torch.zeros(*shape, dtype=torch.int32))


def u8(*shape):
    return cuda(torch.zeros(*shape, dtype=torch.uint8))


def test_append_binding(fake):
    x = dict(k=bf(5, 2, 128), v=bf(5, 2, 128), k_cache=u8(4, 2, 16, 128), v_cache=u8(4, 2, 16, 128),
             k_block_scales=cuda(torch.ones(4, 2)), v_block_scales=cuda(torch.ones(4, 2)), block_tables=i32(3, 6),
             seq_lens=i32(3), row_offsets=i32(4))
    pkv.reshape_and_cache_block_scales(**x)
    name, a = fake.calls.pop()
    assert name == "reshape_and_cache_block_scales"
    assert a[9:20] == (5, 3, 2, 128, 16, 6, 4, 256, 256, pkv.BF16, pkv.FP8_E4M3)
    for key, bad, err in [("row_offsets", i32(3), TypeError), ("k_block_scales", cuda(torch.ones(4, 1)), TypeError),
                          ("v_block_scales", cuda(torch.ones(4, 2, dtype=torch.float64)), TypeError),
                          ("seq_lens", i32(2), ValueError), ("v", bf(4, 2, 128), ValueError),
                          ("v_cache", cuda(torch.zeros(4, 2, 16, 128, dtype=torch.int8)), TypeError),
                          ("block_tables", cuda(torch.zeros(3, 6, dtype=torch.int64)), TypeError)]:
        with pytest.raises(err):
            pkv.reshape_and_cache_block_scales(**{**x, key: bad})
    assert not fake.calls


def test_decode_bindings(fake):
    x = dict(out=bf(3, 8, 128), q=bf(3, 8, 128), k_cache=u8(4, 2, 16, 128), v_cache=u8(4, 2, 16, 128),
             block_tables=i32(3, 6), seq_lens=i32(3), scale=0.5, workspace=u8(1 << 16))
    ks, vs = cuda(torch.ones(4, 2)), cuda(torch.ones(4, 2))
    pkv.paged_attention_decode_block_scales(**x, k_block_scales=ks, v_block_scales=vs, num_partitions=7)
    name, a = fake.calls.pop()
    assert a[6:16] == (3, 8, 2, 128, 16, 0.5, 6, 4, pkv.BF16, pkv.FP8_E4M3) and a[18] == 7
    assert (a[16], a[17]) == (ks.data_ptr(), vs.data_ptr())
    pkv.paged_attention_decode_sparse(**x, selected=i32(3, 2, 5), k_scale=2.0, v_scale=3.0)
    name, a = fake.calls.pop()
    assert a[7:20] == (3, 8, 2, 128, 16, 0.5, 6, 4, 5, pkv.BF16, pkv.FP8_E4M3, 2.0, 3.0)
    assert a[20] is None and a[21] is None
    for bad in (dict(selected=i32(3, 4, 5)), dict(selected=cuda(torch.zeros(3, 2, 5, dtype=torch.int64)))):
        with pytest.raises(TypeError):
            pkv.paged_attention_decode_sparse(**x, **bad)
    with pytest.raises(ValueError):
        pkv.paged_attention_decode_sparse(**x, selected=i32(3, 2, 5), k_block_scales=ks)
    with pytest.raises(TypeError):
        pkv.paged_attention_decode_block_scales(**x, k_block_scales=ks, v_block_scales=cuda(torch.ones(2, 4)))
    assert not fake.calls


def test_select_bindings(fake):
    kb = bf(4, 2, 2, 128)
    pkv.update_key_bounds(kb, bf(4, 2, 16, 128), i32(3, 6), i32(3), i32(4), 9)
    name, a = fake.calls.pop()
    assert a[5:14] == (9, 3, 2, 128, 16, 6, 4, pkv.BF16, 1.0) and a[14] is None
    with pytest.raises(TypeError):
        pkv.update_key_bounds(bf(4, 2, 128, 2), bf(4, 2, 16, 128), i32(3, 6), i32(3), i32(4), 9)
    x = dict(selected=i32(3, 2, 5), q=bf(3, 8, 128), key_bounds=kb, block_tables=i32(3, 6), seq_lens=i32(3),
             block_size=16, workspace=u8(1 << 16))
    pkv.select_blocks(**x, num_sink_blocks=2)
    name, a = fake.calls.pop()
    assert name == "select_blocks" and a[5:15] == (3, 8, 2, 128, 16, 6, 4, 5, 2, 1)
    for bad in (dict(q=cuda(torch.zeros(3, 8, 128))), dict(selected=i32(3, 1, 5)), dict(seq_lens=i32(3, 1))):
        with pytest.raises((TypeError, ValueError)):
            pkv.select_blocks(**{**x, **bad})
    assert not fake.calls


def test_tensors_on_another_device_are_refused(fake):
    far = lambda *shape, dtype=torch.bfloat16: cuda(torch.zeros(*shape, dtype=dtype), 1)
    x = rope_inputs()
    for name, bad in (("q", far(3, 8, 64)), ("v", far(3, 2, 64)), ("cos_sin", far(10, 32, dtype=torch.float32)),
                      ("v_cache", far(4, 2, 16, 64)), ("q_out", far(3, 8, 64))):
        with pytest.raises(ValueError):
            pkv.qk_norm_rope_and_cache(**{**x, name: bad})
    sel = dict(selected=i32(3, 2, 5), q=bf(3, 8, 128), key_bounds=bf(4, 2, 2, 128), block_tables=i32(3, 6), seq_lens=i32(3),
               block_size=16, workspace=u8(1 << 16))
    for name, bad in (("key_bounds", far(4, 2, 2, 128)), ("workspace", far(1 << 16, dtype=torch.uint8)),
                      ("selected", far(3, 2, 5, dtype=torch.int32))):
        with pytest.raises(ValueError):
            pkv.select_blocks(**{**sel, name: bad})
    assert not fake.calls


def test_views_that_are_not_contiguous_are_refused(fake):
    x = rope_inputs()
    with pytest.raises(ValueError):
        pkv.qk_norm_rope_and_cache(**{**x, "q_out": cuda(torch.zeros(3, 8, 128, dtype=torch.bfloat16)[:, :, ::2])})
    with pytest.raises(ValueError):
        pkv.qk_norm_rope_and_cache(**{**x, "k_cache": cuda(torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16).transpose(1, 2))})
    with pytest.raises(ValueError):
        pkv.update_key_bounds(bf(4, 2, 2, 128), bf(4, 2, 16, 128), cuda(torch.zeros(3, 12, dtype=torch.int32)[:, ::2]),
                              i32(3), i32(4), 9)
    assert not fake.calls

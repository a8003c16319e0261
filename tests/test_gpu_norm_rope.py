"""qk_norm_rope and qk_norm_rope_and_cache against the formulas in 64 bits.

Tolerances: an output is rounded once (bf16: half a step is 2^-8 of the value, fp32: 2^-24); before
that the fp32 work is a sum of head_dim squares, a reciprocal square root, three products and a
two-term rotation, each within a few 2^-24 of the row's size: 3e-6 of the largest element of the
pair covers it (a sum of 128 terms in a tree, 2^-24 * (7 + ~10))."""
import pytest
import torch

import paged_kv_cache_462_b200 as pkv
import plain_serving as plain

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
FP32 = 3e-6


def table(rows, rotary, gen):
    ang = torch.rand(rows, rotary // 2, generator=gen, dtype=torch.float64) * 6.28
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def inputs(T, Hq, Hkv, D, R, kind, seed=0, strided=True, positions=40):
    gen = torch.Generator().manual_seed(seed)
    width = (Hq + 2 * Hkv) * D + (16 if strided else 0)
    qkv = (torch.randn(T, width, generator=gen) * torch.exp(torch.randn(T, 1, generator=gen))).to(DT[kind])
    parts = qkv[:, :(Hq + 2 * Hkv) * D].split([Hq * D, Hkv * D, Hkv * D], 1)
    w = [(1 + 0.3 * torch.randn(D, generator=gen)).to(DT[kind]) for _ in range(2)]
    pos = torch.randint(0, positions, (T,), generator=gen)
    dev = qkv.cuda()
    dparts = dev[:, :(Hq + 2 * Hkv) * D].split([Hq * D, Hkv * D, Hkv * D], 1)
    unf = lambda ps: [p.unflatten(1, (-1, D)) for p in ps]
    return unf(parts), unf(dparts), w, table(positions, R, gen), pos


def close(got, want, kind, what):
    got = got.cpu().double()
    row = want.abs().amax(-1, keepdim=True)
    err = (got - want).abs() - HALF[kind] * want.abs() - FP32 * row
    assert float(err.max()) <= 0, (what, float((got - want).abs().max()), float(err.max()))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,il", [
    (1, 32, 8, 128, 128, False), (3, 40, 8, 128, 128, True), (65, 8, 2, 64, 64, False), (7, 5, 1, 128, 64, False),
    (130, 1, 1, 64, 32, True), (5, 3, 2, 128, 8, False), (4, 3, 2, 128, 8, True), (6, 2, 1, 64, 0, False),
    (33, 16, 16, 128, 24, False), (257, 4, 1, 64, 56, False), (2, 7, 7, 128, 120, True)])
def test_norm_rope(kind, T, Hq, Hkv, D, R, il):
    (q, k, _), (dq, dk, _), (qw, kw), cs, pos = inputs(T, Hq, Hkv, D, R, kind)
    qo, ko = torch.empty(T, Hq, D, dtype=DT[kind], device="cuda"), torch.empty(T, Hkv, D, dtype=DT[kind], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.qk_norm_rope(qo, ko, dq, dk, qw.cuda(), kw.cuda(), 1e-6, cs.cuda(), pos.cuda(), il, err)
    close(qo, plain.norm_rope(q, qw, 1e-6, cs, pos, il), kind, "q")
    close(ko, plain.norm_rope(k, kw, 1e-6, cs, pos, il), kind, "k")
    assert err.item() == 0


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,il", [(9001, 3, 1, 64, 64, False), (15000, 1, 1, 128, 64, True), (2501, 40, 8, 128, 128, False),
                                             (1800, 70, 9, 64, 64, False), (3333, 5, 3, 128, 128, False)])
def test_many_tokens(kind, T, Hq, Hkv, D, R, il):
    """CTAs that take several sets of tokens, sets of several tokens, more rows than one pass holds."""
    (q, k, v), (dq, dk, dv), (qw, kw), cs, pos = inputs(T, Hq, Hkv, D, R, kind, seed=8)
    NB = T // 16 + 2
    slots = torch.randperm(NB * 16, generator=torch.Generator().manual_seed(2))[:T]
    slots[T // 2] = -1
    kc = torch.zeros(NB, Hkv, 16, D, dtype=DT[kind], device="cuda")
    vc = torch.zeros_like(kc)
    qo, q2 = (torch.empty(T, Hq, D, dtype=DT[kind], device="cuda") for _ in range(2))
    ko = torch.empty(T, Hkv, D, dtype=DT[kind], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (qw.cuda(), kw.cuda(), 1e-6, cs.cuda(), pos.cuda())
    pkv.qk_norm_rope(qo, ko, dq, dk, *args, il, err)
    pkv.qk_norm_rope_and_cache(q2, dq, dk, dv, *args, kc, vc, slots.cuda(), il, device_error=err)
    close(qo, plain.norm_rope(q, qw, 1e-6, cs, pos, il), kind, "q")
    close(ko, plain.norm_rope(k, kw, 1e-6, cs, pos, il), kind, "k")
    assert torch.equal(qo, q2) and err.item() == 0
    ok = slots >= 0
    at = slots[ok].cuda()
    assert torch.equal(kc[at // 16, :, at % 16], ko[ok.cuda()])
    assert torch.equal(vc[at // 16, :, at % 16], dv[ok.cuda()])


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "e4m3"),
                                        ("bf16", "e5m2"), ("bf16", "int8"), ("f32", "int8")])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,BS,il", [(9, 8, 2, 128, 128, 16, False), (50, 5, 1, 64, 32, 8, True),
                                               (1, 32, 8, 128, 64, 32, False)])
def test_norm_rope_and_cache(kind, cache, T, Hq, Hkv, D, R, BS, il):
    (q, k, v), (dq, dk, dv), (qw, kw), cs, pos = inputs(T, Hq, Hkv, D, R, kind, seed=3)
    gen = torch.Generator().manual_seed(5)
    NB = T // BS + 3
    slots = torch.randperm(NB * BS, generator=gen)[:T]
    if T > 8:
        slots[4] = -1
        slots[7] = NB * BS + 3            # beyond the pool: flagged, not written
    dt = plain.CODE.get(cache, DT[kind])
    kc = torch.zeros(NB, Hkv, BS, D, dtype=dt, device="cuda")
    vc, vref, kref = torch.zeros_like(kc), torch.zeros_like(kc), torch.zeros_like(kc)
    ks, vs = (0.03, 0.02) if cache in plain.CODE else (1.0, 1.0)
    qo = torch.empty(T, Hq, D, dtype=DT[kind], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.qk_norm_rope_and_cache(qo, dq, dk, dv, qw.cuda(), kw.cuda(), 1e-5, cs.cuda(), pos.cuda(), kc, vc, slots.cuda(),
                               il, ks, vs, err)
    assert err.item() == (pkv.DEVERR_SLOT if T > 8 else 0)
    close(qo, plain.norm_rope(q, qw, 1e-5, cs, pos, il), kind, "q")      # padding rows too
    # V: the append that the library has, bit for bit
    pkv.reshape_and_cache(dv.contiguous(), dv.contiguous(), kref, vref, slots.cuda(), vs, vs)
    assert torch.equal(vc.view(torch.uint8), vref.view(torch.uint8))
    want = plain.norm_rope(k, kw, 1e-5, cs, pos, il)
    got = torch.zeros(T, Hkv, D, dtype=torch.float64)
    ok = (slots >= 0) & (slots < NB * BS)
    flat = kc.cpu().float().double()
    got[ok] = flat[slots[ok] // BS, :, slots[ok] % BS]
    want = want[ok] / float(torch.tensor(ks, dtype=torch.float32))
    if cache in plain.CODE:
        y = want.clamp(-plain.QMAX[cache], plain.QMAX[cache])
        room = plain.half_step(y, cache) + 2 * FP32 * want.abs().amax(-1, keepdim=True)
        assert float(((got[ok] - y).abs() - room).max()) <= 0
    else:
        close(got[ok], want, kind, "k")
    written = torch.zeros(NB * BS, dtype=torch.bool)
    written[slots[ok]] = True
    rest = flat.permute(0, 2, 1, 3).reshape(NB * BS, -1)[~written]
    assert not rest.any()                                                  # nothing else in the pool


def test_in_place_and_bad_positions():
    (q, k, _), _, (qw, kw), cs, pos = inputs(6, 8, 2, 128, 128, "bf16", seed=9, strided=False)
    dq, dk = q.contiguous().cuda(), k.contiguous().cuda()
    pos[2], pos[4] = -1, 40
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.qk_norm_rope(dq, dk, dq, dk, qw.cuda(), kw.cuda(), 1e-6, cs.cuda(), pos.cuda(), False, err)
    assert err.item() == pkv.DEVERR_POSITION
    good = (pos >= 0) & (pos < 40)
    p = pos.clamp(0, 39)
    close(dq[good], plain.norm_rope(q, qw, 1e-6, cs, p, False)[good], "bf16", "q")
    close(dk[good], plain.norm_rope(k, kw, 1e-6, cs, p, False)[good], "bf16", "k")
    assert torch.equal(dq.cpu()[~good], q[~good]) and torch.equal(dk.cpu()[~good], k[~good])   # left as they were


def test_overlaps_are_refused():
    (_, _, _), (dq, dk, dv), (qw, kw), cs, pos = inputs(6, 8, 2, 128, 128, "bf16", seed=9)
    ko = torch.empty(6, 2, 128, dtype=torch.bfloat16, device="cuda")
    buf = torch.zeros(8, 8, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pkv.PkvError):       # q_out one token behind q
        pkv.qk_norm_rope(buf[1:7], ko, buf[:6], dk, qw.cuda(), kw.cuda(), 1e-6, cs.cuda(), pos.cuda())
    with pytest.raises(ValueError):         # a strided output
        pkv.qk_norm_rope(dq, ko, dq, dk, qw.cuda(), kw.cuda(), 1e-6, cs.cuda(), pos.cuda())
    empty = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    pkv.qk_norm_rope(empty, empty[:, :2], empty, empty[:, :2], qw.cuda(), kw.cuda(), 1e-6, cs.cuda(),
                     pos[:0].cuda())        # no tokens: nothing to do


def test_extreme_rows():
    """A row of zeros, huge and tiny rows, NaN in one row only."""
    D = 128
    q = torch.zeros(5, 2, D)
    q[1] = 1e18 * torch.randn(2, D, generator=torch.Generator().manual_seed(0))
    q[2] = 1e-18
    q[3] = 1.0
    q[3, 0, 7] = float("nan")
    cs = torch.cat([torch.ones(1, D // 2), torch.zeros(1, D // 2)], 1)
    w = torch.ones(D)
    pos = torch.zeros(5, dtype=torch.int64)
    qo, ko = torch.empty(5, 2, D, device="cuda"), torch.empty(5, 2, D, device="cuda")
    pkv.qk_norm_rope(qo, ko, q.cuda(), q.cuda(), w.cuda(), w.cuda(), 1e-6, cs.cuda(), pos.cuda())
    want = plain.norm_rope(q, w, 1e-6, cs, pos, False)
    assert torch.equal(torch.isnan(qo.cpu()), torch.isnan(want))
    fine = ~torch.isnan(want).any(-1)
    assert float(((qo.cpu().double() - want).abs()[fine] - 4 * FP32 * want.abs().amax(-1)[fine][:, None]).max()) <= 0


def test_captured_and_other_stream():
    (q, k, v), (dq, dk, dv), (qw, kw), cs, pos = inputs(12, 8, 2, 128, 128, "bf16", seed=11)
    kc = torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    qo = torch.empty(12, 8, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(12).cuda()
    args = (qw.cuda(), kw.cuda(), 1e-6, cs.cuda(), pos.cuda())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.qk_norm_rope_and_cache(qo, dq, dk, dv, *args, kc, vc, slots, stream=side)
    side.synchronize()
    first = (qo.clone(), kc.clone(), vc.clone())
    close(qo, plain.norm_rope(q, qw, 1e-6, cs, pos, False), "bf16", "q")
    for t in (qo, kc, vc):
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.qk_norm_rope_and_cache(qo, dq, dk, dv, *args, kc, vc, slots)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (qo, kc, vc)))

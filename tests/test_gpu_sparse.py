"""Key bounds, block selection and the decode over selected blocks, against plain 64-bit forms. Bounds
and selections are exact; the decode's tolerance is derived in check_bf16 (and, for 8-bit caches, in
test_gpu_block_scales)."""
import itertools
import math

import pytest
import torch

import paged_kv_cache_462_b200 as pkv
import plain_serving as plain
from test_gpu_block_scales import check_decode

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ bounds

@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2", "int8"])
@pytest.mark.parametrize("D,block,heads", [(128, 16, 2), (64, 8, 3), (128, 32, 1), (64, 32, 2), (128, 8, 8), (64, 16, 1)])
@pytest.mark.parametrize("with_scales", [False, True])
def test_bounds(kind, D, block, heads, with_scales):
    if kind == "bf16" and with_scales:
        pytest.skip("bf16 caches have no scales")
    lens = [1, block, block + 1, 5 * block - 1, 0, 77]
    new = [1, block, 2, 3 * block, 0, 1]
    gen = torch.Generator().manual_seed(7)
    table, pool = plain.tables(lens, block, gen)
    x = torch.randn(pool, heads, block, D, generator=gen) * 3
    k = x.to(torch.bfloat16) if kind == "bf16" else \
        (x * plain.QMAX[kind] / 15).clamp(-plain.QMAX[kind], plain.QMAX[kind]).to(plain.CODE[kind])
    for s, L in enumerate(lens):                        # what lies behind the last token is not looked at
        if L % block:
            p = int(table[s, L // block])
            if kind == "bf16":
                k[p, :, L % block:] = float("nan")
            else:
                k.view(torch.uint8)[p, :, L % block:] = 0x7f
    scales = torch.rand(pool, heads, generator=gen) + 0.01
    old = torch.full((pool, heads, 2, D), 5.0, dtype=torch.bfloat16)
    b = old.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    off = list(itertools.accumulate([0] + new))
    pkv.update_key_bounds(b, k.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                          torch.tensor(off, dtype=torch.int32).cuda(), off[-1], 0.37,
                          scales.cuda() if with_scales else None, err)
    want = old.clone()
    for s, L in enumerate(lens):
        for j in range((L - new[s]) // block, -(-L // block)) if new[s] else ():
            p = int(table[s, j])
            y = k[p, :, :min(block, L - j * block)].float()
            f = torch.ones(heads) if kind == "bf16" else scales[p] if with_scales else torch.full((heads,), 0.37)
            want[p, :, 0] = (y.amax(1) * f[:, None]).to(torch.bfloat16)
            want[p, :, 1] = (y.amin(1) * f[:, None]).to(torch.bfloat16)
    assert torch.equal(b.cpu(), want)
    assert err.item() == 0


def test_bounds_nan_keys_and_flags():
    k = torch.zeros(3, 1, 16, 64, dtype=torch.bfloat16)
    k[0, 0, 3, 9] = float("nan")
    b = torch.zeros(3, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()
    run = lambda t, l, o, n: pkv.update_key_bounds(b, k.cuda(), torch.tensor(t, dtype=torch.int32).cuda(), i32(*l), i32(*o), n,
                                                   device_error=err)
    run([[0, 1]], [20], [0, 20], 20)
    got = b.cpu()
    assert bool(torch.isnan(got[0, 0, :, 9]).all()) and int(torch.isnan(got).sum()) == 2 and err.item() == 0
    for t, l, o, n, want in ([[[0, 7]], [20], [0, 20], 20, pkv.DEVERR_BLOCK_ID], [[[0, 1]], [20], [0, 21], 21, pkv.DEVERR_SEQ_LEN],
                             [[[0, 1]], [20], [0, 20], 10, pkv.DEVERR_ROWS], [[[0, 1]], [33], [0, 1], 1, pkv.DEVERR_SEQ_LEN]):
        err.zero_()
        run(t, l, o, n)
        assert err.item() == want


# ------------------------------------------------------------------ selection

def bounds_like(pool, heads, D, gen, step=None):
    mid, half = torch.randn(pool, heads, 1, D, generator=gen), 1.5 + torch.rand(pool, heads, 1, D, generator=gen)
    b = torch.cat([mid + half, mid - half], 2)
    if step is not None:
        b = (b / step).round() * step                  # few distinct scores: ties
    return b.to(torch.bfloat16)


def run_select(q, b, table, lens, block, keep, sink, recent, ws=None):
    S, Hkv = q.shape[0], b.shape[1]
    out = torch.full((S, Hkv, keep), -7, dtype=torch.int32, device="cuda")
    ws = pkv.new_select_workspace(S, Hkv, table.shape[1]) if ws is None else ws
    pkv.select_blocks(out, q.cuda(), b.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), block, sink,
                      recent, workspace=ws)
    return out.cpu(), pkv.read_device_error(ws, clear=True)


def check_select(lens, Hq, Hkv, D, block, keep, sink=1, recent=1, step=None, seed=0, q=None, b=None):
    gen = torch.Generator().manual_seed(seed)
    table, pool = plain.tables(lens, block, gen)
    if q is None:
        q = torch.randn(len(lens), Hq, D, generator=gen).to(torch.bfloat16)
    b = bounds_like(pool, Hkv, D, gen, step) if b is None else b(pool, gen)
    got, err = run_select(q, b, table, lens, block, keep, sink, recent)
    want = torch.tensor(plain.select(q, b, table, lens, block, keep, sink, recent), dtype=torch.int32)
    assert torch.equal(got, want), (got != want).nonzero()[:5].tolist()
    assert err == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (40, 8, 128), (3, 3, 64), (16, 2, 64), (2, 1, 128), (5, 1, 64)])
@pytest.mark.parametrize("keep,sink,recent", [(6, 1, 1), (1, 0, 0), (5, 0, 2), (4, 2, 2), (33, 1, 1), (300, 4, 8)])
def test_select(Hq, Hkv, D, keep, sink, recent):
    block = 16
    check_select([0, 1, 16, 17, 16 * keep, 16 * keep + 1, 16 * keep + 17, 5000, 2049], Hq, Hkv, D, block, keep, sink, recent)


@pytest.mark.parametrize("block", [8, 32])
@pytest.mark.parametrize("step", [0.5, 2.0, 100.0])
def test_select_ties_go_to_the_lowest_index(block, step):
    """Coarse bounds and a coarse query: many equal scores, up to all of them (step 100)."""
    gen = torch.Generator().manual_seed(3)
    q = torch.randn(3, 8, 64, generator=gen).sign().to(torch.bfloat16)
    check_select([3000, 700, 1025], 8, 2, 64, block, 20, 1, 1, step=step, q=q)
    check_select([3000, 700, 1025], 8, 2, 64, block, 20, 0, 0, step=step, q=q)


def test_select_scores_that_fp32_cannot_tell_apart():
    """Large products that cancel and one small difference: blocks differ by 2^-9 in sums whose terms
    are 2^17, below the last bit of any fp32 sum of them. Shuffled, so that ties' order is no help."""
    D, n = 128, 900
    gen = torch.Generator().manual_seed(5)

    def b(pool, gen):
        x = torch.zeros(pool, 1, 2, D)
        big = torch.full((D // 2,), 4096.0)
        x[:, 0, :, 0:D - 2:2], x[:, 0, :, 1:D - 2:2] = big[:-1], -big[:-1]
        rank = torch.randperm(pool, generator=gen).float() % 120
        x[:, 0, :, D - 2] = ((1 + rank) * 2.0 ** -7)[:, None]
        return x.to(torch.bfloat16)

    q = torch.full((1, 2, D), 32.0)
    q[:, :, D - 2:] = 0.25
    check_select([16 * n], 2, 1, D, 16, 50, 1, 1, q=q.to(torch.bfloat16), b=b)
    check_select([16 * n], 2, 1, D, 16, 333, 0, 3, q=q.to(torch.bfloat16), b=b)


@pytest.mark.parametrize("blocks", [2048, 2049, 8192, 8193, 16384, 16385, 20001])
def test_select_long_sequences(blocks):
    """Around and beyond the streams that are selected in registers."""
    check_select([16 * blocks - 5], 4, 1, 64, 16, 100)
    check_select([16 * blocks], 4, 1, 64, 16, 700, 0, 0, step=4.0, seed=2)


def test_select_values_that_are_not_finite_and_bad_tables():
    gen = torch.Generator().manual_seed(8)
    lens, block = [16 * 200], 16
    table, pool = plain.tables(lens, block, gen)
    b = bounds_like(pool, 2, 64, gen)
    q = torch.randn(1, 8, 64, generator=gen).to(torch.bfloat16)
    q[q == 0] = 1
    b[table[0, 50].long(), 0, 0, 3] = float("nan")
    b[table[0, 51].long(), 1, :, 3] = float("inf")
    b[table[0, 60].long()] = float("inf")
    b[table[0, 61].long(), :, 1] = -float("inf")
    got, err = run_select(q, b, table, lens, block, 10, 1, 1)
    want = torch.tensor(plain.select(q, b, table, lens, block, 10, 1, 1), dtype=torch.int32)
    assert torch.equal(got, want) and err == 0
    for h in range(2):
        assert {60, 61} <= set(got[0, h].tolist())
    # more blocks that are not finite than places: the first of them
    b[table[0, 20:190].long()] = float("nan")
    got, err = run_select(q, b, table, lens, block, 10, 1, 1)
    assert got[0].tolist() == [[0] + list(range(20, 28)) + [199]] * 2
    # a NaN query: every block alike
    q[0, 0, 5] = float("nan")
    b = bounds_like(pool, 2, 64, gen)
    got, err = run_select(q, b, table, lens, block, 10, 1, 1)
    assert got[0, 0].tolist() == list(range(9)) + [199]
    # bad ids rank last, and are chosen when nothing else is left
    q[0, 0, 5] = 1
    bad = table.clone()
    bad[0, 10:190] = 1 << 20
    bad[0, 100] = -3
    got, err = run_select(q, b, bad, lens, block, 40, 0, 0)
    assert err == pkv.DEVERR_BLOCK_ID
    for h in range(2):
        assert got[0, h].tolist() == list(range(30)) + list(range(190, 200))
    # a length beyond the table is taken as the table's, whose last column holds -1 here
    got, err = run_select(q, b, table, [5000], block, 10, 1, 1)
    assert err == pkv.DEVERR_SEQ_LEN | pkv.DEVERR_BLOCK_ID


def test_select_workspace_serves_calls_of_other_sizes():
    """One workspace for a wide batch, a long sequence and the batch again, and the kept one."""
    gen = torch.Generator().manual_seed(9)
    ws = pkv.new_select_workspace(64, 8, 3000)
    for S, Hkv, n, ws_ in [(64, 8, 90, ws), (1, 1, 3000, ws), (40, 2, 500, ws), (64, 8, 90, ws), (3, 2, 300, None), (30, 8, 200, None)]:
        lens = [16 * n - 3 * s for s in range(S)]
        table, pool = plain.tables(lens, 16, gen)
        b = bounds_like(pool, Hkv, 64, gen)
        q = torch.randn(S, Hkv * 2, 64, generator=gen).to(torch.bfloat16)
        want = torch.tensor(plain.select(q, b, table, lens, 16, 12, 1, 1), dtype=torch.int32)
        if ws_ is None:
            got = torch.empty(S, Hkv, 12, dtype=torch.int32, device="cuda")
            pkv.select_blocks(got, q.cuda(), b.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 16)
            got = got.cpu()
        else:
            got, err = run_select(q, b, table, lens, 16, 12, 1, 1, ws_)
            assert err == 0
        assert torch.equal(got, want)


# ------------------------------------------------------------------ sparse decode

def lists(lens, block, heads, width, gen, wild=False):
    out = []
    for L in lens:
        n = -(-L // block)
        row = []
        for _ in range(heads):
            js = torch.randperm(n, generator=gen).tolist()[:width] if n else []
            if not wild:
                js = sorted(js)
            elif js:
                js[0] = js[-1]                             # one twice
                js = [(-1 if i % 5 == 3 else j) for i, j in enumerate(js)]
            row.append(js + [-1] * (width - len(js)))
        out.append(row)
    return out


def check_bf16(lens, Hq, Hkv, D, block, width, wild, partitions=(0,), seed=0):
    """Room: the output's and the weights' rounding to bf16 (2^-8 each, the latter on the size of the
    terms), 1e-5 for fp32 scores and sums."""
    gen = torch.Generator().manual_seed(seed)
    table, pool = plain.tables(lens, block, gen)
    k, v = (torch.randn(pool, Hkv, block, D, generator=gen).to(torch.bfloat16) for _ in range(2))
    for s, L in enumerate(lens):
        if L % block:
            p = int(table[s, L // block])
            k[p, :, L % block:], v[p, :, L % block:] = float("nan"), float("inf")
    q = torch.randn(len(lens), Hq, D, generator=gen).to(torch.bfloat16)
    sel = lists(lens, block, Hkv, width, gen, wild)
    want, size = plain.decode(q, k, v, table, lens, 0.11, block, sel)
    for parts in partitions:
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        ws = pkv.new_workspace(len(lens), Hq, Hkv, D, parts)
        pkv.paged_attention_decode_sparse(out, q.cuda(), k.cuda(), v.cuda(), table.cuda(),
                                          torch.tensor(lens, dtype=torch.int32).cuda(),
                                          torch.tensor(sel, dtype=torch.int32).cuda(), 0.11, num_partitions=parts,
                                          workspace=ws)
        err = (out.cpu().double() - want).abs() - 2.0 ** -8 * (want.abs() + size) - 1e-5 * size
        assert float(err.max()) <= 0, (parts, float(err.max()))
        assert pkv.read_device_error(ws) == 0


@pytest.mark.parametrize("wild", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,block", [(8, 2, 128, 16), (40, 8, 128, 16), (3, 3, 64, 32), (16, 2, 64, 16), (4, 1, 128, 32),
                                           (12, 6, 128, 32), (5, 1, 64, 16), (64, 8, 128, 16)])
@pytest.mark.parametrize("width", [1, 7, 40])
def test_sparse_bf16(wild, Hq, Hkv, D, block, width):
    check_bf16([0, 1, block, block + 1, 777, 2000, 3 * block - 1], Hq, Hkv, D, block, width, wild, (0, 1, 33))


@pytest.mark.parametrize("kind", ["e4m3", "e5m2", "int8"])
@pytest.mark.parametrize("block_scales", [False, True])
@pytest.mark.parametrize("Hq,Hkv,block", [(8, 2, 16), (40, 8, 32), (4, 1, 16)])
def test_sparse_8bit(kind, block_scales, Hq, Hkv, block):
    lens = [0, 1, 5 * block + 3, 900, 40 * block]
    sel = lists(lens, block, Hkv, 11, torch.Generator().manual_seed(6), wild=True)
    check_decode(lens, Hq, Hkv, block, kind, 1.0 if block_scales else 0.0, (0, 9), selected=sel, block_scales=block_scales)


def test_sparse_all_blocks_is_the_dense_decode():
    lens, gen = [333, 16, 1000], torch.Generator().manual_seed(1)
    table, pool = plain.tables(lens, 16, gen)
    k, v = (torch.randn(pool, 2, 16, 128, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(3, 8, 128, generator=gen).to(torch.bfloat16).cuda()
    sl = torch.tensor(lens, dtype=torch.int32).cuda()
    sel = torch.arange(63, dtype=torch.int32).expand(3, 2, 63).contiguous().cuda()
    a, b = torch.empty_like(q), torch.empty_like(q)
    pkv.paged_attention_decode(a, q, k, v, table.cuda(), sl, 0.09, num_partitions=16)
    pkv.paged_attention_decode_sparse(b, q, k, v, table.cuda(), sl, sel, 0.09, num_partitions=16)
    assert torch.equal(a, b)


def test_sparse_flags_and_empty_lists():
    k = torch.randn(6, 2, 16, 128).to(torch.bfloat16).cuda()
    q = torch.ones(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    t = torch.tensor([[0, 1, 2], [3, 50, 5]], dtype=torch.int32).cuda()
    sl = torch.tensor([40, 48], dtype=torch.int32).cuda()
    ws = pkv.new_workspace(2, 4, 2, 128)
    out = torch.empty_like(q)

    def run(sel):
        out.fill_(float("nan"))
        pkv.paged_attention_decode_sparse(out, q, k, k, t, sl, torch.tensor(sel, dtype=torch.int32).cuda(), 0.1, workspace=ws)
        return pkv.read_device_error(ws, clear=True)

    assert run([[[-1, -1], [-1, -5]], [[-1, -1], [0, -1]]]) == 0
    got = out.cpu().float()
    assert not got[0].any() and not got[1, :2].any() and bool(torch.isfinite(got).all()) and bool(got[1, 2:].any())
    assert run([[[0, 3], [1, 2]], [[0, 2], [2, 2]]]) == pkv.DEVERR_SELECTION      # block 3 of three
    assert bool(torch.isfinite(out).all())
    assert run([[[0, 1], [1, 2]], [[0, 1], [2, 2]]]) == pkv.DEVERR_BLOCK_ID       # the table's 50
    assert bool(torch.isfinite(out).all())


# ------------------------------------------------------------------ all of them, as a server runs them

@pytest.mark.parametrize("cache", ["e4m3", "int8", "bf16"])
def test_steps_of_a_server(cache):
    """Prompts, then decode steps: norm + rotation, append, bounds, selection, attention, the last three
    checked against plain forms on what the cache holds; short sequences see the dense decode."""
    Hq, Hkv, D, block, keep = 8, 2, 128, 16, 8
    gen = torch.Generator().manual_seed(12)
    lens = [300, 5, 64, 129]
    steps = 3
    table, pool = plain.tables([n + steps for n in lens], block, gen)
    dt = table.cuda()
    coded = cache != "bf16"
    kc = torch.zeros(pool, Hkv, block, D, dtype=plain.CODE.get(cache, torch.bfloat16), device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = torch.zeros(pool, Hkv, device="cuda"), torch.zeros(pool, Hkv, device="cuda")
    kb = torch.zeros(pool, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    ang = torch.arange(512, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    have = [0] * len(lens)
    for step in range(1 + steps):
        new = lens if step == 0 else [1] * len(lens)
        off = list(itertools.accumulate([0] + new))
        T = off[-1]
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen).to(torch.bfloat16).cuda()
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        pos = torch.cat([torch.arange(h, h + n) for h, n in zip(have, new)])
        seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(new))
        slots = (table[seq, pos // block].long() * block + pos % block).cuda()
        have = [h + n for h, n in zip(have, new)]
        sl = torch.tensor(have, dtype=torch.int32).cuda()
        ro = torch.tensor(off, dtype=torch.int32).cuda()
        qo = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        ko = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
        scales = {}
        if coded:
            pkv.qk_norm_rope(qo, ko, q, k, w, w, 1e-6, cs, pos.cuda(), device_error=err)
            pkv.reshape_and_cache_block_scales(ko, v, kc, vc, ks, vs, dt, sl, ro, device_error=err)
            scales = dict(k_block_scales=ks, v_block_scales=vs)
        else:
            pkv.qk_norm_rope_and_cache(qo, q, k, v, w, w, 1e-6, cs, pos.cuda(), kc, vc, slots, device_error=err)
        pkv.update_key_bounds(kb, kc, dt, sl, ro, T, k_block_scales=ks if coded else None, device_error=err)
        if step == 0:
            continue
        sel = torch.empty(len(lens), Hkv, keep, dtype=torch.int32, device="cuda")
        out, dense = torch.empty_like(qo), torch.empty_like(qo)
        pkv.select_blocks(sel, qo, kb, dt, sl, block)
        pkv.paged_attention_decode_sparse(out, qo, kc, vc, dt, sl, sel, D ** -0.5, **scales)
        if coded:
            pkv.paged_attention_decode_block_scales(dense, qo, kc, vc, dt, sl, D ** -0.5, ks, vs)
        else:
            pkv.paged_attention_decode(dense, qo, kc, vc, dt, sl, D ** -0.5)
        kv, vv = (plain.values(x) if coded else x.cpu().double() for x in (kc, vc))
        f = dict(ks=ks.cpu(), vs=vs.cpu()) if coded else {}
        full = kv * ks.cpu().double()[..., None, None] if coded else kv
        for s, L in enumerate(have):
            for j in range(-(-L // block)):
                x = full[table[s, j], :, :min(block, L - j * block)]
                assert torch.equal(kb[table[s, j]].cpu().double()[:, 0], x.amax(1).to(torch.bfloat16).double())
                assert torch.equal(kb[table[s, j]].cpu().double()[:, 1], x.amin(1).to(torch.bfloat16).double())
        want_sel = plain.select(qo, kb, table, have, block, keep, 1, 1)
        assert sel.tolist() == want_sel
        want, size = plain.decode(qo, kv, vv, table, have, D ** -0.5, block, want_sel, **f)
        room = 2.0 ** -8 * (want.abs() + size) + 1e-5 * size
        if cache == "int8":
            room = room + 2 * D ** -0.5 * float(full.abs().sum(-1).max()) * float(qo.abs().max()) * 2.0 ** -14 * size
        assert float(((out.cpu().double() - want).abs() - room).max()) <= 0
        short = [s for s, L in enumerate(have) if L <= keep * block]
        assert short and float((out[short].float() - dense[short].float()).abs().max()) <= 2.0 ** -7 * float(dense.float().abs().max())
    assert err.item() == 0


def test_far_blocks():
    """Blocks beyond 2^31 elements of the caches: appended, bounded, selected and attended like near ones."""
    S, Hq, Hkv, D, block = 2, 8, 8, 128, 16
    NB = 140000                                            # 2.29e9 elements a cache
    lens = [75, 200]
    gen = torch.Generator().manual_seed(21)
    n = [-(-L // block) for L in lens]
    table = torch.full((S, max(n)), -1, dtype=torch.int32)
    far = NB - 1 - torch.arange(sum(n), dtype=torch.int32)
    for s in range(S):
        table[s, :n[s]] = far[sum(n[:s]):sum(n[:s + 1])]
    near = torch.where(table >= 0, NB - 1 - table, table)   # the same blocks at the pool's start
    T = sum(lens)
    k, v = (torch.randn(T, Hkv, D, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(S, Hq, D, generator=gen).to(torch.bfloat16).cuda()
    sl = torch.tensor(lens, dtype=torch.int32).cuda()
    ro = torch.tensor([0, lens[0], T], dtype=torch.int32).cuda()
    res = []
    for t, pool in ((table, NB), (near, sum(n))):
        dt = t.cuda()
        kc = torch.zeros(pool, Hkv, block, D, dtype=torch.float8_e4m3fn, device="cuda")
        vc = torch.zeros_like(kc)
        ks, vs = torch.zeros(pool, Hkv, device="cuda"), torch.zeros(pool, Hkv, device="cuda")
        kb = torch.zeros(pool, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
        sel = torch.empty(S, Hkv, 4, dtype=torch.int32, device="cuda")
        o1, o2 = torch.empty_like(q), torch.empty_like(q)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.reshape_and_cache_block_scales(k, v, kc, vc, ks, vs, dt, sl, ro, device_error=err)
        pkv.update_key_bounds(kb, kc, dt, sl, ro, T, k_block_scales=ks, device_error=err)
        pkv.select_blocks(sel, q, kb, dt, sl, block)
        pkv.paged_attention_decode_sparse(o1, q, kc, vc, dt, sl, sel, 0.1, k_block_scales=ks, v_block_scales=vs, num_partitions=4)
        pkv.paged_attention_decode_block_scales(o2, q, kc, vc, dt, sl, 0.1, ks, vs, num_partitions=4)
        # and the fused norm + append into a bf16 pool of that many blocks, one row in the last block
        kc16 = torch.zeros(pool, Hkv, block, D, dtype=torch.bfloat16, device="cuda")
        vc16 = torch.zeros_like(kc16)
        w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
        slot = torch.tensor([(pool - 1 if pool == NB else 0) * block + 3], device="cuda")
        pkv.qk_norm_rope_and_cache(torch.empty_like(q[:1]), q[:1], k[:1], v[:1], w, w, 1e-6,
                                   torch.ones(1, D, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"),
                                   kc16, vc16, slot, device_error=err)
        assert err.item() == 0
        at = t[t >= 0].long().cuda()
        b = int(slot) // block
        res.append([x.clone() for x in (kc.view(torch.uint8)[at], vc.view(torch.uint8)[at], ks[at], vs[at], kb[at], sel,
                                        o1, o2, kc16[b], vc16[b])])
        del kc, vc, kc16, vc16, kb
    torch.cuda.empty_cache()
    for a, b in zip(*res):
        assert torch.equal(a, b)
    assert bool(res[0][8].any())


def test_two_streams_at_once():
    """Selection and sparse decode on two streams at the same time, without workspaces of their own."""
    gen = torch.Generator().manual_seed(31)
    lens = [3000, 700, 1999, 40, 2500, 16]
    table, pool = plain.tables(lens, 16, gen)
    b = bounds_like(pool, 2, 128, gen).cuda()
    k, v = (torch.randn(pool, 2, 16, 128, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    dt, sl = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    qs = [torch.randn(6, 8, 128, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]

    def run(q):
        sel = torch.empty(6, 2, 24, dtype=torch.int32, device="cuda")
        out = torch.empty_like(q)
        pkv.select_blocks(sel, q, b, dt, sl, 16)
        pkv.paged_attention_decode_sparse(out, q, k, v, dt, sl, sel, 0.1)
        return sel, out

    want = [run(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(qs[i]))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for x in g:
            assert torch.equal(x[0], w[0]) and torch.equal(x[1], w[1])


def test_a_step_captured_and_replayed():
    """Norm, append, bounds, selection and attention in one graph, replayed with other queries and
    lengths: the same as the calls made one by one."""
    S, Hq, Hkv, D, block, keep = 3, 8, 2, 128, 16, 6
    gen = torch.Generator().manual_seed(41)
    final = [400, 130, 260]
    table, pool = plain.tables(final, block, gen)
    dt = table.cuda()
    cs = torch.randn(512, D, generator=gen).cuda()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    ro = torch.arange(S + 1, dtype=torch.int32, device="cuda")

    class Run:
        def __init__(self):
            g = torch.Generator(device="cuda").manual_seed(5)
            code = lambda: (torch.randn(pool, Hkv, block, D, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)
            self.kc, self.vc = code(), code()
            self.ks = torch.full((pool, Hkv), 2.0 ** -6, device="cuda")
            self.vs = self.ks.clone()
            self.kb = torch.zeros(pool, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
            self.sl = torch.tensor([f - 8 for f in final], dtype=torch.int32, device="cuda")
            pkv.update_key_bounds(self.kb, self.kc, dt, self.sl, torch.cat([ro[:1], self.sl.cumsum(0).to(torch.int32)]),
                                  int(self.sl.sum()), k_block_scales=self.ks)
            self.qkv = torch.zeros(S, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda")
            self.pos = torch.zeros(S, dtype=torch.int64, device="cuda")
            self.qo = torch.empty(S, Hq, D, dtype=torch.bfloat16, device="cuda")
            self.ko = torch.empty(S, Hkv, D, dtype=torch.bfloat16, device="cuda")
            self.sel = torch.empty(S, Hkv, keep, dtype=torch.int32, device="cuda")
            self.out = torch.empty_like(self.qo)

        def step(self):
            q, k, v = (x.unflatten(1, (-1, D)) for x in self.qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
            pkv.qk_norm_rope(self.qo, self.ko, q, k, w, w, 1e-6, cs, self.pos)
            pkv.reshape_and_cache_block_scales(self.ko, v, self.kc, self.vc, self.ks, self.vs, dt, self.sl, ro)
            pkv.update_key_bounds(self.kb, self.kc, dt, self.sl, ro, S, k_block_scales=self.ks)
            pkv.select_blocks(self.sel, self.qo, self.kb, dt, self.sl, block)
            pkv.paged_attention_decode_sparse(self.out, self.qo, self.kc, self.vc, dt, self.sl, self.sel, 0.1,
                                              k_block_scales=self.ks, v_block_scales=self.vs)

        def feed(self, i):
            g = torch.Generator(device="cuda").manual_seed(100 + i)
            self.qkv.copy_(torch.randn(self.qkv.shape, generator=g, device="cuda"))
            self.sl += 1
            self.pos.copy_(self.sl.long() - 1)

    eager, other = Run(), Run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.step()
    for i in range(6):
        eager.feed(i)
        eager.step()
        other.feed(i)
        graph.replay()
        for x in ("qo", "sel", "out", "ks", "vs", "kb"):
            assert torch.equal(getattr(eager, x), getattr(other, x)), x
        assert torch.equal(eager.kc.view(torch.uint8), other.kc.view(torch.uint8))


def test_the_binding_without_its_hot_path(monkeypatch):
    """The same calls through ctypes and the step-by-step checks, as where _fastcall is not built."""
    gen = torch.Generator().manual_seed(51)
    lens, new = [300, 17, 64], [300, 17, 64]
    table, pool = plain.tables(lens, 16, gen)
    dt, sl = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    ro = torch.tensor([0, 300, 317, 381], dtype=torch.int32).cuda()
    qkv = torch.randn(381, 12 * 128, generator=gen).to(torch.bfloat16).cuda()
    q, k, v = (x.unflatten(1, (-1, 128)) for x in qkv.split([1024, 256, 256], 1))
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    cs, pos = torch.randn(400, 128, generator=gen).cuda(), torch.arange(381, device="cuda")

    def run():
        kc = torch.zeros(pool, 2, 16, 128, dtype=torch.int8, device="cuda")
        vc, ks, vs = torch.zeros_like(kc), torch.zeros(pool, 2, device="cuda"), torch.zeros(pool, 2, device="cuda")
        kb = torch.zeros(pool, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
        k16, v16 = (torch.zeros(pool + 9, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        qo, ko = torch.empty(381, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(381, 2, 128, dtype=torch.bfloat16, device="cuda")
        pkv.qk_norm_rope(qo, ko, q, k, w, w, 1e-6, cs, pos)
        pkv.qk_norm_rope_and_cache(torch.empty_like(qo), q, k, v, w, w, 1e-6, cs, pos, k16, v16, pos)
        pkv.reshape_and_cache_block_scales(ko, v, kc, vc, ks, vs, dt, sl, ro)
        pkv.update_key_bounds(kb, kc, dt, sl, ro, 381, k_block_scales=ks)
        qq = qo[[299, 316, 380]].contiguous()
        sel = torch.empty(3, 2, 5, dtype=torch.int32, device="cuda")
        o1, o2, o3 = torch.empty_like(qq), torch.empty_like(qq), torch.empty_like(qq)
        pkv.select_blocks(sel, qq, kb, dt, sl, 16)
        pkv.paged_attention_decode_block_scales(o1, qq, kc, vc, dt, sl, 0.1, ks, vs)
        pkv.paged_attention_decode_sparse(o2, qq, kc, vc, dt, sl, sel, 0.1, k_block_scales=ks, v_block_scales=vs)
        pkv.paged_attention_decode_sparse(o3, qq, kc, vc, dt, sl, sel, 0.1, 0.02, 0.02)
        return kc, vc, ks, vs, kb, qo, ko, k16, v16, sel, o1, o2, o3

    pkv.load_library()
    assert pkv._fast is not None, "csrc/fastcall.cpp is not built"
    want = run()
    monkeypatch.setattr(pkv, "_fast", None)
    monkeypatch.setattr(pkv, "_lib", None)
    monkeypatch.setattr(pkv, "_bind_fast", lambda lib: None)
    got = run()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_streams_given_by_argument(monkeypatch):
    """A stream that is not the current one: another stream's object, its handle, and the legacy default
    stream from within a side stream; the kept workspaces are made on the stream that uses them."""
    monkeypatch.setattr(pkv, "_op_ws", {})
    gen = torch.Generator().manual_seed(61)
    lens = [900, 33]
    table, pool = plain.tables(lens, 16, gen)
    b = bounds_like(pool, 2, 128, gen).cuda()
    k = torch.randn(pool, 2, 16, 128, generator=gen).to(torch.bfloat16).cuda()
    dt, sl = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    q = torch.randn(2, 8, 128, generator=gen).to(torch.bfloat16).cuda()

    def run(stream):
        sel, out = torch.empty(2, 2, 9, dtype=torch.int32, device="cuda"), torch.empty_like(q)
        torch.cuda.synchronize()
        pkv.select_blocks(sel, q, b, dt, sl, 16, stream=stream)
        pkv.paged_attention_decode_sparse(out, q, k, k, dt, sl, sel, 0.1, stream=stream)
        torch.cuda.synchronize()
        return sel, out

    want = run(None)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    got = [run(side), run(side.cuda_stream)]
    with torch.cuda.stream(other):
        got += [run(None), run(0), run(side)]
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(ValueError):                       # which stream's graph would hold the workspace?
        with torch.cuda.graph(graph):
            pkv.select_blocks(want[0], q, b, dt, sl, 16, stream=side)

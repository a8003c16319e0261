"""An 8-bit cache with a scale for each block and KV head: the append is exact (scales are powers of
two), the decode is held to the 64-bit softmax.

Decode tolerance, on the size A = sum p |v| of an output's terms: the output's rounding (bf16, 2^-8
of the value), the weights' (f16, 2^-11), and what the scores are off: q is exact in f16 (E4M3 and
E5M2), and for INT8 rounded to 2^-13 of its largest element, which moves a score by at most
scale * sum |k_d| * max|q| * 2^-14 and a weight by twice that (its sum moves too).
Weights below f16's smallest normal number are off by up to half its smallest step, 2^-25, whatever their
size: with w = 2^(s + log2 vs - m) the kernel's weights, an output is sum w code / sum (w / vs), the largest
w is at least 1, so the lower sum is at least 1 / vs of its block, and the output is off by at most
2^-25 * max vs * sum |code|. (It shows where the token with all the weight holds a zero.)"""
import itertools
import math

import pytest
import torch

import paged_kv_cache_462_b200 as pkv
import plain_serving as plain

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Cache:
    """A cache on the device and its 64-bit model."""

    def __init__(self, lens, block, heads, dim, kind, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.block, self.kind = block, kind
        self.table, pool = plain.tables(lens, block, gen)
        shape = (pool, heads, block, dim)
        codes = (torch.randn(shape, generator=gen) * plain.QMAX[kind] / 4).clamp(-plain.QMAX[kind], plain.QMAX[kind])
        self.kc = codes.to(plain.CODE[kind]).cuda()
        self.vc = codes.flip(0).contiguous().to(plain.CODE[kind]).cuda()
        # what lies in the pool before: scales that must not leak into new blocks
        self.ks = torch.full((pool, heads), 1024.0, device="cuda")
        self.vs = torch.full((pool, heads), 2.0 ** -40, device="cuda")
        self.model = [plain.values(self.kc), plain.values(self.vc), self.ks.cpu().double(), self.vs.cpu().double()]
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dtable = self.table.cuda()

    def append(self, k, v, lens, offsets, **kw):
        pkv.reshape_and_cache_block_scales(k.cuda(), v.cuda(), self.kc, self.vc, self.ks, self.vs, self.dtable,
                                           torch.tensor(lens, dtype=torch.int32).cuda(),
                                           torch.tensor(offsets, dtype=torch.int32).cuda(), device_error=self.err, **kw)
        plain.append_block_scales(k, self.model[0], self.model[2], self.table, lens, offsets, self.block, self.kind)
        plain.append_block_scales(v, self.model[1], self.model[3], self.table, lens, offsets, self.block, self.kind)

    def check(self):
        got = [plain.values(self.kc), plain.values(self.vc), self.ks.cpu().double(), self.vs.cpu().double()]
        for name, a, b in zip(("k codes", "v codes", "k scales", "v scales"), got, self.model):
            same = (a == b) | (torch.isnan(a) & torch.isnan(b))
            assert bool(same.all()), (name, (~same).nonzero()[:4].tolist())


@pytest.mark.parametrize("kind", ["e4m3", "e5m2", "int8"])
@pytest.mark.parametrize("rows,dim,block,heads", [("bf16", 128, 16, 2), ("f32", 128, 16, 1), ("bf16", 64, 8, 3),
                                                 ("f32", 64, 32, 2), ("bf16", 128, 32, 5), ("f32", 128, 8, 1)])
def test_append_in_steps(kind, rows, dim, block, heads):
    """Prompts of many lengths, then chunks and single tokens, sequences without new rows among them;
    token sizes vary so that blocks' scales grow."""
    final = [1, 2, block - 1, block, block + 1, 3 * block + 5, 70, 129]
    c = Cache(final, block, heads, dim, kind)
    gen = torch.Generator().manual_seed(1)
    have = [0] * len(final)
    step = 0
    while have != final:
        new = []
        for s, (h, f) in enumerate(zip(have, final)):
            n = [f // 2 + 1, 1, 0, 2, block, 3][(step + s) % 6] if step < 30 else f - h
            new.append(min(n, f - h))
        off = list(itertools.accumulate([0] + new))
        T = off[-1] + 2                                     # rows behind the last sequence: not read
        x = [(torch.randn(T, heads, dim, generator=gen) * torch.exp(1.5 * torch.randn(T, heads, 1, generator=gen))).to(DT[rows])
             for _ in range(2)]
        x[0][off[-1]:] = float("nan")
        have = [h + n for h, n in zip(have, new)]
        c.append(*x, have, off)
        c.check()
        step += 1
    assert c.err.item() == 0


@pytest.mark.parametrize("kind", ["e4m3", "e5m2", "int8"])
def test_append_special_values(kind):
    """Zeros, infinities, NaN, values beyond the largest scale and below the smallest, exact borders."""
    top = plain.QMAX[kind]
    rows = torch.zeros(64, 1, 64)
    rows[1] = float("inf")
    rows[2, 0, :3] = torch.tensor([float("nan"), 1.0, -float("inf")])
    rows[16:32] = 3e38                                      # beyond qmax * 2^50: saturates
    rows[32:48] = 1e-38                                     # below 2^-50 of anything
    rows[48, 0] = top * 2.0 ** -3                           # exactly qmax * 2^-3
    rows[49, 0, 5] = -top * 2.0 ** -3 * (1 + 2.0 ** -20)    # just above: the next power
    rows[50, 0, :4] = torch.tensor([0.5, 1.5, 2.5, -0.5]) * 2.0 ** -2
    c = Cache([64], 16, 1, 64, kind)
    c.append(rows, -rows, [64], [0, 64])
    c.check()
    c2 = Cache([20], 16, 1, 64, kind)
    one = torch.ones(1, 1, 64)
    for i in range(20):                                     # token by token, each larger than the last
        c2.append(one * 2.0 ** (i % 17) * 1.01, one * 2.0 ** -(i % 17), [i + 1], [0, 1])
        c2.check()
    assert c.err.item() == 0 and c2.err.item() == 0


def test_append_strided_rows_and_bad_batches():
    gen = torch.Generator().manual_seed(2)
    c = Cache([40, 33, 20, 50], 16, 2, 128, "e4m3")
    qkv = torch.randn(30, 3 * 256 + 8, generator=gen).to(torch.bfloat16)
    k, v = qkv[:, 256:512].unflatten(1, (2, 128)), qkv[:, 512:768].unflatten(1, (2, 128))
    d = qkv.cuda()
    lens, off = [10, 5, 15, 0], [0, 10, 15, 30, 30]
    pkv.reshape_and_cache_block_scales(d[:, 256:512].unflatten(1, (2, 128)), d[:, 512:768].unflatten(1, (2, 128)), c.kc,
                                       c.vc, c.ks, c.vs, c.dtable, torch.tensor(lens, dtype=torch.int32).cuda(),
                                       torch.tensor(off, dtype=torch.int32).cuda(), device_error=c.err)
    plain.append_block_scales(k, c.model[0], c.model[2], c.table, lens, off, 16, "e4m3")
    plain.append_block_scales(v, c.model[1], c.model[3], c.table, lens, off, 16, "e4m3")
    c.check()
    assert c.err.item() == 0

    def bad(lens, off, want, table=None):
        c.err.zero_()
        pkv.reshape_and_cache_block_scales(k.cuda().contiguous(), v.cuda().contiguous(), c.kc, c.vc, c.ks, c.vs,
                                           c.dtable if table is None else table,
                                           torch.tensor(lens, dtype=torch.int32).cuda(),
                                           torch.tensor(off, dtype=torch.int32).cuda(), device_error=c.err)
        assert c.err.item() == want
        c.check()                                            # nothing written

    bad([10, 10, 10, 10], [5, 3, 3, 3, 2], pkv.DEVERR_ROWS)           # descending
    bad([10, 10, 10, 10], [0, 0, 0, 0, 31], pkv.DEVERR_ROWS)          # beyond the rows
    bad([10, 10, 10, 10], [-1, 0, 0, 0, 0], pkv.DEVERR_ROWS)
    bad([3, 0, 0, 0], [0, 4, 4, 4, 4], pkv.DEVERR_SEQ_LEN)            # more rows than tokens
    bad([1 << 20, -5, 0, 0], [0, 4, 4, 4, 4], pkv.DEVERR_SEQ_LEN)
    t = c.table.clone()
    t[0, 0] = 1 << 20
    bad([4, 0, 0, 0], [0, 4, 4, 4, 4], pkv.DEVERR_BLOCK_ID, t.cuda())


# ------------------------------------------------------------------ decode

def scales(shape, gen, spread):
    return 2.0 ** (spread * torch.randn(shape, generator=gen)) * 0.01


def check_decode(lens, Hq, Hkv, block, kind, spread, partitions=(0,), selected=None, seed=0, block_scales=True):
    gen = torch.Generator().manual_seed(seed)
    table, pool = plain.tables(lens, block, gen)
    D, S = 128, len(lens)
    unit = plain.QMAX[kind] / 4.2
    code = lambda: (torch.randn(pool, Hkv, block, D, generator=gen) * unit).clamp(-plain.QMAX[kind], plain.QMAX[kind]).to(plain.CODE[kind])
    k, v = code(), code()
    for s, L in enumerate(lens):                             # NaN behind the last token, where there is one
        if L % block and kind != "int8":
            p = int(table[s, L // block])
            k.view(torch.uint8)[p, :, L % block:] = 0x7f
            v.view(torch.uint8)[p, :, L % block:] = 0x7f
    q = torch.randn(S, Hq, D, generator=gen).to(torch.bfloat16)
    ks, vs = (scales((pool, Hkv), gen, spread) / unit * 100 for _ in range(2))
    dev = dict(q=q.cuda(), k_cache=k.cuda(), v_cache=v.cuda(), block_tables=table.cuda(),
               seq_lens=torch.tensor(lens, dtype=torch.int32).cuda(), scale=D ** -0.5)
    one = float(ks[0, 0])
    if not block_scales:
        ks, vs = torch.full_like(ks, one), torch.full_like(vs, one)
    want, size = plain.decode(q, plain.values(k), plain.values(v), table, lens, D ** -0.5, block, selected, ks, vs)
    room = 2.0 ** -8 * want.abs() + 2.0 ** -11 * size + 1e-5 * size
    tiny = torch.zeros_like(want)
    for s, L in enumerate(lens):
        n = -(-L // block)
        for h in range(Hkv):
            js = list(range(n)) if selected is None else [j for j in selected[s][h][:n] if j >= 0]
            if js:
                ids = table[s, js].long()
                codes = plain.values(v)[ids, h].abs().nan_to_num(0.0).sum((0, 1))
                tiny[s, h * Hq // Hkv:(h + 1) * Hq // Hkv] = 2.0 ** -25 * float(vs[ids, h].max()) * codes
    room = room + tiny
    if kind == "int8":
        big_k = float((plain.values(k).abs().sum(-1) * ks.double()[..., None]).max())
        room = room + 2 * (D ** -0.5) * big_k * float(q.abs().max()) * 2.0 ** -14 * size
    for parts in partitions:
        out = torch.full((S, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        ws = pkv.new_workspace(S, Hq, Hkv, D, parts)
        if selected is not None:
            sel = torch.tensor(selected, dtype=torch.int32).cuda()
            kw = dict(k_block_scales=ks.cuda(), v_block_scales=vs.cuda()) if block_scales else dict(k_scale=one, v_scale=one)
            pkv.paged_attention_decode_sparse(out, **dev, selected=sel, num_partitions=parts, workspace=ws, **kw)
        else:
            pkv.paged_attention_decode_block_scales(out, **dev, k_block_scales=ks.cuda(), v_block_scales=vs.cuda(),
                                                    num_partitions=parts, workspace=ws)
        err = (out.cpu().double() - want).abs() - room
        assert float(err.max()) <= 0, (parts, float((out.cpu().double() - want).abs().max()), float(err.max()))
        assert pkv.read_device_error(ws) == 0
    return out


@pytest.mark.parametrize("kind", ["e4m3", "e5m2", "int8"])
@pytest.mark.parametrize("Hq,Hkv,block", [(8, 2, 16), (40, 8, 16), (3, 3, 32), (16, 2, 32), (4, 1, 16), (12, 6, 16),
                                         (10, 2, 32), (8, 8, 16)])
def test_decode(kind, Hq, Hkv, block):
    check_decode([0, 1, block - 1, block, block + 1, 3 * block - 1, 97, 200, 1100], Hq, Hkv, block, kind, 1.0, (0, 1, 7))


@pytest.mark.parametrize("kind", ["e4m3", "e5m2", "int8"])
@pytest.mark.parametrize("spread", [0.0, 5.0])
def test_decode_scales_far_apart(kind, spread):
    """Blocks whose scales differ by factors of 2^20 and more, split over many partitions."""
    check_decode([333, 64, 700], 8, 2, 16, kind, spread, (0, 64))


def test_decode_tiny_v_blocks_keep_their_weight():
    """A block of zeros (the append's smallest scale) takes its share of the softmax all the same."""
    L, D = 32, 128
    k = torch.zeros(2, 1, 16, D).to(torch.float8_e4m3fn).cuda()
    v = torch.zeros(2, 1, 16, D)
    v[0] = 8.0
    v = v.to(torch.float8_e4m3fn).cuda()
    ks = torch.ones(2, 1, device="cuda")
    for big in (1.0, 2.0 ** 40):
        vs = torch.tensor([[big], [2.0 ** -50]], device="cuda")
        out = torch.empty(1, 1, D, dtype=torch.bfloat16, device="cuda")
        pkv.paged_attention_decode_block_scales(out, torch.ones(1, 1, D, dtype=torch.bfloat16, device="cuda"), k, v,
                                                torch.tensor([[0, 1]], dtype=torch.int32).cuda(),
                                                torch.tensor([L], dtype=torch.int32).cuda(), 1.0, ks, vs)
        assert torch.equal(out.cpu().float(), torch.full((1, 1, D), 4.0 * big))


def test_decode_bad_tables_are_flagged():
    k = torch.zeros(4, 2, 16, 128, dtype=torch.uint8, device="cuda")
    s = torch.ones(4, 2, device="cuda")
    q = torch.ones(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = pkv.new_workspace(2, 4, 2, 128)
    out = torch.empty_like(q)
    pkv.paged_attention_decode_block_scales(out, q, k, k.clone(), torch.tensor([[0, 99], [2, -1]], dtype=torch.int32).cuda(),
                                            torch.tensor([20, 1000], dtype=torch.int32).cuda(), 1.0, s, s, workspace=ws)
    assert pkv.read_device_error(ws) == pkv.DEVERR_BLOCK_ID | pkv.DEVERR_SEQ_LEN
    assert bool(torch.isfinite(out).all())


def test_decode_captured_twice_on_one_stream():
    """Two graphs and eager calls, replayed in turn with new inputs: each has its own workspace, and a
    replay does not take the replay before for itself."""
    lens, D = [900, 37, 2000, 512], 128
    gen = torch.Generator().manual_seed(4)
    table, pool = plain.tables(lens, 16, gen)
    code = lambda: (torch.randn(pool, 2, 16, D, generator=gen) * 60).to(torch.float8_e4m3fn).cuda()
    k, v = code(), code()
    s = (torch.rand(pool, 2, generator=gen) * 0.02 + 0.005).cuda()
    dt, dl = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    qs = [torch.randn(4, 8, D, generator=gen).to(torch.bfloat16).cuda() for _ in range(6)]
    run = lambda o, x: pkv.paged_attention_decode_block_scales(o, x, k, v, dt, dl, 0.3, s, s)
    want = []
    for x in qs:
        o = torch.empty_like(x)
        run(o, x)
        want.append(o)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        x, o = torch.zeros_like(qs[0]), torch.zeros_like(qs[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            run(o, x)
        graphs.append((g, x, o))
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(0, 6, 2):
        for (g, x, o), side, j in zip(graphs, sides, (i, i + 1)):
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                x.copy_(qs[j])
                g.replay()
        torch.cuda.synchronize()
        for (g, x, o), j in zip(graphs, (i, i + 1)):
            assert torch.equal(o, want[j])


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("Hq,Hkv,block", [(4, 1, 16), (15, 3, 16), (8, 1, 32)])
def test_decode_many_sequences_of_few_heads(kind, Hq, Hkv, block):
    """One KV head to a unit and enough streams for more than three runs an SM."""
    lens = [(37 * i * i + 11) % 1100 for i in range(110)]
    check_decode(lens, Hq, Hkv, block, kind, 1.0, (0,))
    sel = [[[j for j in range(h, 60, 3)] + [-1] * 2 for h in range(Hkv)] for _ in lens]
    width = max(len(r) for row in sel for r in row)
    sel = [[(r + [-1] * width)[:width] for r in row] for row in sel]
    sel = [[[j if j < -(-L // block) else -1 for j in r] for r in row] for row, L in zip(sel, lens)]
    check_decode(lens, Hq, Hkv, block, kind, 1.0, (0,), selected=sel)

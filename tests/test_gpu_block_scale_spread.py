"""V scales that differ by orders of magnitude within a sequence: a block with one large element, or with a scale that
is far too large for what it holds, leaves the other blocks their share."""
import pytest
import torch

import paged_kv_cache_462_b200 as pkv
import plain_serving as plain

pytestmark = pytest.mark.gpu
D = 128


def check(q, k, v, ks, vs, table, lens, parts):
    """Room: the output's bf16, fp32 scores and sums (1e-5), and the weights' f16: 2^-11 of a weight, and half its
    smallest step, 2^-25, where the largest weight times scale, W, is 2^7 at least."""
    want, size = plain.decode(q, plain.values(k), plain.values(v), table, lens, 1.0, 16, None, ks, vs)
    Hkv, G = k.shape[1], q.shape[1] // k.shape[1]
    room = 2.0 ** -8 * want.abs() + 2.0 ** -11 * size + 1e-5 * size
    for s, L in enumerate(lens):
        ids = table[s, :-(-L // 16)].long()
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            keys = (plain.values(k)[ids, h] * ks[ids, h].double()[:, None, None]).flatten(0, 1)[:L]
            p = torch.softmax(q[s, heads].double() @ keys.T, -1)
            top = (p * vs[ids, h].double().repeat_interleave(16)[:L]).amax(-1)
            room[s, heads] += 2.0 ** -32 * top[:, None] * plain.values(v)[ids, h].abs().flatten(0, 1)[:L].sum(0)
    for n in parts:
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        sl = torch.tensor(lens, dtype=torch.int32).cuda()
        pkv.paged_attention_decode_block_scales(out, q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl, 1.0, ks.cuda(), vs.cuda(), n)
        err = (out.cpu().double() - want).abs() - room
        assert float(err.max()) <= 0, (n, float(err.max()), float((out.cpu().double() - want).abs().max()))


@pytest.mark.parametrize("kind", ["e4m3", "e5m2", "int8"])
@pytest.mark.parametrize("power", [0, 10, 16, 20, 24])
def test_a_block_whose_scale_is_too_large(kind, power):
    """All-zero V codes under a scale 2^power times the others', which alone decide the output."""
    gen = torch.Generator().manual_seed(power)
    lens = [16 * 40, 700]
    table, pool = plain.tables(lens, 16, gen)
    code = lambda: (torch.randn(pool, 2, 16, D, generator=gen) * plain.QMAX[kind] / 4.2).clamp(
        -plain.QMAX[kind], plain.QMAX[kind]).to(plain.CODE[kind])
    k, v = code(), code()
    q = (torch.randn(2, 8, D, generator=gen) * 2.0 ** -4).to(torch.bfloat16)
    ks = torch.full((pool, 2), 0.25 / plain.QMAX[kind])
    vs = torch.full((pool, 2), 2.0 ** -7)
    for s in range(2):
        v.view(torch.uint8)[int(table[s, 5])] = 0
        vs[int(table[s, 5])] *= 2.0 ** power
    check(q, k, v, ks, vs, table, lens, (0, 1, 17))


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("power", [8, 14, 18])
def test_one_large_element(kind, power):
    """Appended rows, one element of one token 2^power times the others: the other dimensions are as they would be
    without it, to the codes' precision."""
    gen = torch.Generator().manual_seed(power)
    L, Hkv = 1000, 2
    table, pool = plain.tables([L], 16, gen)
    k, v = (torch.randn(L, Hkv, D, generator=gen).to(torch.bfloat16) for _ in range(2))
    v[345, 1, 77] = 3.0 * 2.0 ** power
    kc, vc = (torch.zeros(pool, Hkv, 16, D, dtype=plain.CODE[kind], device="cuda") for _ in range(2))
    ks, vs = torch.zeros(pool, Hkv, device="cuda"), torch.zeros(pool, Hkv, device="cuda")
    pkv.reshape_and_cache_block_scales(k.cuda(), v.cuda(), kc, vc, ks, vs, table.cuda(), torch.tensor([L], dtype=torch.int32).cuda(),
                                       torch.tensor([0, L], dtype=torch.int32).cuda())
    q = (torch.randn(1, 8, D, generator=gen) * 0.08).to(torch.bfloat16)
    check(q, kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu(), table, [L], (0, 1, 9))

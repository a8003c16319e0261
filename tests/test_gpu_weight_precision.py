"""bf16 caches, up to four query heads to a KV head: the softmax weights enter p.V with more than bf16's eight bits."""
import pytest
import torch

import paged_kv_cache_462_b200 as pkv
import plain_serving as plain

pytestmark = pytest.mark.gpu


def inputs(lens, Hq, Hkv, D, block, seed=0):
    gen = torch.Generator().manual_seed(seed)
    table, pool = plain.tables(lens, block, gen)
    k, v = (torch.randn(pool, Hkv, block, D, generator=gen).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(len(lens), Hq, D, generator=gen).to(torch.bfloat16)
    return q, k, v, table


def run(form, q, k, v, table, lens, block, parts=0):
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32).cuda()
    args = (out, q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl)
    if form == "dense":
        pkv.paged_attention_decode(*args, 0.1, num_partitions=parts)
    else:
        n = max(-(-L // block) for L in lens)
        sel = torch.arange(n, dtype=torch.int32, device="cuda").expand(len(lens), k.shape[1], n).contiguous()
        pkv.paged_attention_decode_sparse(*args, sel, 0.1, num_partitions=parts)
    return out.cpu()


CASES = [("dense", 3, 3, 128, 16), ("dense", 4, 2, 64, 16), ("dense", 32, 8, 128, 16), ("dense", 8, 2, 128, 32),
         ("sparse", 3, 3, 64, 32), ("sparse", 4, 2, 128, 16), ("sparse", 16, 4, 128, 16), ("sparse", 32, 8, 64, 32),
         ("sparse", 4, 1, 128, 16), ("sparse", 2, 2, 64, 16)]


@pytest.mark.parametrize("form,Hq,Hkv,D,block", CASES)
def test_weights(form, Hq, Hkv, D, block):
    """Room: the output's bf16, 2^-8; a weight's upper 16 bits leave less than 2^-7 of it, rounded by 2^-8 of that;
    1e-5 for fp32 scores and sums."""
    lens = [1, 2, 3, 5, 9, 17, 40, block, 333, 2000]
    q, k, v, table = inputs(lens, Hq, Hkv, D, block)
    want, size = plain.decode(q, k, v, table, lens, 0.1, block)
    for parts in (0, 1, 19):
        got = run(form, q, k, v, table, lens, block, parts).double()
        err = (got - want).abs() - 2.0 ** -8 * want.abs() - (2.0 ** -15 + 1e-5) * size
        assert float(err.max()) <= 0, (parts, float(err.max()))


@pytest.mark.parametrize("form,Hq,Hkv,D,block", CASES)
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_an_infinite_v(form, Hq, Hkv, D, block, value):
    """It makes its dimension infinite and leaves the others alone, with weights of one and of less."""
    lens = [1, 40, 700]
    q, k, v, table = inputs(lens, Hq, Hkv, D, block, seed=1)
    want, size = plain.decode(q, k, v, table, lens, 0.1, block)
    for s, at in ((0, 0), (1, 37), (2, 400)):
        v[int(table[s, at // block]), :, at % block, 9] = value
    for parts in (0, 1, 19):
        got = run(form, q, k, v, table, lens, block, parts).double()
        assert bool((got[..., 9] == value).all())
        got[..., 9] = want[..., 9]
        assert float(((got - want).abs() - 2.0 ** -8 * want.abs() - (2.0 ** -15 + 1e-5) * size).max()) <= 0

"""Selection where products fall below fp32's normal range: blocks are still ranked by the exact scores."""
import pytest
import torch

import paged_kv_cache_462_b200 as pkv
import plain_serving as plain

pytestmark = pytest.mark.gpu


def check(q, b, table, n, keep, block=16):
    lens = [block * n]
    got = torch.empty(1, b.shape[1], keep, dtype=torch.int32, device="cuda")
    pkv.select_blocks(got, q.cuda(), b.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), block)
    want = plain.select(q, b, table, lens, block, keep, 1, 1)
    assert got.tolist() == want


@pytest.mark.parametrize("exponent", [-58, -63, -66, -69, -72, -75, -80])
@pytest.mark.parametrize("n,keep,D", [(700, 40, 128), (150, 75, 64), (5000, 300, 64)])
def test_tiny_products(exponent, n, keep, D):
    gen = torch.Generator().manual_seed(-exponent)
    table, pool = plain.tables([16 * n], 16, gen)
    b = ((torch.rand(pool, 2, 2, D, generator=gen) + 0.5).sort(2, descending=True)[0] * 2.0 ** exponent).to(torch.bfloat16)
    q = (torch.randn(1, 8, D, generator=gen) * 2.0 ** exponent).to(torch.bfloat16)
    check(q, b, table, n, keep)


def test_tiny_and_ordinary_products_together():
    """Half the blocks score about 2^-136, the others about 1 or -1: the border lies among the tiny ones."""
    gen = torch.Generator().manual_seed(2)
    n, D = 900, 128
    table, pool = plain.tables([16 * n], 16, gen)
    b = (torch.rand(pool, 1, 2, D, generator=gen) + 0.5).sort(2, descending=True)[0] * 2.0 ** -72
    big = torch.randperm(n, generator=gen)[:n // 2]
    b[table[0, big[:200]].long()] += 1.0
    b[table[0, big[200:]].long()] -= 1.0
    q = (torch.rand(1, 4, D, generator=gen) + 0.5) * 2.0 ** -72
    check(q.to(torch.bfloat16), b.to(torch.bfloat16), table, n, 400)

"""What the header says of offsets out of order and of bounds that are not finite."""
import pytest
import torch

import paged_kv_cache_462_b200 as pkv
import plain_serving as plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offsets", [[0, 100, 3, 40, 90], [0, 60, 50, 120, 200], [5, 0, 200, 100, 150], [0, -4, 90, 20, 110],
                                     [0, 1 << 30, 90, 100, 120]])
def test_offsets_out_of_order(offsets):
    """Blocks are written as the sequence's own (valid) entries say or not at all, and the call is flagged."""
    lens, T, D, block = [200, 130, 160, 170], 200, 64, 16
    gen = torch.Generator().manual_seed(1)
    table, pool = plain.tables(lens, block, gen)
    k, v = (torch.randn(T, 2, D, generator=gen).to(torch.bfloat16) for _ in range(2))
    kc, vc = (torch.full((pool, 2, block, D), 7, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = torch.full((pool, 2), 2.0 ** -3, device="cuda"), torch.full((pool, 2), 2.0 ** -3, device="cuda")
    kb = torch.full((pool, 2, 2, D), 5.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sl, ro = torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(offsets, dtype=torch.int32).cuda()
    pkv.reshape_and_cache_block_scales(k.cuda(), v.cuda(), kc, vc, ks, vs, table.cuda(), sl, ro, device_error=err)
    assert err.item() & pkv.DEVERR_ROWS
    err.zero_()
    pkv.update_key_bounds(kb, kc, table.cuda(), sl, ro, T, k_block_scales=ks, device_error=err)
    assert err.item() & pkv.DEVERR_ROWS
    got_k, got_s, got_b = plain.values(kc), ks.cpu().double(), kb.cpu().double()
    for s, L in enumerate(lens):
        codes, scales = torch.full((pool, 2, block, D), 7.0, dtype=torch.float64), torch.full((pool, 2), 2.0 ** -3, dtype=torch.float64)
        a, b = offsets[s], offsets[s + 1]
        good = 0 <= a <= b <= T and b - a <= L
        if good:
            own = [0] * (s + 1) + [b - a] * (len(lens) - s)
            plain.append_block_scales(k[a:b], codes, scales, table, [L if i == s else 0 for i in range(len(lens))], own, block, "int8")
        for j in range(-(-L // block)):
            p = int(table[s, j])
            old = bool((got_k[p] == 7).all())
            if not old:
                assert good and torch.equal(got_k[p], codes[p]) and torch.equal(got_s[p], scales[p])
            if not bool((got_b[p] == 5).all()):
                x = (got_k[p] * got_s[p][:, None, None])[:, :min(block, L - j * block)]
                assert good and torch.equal(got_b[p, :, 0], x.amax(1).to(torch.bfloat16).double())
                assert torch.equal(got_b[p, :, 1], x.amin(1).to(torch.bfloat16).double())
    spare = sorted(set(range(pool)) - set(table[table >= 0].tolist()))
    assert bool((got_k[spare] == 7).all()) and bool((got_b[spare] == 5).all())


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("side", [0, 1])
def test_a_bound_that_is_not_finite_ranks_first(value, side):
    """Whatever the query's sign makes of it."""
    gen = torch.Generator().manual_seed(2)
    table, pool = plain.tables([16 * 300], 16, gen)
    b = torch.randn(pool, 1, 2, 64, generator=gen).sort(2, descending=True)[0].to(torch.bfloat16)
    for j, d in ((40, 0), (77, 1), (150, 2)):
        b[int(table[0, j]), 0, side, d] = value
    q = torch.randn(1, 4, 64, generator=gen).to(torch.bfloat16)
    q[0, :, 0], q[0, :, 1], q[0, :, 2] = 1.0, -1.0, 0.0
    sel = torch.empty(1, 1, 5, dtype=torch.int32, device="cuda")
    pkv.select_blocks(sel, q.cuda(), b.cuda(), table.cuda(), torch.tensor([16 * 300], dtype=torch.int32).cuda(), 16)
    assert sel[0, 0].tolist() == [0, 40, 77, 150, 299]

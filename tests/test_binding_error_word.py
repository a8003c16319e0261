"""device_error is an int32 word: anything the kernels' 4-byte atomics could miss or overrun is refused."""
import pytest
import torch

import paged_kv_cache_462_b200 as pkv
from test_binding_cpu import cuda, fake  # noqa: F401 (fixture)
from test_serving_refusals import bf, i32, rope_inputs, u8


def calls():
    k, kc = bf(5, 2, 128), u8(4, 2, 16, 128)
    slots, ones, scales = cuda(torch.zeros(5, dtype=torch.int64)), cuda(torch.ones(2)), cuda(torch.ones(4, 2))
    x = rope_inputs()
    plain = {n: x[n] for n in ("q_out", "q", "k", "q_weight", "k_weight", "eps", "cos_sin", "positions")}
    return {
        "append": lambda e: pkv.reshape_and_cache(k, k, kc, kc, slots, device_error=e),
        "head_scales": lambda e: pkv.reshape_and_cache_head_scales(k, k, kc, kc, slots, ones, ones, device_error=e),
        "block_scales": lambda e: pkv.reshape_and_cache_block_scales(k, k, kc, kc, scales, scales, i32(3, 6), i32(3),
                                                                     i32(4), device_error=e),
        "bounds": lambda e: pkv.update_key_bounds(bf(4, 2, 2, 128), bf(4, 2, 16, 128), i32(3, 6), i32(3), i32(4), 9,
                                                  device_error=e),
        "norm": lambda e: pkv.qk_norm_rope(**plain, k_out=bf(*x["k"].shape), device_error=e),
        "norm_cache": lambda e: pkv.qk_norm_rope_and_cache(**x, device_error=e),
    }


@pytest.fixture
def lib(fake, monkeypatch):  # noqa: F811
    monkeypatch.setattr(pkv, "_fast", None)
    monkeypatch.setattr(pkv, "_current_raw_stream", lambda dev: 0)
    return fake


@pytest.mark.parametrize("name", sorted(calls()))
def test_the_error_word(lib, name):
    call = calls()[name]
    for good in (None, i32(1), i32(7)):
        call(good)
    given = [a[-2] for n, a in lib.calls]
    assert [bool(getattr(p, "value", p)) for p in given] == [False, True, True]
    n = len(lib.calls)
    for bad in (u8(8)[1:2], u8(4), cuda(torch.zeros(1, dtype=torch.int64)), cuda(torch.zeros(1)), i32(0),
                cuda(torch.zeros(1, dtype=torch.bool))):
        with pytest.raises(TypeError):
            call(bad)
    for bad in (torch.zeros(1, dtype=torch.int32), cuda(torch.zeros(1, dtype=torch.int32), 1), i32(4)[::2]):
        with pytest.raises(ValueError):
            call(bad)
    assert len(lib.calls) == n

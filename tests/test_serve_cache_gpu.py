"""GPU tests of what the 8-bit cache does to what it holds already: codes that move to a larger
scale, and pages mapped ahead through an eviction."""
import math

import pytest
import torch

import serve_ref as ref
from block_sparse_attention_vsa_gb300 import binding

pytestmark = pytest.mark.gpu

D = 128
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("steps", [[1], [4], [1, 1, 1], [2, 7]])
def test_codes_that_move_round_only_below_the_normal_range(steps):
    """Every code there is, moved by powers of two one after another."""
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 0x7f) != 0x7f].view(torch.float8_e4m3fn).double()  # without NaN
    row = torch.zeros(2, D, dtype=torch.float64)
    row.view(-1)[:len(codes)] = codes
    row[1, -1] = 448.0
    cache = binding.new_cache8(1, 64, DEV)
    table = i32([[[0]]])
    x = row.to(torch.bfloat16)[None, None].to(DEV)
    binding.vsa_cache_write(cache, x, x, table, i32([0]))
    held, at, scale = row.clone(), 2, 1.0
    assert torch.equal(cache.k[0, :2].cpu().double(), held)
    for m in steps:
        scale *= 2.0 ** m
        top = torch.full((1, 1, 1, D), 448.0 * scale, dtype=torch.bfloat16, device=DEV)
        binding.vsa_cache_write(cache, top, top, table, i32([at]))
        at += 1
        moved = held * 2.0 ** -m
        held = ref.e4m3(moved)
        normal = moved.abs() >= 2.0 ** -6
        assert torch.equal(held[normal], moved[normal])
        for t in (cache.k, cache.v):
            assert torch.equal(t[0, :2].cpu().double(), held)
        assert cache.k_scale[0] == scale == cache.v_scale[0]
    # one step of the subnormal range in all
    total = row * 2.0 ** -sum(steps)
    assert (held - total).abs().max() <= 2.0 ** -9
    if steps == [1]:  # nine steps of 2^-9 halved: above the smallest subnormal, and rounded
        was = 1.125 * 2.0 ** -6
        assert (held[row == was] == 4 * 2.0 ** -9).all() and was / 2 > 2.0 ** -9


def test_an_infinity_counts_by_the_scale_of_its_time():
    cache, table = binding.new_cache8(1, 64, DEV), i32([[[0]]])
    x = torch.ones((1, 1, 2, D), dtype=torch.bfloat16, device=DEV)
    x[0, 0, 0, 0], x[0, 0, 1] = math.inf, 400.0
    binding.vsa_cache_write(cache, x[:, :, :1].contiguous(), x[:, :, :1].contiguous(), table,
                            i32([0]))
    s = cache.k_scale[0].item()
    assert cache.k[0, 0, 0].item() == 448.0 and s == 2.0 ** -8
    binding.vsa_cache_write(cache, x[:, :, 1:].contiguous(), x[:, :, 1:].contiguous(), table,
                            i32([1]))
    assert cache.k[0, 0, 0].double().item() * cache.k_scale[0].item() == 448.0 * s

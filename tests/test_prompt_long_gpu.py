"""Walks over many keys: longer than a second, the limit of a wait inside most kernels, and sums of
many like terms."""
import math

import pytest
import torch

from block_sparse_attention_vsa_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 128


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("Sq", [1, 129])
def test_the_half_of_an_item_without_queries_waits_for_the_other(Sq):
    """One item, uncut, over 2^27 keys (34 GB): with one query its second tile has none, and the
    first takes a million key tiles."""
    n = 1 << 27
    q = torch.full((1, 1, Sq, D), 2.0, dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros((1, 1, n, D), dtype=torch.bfloat16, device=DEV)
    kv[:, :, 0] = 1.0
    kv[:, :, 0, 1::2] = 3.0  # a score of 512 / sqrt(128), 2^65 times the others' weights
    torch.cuda.synchronize()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    out, lse = binding.vsa_fwd_prompt(q, kv, kv, causal=False, workspace=False)
    b.record()
    code, detail = binding.vsa_device_status()
    assert code == binding.VSA_OK, hex(detail)
    assert a.elapsed_time(b) > 1000.0
    # (2^-38 of the first key's weight in all the others: nothing in either type)
    score = 2.0 * (1.0 + 3.0) * D / 2 / math.sqrt(D) / math.log(2.0)
    assert torch.equal(out, kv[:, :, :1].expand(1, 1, Sq, D))
    assert ((lse.double() - score).abs() <= 2.0 ** -15 * score).all()
    del kv
    torch.cuda.empty_cache()


def test_sums_of_many_like_terms():
    """Flat weights over 2^18 keys in one walk, v of one sign: what the tensor core drops of small
    terms beside a large sum stays below a thousandth.  The columns have means of 0.65 to 2.6, all
    over two octaves of bf16, so that their roundings -- 2^-8 at most, 0.0012 in the mean square -- are
    not the same one 128 times over and a mean of them is within three times 0.0012 / sqrt(128)."""
    n = 1 << 18
    g = torch.Generator().manual_seed(80)
    v = torch.rand((1, 1, n, D), generator=g) * 0.7 + 0.3
    v = (v * torch.linspace(1.0, 4.0, D)).to(torch.bfloat16).to(DEV)
    zero = torch.zeros_like(v)
    out, lse = binding.vsa_fwd_prompt(zero[:, :, :3], zero, v, causal=False, workspace=False)
    code, detail = binding.vsa_device_status()
    assert code == binding.VSA_OK, hex(detail)
    want = v.double().mean(2, keepdim=True)
    off = (out.double() - want) / want
    assert (lse == 18.0).all() and off.abs().max() <= 2.0 ** -8 + 0.001
    assert off.mean().abs() <= 0.001 + 3 * 0.0012 / math.sqrt(D)

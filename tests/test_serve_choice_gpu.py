"""GPU tests of the choice of blocks where its slow path decides: more than 32 blocks inside
the error band of the fp32 sums.  Chosen blocks are whole numbers and compared for equality."""
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


def check(q, k, topk, **kw):
    got = binding.vsa_select_blocks(q.to(DEV), k.to(DEV), topk, **kw)
    want = ref.select_blocks(q, k, topk, **kw)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])


@pytest.mark.parametrize("far", [8, 16, 40])
def test_equal_rows_choose_alike_whatever_their_path(far):
    """Scores 2^60 + small_j - 2^60: an fp64 sum in one order has small_j, in another 0.  Of
    rows with equal q, those that see up to 32 such blocks score candidates, those that see
    more score every block; both have to find the same blocks among the ones that both see."""
    g = torch.Generator().manual_seed(far)
    nk = 48
    k = torch.zeros(1, 1, nk, D)
    k[..., 0], k[..., far] = 2.0 ** 30, -2.0 ** 30
    # small_j in lane 1's columns, 1 .. 48 shuffled, larger for the first 20 blocks
    small = torch.cat([100 + torch.randperm(20, generator=g), 1 + torch.randperm(28, generator=g)])
    k[0, 0, :, 9] = small.float()
    q = torch.zeros(1, 1, nk, D)
    q[..., 0], q[..., far], q[..., 9] = 2.0 ** 30, 2.0 ** 30, 1.0
    q, k = q.to(torch.bfloat16), k.to(torch.bfloat16)
    idx, num = binding.vsa_select_blocks(q.to(DEV), k.to(DEV), 6, causal=True)
    want = sorted(small[:20].argsort(descending=True)[:6].tolist())
    rows = idx[0, 0].tolist()
    assert all(row == rows[-1] for row in rows[20:]), [r for r in rows[20:] if r != rows[-1]][:2]
    if far == 16:  # lanes 0 and 2 cancel before lane 1 is added: the real numbers' order
        assert rows[-1] == want


@pytest.mark.parametrize("nk", [33, 200, 700, 1536, 2048])
def test_many_equal_means(nk):
    """Blocks of a few kinds, more than 32 of a kind: ties go to the lowest index."""
    g = torch.Generator().manual_seed(nk)
    kinds = torch.randn((1, 2, 3, D), generator=g).to(torch.bfloat16)
    k = kinds[:, :, torch.randint(0, 3, (nk,), generator=g)]
    q = torch.randn((1, 2, 20, D), generator=g).to(torch.bfloat16)
    check(q, k, min(nk, 1 + nk // 3), n_near=1)
    check(q, k, 1)


def test_means_with_a_common_offset():
    """Two outlier channels that all key means share: the scores differ far less than they
    are large, so many lie inside the band."""
    g = torch.Generator().manual_seed(9)
    k = torch.randn((1, 1, 600, D), generator=g) * 0.02
    k[..., 3] += 14.0
    k[..., 77] -= 11.0
    q = torch.randn((1, 1, 40, D), generator=g)
    check(q.to(torch.bfloat16), k.to(torch.bfloat16), 60, n_first=1, n_near=1)

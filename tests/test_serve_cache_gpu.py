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


def grown(kept, table, block):
    """The table to go on with: what stays, the pages that went, those mapped ahead."""
    j = torch.arange(table.shape[2], device=table.device)
    held, n_freed = ((kept.lens + block - 1) // block)[:, None, None], kept.n_freed[:, None, None]
    back = kept.freed.gather(2, (j - held).clamp(min=0).expand(table.shape))
    return torch.where(j < held, kept.table, torch.where(j < held + n_freed, back, table))


@pytest.mark.parametrize("block", [64, 128])
def test_pages_mapped_ahead_through_an_eviction(block):
    """Sequences that lose nothing, some blocks, and hold nothing; all with pages mapped ahead.
    Mapped again, every page is there once, and the tokens after land where they should;
    without it the ones that open a block are dropped."""
    g = torch.Generator().manual_seed(block)
    B, H, mb = 3, 2, 12
    held = [2 * block, 7 * block, 0]
    table = torch.randperm(B * H * mb, generator=g).to(torch.int32).view(B, H, mb)

    def bf16(T):
        return torch.randn((B, H, T, D), generator=g).to(torch.bfloat16)

    state = {t: torch.zeros(B * H * mb, block, D).double() for t in "kv"}
    state.update({t: torch.zeros(B * H * mb).double() for t in ("k_scale", "v_scale")})
    state["k_mean"] = torch.zeros(B * H * mb, D).double()
    cache = binding.new_cache8(B * H * mb, block, DEV)
    k, v, zero, n = bf16(7 * block), bf16(7 * block), torch.zeros(B, dtype=torch.int32), i32(held)
    binding.vsa_cache_write(cache, k.to(DEV), v.to(DEV), table.to(DEV), zero.to(DEV), n)
    ref.cache_write(state, k, v, table, zero, n.cpu(), block)
    weight = torch.rand((B, H, mb), generator=g)
    kept = binding.vsa_cache_evict(weight.to(DEV), table.to(DEV), n, 4, block=block, n_last=1)
    want = ref.evict(weight, table, n.cpu(), 4, block, 0, 1)
    assert kept.n_freed.tolist() == [0, 3, 0] and kept.lens.tolist() == [2 * block, 4 * block, 0]
    # (nothing behind what stays)
    for b, at in enumerate((2, 4, 0)):
        assert (kept.table[b, :, at:] == -1).all()
    new = grown(kept, table.to(DEV), block)
    assert new.dtype == torch.int32
    assert torch.equal(new.flatten(1).sort(-1).values, table.to(DEV).flatten(1).sort(-1).values)
    assert torch.equal(new[:, :, :4].cpu()[1], want[0][1, :, :4])
    k, v = bf16(block + 9), bf16(block + 9)
    lost = [t.clone() for t in (cache.k.view(torch.uint8), cache.k_scale)]
    binding.vsa_cache_write(cache, k.to(DEV), v.to(DEV), kept.table, kept.lens)
    assert torch.equal(cache.k.view(torch.uint8), lost[0]) and torch.equal(cache.k_scale, lost[1])
    binding.vsa_cache_write(cache, k.to(DEV), v.to(DEV), new, kept.lens)
    ref.cache_write(state, k, v, new.cpu(), kept.lens.cpu(), None, block)
    for t in "kv":
        assert torch.equal(getattr(cache, t).cpu().double(), state[t])
        assert torch.equal(getattr(cache, t + "_scale").cpu().double(), state[t + "_scale"])
    # attention over the new tokens' blocks finds them
    q, lens = torch.randn((B, 4, 1, D), generator=g).to(torch.bfloat16), kept.lens + block + 9
    from test_serve_gpu import check_attend
    out, lse = binding.vsa_fwd_cache(q.to(DEV), cache, new, lens)
    check_attend(ref.attend(q, state, new.cpu(), lens.cpu(), block), out, lse)


@pytest.mark.parametrize("key,value,query", [(80, 80, -80), (-80, -40, 40), (0, 80, 0),
                                             (80, 0, -100)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_attention_at_the_ends_of_the_scales_range(key, value, query, sign):
    """Scales of 2^+-80 and of either sign, with queries that bring the scores back to size."""
    from test_serve_gpu import cache_case, check_attend, to_cache
    g, table, lens, pages, state = cache_case(81, 2, 2, [700, 70], 64)
    state["k_scale"] = state["k_scale"] * sign * 2.0 ** key
    state["v_scale"] = state["v_scale"] * sign * 2.0 ** value
    q = (torch.randn((2, 8, 1, D), generator=g).double() * 2.0 ** query).to(torch.bfloat16)
    weight = torch.zeros(table.shape, device=DEV)
    out, lse = binding.vsa_fwd_cache(q.to(DEV), to_cache(state), table.to(DEV), lens.to(DEV),
                                     weight=weight)
    check_attend(ref.attend(q, state, table, lens, 64), out, lse, weight)


@pytest.mark.parametrize("tokens", [1, 64, 5000])
@pytest.mark.parametrize("block", [64, 128])
def test_scores_of_minus_infinity_are_not_an_empty_row(tokens, block):
    """A query head whose every score is -infinity (an infinite element against keys of one
    sign) attends tokens: the softmax is not a number, and that shows.  Heads beside it, and a
    sequence that holds nothing, are as ever."""
    from test_serve_gpu import cache_case, check_attend, to_cache
    g, table, lens, pages, state = cache_case(82, 3, 2, [tokens, tokens, 0], block)
    state["k"][..., 5] = state["k"][..., 5].abs().clamp(min=1.0)
    q = torch.randn((3, 8, 1, D), generator=g).to(torch.bfloat16)
    clean = ref.attend(q, state, table, lens, block)
    bad = q.clone()
    bad[0, 2, 0, 5] = -math.inf
    weight = torch.zeros(table.shape, device=DEV)
    out, lse = binding.vsa_fwd_cache(bad.to(DEV), to_cache(state), table.to(DEV), lens.to(DEV),
                                     weight=weight)
    assert out[0, 2].isnan().all() and lse[0, 2].isnan().all()
    assert weight[0, 0, :-(-tokens // block)].isnan().all()
    out, lse, weight = out.cpu(), lse.cpu(), weight.cpu()
    out[0, 2], lse[0, 2] = clean["out"][0, 2].to(torch.bfloat16), clean["lse"][0, 2].float()
    weight[0, 0] = clean["weight"][0, 0].float()
    check_attend(clean, out, lse, weight)
    # weights of nothing in some of the row's parts are nothing: one finite score is enough
    bad[0, 2, 0, 5] = -3e38
    far = dict(state, k=state["k"].clone())
    far["k"][int(table[0, 0, (tokens - 1) // block]), (tokens - 1) % block, 5] = 0.0
    out, lse = binding.vsa_fwd_cache(bad.to(DEV), to_cache(far), table.to(DEV), lens.to(DEV),
                                     scale=1.0)
    last = far["v"][int(table[0, 0, (tokens - 1) // block]), (tokens - 1) % block]
    want = last * state["v_scale"][int(table[0, 0, (tokens - 1) // block])]
    # one weight of 1, all others 0: the value, rounded once
    assert ((out[0, 2, 0].cpu().double() - want).abs() <= 2.0 ** -8 * want.abs()).all()
    assert lse[0, 2].isfinite().all()

"""GPU tests of the operators around the attention -- block means, the choice of blocks, the
8-bit cache and eviction -- against their plain 64-bit forms (tests/serve_ref.py).

Whole numbers (chosen blocks, codes, scales, tables) are compared for equality: the choice
is that of the real numbers, scales are powers of two, codes are correctly rounded.  Floating
results are held to bounds derived from the roundings they go through:

  half steps, relative: bf16 2^-8, fp16 2^-11, fp32 2^-24
  mean    bf16 once, and an fp32 sum of n <= 128 terms: 2^-8 |m| + 128 * 2^-24 * mean|x|
  score   fp32 sum of 128 products that are exact in fp32, the tensor cores' sums being off
          by at most 2^-15 of sum |q||k| in all: ds = 2^-15 * max_j sum |q||k_j| * scale
          (natural units), 4 * 2^-24 of |lse| more for scaling and subtracting
  out     sum of p v: each p is off by 2^-11 (fp16) + 2 ds (numerator and sum) + 2^-20
          (exp2, sums); p below fp16's smallest are lost: 2^-28 of the largest p each;
          bf16 once: 2^-8 |out| + (2^-11 + 2 ds + 2^-20) sum p|v| + n 2^-28 max|v|
  lse     ds * log2(e) + 2^-20 + 4 * 2^-24 |lse|
  weight  relative 2 ds + 2^-18 + 8 * 2^-24 |lse|
"""
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
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(shape, g, mul=1.0):
    return (torch.randn(shape, generator=g) * mul).to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


def same(got, want):
    for x, y in zip(got, want):
        assert torch.equal(x.cpu(), y)


# ------------------------------------------------------------------ block means
@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("B,H,S", [(1, 1, 1), (2, 3, 64), (1, 2, 127), (1, 1, 129),
                                   (2, 2, 1000), (1, 5, 4096)])
def test_block_mean(block, B, H, S):
    g = gen(S + block)
    x = randn((B, H, S, D), g)
    nb = -(-S // block)
    sizes = torch.randint(-3, block + 9, (nb,), generator=g, dtype=torch.int32)
    for sz in (None, sizes):
        got = binding.vsa_block_mean(x.to(DEV), None if sz is None else sz.to(DEV), block=block)
        want, mag = ref.block_mean(x, sz, block)
        assert got.shape == (B, H, nb, D) and got.dtype == torch.bfloat16
        bound = 2.0 ** -8 * want.abs() + 128 * 2.0 ** -24 * mag
        assert ((got.cpu().double() - want).abs() <= bound).all()


def test_block_mean_does_not_read_masked_tokens():
    x = randn((1, 2, 256, D), gen(1))
    x[:, :, 40:64] = math.nan
    x[:, :, 128:192] = math.inf
    x[:, :, 192] = math.nan
    got = binding.vsa_block_mean(x.to(DEV), i32([40, 64, 0, 0]).to(DEV), block=64).cpu()
    assert got.isfinite().all() and (got[:, :, 2:] == 0).all()
    assert binding.vsa_block_mean(x.to(DEV), block=64)[:, :, 0].isnan().all()


# ------------------------------------------------------------------ choosing blocks
SELECT = [
    dict(B=1, Hq=1, Hkv=1, nq=1, nk=1, topk=1),
    dict(B=2, Hq=4, Hkv=2, nq=33, nk=65, topk=7),
    dict(B=1, Hq=3, Hkv=1, nq=31, nk=512, topk=511),
    dict(B=1, Hq=2, Hkv=2, nq=64, nk=513, topk=64, n_near=2),
    dict(B=1, Hq=2, Hkv=1, nq=40, nk=1024, topk=1, n_first=1, n_near=3),
    dict(B=1, Hq=1, Hkv=1, nq=32, nk=1025, topk=100, causal=True),
    dict(B=1, Hq=1, Hkv=1, nq=48, nk=1536, topk=128, n_near=1),
    dict(B=1, Hq=1, Hkv=1, nq=16, nk=2047, topk=300, n_first=4),
    dict(B=1, Hq=1, Hkv=1, nq=8, nk=2048, topk=2048),
    dict(B=2, Hq=2, Hkv=1, nq=50, nk=20, topk=5, causal=True, n_near=2),  # empty rows
    dict(B=1, Hq=2, Hkv=2, nq=20, nk=10, topk=32),                        # topk > nk
    dict(B=1, Hq=1, Hkv=1, nq=5, nk=0, topk=3),
]


def check_select(q, k, c, sizes=None):
    kw = {x: c[x] for x in ("causal", "n_first", "n_near") if x in c}
    got = binding.vsa_select_blocks(q.to(DEV), k.to(DEV), c["topk"],
                                    sizes=None if sizes is None else sizes.to(DEV), **kw)
    same(got, ref.select_blocks(q, k, c["topk"], sizes, **kw))


@pytest.mark.parametrize("c", SELECT, ids=lambda c: f"nq{c['nq']}_nk{c['nk']}_k{c['topk']}")
def test_select_blocks(c):
    g = gen(c["nk"] * 7 + c["nq"])
    q, k = randn((c["B"], c["Hq"], c["nq"], D), g), randn((c["B"], c["Hkv"], c["nk"], D), g)
    check_select(q, k, c)
    if c["nk"]:
        check_select(q, k, c, torch.randint(0, 3, (c["nk"],), generator=g, dtype=torch.int32))
        check_select(q, k, c, torch.zeros(c["nk"], dtype=torch.int32))


def test_select_blocks_equal_scores_go_to_the_lower_index():
    g = gen(3)
    c = dict(topk=9, n_near=1)
    q = randn((1, 1, 40, D), g)
    # 300 key blocks in 3 kinds; then whole numbers, whose scores tie exactly
    k = randn((1, 1, 3, D), g)[:, :, torch.arange(300) % 3]
    check_select(q, k, c)
    qi = torch.randint(-2, 3, (1, 1, 40, D), generator=g).to(torch.bfloat16)
    ki = torch.randint(-2, 3, (1, 1, 700, D), generator=g).to(torch.bfloat16)
    check_select(qi, ki, c)
    check_select(torch.zeros_like(q), k, c)
    check_select(q, torch.zeros_like(k), c)
    check_select(torch.ones_like(q), torch.ones_like(k), c)


def test_select_blocks_close_scores():
    """Scores that differ by less than fp32 sums tell: equal but for one small element."""
    g = gen(4)
    base = randn((1, 1, 1, D), g, 4.0)
    k = base.expand(1, 1, 64, D).clone()
    k[0, 0, :, 5] = torch.randint(-500, 500, (64,), generator=g).to(torch.bfloat16) * 2.0 ** -24
    q = randn((1, 1, 33, D), g, 4.0)
    for topk in (1, 10, 63):
        check_select(q, k, dict(topk=topk))
    # 20 such blocks among others, so that the border of some rows falls inside them
    k2 = randn((1, 1, 200, D), g, 4.0)
    k2[0, 0, 60:80] = k[0, 0, :20]
    for topk in (5, 50, 100, 150):
        check_select(q, k2, dict(topk=topk))


def test_select_blocks_wide_range():
    """Scores beyond fp32 and below its normal range; rows of very different magnitude."""
    g = gen(5)
    q, k = randn((1, 1, 40, D), g), randn((1, 1, 130, D), g)
    q = (q.double() * 10.0 ** torch.randint(-38, 38, (1, 1, 40, 1), generator=g)).to(torch.bfloat16)
    for mul in (1e-30, 1e-5, 1e30):
        check_select(q, (k.double() * mul).to(torch.bfloat16), dict(topk=17))


def test_select_blocks_nan_and_infinity():
    g = gen(6)
    q, k = randn((1, 1, 33, D), g), randn((1, 1, 100, D), g)
    k[0, 0, 3, 7] = math.nan
    k[0, 0, 50, 1] = math.inf
    k[0, 0, 51, 1] = -math.inf
    q[0, 0, 5, 9] = math.nan
    for c in (dict(topk=10), dict(topk=98), dict(topk=100), dict(topk=12, n_first=5, n_near=2)):
        check_select(q, k, c)
    # a NaN in a block that may not be chosen
    sizes = torch.ones(100, dtype=torch.int32)
    sizes[3] = 0
    check_select(q[:, :, 6:].contiguous(), k, dict(topk=10), sizes)


def cache_case(seed, B, Hkv, lens, block, spare=0, codes=True):
    """A table over shuffled pages (extra pages unused), entries past the end poisoned."""
    g = gen(seed)
    need = [-(-n // block) for n in lens]
    mb = max(max(need) + spare, 1)
    pages = Hkv * sum(n + spare for n in need) + 3
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((B, Hkv, mb), 2 ** 31 - 1, dtype=torch.int32)
    at = 0
    for b in range(B):
        for h in range(Hkv):
            n = need[b] + spare
            table[b, h, :n] = perm[at:at + n]
            at += n
    state = None
    if codes:
        state = {t: ref.e4m3(torch.randn((pages, block, D), generator=g) * 60) for t in "kv"}
        for t in ("k_scale", "v_scale"):
            state[t] = torch.exp2(torch.randint(-9, -4, (pages,), generator=g).double())
        state["k_mean"] = randn((pages, D), g).double()
    return g, table, i32(lens), pages, state


def to_cache(state):
    return binding.Cache8(*(state[t].float().to(torch.float8_e4m3fn).to(DEV) for t in "kv"),
                          state["k_scale"].float().to(DEV), state["v_scale"].float().to(DEV),
                          state["k_mean"].to(torch.bfloat16).to(DEV))


CSELECT = [
    dict(B=1, Hq=1, Hkv=1, lens=[1], topk=1),
    dict(B=3, Hq=8, Hkv=2, lens=[0, 64, 65], topk=2),
    dict(B=2, Hq=32, Hkv=2, lens=[5000, 700], topk=20, n_first=2, n_near=3),  # 16 heads a group
    dict(B=1, Hq=3, Hkv=1, lens=[131072], topk=129, n_near=0),                # 2048 blocks
    dict(B=2, Hq=12, Hkv=1, lens=[20000, 64 * 300], topk=299, n_near=1),
    dict(B=1, Hq=4, Hkv=4, lens=[300], topk=40),
]


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("c", CSELECT, ids=lambda c: f"len{max(c['lens'])}_k{c['topk']}")
def test_cache_select(c, block):
    kw = {x: c[x] for x in ("n_first", "n_near") if x in c}
    g, table, lens, pages, _ = cache_case(11, c["B"], c["Hkv"], c["lens"], block, codes=False)
    if c["lens"][0] > 4000:
        table[0, 0, 3] = -1
        table[0, 0, 4] = pages
    q, mean = randn((c["B"], c["Hq"], 1, D), g), randn((pages, D), g)

    def check(q, mean):
        got = binding.vsa_cache_select(q.to(DEV), mean.to(DEV), table.to(DEV), lens.to(DEV),
                                       c["topk"], block=block, **kw)
        same(got, ref.cache_select(q, mean, table, lens, c["topk"], block, **kw))

    check(q, mean)
    check(q, mean[torch.arange(pages) % 2])          # two kinds of blocks: ties
    check(torch.zeros_like(q), mean)
    check(q, torch.ones_like(mean))
    check((q.double() * 1e30).to(torch.bfloat16), (mean.double() * 1e20).to(torch.bfloat16))
    check((q.double() * 1e-30).to(torch.bfloat16), (mean.double() * 1e-20).to(torch.bfloat16))
    bad = mean.clone()
    bad[int(table[0, 0, 0]) if c["lens"][0] else 0, 3] = math.nan
    bad[-1, 4] = math.inf
    check(q, bad)


# ------------------------------------------------------------------ writing the cache
def check_cache(cache, state, mean=True):
    for t in "kv":
        assert torch.equal(getattr(cache, t).cpu().double().nan_to_num(nan=1e9),
                           state[t].nan_to_num(nan=1e9)), t
        assert torch.equal(getattr(cache, t + "_scale").cpu().double(), state[t + "_scale"])
    if mean:
        got, want = cache.k_mean.cpu().double(), state["k_mean"]
        # codes sum exactly; one division, one rounding to fp32 and one to bf16
        assert ((got - want).abs() <= (2.0 ** -8 + 2.0 ** -22) * want.abs()).all()


WRITE = [
    dict(B=1, Hkv=1, T=1, lens=[0], n_new=None),
    dict(B=2, Hkv=2, T=1, lens=[63, 64], n_new=None),
    dict(B=3, Hkv=2, T=1, lens=[1, 127, 200], n_new=[1, 0, 1]),
    dict(B=2, Hkv=3, T=300, lens=[0, 37], n_new=[300, 123]),
    dict(B=2, Hkv=1, T=129, lens=[130, 60], n_new=[200, -4]),   # counts clamped
    dict(B=1, Hkv=2, T=257, lens=[64], n_new=None),
]


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("c", WRITE, ids=lambda c: f"T{c['T']}_at{c['lens'][0]}")
def test_cache_write(c, block):
    g, table, lens, pages, state = cache_case(21, c["B"], c["Hkv"], c["lens"], block,
                                              spare=c["T"] // block + 2)
    shape = (c["B"], c["Hkv"], c["T"], D)
    # rows of different magnitude, so that some raise their page's scale and some do not
    k, v = (randn(shape, g, 1.0).float() * torch.exp2(
        torch.randint(-6, 7, shape[:3] + (1,), generator=g).float()) for _ in range(2))
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    n_new = None if c["n_new"] is None else i32(c["n_new"])
    if n_new is not None:  # what a padded batch holds behind its tokens
        for b, n in enumerate(c["n_new"]):
            k[b, :, max(n, 0):] = math.nan
            v[b, :, max(n, 0):] = math.inf
    cache = to_cache(state)
    binding.vsa_cache_write(cache, k.to(DEV), v.to(DEV), table.to(DEV), lens.to(DEV),
                            None if n_new is None else n_new.to(DEV))
    ref.cache_write(state, k, v, table, lens, n_new, block)
    check_cache(cache, state)


def test_cache_write_special_values_bad_pages_and_overflow():
    block = 64
    g, table, lens, pages, state = cache_case(22, 1, 4, [70], block, spare=2)
    k, v = randn((1, 4, 200, D), g), randn((1, 4, 200, D), g)
    k[0, 0, 3, 5], k[0, 0, 4, 6], v[0, 1, 90, 7] = math.nan, math.inf, -math.inf
    k[0, 2] = 0.0
    v[0, 2] = 1e-38
    k[0, 3, 0:58] = 3.38e38
    table[0, 1, 1], table[0, 3, 2] = -1, pages + 5
    # the table ends at 4 blocks: tokens from 256 on are dropped
    table = table[:, :, :4].contiguous()
    cache = to_cache(state)
    binding.vsa_cache_write(cache, k.to(DEV), v.to(DEV), table.to(DEV), lens.to(DEV))
    ref.cache_write(state, k, v, table, lens, None, block)
    check_cache(cache, state, mean=False)


def test_cache_write_token_by_token_ends_like_at_once():
    """Scales are powers of two: a page filled token by token holds what one filled at once
    does, but for codes that went below the smallest subnormal on the way."""
    g = gen(23)
    k = (torch.randn((1, 2, 130, D), generator=g) * torch.exp2(
        torch.randint(-2, 3, (1, 2, 130, 1), generator=g).float())).to(torch.bfloat16).to(DEV)
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(1, 2, 3)
    one, many = binding.new_cache8(6, 64, DEV), binding.new_cache8(6, 64, DEV)
    binding.vsa_cache_write(one, k, k, table, i32([0]).to(DEV))
    for t in range(130):
        binding.vsa_cache_write(many, k[:, :, t:t + 1].contiguous(),
                                k[:, :, t:t + 1].contiguous(), table, i32([t]).to(DEV))
    assert torch.equal(one.k_scale, many.k_scale) and torch.equal(one.v_scale, many.v_scale)
    a, b = one.k.double(), many.k.double()
    # a code of 2^-6 or more never was subnormal on the way to it; below, one rounding more
    # of half a subnormal step per move, each halved by the moves after it: one step in all
    big = a.abs() > 2.0 ** -6
    assert torch.equal(a[big], b[big])
    assert (a - b).abs().max() <= 2.0 ** -9
    assert torch.equal(many.k.view(torch.uint8), many.v.view(torch.uint8))


# ------------------------------------------------------------------ attention over the cache
def check_attend(r, out, lse=None, weight=None, past=None, keep=0.0):
    ds = 2.0 ** -15 * r["qk"]
    err = (out.cpu().double() - r["out"]).abs()
    bound = (2.0 ** -8 * r["out"].abs() + (2.0 ** -11 + 2 * ds + 2.0 ** -20)[..., None] * r["mag"]
             + (r["count"] * 2.0 ** -28 * r["vmax"])[..., None])
    assert (err <= bound).all(), (err - bound).max()
    empty = r["lse"] == ref.LSE_EMPTY
    assert (out.cpu()[empty] == 0).all()
    if lse is not None:
        got = lse.cpu().double()
        assert (got[empty] == ref.LSE_EMPTY).all()
        bound = ds * math.log2(math.e) + 2.0 ** -20 + 2.0 ** -22 * r["lse"].abs()
        assert ((got - r["lse"]).abs()[~empty] <= bound[~empty]).all()
    if weight is not None:
        Hkv = weight.shape[1]
        B, Hq = r["out"].shape[:2]
        top = lambda x: x.view(B, Hkv, Hq // Hkv).amax(-1, keepdim=True)  # noqa: E731
        rel = 2 * top(ds) + 2.0 ** -18 + 2.0 ** -21 * top(torch.where(empty, 0.0, r["lse"].abs()))
        want = r["weight"] + (0.0 if past is None else keep * past.double())
        bound = rel * r["weight"] + 2.0 ** -23 * want + 1e-30
        assert ((weight.cpu().double() - want).abs() <= bound).all()


ATTEND = [
    dict(B=1, Hq=1, Hkv=1, lens=[1]),
    dict(B=3, Hq=4, Hkv=2, lens=[0, 31, 64]),
    dict(B=2, Hq=16, Hkv=2, lens=[129, 1000]),
    dict(B=1, Hq=10, Hkv=1, lens=[333]),           # two chunks of heads, the last of two
    dict(B=1, Hq=48, Hkv=2, lens=[2000]),          # three chunks
    dict(B=5, Hq=6, Hkv=2, lens=[1, 65, 127, 128, 4097]),
    dict(B=1, Hq=2, Hkv=1, lens=[131072]),         # the longest table
]


def random_listing(g, B, Hkv, mb, width):
    """Listings with duplicates, entries outside the sequence, and odd counts."""
    idx = torch.randint(-2, mb + 3, (B, Hkv, width), generator=g, dtype=torch.int32)
    num = torch.randint(-1, width + 3, (B, Hkv), generator=g, dtype=torch.int32)
    return idx, num


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("c", ATTEND, ids=lambda c: f"B{c['B']}_H{c['Hq']}_{max(c['lens'])}")
def test_fwd_cache(c, block):
    g, table, lens, pages, state = cache_case(31, c["B"], c["Hkv"], c["lens"], block)
    mb = table.shape[2]
    if mb > 8:
        table[0, 0, 5] = -7
        table[0, c["Hkv"] - 1, 6] = pages
    q = randn((c["B"], c["Hq"], 1, D), g, 1.5)
    cache = to_cache(state)
    args = (q.to(DEV), cache, table.to(DEV), lens.to(DEV))
    ws = binding.new_cache_workspace(c["B"], c["Hq"], c["Hkv"], mb, True, DEV)
    past = torch.rand((c["B"], c["Hkv"], mb), generator=g)
    for width in (0, 1, 7, 40):
        idx = num = None
        if width:
            idx, num = random_listing(g, c["B"], c["Hkv"], mb, width)
        kw = dict(idx=None if idx is None else idx.to(DEV), num=None if num is None else num.to(DEV))
        r = ref.attend(q, state, table, lens, block, idx, num)
        out, lse = binding.vsa_fwd_cache(*args, **kw)
        check_attend(r, out, lse)
        weight = past.to(DEV)
        out2, lse2 = binding.vsa_fwd_cache(*args, weight=weight, keep=0.75, workspace=ws, **kw)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
        check_attend(r, out2, lse2, weight, past, 0.75)
        assert int(ws[:65536].abs().sum()) == 0, "counters not returned to zero"
        weight.fill_(math.nan)
        out3, none = binding.vsa_fwd_cache(*args, weight=weight, keep=0.0, lse=None, workspace=ws,
                                           **kw)
        assert none is None and torch.equal(out, out3)
        check_attend(r, out3, None, weight)


@pytest.mark.parametrize("mul", [0.01, 8.0, 40.0])
def test_fwd_cache_peaky_and_flat(mul):
    g, table, lens, pages, state = cache_case(32, 2, 2, [700, 90], 64)
    q = randn((2, 8, 1, D), g, mul)
    cache = to_cache(state)
    weight = torch.zeros(table.shape, device=DEV)
    out, lse = binding.vsa_fwd_cache(q.to(DEV), cache, table.to(DEV), lens.to(DEV), weight=weight)
    check_attend(ref.attend(q, state, table, lens, 64), out, lse, weight)


def test_fwd_cache_scales_of_any_size():
    """Pages whose value scales differ by 2^60, a zero scale, scales that are no power of two."""
    g, table, lens, pages, state = cache_case(33, 1, 2, [640], 64)
    state["v_scale"] = torch.exp2(torch.randint(-60, 1, (pages,), generator=g).double())
    state["v_scale"][int(table[0, 0, 2])] = 0.0
    state["k_scale"] = (state["k_scale"] * 1.3).float().double()
    state["v_scale"] = (state["v_scale"] * 0.7).float().double()
    q = randn((1, 4, 1, D), g)
    out, lse = binding.vsa_fwd_cache(q.to(DEV), to_cache(state), table.to(DEV), lens.to(DEV))
    check_attend(ref.attend(q, state, table, lens, 64), out, lse)
    # queries of very different magnitude, one of zeros
    q = (randn((1, 4, 1, D), g).double() * torch.tensor([1e-30, 1e-3, 1.0, 0.0]).view(1, 4, 1, 1)
         ).to(torch.bfloat16)
    out, lse = binding.vsa_fwd_cache(q.to(DEV), to_cache(state), table.to(DEV), lens.to(DEV))
    check_attend(ref.attend(q, state, table, lens, 64), out, lse)


def test_fwd_cache_does_not_read_past_the_sequence():
    """NaN codes behind the last token of a page, and in pages that are not listed."""
    g, table, lens, pages, state = cache_case(34, 2, 2, [70, 161], 64)
    q = randn((2, 4, 1, D), g)
    clean = ref.attend(q, state, table, lens, 64)
    used = set()
    for b in range(2):
        for h in range(2):
            for j in range(-(-int(lens[b]) // 64)):
                p = int(table[b, h, j])
                used.add(p)
                for t in "kv":
                    state[t][p, max(0, min(64, int(lens[b]) - 64 * j)):] = math.nan
    for p in set(range(pages)) - used:
        state["k"][p] = state["v"][p] = math.nan
        state["k_scale"][p] = math.nan
    out, lse = binding.vsa_fwd_cache(q.to(DEV), to_cache(state), table.to(DEV), lens.to(DEV))
    check_attend(clean, out, lse)


def test_fwd_cache_rows_of_nothing():
    """Many rows a piece, every other one without a token: a warp may be at the next row's
    end before another has read this one's statistics."""
    lens = [(j * 7) % 130 if j % 2 == 0 else 0 for j in range(160)]
    g, table, lens, pages, state = cache_case(41, 160, 8, lens, 64)
    q = randn((160, 8, 1, D), g)
    args = (q.to(DEV), to_cache(state), table.to(DEV), lens.to(DEV))
    out, lse = binding.vsa_fwd_cache(*args)
    check_attend(ref.attend(q, state, table, lens, 64), out, lse)
    ws = binding.new_cache_workspace(160, 8, 8, table.shape[2])
    for _ in range(20):
        again = binding.vsa_fwd_cache(*args, workspace=ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_calls_on_another_stream_while_the_current_one_is_busy():
    """What a call with a stream allocates (a zeroed workspace among it) is ready on that
    stream, not behind the current one's work."""
    g, table, lens, pages, state = cache_case(42, 2, 2, [3000, 500], 64)
    q = randn((2, 8, 1, D), g).to(DEV)
    cache, table, lens = to_cache(state), table.to(DEV), lens.to(DEV)
    weight = torch.rand(table.shape, generator=g).to(DEV)
    x = randn((1, 2, 1000, D), g).to(DEV)

    def calls(stream):
        m = binding.vsa_block_mean(x, stream=stream)
        return (m, *binding.vsa_select_blocks(m, m, 4, stream=stream),
                *binding.vsa_cache_select(q, cache.k_mean, table, lens, 5, stream=stream),
                *binding.vsa_fwd_cache(q, cache, table, lens, stream=stream),
                *binding.vsa_cache_evict(weight, table, lens, 5, stream=stream))

    want = calls(None)
    busy = torch.ones(4096, 4096, device=DEV)
    # blocks for the current stream's allocator to hand out, full of ones
    filled = [torch.ones(1 << 18, dtype=torch.int32, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    del filled
    for _ in range(20):
        busy = busy @ busy
    side = torch.cuda.Stream()
    got = calls(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_fwd_cache_shared_workspace_streams_and_graphs():
    """One workspace for two shapes in turn, a call on another stream, a captured call
    replayed on new contents: the same bits each time."""
    cases = [cache_case(35, 3, 2, [3000, 100, 1], 64), cache_case(36, 1, 1, [9000], 64)]
    runs = []
    for g, table, lens, pages, state in cases:
        q = randn((table.shape[0], table.shape[1] * 4, 1, D), g).to(DEV)
        runs.append((q, to_cache(state), table.to(DEV), lens.to(DEV)))
    n = max(binding.cache_workspace_bytes(r[0].shape[0], r[0].shape[1], r[2].shape[1],
                                          r[2].shape[2], True) for r in runs)
    ws = torch.zeros(n // 4 + 4, dtype=torch.int32, device=DEV)
    weights = [torch.zeros(r[2].shape, device=DEV) for r in runs]
    first = [binding.vsa_fwd_cache(*r) for r in runs]
    for _ in range(3):
        for r, w, f in zip(runs, weights, first):
            got = binding.vsa_fwd_cache(*r, weight=w, keep=0.0, workspace=ws)
            assert torch.equal(got[0], f[0]) and torch.equal(got[1], f[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.vsa_fwd_cache(*runs[0], stream=side, workspace=ws)
    side.synchronize()
    assert torch.equal(got[0], first[0][0])
    q, cache, table, lens = runs[0]
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        binding.vsa_fwd_cache(q, cache, table, lens, out=out, lse=lse, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0][0]) and torch.equal(lse, first[0][1])
    lens.copy_(torch.minimum(i32([100, 90, 1]).to(DEV), lens))
    q.neg_()
    graph.replay()
    torch.cuda.synchronize()
    want = binding.vsa_fwd_cache(q, cache, table, lens)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_far_pages_pass_32_bit_offsets():
    """Pages beyond 2^32 bytes of codes (524,288 pages of 8 KB and more)."""
    pages, block = 530000, 64
    g = gen(37)
    cache = binding.new_cache8(pages, block, DEV)
    table = i32([[[529999, 0, 524289]], [[7, 529998, -1]]]).to(DEV)
    k, v = randn((2, 1, 150, D), g), randn((2, 1, 150, D), g)
    n_new = i32([150, 120])
    binding.vsa_cache_write(cache, k.to(DEV), v.to(DEV), table, i32([0, 0]).to(DEV), n_new.to(DEV))
    order = [529999, 0, 524289, 7, 529998]
    near = i32([[[0, 1, 2]], [[3, 4, -1]]])  # the same pages, renumbered
    state = {t: torch.zeros(5, block, D, dtype=torch.float64) for t in "kv"}
    state.update(k_scale=torch.zeros(5).double(), v_scale=torch.zeros(5).double(),
                 k_mean=torch.zeros(5, D).double())
    ref.cache_write(state, k, v, near, i32([0, 0]), n_new, block)
    pick = torch.tensor(order, device=DEV)
    k8, v8 = (x.view(torch.uint8)[pick].view(torch.float8_e4m3fn) for x in (cache.k, cache.v))
    small = binding.Cache8(k8, v8, cache.k_scale[pick], cache.v_scale[pick], cache.k_mean[pick])
    check_cache(small, state)
    q = randn((2, 2, 1, D), g)
    lens = i32([150, 120])
    out, lse = binding.vsa_fwd_cache(q.to(DEV), cache, table, lens.to(DEV))
    check_attend(ref.attend(q, state, near, lens, block), out, lse)
    same(binding.vsa_cache_select(q.to(DEV), cache.k_mean, table, lens.to(DEV), 1, n_near=0),
         ref.cache_select(q, small.k_mean.cpu(), near, lens, 1, block, n_near=0))


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("budget,n_first,n_last", [(1, 0, 1), (5, 1, 2), (40, 0, 1), (64, 3, 61),
                                                   (2048, 0, 1)])
def test_cache_evict(block, budget, n_first, n_last):
    lens = [0, 1, block * 40, block * 41 + 1, block * 200 - 3, block * 2048]
    g, table, lens_t, pages, _ = cache_case(41, len(lens), 2, lens, block, codes=False)
    weight = torch.rand(table.shape, generator=g)
    weight[2] = (weight[2] * 4).floor()        # ties
    weight[3, 0, 5], weight[3, 0, 7], weight[3, 0, 9] = math.nan, math.inf, -math.inf
    weight[3, 1, 3], weight[3, 1, 4] = 0.0, -0.0
    got = binding.vsa_cache_evict(weight.to(DEV), table.to(DEV), lens_t.to(DEV), budget,
                                  block=block, n_first=n_first, n_last=n_last)
    want = ref.evict(weight, table, lens_t, budget, block, n_first, n_last)
    assert torch.equal(got.weight.cpu().nan_to_num(nan=7e7), want[1].nan_to_num(nan=7e7))
    same((got.table, got.lens, got.freed, got.n_freed), (want[0], want[2], want[3], want[4]))


# ------------------------------------------------------------------ runs of them together
@pytest.mark.parametrize("block", [64, 128])
def test_choose_then_attend_and_its_gradient(block):
    """block means -> LUT -> forward -> backward, as a training step uses them: the LUT is
    the exact choice on the means, and the gradients those of attention over it, by the
    formula (autograd in fp64) and by differences along a direction."""
    from gpu_util import OUT_MAX, OUT_MEAN
    g = gen(51)
    B, Hq, Hkv, nb, topk = 1, 4, 2, 9, 4
    S = nb * block
    q, k, v = randn((B, Hq, S, D), g), randn((B, Hkv, S, D), g), randn((B, Hkv, S, D), g)
    sizes = torch.full((nb,), block, dtype=torch.int32)
    sizes[-1] = 17
    qd, kd, vd, sd = q.to(DEV), k.to(DEV), v.to(DEV), sizes.to(DEV)
    qm, km = binding.vsa_block_mean(qd, block=block), binding.vsa_block_mean(kd, sd, block=block)
    idx, num = binding.vsa_select_blocks(qm, km, topk, sizes=sd, n_near=1)
    same((idx, num), ref.select_blocks(qm.cpu(), km.cpu(), topk, sizes, n_near=1))
    out, lse = binding.vsa_fwd_gqa(qd, kd, vd, idx, num, sd, block=block)
    dout = randn(out.shape, g)
    grads = binding.vsa_bwd(qd, kd, vd, out, dout.to(DEV), lse, idx, num, sd, block=block)

    mask = torch.zeros(B, Hq, S, S, dtype=torch.bool)
    ic = idx.cpu()
    for h in range(Hq):
        for i in range(nb):
            for j in ic[0, h, i].tolist():
                if j >= 0:
                    mask[0, h, i * block:(i + 1) * block, j * block:j * block + int(sizes[j])] = True

    def attention(q, k, v):
        kk, vv = k.repeat_interleave(Hq // Hkv, 1), v.repeat_interleave(Hq // Hkv, 1)
        s = (q @ kk.transpose(-1, -2) / math.sqrt(D)).masked_fill(~mask, -math.inf)
        return torch.softmax(s, -1) @ vv

    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    want = attention(*leaves)
    err = (out.cpu().double() - want).abs()
    assert err.max() <= OUT_MAX and err.mean() <= OUT_MEAN
    exact = torch.autograd.grad(want, leaves, dout.double())
    for got, w in zip(grads, exact):
        assert (got.cpu().double() - w).abs().max() <= 2e-2 * w.abs().max()
    # along random directions: (f(x + e d) - f(x - e d)) / 2e against grad . d
    for n, (t, got, w) in enumerate(zip(leaves, grads, exact)):
        d = torch.randn(t.shape, generator=g, dtype=torch.float64)
        e = 1e-4
        args = [x.detach() for x in leaves]
        hi, lo = list(args), list(args)
        hi[n], lo[n] = args[n] + e * d, args[n] - e * d
        with torch.no_grad():
            slope = ((attention(*hi) - attention(*lo)) * dout.double()).sum() / (2 * e)
        dot = (got.cpu().double() * d).sum()
        # each gradient element is off by at most 2e-2 of the largest (above); a random
        # direction adds such errors up with their root, 4 of its deviations at most
        assert (dot - slope).abs() <= 2e-2 * w.abs().max() * math.sqrt(d.numel()) * 4


def test_a_server_run():
    """A prompt written into the cache, then tokens one by one: written, blocks chosen,
    attended with accumulating weights, and evicted over a budget -- each step against the
    plain forms on a reference cache kept beside it."""
    block, B, Hkv, G = 64, 2, 2, 4
    g, table, _, pages, state = cache_case(52, B, Hkv, [600, 300], block, spare=2)
    for t in state:
        state[t].zero_()
    cache = to_cache(state)
    mb = table.shape[2]
    weight = torch.zeros(table.shape, device=DEV)
    table_d, lens_d = table.to(DEV), i32([0, 0]).to(DEV)
    ws = binding.new_cache_workspace(B, Hkv * G, Hkv, mb, True, DEV)
    n_new = i32([550, 250])
    for step in range(40):
        T = 550 if step == 0 else 1
        k, v = randn((B, Hkv, T, D), g), randn((B, Hkv, T, D), g)
        n = n_new if step == 0 else i32([1, 1])
        binding.vsa_cache_write(cache, k.to(DEV), v.to(DEV), table_d, lens_d, n.to(DEV))
        ref.cache_write(state, k, v, table_d.cpu(), lens_d.cpu(), n, block)
        lens_d = lens_d + n.to(DEV)
        check_cache(cache, state)
        q = randn((B, Hkv * G, 1, D), g)
        idx, num = binding.vsa_cache_select(q.to(DEV), cache.k_mean, table_d, lens_d, 4,
                                            n_first=1, n_near=1)
        same((idx, num), ref.cache_select(q, cache.k_mean.cpu(), table_d.cpu(), lens_d.cpu(), 4,
                                          block, 1, 1))
        past = weight.cpu()
        out, lse = binding.vsa_fwd_cache(q.to(DEV), cache, table_d, lens_d, idx=idx, num=num,
                                         weight=weight, workspace=ws)
        r = ref.attend(q, state, table_d.cpu(), lens_d.cpu(), block, idx.cpu(), num.cpu())
        check_attend(r, out, lse, weight, past, 1.0)
        if step % 16 == 15:
            got = binding.vsa_cache_evict(weight, table_d, lens_d, 7 - step // 16, n_first=1,
                                          n_last=1)
            want = ref.evict(weight.cpu(), table_d.cpu(), lens_d.cpu(), 7 - step // 16, block, 1, 1)
            same(got, want)
            assert int(got.n_freed[0]) > 0
            table_d, weight, lens_d = got.table.clone(), got.weight, got.lens
            # the freed pages are the pool to grow from
            for b in range(B):
                held = -(-int(lens_d[b]) // block)
                for h in range(Hkv):
                    back = got.freed[b, h, :int(got.n_freed[b])]
                    table_d[b, h, held:held + len(back)] = back


def test_one_launch_each():
    g, table, lens, pages, state = cache_case(61, 1, 2, [300], 64, spare=1)
    cache, table, lens = to_cache(state), table.to(DEV), lens.to(DEV)
    x = randn((1, 2, 64, D), g).to(DEV)
    q = randn((1, 4, 1, D), g).to(DEV)
    weight = torch.zeros(table.shape, device=DEV)
    for call in (lambda: binding.vsa_block_mean(x), lambda: binding.vsa_select_blocks(x, x, 4),
                 lambda: binding.vsa_cache_select(q, cache.k_mean, table, lens, 2),
                 lambda: binding.vsa_cache_write(cache, x, x, table, lens),
                 lambda: binding.vsa_fwd_cache(q, cache, table, lens, weight=weight),
                 lambda: binding.vsa_cache_evict(weight, table, lens, 2)):
        call()
        assert binding.vsa_last_launch_count() == 1
    torch.cuda.synchronize()


# ------------------------------------------------------------------ refusals of the binding
def test_refusals():
    g, table, lens, pages, state = cache_case(62, 1, 2, [300], 64)
    cache, table, lens = to_cache(state), table.to(DEV), lens.to(DEV)
    q = randn((1, 4, 1, D), g).to(DEV)
    x = randn((1, 2, 64, D), g).to(DEV)
    bad = [
        lambda: binding.vsa_block_mean(x.float()),
        lambda: binding.vsa_block_mean(x.cpu()),
        lambda: binding.vsa_block_mean(x, i32([1, 2]).to(DEV)),
        lambda: binding.vsa_block_mean(x.transpose(1, 2)),
        lambda: binding.vsa_select_blocks(x, x[:, :, :, :64].contiguous(), 3),
        lambda: binding.vsa_cache_select(x, cache.k_mean, table, lens, 2),      # not one token
        lambda: binding.vsa_cache_write(cache, x, x[:, :1].contiguous(), table, lens),
        lambda: binding.vsa_cache_write(cache, x, x, table, lens.long()),
        lambda: binding.vsa_fwd_cache(q, cache, table, lens, idx=table),        # no num
        lambda: binding.vsa_fwd_cache(q, cache._replace(k_scale=cache.k_scale[1:]), table, lens),
        lambda: binding.vsa_fwd_cache(q, cache, table, lens, weight=cache.k_scale),
        lambda: binding.vsa_fwd_cache(q, cache, table, lens.cpu()),
        lambda: binding.vsa_fwd_cache(q[:, :3].contiguous(), cache, table, lens),
        lambda: binding.vsa_cache_evict(cache.k_scale, table, lens, 2),
    ]
    for call in bad:
        with pytest.raises((ValueError, TypeError)):
            call()
    weight = torch.zeros(table.shape, device=DEV)
    refused = [
        lambda: binding.vsa_select_blocks(x, x, 0),
        lambda: binding.vsa_select_blocks(x[:, :1].contiguous(), x, 2),         # 1 % 2 heads
        lambda: binding.vsa_fwd_cache(q, cache, table, lens, scale=0.0),
        lambda: binding.vsa_fwd_cache(q, cache, table, lens, weight=weight, keep=math.nan),
        lambda: binding.vsa_fwd_cache(q, cache, table, lens,
                                      workspace=torch.zeros(64, dtype=torch.int32, device=DEV)),
        lambda: binding.vsa_fwd_cache(q, cache, table, lens, out=q),
        lambda: binding.vsa_cache_evict(weight, table, lens, 2, n_first=2, n_last=1),
        lambda: binding.vsa_cache_evict(weight, table, lens, 2, n_last=0),
    ]
    for call in refused:
        with pytest.raises(binding.VsaError):
            call()
    torch.cuda.synchronize()


def test_short_and_long_way_agree():
    """A call without a stream goes the short way through C++, one with the current stream the
    long way through Python: the same results, and the same refusals (above)."""
    g, table, lens, pages, state = cache_case(63, 2, 2, [300, 70], 64, spare=2)
    cache, table, lens = to_cache(state), table.to(DEV), lens.to(DEV)
    other = binding.Cache8(*(t.view(torch.uint8).clone().view(t.dtype) if i < 2 else t.clone()
                             for i, t in enumerate(cache)))
    x = randn((2, 2, 80, D), g).to(DEV)
    q = randn((2, 4, 1, D), g).to(DEV)
    sizes = i32([64, 11]).to(DEV)
    now = torch.cuda.current_stream()
    means = [binding.vsa_block_mean(x, sizes, stream=s) for s in (None, now)]
    assert torch.equal(*means)
    for a, b in zip(*(binding.vsa_select_blocks(m, m, 3, sizes=sizes, causal=True, n_near=1,
                                                stream=s) for m, s in zip(means, (None, now)))):
        assert torch.equal(a, b)
    n_new = i32([80, 5]).to(DEV)
    for c, s in ((cache, None), (other, now)):
        binding.vsa_cache_write(c, x, x, table, lens, n_new, stream=s)
    for a, b in zip(cache, other):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    lens = lens + n_new
    picks = [binding.vsa_cache_select(q, cache.k_mean, table, lens, 3, n_first=1, stream=s)
             for s in (None, now)]
    ws = binding.new_cache_workspace(2, 4, 2, table.shape[2], True, DEV)
    outs = []
    for (idx, num), s in zip(picks, (None, now)):
        weight = torch.ones(table.shape, device=DEV)
        out = binding.vsa_fwd_cache(q, cache, table, lens, idx=idx, num=num, scale=0.1,
                                    weight=weight, keep=0.5, workspace=ws, stream=s)
        outs.append((idx, num) + out + (weight,) +
                    tuple(binding.vsa_cache_evict(weight, table, lens, 4, n_first=1, stream=s)))
    for a, b in zip(*outs):
        assert a.dtype == b.dtype and torch.equal(a, b)
    kept = binding.vsa_cache_evict(weight, table, lens, 4)
    assert kept.n_freed.tolist() == [2, 0] and kept.lens.tolist() == [380 - 128, 75]
    # outputs given are the ones returned
    out, lse = torch.empty_like(q), torch.empty((2, 4, 1), device=DEV)
    got = binding.vsa_fwd_cache(q, cache, table, lens, out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse
    assert binding.vsa_fwd_cache(q, cache, table, lens, lse=False, workspace=ws)[1] is None


def test_an_empty_listing_is_refused_and_an_empty_row_is_empty():
    g, table, lens, pages, state = cache_case(64, 2, 2, [300, 70], 64)
    cache, table, lens = to_cache(state), table.to(DEV), lens.to(DEV)
    q = randn((2, 4, 1, D), g).to(DEV)
    ws = binding.new_cache_workspace(2, 4, 2, table.shape[2], False, DEV)
    none = torch.zeros((2, 2, 0), dtype=torch.int32, device=DEV)
    num = torch.zeros((2, 2), dtype=torch.int32, device=DEV)
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises(ValueError):
            binding.vsa_fwd_cache(q, cache, table, lens, idx=none, num=num, workspace=ws,
                                  stream=stream)
    out, lse = binding.vsa_fwd_cache(q, cache, table, lens, idx=none.new_zeros((2, 2, 3)), num=num,
                                     workspace=ws)
    assert (out == 0).all() and (lse == ref.LSE_EMPTY).all()


@pytest.mark.parametrize("tokens", [1, 64, 5000])
def test_fwd_cache_nan_in_an_attended_token(tokens):
    """A NaN among the attended keys or values makes the row NaN, never an empty one; other
    sequences and heads do not see it."""
    g, table, lens, pages, state = cache_case(65, 2, 2, [tokens, tokens], 64)
    for t in "kv":
        bad = {x: y.clone() for x, y in state.items()}
        bad[t][int(table[0, 1, (tokens - 1) // 64]), (tokens - 1) % 64] = math.nan
        q = randn((2, 4, 1, D), g)
        weight = torch.zeros(table.shape, device=DEV)
        out, lse = binding.vsa_fwd_cache(q.to(DEV), to_cache(bad), table.to(DEV), lens.to(DEV),
                                         weight=weight)
        assert out[0, 2:].isnan().all()
        assert lse[0, 2:].isnan().all() == (t == "k")
        clean = ref.attend(q, state, table, lens, 64)
        keep = torch.ones(2, 4, 1, dtype=torch.bool)
        keep[0, 2:] = False
        ok, want = out.cpu().double()[keep], clean["out"][keep]
        assert ok.isfinite().all() and (ok - want).abs().max() <= 2.0 ** -7 * clean["vmax"].max()


def test_cache_write_without_means():
    g, table, lens, pages, state = cache_case(66, 1, 2, [50], 64, spare=2)
    k, v = randn((1, 2, 90, D), g), randn((1, 2, 90, D), g)
    cache = to_cache(state)
    for c in (cache._replace(k_mean=None),):
        binding.vsa_cache_write(c, k.to(DEV), v.to(DEV), table.to(DEV), lens.to(DEV))
    before = state["k_mean"].clone()
    ref.cache_write(state, k, v, table, lens, None, 64)
    check_cache(cache, state, mean=False)
    assert torch.equal(cache.k_mean.cpu().double(), before)


@pytest.mark.parametrize("topk,n_first,n_near", [(1, 2, 3), (3, 1, 3), (4, 3, 3), (2, 0, 40)])
def test_cache_select_with_more_forced_blocks_than_places(topk, n_first, n_near):
    """The lowest of the forced blocks are chosen, and nothing is written past a row's end."""
    g, table, lens, pages, _ = cache_case(67, 3, 2, [700, 64, 5000], 64, codes=False)
    q, mean = randn((3, 6, 1, D), g), randn((pages, D), g)
    got = binding.vsa_cache_select(q.to(DEV), mean.to(DEV), table.to(DEV), lens.to(DEV), topk,
                                   n_first=n_first, n_near=n_near)
    same(got, ref.cache_select(q, mean, table, lens, topk, 64, n_first, n_near))

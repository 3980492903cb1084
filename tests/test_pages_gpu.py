"""The pages of the 8-bit cache against plain forms, one entry at a time: reserving, letting go,
forking, closing up, and a server's run through all of them."""
import random

import pytest
import torch

import prompt_ref as ref
import serve_ref
from block_sparse_attention_vsa_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 128


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def words(refs):
    return [w - (1 << 32) if w >> 31 else w for w in ref.bits(refs)]


def to_pool(refs):
    return binding.Pages(i32(refs), i32(words(refs)))


def same_pool(pool, refs):
    assert pool.refs.tolist() == refs
    n = len(refs)
    got = [w & 0xffffffff for w in pool.free.tolist()]
    if n % 32 and got:  # bits past the pool are anyone's
        got[-1] &= (1 << n % 32) - 1
    assert got == ref.bits(refs)


def state(seed, B, H, mb, block, pages, lens, share=0):
    """A table with pages for every block held, in shuffled order, and the counts; `share` rows
    name a page of another one."""
    r = random.Random(seed)
    perm = list(range(pages))
    r.shuffle(perm)
    refs = [0] * pages
    table = [[[-1] * mb for _ in range(H)] for _ in range(B)]
    for b in range(B):
        for h in range(H):
            for j in range(-(-lens[b] // block)):
                table[b][h][j] = perm.pop()
                refs[table[b][h][j]] += 1
    for _ in range(share):
        b, c, h = r.randrange(B), r.randrange(B), r.randrange(H)
        n = min(lens[b], lens[c]) // block
        if b != c and n:
            j = r.randrange(n)
            refs[table[b][h][j]] -= 1
            table[b][h][j] = table[c][h][j]
            refs[table[b][h][j]] += 1
    return table, refs


def cache(seed, pages, block, mean=True):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (2, pages, block, D), generator=g, dtype=torch.uint8)
    scale = torch.rand((2, pages), generator=g) + 0.5
    km = torch.randn((pages, D), generator=g).to(torch.bfloat16)
    c = codes.to(DEV).view(torch.float8_e4m3fn)
    s = scale.to(DEV)
    return binding.Cache8(c[0], c[1], s[0], s[1], km.to(DEV) if mean else None)


def raw(c):
    return [None if t is None else t.view(torch.uint8 if t.dtype == torch.float8_e4m3fn
                                          else t.dtype).clone() for t in c]


CASES = [  # B, H, mb, block, pages, longest
    (1, 1, 1, 64, 1, 64), (3, 2, 9, 64, 200, 500), (5, 3, 40, 128, 1000, 4000),
    (2, 1, 70, 64, 33, 900), (9, 8, 33, 64, 5000, 2000), (300, 1, 3, 64, 700, 128),
    (4, 2, 600, 64, 31, 0), (2, 2, 1200, 64, 40_000, 70_000)]


def lengths(c, seed):
    B, H, mb, block, pages, longest = c
    r = random.Random(seed)
    room = pages // (B * H) if B * H else 0
    return [min(r.randint(0, longest), room * block, mb * block) for _ in range(B)]


@pytest.mark.parametrize("c", CASES, ids=str)
@pytest.mark.parametrize("more", ["one", "some", "all"])
def test_reserve(c, more):
    B, H, mb, block, pages, _ = c
    lens = lengths(c, 1)
    table, refs = state(2, B, H, mb, block, pages, lens)
    r = random.Random(3)
    new = None if more == "one" else [r.randint(-2, 200) if more == "some" else mb * block
                                      for _ in range(B)]
    pool, t = to_pool(refs), i32(table)
    lacking = binding.vsa_pages_reserve(pool, t, i32(lens), None if new is None else i32(new),
                                        block=block)
    want = ref.reserve(refs, table, lens, new, block)
    assert lacking.tolist() == want and t.tolist() == table
    same_pool(pool, refs)


@pytest.mark.parametrize("c", CASES, ids=str)
@pytest.mark.parametrize("trim", [True, False], ids=["ahead", "all"])
def test_free(c, trim):
    B, H, mb, block, pages, _ = c
    lens = lengths(c, 4)
    table, refs = state(5, B, H, mb, block, pages, lens, share=20)
    back = [max(-3, n - random.Random(n).randint(0, 300)) for n in lens] if trim else None
    pool, t = to_pool(refs), i32(table)
    binding.vsa_pages_free(pool, t, None if back is None else i32(back), block=block)
    ref.free(refs, table, back, block)
    assert t.tolist() == table
    same_pool(pool, refs)


def test_free_takes_what_names_no_page_and_pages_given_up_too_often():
    refs = [1, 2, 0, 1] + [0] * 30
    table = [[[0, 1, 1, 1, -1, -7, 34, 1 << 30, 2, 2, 0]]]
    pool, t = to_pool(refs), i32(table)
    binding.vsa_pages_free(pool, t)
    ref.free(refs, table, None, 64)
    assert t.tolist() == table and refs[:4] == [0, 0, 0, 1]
    same_pool(pool, refs)


def test_reserve_replaces_what_names_no_page():
    refs = [0] * 40
    table = [[[-1, 99, -5, 7, -1]]]
    refs[7] = 1
    pool, t = to_pool(refs), i32(table)
    binding.vsa_pages_reserve(pool, t, i32([0]), i32([300]))
    assert t.tolist() == [[[0, 1, 2, 7, 3]]]
    ref.reserve(refs, table, [0], [300], 64)
    same_pool(pool, refs)


@pytest.mark.parametrize("c", CASES, ids=str)
@pytest.mark.parametrize("N", [1, 4, 37])
def test_fork(c, N):
    B, H, mb, block, pages, _ = c
    lens = lengths(c, 6)
    table, refs = state(7, B, H, mb, block, pages, lens, share=5)
    r = random.Random(8)
    parent = [r.randint(-1, B) if r.random() < 0.2 else r.randrange(B) for _ in range(N)]
    kv = cache(9, pages, block, mean=N != 4)
    pool, t = to_pool(refs), i32(table)
    want_codes = raw(kv)
    got = binding.vsa_cache_fork(kv, pool, t, i32(lens), i32(parent))
    out, n_out, lacking, copies = ref.fork(refs, table, lens, parent, block, mb)
    assert got.table.tolist() == out and got.lens.tolist() == n_out
    assert got.lacking.tolist() == lacking and t.tolist() == table
    same_pool(pool, refs)
    for src, dst, n in copies:
        for x in want_codes[:2]:
            x[dst, :n] = x[src, :n]
        for x in want_codes[2:]:
            if x is not None:
                x[dst] = x[src]
    for x, y in zip(raw(kv), want_codes):
        assert x is None and y is None or torch.equal(x, y)


# divided among several CTAs: many rows, and rows of many blocks
MANY = [(140, 8, 6, 64, 4000, 300), (17, 8, 1000, 64, 6000, 1000)]


@pytest.mark.parametrize("c,more", [(MANY[0], "one"), (MANY[0], "some"), (MANY[0], "all"),
                                    (MANY[1], "one"), (MANY[1], "some")], ids=str)
def test_reserve_of_large_tables(c, more):
    test_reserve(c, more)


def test_reserve_of_long_prompts():
    """Among short ones, out of a pool with holes of all sizes, whose end some do not get."""
    B, H, mb, pages = 17, 8, 1000, 9000
    r = random.Random(21)
    refs = [int(r.random() < (p % 1000) / 1000) for p in range(pages)]
    held = [p for p in range(pages) if refs[p]]
    table = [[[-1] * mb for _ in range(H)] for _ in range(B)]
    for p in held[:2000]:  # entries that have a page already, anywhere
        b, h, j = r.randrange(B), r.randrange(H), r.randrange(60)
        if table[b][h][j] < 0:
            table[b][h][j] = p
    lens = [r.randint(0, 2000) for _ in range(B)]
    new = [r.choice([0, 1, 70, 300, 9000, 40_000]) for _ in range(B)]
    pool, t = to_pool(refs), i32(table)
    lacking = binding.vsa_pages_reserve(pool, t, i32(lens), i32(new))
    want = ref.reserve(refs, table, lens, new, 64)
    assert sum(want) > 0 and lacking.tolist() == want and t.tolist() == table
    same_pool(pool, refs)


def test_fork_of_many_rows():
    test_fork(MANY[0], 150)


@pytest.mark.parametrize("c", CASES, ids=str)
@pytest.mark.parametrize("full", [False, True], ids=["holes", "full"])
def test_compact(c, full):
    B, H, mb, block, pages, _ = c
    lens = lengths(c, 10)
    table, refs = state(11, B, H, mb, block, pages, lens, share=7)
    if full:  # every page in use, by another table
        refs = [n or 1 for n in refs]
    table[0][0][mb - 1] = pages + 3 if lens[0] <= (mb - 1) * block else table[0][0][mb - 1]
    kv = cache(12, pages, block, mean=not full)
    pool, t = to_pool(refs), i32(table)
    before = raw(kv)
    to, n_used = binding.vsa_cache_compact(kv, pool, t)
    want_to, used = ref.compact(refs, table)
    assert to.tolist() == want_to and n_used.tolist() == [used] and t.tolist() == table
    same_pool(pool, refs)
    src = [p for p, x in enumerate(want_to) if x >= 0]
    dst = [want_to[p] for p in src]
    for x, y in zip(raw(kv), before):
        assert x is None and y is None or torch.equal(x[dst], y[src])


def test_a_large_pool():
    """Bitmaps of many words a thread, and what one call asks for past them."""
    pages = 3_000_001
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[::3] = 1
    refs[:1_000_000] = 1
    bit = torch.nn.functional.pad((refs == 0).long(), (0, -pages % 32)).view(-1, 32)
    w = (bit << torch.arange(32, device=DEV)).sum(-1)
    free = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
    pool = binding.Pages(refs.clone(), free.clone())
    t = torch.full((40, 8, 1500), -1, dtype=torch.int32, device=DEV)
    lacking = binding.vsa_pages_reserve(pool, t, i32([0] * 40), i32([96_000] * 40))
    want = torch.nonzero(refs == 0)[:40 * 8 * 1500, 0].to(torch.int32)
    assert torch.equal(t.flatten(), want) and (lacking == 0).all()
    binding.vsa_pages_free(pool, t)
    assert torch.equal(pool.refs, refs) and torch.equal(pool.free, free) and (t == -1).all()


def test_far_pages_pass_32_bit_offsets():
    """Pages whose codes lie more than 2^32 bytes into the pool."""
    pages, block = 600_000, 64  # 4.9 GB a tensor
    kv = binding.new_cache8(pages, block)
    src = pages - 1
    kv.k[src].view(torch.uint8).fill_(7)
    kv.v[src].view(torch.uint8).fill_(9)
    kv.k_scale[src], kv.v_scale[src], kv.k_mean[src] = 2.0, 4.0, 1.0
    refs = [0] * pages
    refs[src] = 1
    pool = to_pool(refs)
    t = i32([[[src, -1]]])
    got = binding.vsa_cache_fork(kv, pool, t, i32([40]), i32([0]))
    assert got.table.tolist() == [[[0, -1]]]
    assert (kv.k[0, :40].view(torch.uint8) == 7).all() and (kv.k[0, 40:].view(torch.uint8) == 0).all()
    to, n_used = binding.vsa_cache_compact(kv, pool, t)
    assert t.tolist() == [[[1, -1]]] and n_used.item() == 2 and to[src].item() == 1
    assert (kv.k[1].view(torch.uint8) == 7).all() and (kv.v[1].view(torch.uint8) == 9).all()
    assert kv.k_scale[1] == 2.0 and kv.v_scale[1] == 4.0 and (kv.k_mean[1] == 1.0).all()


def bf16(shape, g):
    return torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV)


def test_a_server_from_prompt_to_eviction():
    """reserve -> attention over the prompts and their writing -> fork -> tokens -> evict ->
    free -> compact: what a child attends is its parent's past and its own tokens."""
    g = torch.Generator().manual_seed(30)
    B, Hq, H, mb, block, pages = 2, 4, 2, 8, 64, 64
    n = [150, 64]
    kv, pool = binding.new_cache8(pages, block), binding.new_pages(pages)
    table = torch.full((B, H, mb), -1, dtype=torch.int32, device=DEV)
    lens = i32([0, 0])
    k, v, q = bf16((B, H, 150, D), g), bf16((B, H, 150, D), g), bf16((B, Hq, 150, D), g)
    assert (binding.vsa_pages_reserve(pool, table, lens, i32(n)) == 0).all()
    out, _ = binding.vsa_fwd_prompt(q, k, v, i32(n), i32(n))
    binding.vsa_cache_write(kv, k, v, table, lens, i32(n))
    lens += i32(n)
    for b in range(B):
        want, bound = ref.attend(q[b], k[b], v[b], [n[b]], [n[b]], [0], [0])
        there = ~want["out"].isnan()
        assert ((out[b].double() - want["out"]).abs() <= bound["out"])[there].all()
    # two samples of the first prompt, one of the second; the prompts' own rows end
    kids = binding.vsa_cache_fork(kv, pool, table, lens, i32([0, 0, 1]))
    binding.vsa_pages_free(pool, table)
    assert kids.lens.tolist() == [150, 150, 64] and (kids.lacking == 0).all()
    assert torch.equal(kids.table[0, :, :2], kids.table[1, :, :2])
    assert (kids.table[0, :, 2] != kids.table[1, :, 2]).all()
    # a token each, with tokens of their own
    table, lens = kids.table, kids.lens
    assert (binding.vsa_pages_reserve(pool, table, lens) == 0).all()
    k1, v1, q1 = bf16((3, H, 1, D), g), bf16((3, H, 1, D), g), bf16((3, Hq, 1, D), g)
    binding.vsa_cache_write(kv, k1, v1, table, lens)
    lens = lens + 1
    weight = torch.zeros((3, H, mb), device=DEV)
    o1, l1 = binding.vsa_fwd_cache(q1, kv, table, lens, weight=weight)

    def dense(q1, table, lens):
        state = {x: t.cpu().double() for x, t in zip(("k", "v", "k_scale", "v_scale", "k_mean"), kv)}
        return serve_ref.attend(q1.cpu(), state, table.cpu(), lens.cpu(), block, None, None)

    want = dense(q1, table, lens)  # (how near that attention comes, its own tests say)
    assert ((o1.cpu().double() - want["out"]).abs() <= 2.0 ** -6 * (1 + want["out"].abs())).all()
    # the new tokens are the children's own
    a, b = (table[i, 0, 2].item() for i in (0, 1))
    assert not torch.equal(kv.k[a, 22].view(torch.uint8), kv.k[b, 22].view(torch.uint8))
    # evicted to two blocks, what goes is let go, the rest closed up: the same attention
    gone = binding.vsa_cache_evict(weight, table, lens, budget=2)
    binding.vsa_pages_free(pool, gone.freed)
    o2, _ = binding.vsa_fwd_cache(q1, kv, gone.table, gone.lens)
    to, n_used = binding.vsa_cache_compact(kv, pool, gone.table)
    o3, _ = binding.vsa_fwd_cache(q1, kv, gone.table, gone.lens)
    torch.cuda.synchronize()
    assert torch.equal(o2, o3)
    named = gone.table[gone.table >= 0]
    assert named.max().item() < n_used.item() and n_used.item() == len(set(named.tolist()))
    count = torch.bincount(named.long(), minlength=pages)
    assert torch.equal(count.int(), pool.refs)
    binding.vsa_pages_free(pool, gone.table)
    same_pool(pool, [0] * pages)


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "graph"])
def test_a_step_behind_a_busy_stream(captured):
    """free -> reserve -> fork -> free -> compact with nothing between, on buffers that hold
    another (valid) state until the moment the step's own is put there."""
    c = (4, 2, 12, 64, 150, 700)
    B, H, mb, block, pages, _ = c
    sets = []
    for seed in (40, 41):
        lens = lengths(c, seed)
        table, refs = state(seed, B, H, mb, block, pages, lens)
        sets.append((table, refs, lens))
    kv = cache(42, pages, block)
    start = raw(kv)
    t, pool, n = i32(sets[1][0]), to_pool(sets[1][1]), i32(sets[1][2])
    src = [i32(sets[0][0]), *to_pool(sets[0][1]), i32(sets[0][2])]
    back = (i32(sets[0][2]) - 70).clamp(min=0)
    parent, new = i32([3, 0, 0, 2]), i32([90, 1, 0, 65])

    def step():
        for dst, s in zip((t, *pool, n), src):
            dst.copy_(s)
        n.copy_(back)
        binding.vsa_pages_free(pool, t, n)
        lacking = binding.vsa_pages_reserve(pool, t, n, new)
        kids = binding.vsa_cache_fork(kv, pool, t, n, parent)
        binding.vsa_pages_free(pool, t)
        to, used = binding.vsa_cache_compact(kv, pool, kids.table)
        return lacking, kids, to, used

    step()
    torch.cuda.synchronize()
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
    for x, y in zip(kv, start):
        x.view(y.dtype).copy_(y)
    for dst, s in zip((t, *pool), (i32(sets[1][0]), *to_pool(sets[1][1]))):
        dst.copy_(s)
    busy = torch.ones(4096, 4096, device=DEV, dtype=torch.bfloat16)
    for _ in range(20):
        busy = busy @ busy * 1e-4
    if captured:
        graph.replay()
    else:
        got = step()
    lacking, kids, to, used = got
    table, refs, lens = sets[0][0], sets[0][1], back.tolist()
    ref.free(refs, table, lens, block)
    assert lacking.tolist() == ref.reserve(refs, table, lens, new.tolist(), block)
    out, n_out, none, _ = ref.fork(refs, table, lens, parent.tolist(), block, mb)
    ref.free(refs, table, None, block)
    want_to, want_used = ref.compact(refs, out)
    assert kids.table.tolist() == out and kids.lens.tolist() == n_out
    assert kids.lacking.tolist() == none
    assert to.tolist() == want_to and used.tolist() == [want_used]
    same_pool(pool, refs)


def test_short_and_long_way_agree(monkeypatch):
    c = (3, 2, 9, 64, 200, 500)
    B, H, mb, block, pages, _ = c
    lens = lengths(c, 50)
    runs = []
    for fast in (True, False):
        if not fast:
            monkeypatch.setattr(binding, "_fast", False)
        table, refs = state(51, B, H, mb, block, pages, lens)
        kv, pool, t = cache(52, pages, block), to_pool(refs), i32(table)
        lacking = binding.vsa_pages_reserve(pool, t, i32(lens), i32([70, 1, 0]))
        kids = binding.vsa_cache_fork(kv, pool, t, i32(lens), i32([0, 2]))
        binding.vsa_pages_free(pool, t, i32(lens))
        to, used = binding.vsa_cache_compact(kv, pool, t)
        runs.append([lacking, *kids, to, used, t, *pool])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_another_stream_and_launches():
    pool = binding.new_pages(40)
    t = torch.full((2, 1, 4), -1, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    binding.vsa_pages_reserve(pool, t, i32([0, 0]), i32([256, 64]))
    assert binding.vsa_last_launch_count() == 1
    torch.cuda.synchronize()
    kv = binding.new_cache8(40)
    kids = binding.vsa_cache_fork(kv, pool, t, i32([250, 64]), i32([0]), stream=side)
    assert binding.vsa_last_launch_count() == 2
    binding.vsa_pages_free(pool, t, stream=side)
    assert binding.vsa_last_launch_count() == 1
    to, used = binding.vsa_cache_compact(kv, pool, kids.table, stream=side)
    assert binding.vsa_last_launch_count() == 2
    side.synchronize()
    assert kids.table.tolist() == [[[0, 1, 2, 3]]] and used.item() == 4


def test_nothing_to_do():
    kv, pool = binding.new_cache8(10), binding.new_pages(10)
    none = torch.empty((0, 2, 3), dtype=torch.int32, device=DEV)
    assert binding.vsa_pages_reserve(pool, none, i32([])).shape == (0,)
    binding.vsa_pages_free(pool, none)
    kids = binding.vsa_cache_fork(kv, pool, none, i32([]), i32([0, -1]))
    assert kids.lens.tolist() == [0, 0] and (kids.table == -1).all()
    kids = binding.vsa_cache_fork(kv, pool, none, i32([]), i32([]))
    assert kids.table.shape == (0, 2, 3)
    to, used = binding.vsa_cache_compact(kv, pool, none)
    assert used.item() == 0 and (to == -1).all()
    empty = binding.new_pages(0)
    t = torch.full((1, 1, 2), -1, dtype=torch.int32, device=DEV)
    assert binding.vsa_pages_reserve(empty, t, i32([0]), i32([100])).tolist() == [2]
    same_pool(pool, [0] * 10)


def test_refusals():
    kv, pool = binding.new_cache8(40), binding.new_pages(40)
    t = torch.full((2, 1, 4), -1, dtype=torch.int32, device=DEV)
    lens, parent = i32([0, 0]), i32([0])
    for call in (
            lambda: binding.vsa_pages_reserve(pool, t.long(), lens),
            lambda: binding.vsa_pages_reserve(pool, t.cpu(), lens),
            lambda: binding.vsa_pages_reserve(pool, t, i32([0])),
            lambda: binding.vsa_pages_reserve(pool, t, lens, i32([0])),
            lambda: binding.vsa_pages_reserve(pool, t, lens, block=1 << 40),
            lambda: binding.vsa_pages_reserve(binding.Pages(pool.refs, pool.refs), t, lens),
            lambda: binding.vsa_pages_free(pool, t[:, :, ::2]),
            lambda: binding.vsa_cache_fork(kv, binding.new_pages(41), t, lens, parent),
            lambda: binding.vsa_cache_fork(kv, pool, t, lens, parent.long()),
            lambda: binding.vsa_cache_fork(kv, pool, t, lens, parent, table_out=t),
            lambda: binding.vsa_cache_compact(kv, binding.new_pages(39), t)):
        with pytest.raises((ValueError, TypeError)):
            call()
    for call in (lambda: binding.vsa_pages_reserve(pool, t, lens, block=32),
                 lambda: binding.vsa_pages_free(pool, pool.refs[:8].view(2, 1, 4)),
                 lambda: binding.vsa_cache_fork(kv, pool, t, lens, parent, table_out=t[:1]),
                 lambda: binding.vsa_pages_reserve(pool, t, t[:, 0, 0].as_strided((2,), (1,)))):
        with pytest.raises(binding.VsaError):
            call()
    same_pool(pool, [0] * 40)

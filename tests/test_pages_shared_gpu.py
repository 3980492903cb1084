"""Pages that several entries name, and sequences whose length is set back into one."""
import random

import pytest
import torch

import prompt_ref as ref
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


def to_pool(refs):
    return binding.Pages(i32(refs), i32([w - (1 << 32) if w >> 31 else w for w in ref.bits(refs)]))


def same_pool(pool, refs):
    assert pool.refs.tolist() == refs
    got = [w & 0xffffffff for w in pool.free.tolist()]
    if len(refs) % 32:  # bits past the pool are anyone's
        got[-1] &= (1 << len(refs) % 32) - 1
    assert got == ref.bits(refs)


def reserve(refs, table, lens, n_new, block):
    """The plain form, and next tokens' blocks whose page others name too."""
    shared = []
    for b, rows in enumerate(table):
        n = max(0, lens[b])
        more = 1 if n_new is None else max(0, n_new[b])
        shared.append(sum(0 <= p < len(refs) and refs[p] > 1 for row in rows
                          for p in row[n // block:min(len(row), -(-(n + more) // block))][:1]))
    return [x + y for x, y in zip(ref.reserve(refs, table, lens, n_new, block), shared)]


@pytest.mark.parametrize("B,H,mb,block,most", [
    (1, 1, 1, 64, 64), (3, 2, 9, 64, 500), (5, 3, 40, 128, 4000), (300, 1, 3, 64, 128),
    (140, 8, 6, 64, 300), (17, 8, 1000, 64, 3000), (1100, 9, 2, 64, 100)], ids=str)
@pytest.mark.parametrize("more", ["one", "some", "all"])
def test_reserve_reports_shared_pages(B, H, mb, block, most, more):
    """Tables whose entries name one another's pages, at lengths and ranges of all kinds, out of a
    pool that may be too small: what is there stays, and is counted."""
    r = random.Random(B * mb + block)
    lens = [min(r.randint(0, most), mb * block) for _ in range(B)]
    pages = H * sum(-(-n // block) + r.randint(0, 2) for n in lens) + 40
    perm = list(range(pages))
    r.shuffle(perm)
    refs, table = [0] * pages, [[[-1] * mb for _ in range(H)] for _ in range(B)]
    held = []
    for b in range(B):
        for h in range(H):
            for j in range(-(-lens[b] // block)):
                p = r.choice(held) if held and r.random() < 0.3 else perm.pop()
                held.append(p)
                table[b][h][j] = p
                refs[p] += 1
    back = [max(0, n - r.choice([0, 0, 1, block, 3 * block])) for n in lens]
    new = None if more == "one" else [r.randint(-2, 200) if more == "some" else mb * block
                                      for _ in range(B)]
    pool, t = to_pool(refs), i32(table)
    lacking = binding.vsa_pages_reserve(pool, t, i32(back), None if new is None else i32(new),
                                        block=block)
    want = reserve(refs, table, back, new, block)
    assert lacking.tolist() == want and t.tolist() == table
    same_pool(pool, refs)


def codes(kv, page, n):
    return [x[page, :n].view(torch.uint8).clone() for x in kv[:2]]


@pytest.mark.parametrize("who", ["parent", "child"])
def test_rejected_drafts_behind_a_fork(who):
    """62 tokens and 4 drafts, forked at 66, one side's drafts rejected: its next tokens would go
    into the block that both hold.  That is reported; its own fork writes a copy, and what the
    other side attends stays what it was."""
    g = torch.Generator().manual_seed(70)
    H, Hq, mb, block = 2, 4, 4, 64

    def bf16(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV)

    kv, pool = binding.new_cache8(32, block), binding.new_pages(32)
    table = torch.full((1, H, mb), -1, dtype=torch.int32, device=DEV)
    k, v, q = bf16(1, H, 66, D), bf16(1, H, 66, D), bf16(1, Hq, 1, D)
    assert binding.vsa_pages_reserve(pool, table, i32([0]), i32([66])).tolist() == [0]
    binding.vsa_cache_write(kv, k, v, table, i32([0]), i32([66]))
    kid = binding.vsa_cache_fork(kv, pool, table, i32([66]), i32([0]))
    back, stay = (table, kid.table) if who == "parent" else (kid.table, table)
    before, lse = binding.vsa_fwd_cache(q, kv, stay, i32([66]))
    block0 = codes(kv, stay[0, 0, 0].item(), 64)

    held = i32([63])
    binding.vsa_pages_free(pool, back, held)
    assert torch.equal(back[:, :, 0], stay[:, :, 0]) and (back[:, :, 1:] == -1).all()
    room = binding.vsa_pages_reserve(pool, back, held, i32([3]))
    assert room.tolist() == [H]           # the shared block, in each head; the other has its page
    assert torch.equal(back[:, :, 0], stay[:, :, 0]) and (back[:, :, 1] >= 0).all()
    # the way on: a fork of it in its place
    binding.vsa_pages_free(pool, back, held)
    own = binding.vsa_cache_fork(kv, pool, back, held, i32([0]))
    binding.vsa_pages_free(pool, back)
    assert binding.vsa_pages_reserve(pool, own.table, own.lens, i32([3])).tolist() == [0]
    assert (own.table[:, :, 0] != stay[:, :, 0]).all()
    k2, v2 = bf16(1, H, 3, D) * 30, bf16(1, H, 3, D) * 30  # larger: the block's scale moves
    binding.vsa_cache_write(kv, k2, v2, own.table, own.lens, i32([3]))
    after, lse2 = binding.vsa_fwd_cache(q, kv, stay, i32([66]))
    assert torch.equal(before, after) and torch.equal(lse, lse2)
    for x, y in zip(block0, codes(kv, stay[0, 0, 0].item(), 64)):
        assert torch.equal(x, y)
    named = torch.cat([own.table.flatten(), stay.flatten()])
    count = torch.bincount(named[named >= 0].long(), minlength=32).int()
    assert torch.equal(count, pool.refs) and count.max().item() == 1


def test_shared_pages_in_front_are_nobodys_matter():
    """Children that go on behind what they share lack nothing."""
    kv, pool = binding.new_cache8(64), binding.new_pages(64)
    table = torch.full((1, 2, 6), -1, dtype=torch.int32, device=DEV)
    for n in (128, 130):
        assert binding.vsa_pages_reserve(pool, table, i32([0]), i32([n])).tolist() == [0]
        kids = binding.vsa_cache_fork(kv, pool, table, i32([n]), i32([0, 0, 0]))
        for _ in range(2):  # (asking twice takes nothing twice)
            lacking = binding.vsa_pages_reserve(pool, kids.table, kids.lens, i32([1, 70, 200]))
            assert lacking.tolist() == [0, 0, 0]
        binding.vsa_pages_free(pool, kids.table)
    binding.vsa_pages_free(pool, table)
    same_pool(pool, [0] * 64)


def test_other_tables_follow_when_a_pool_is_closed_up():
    """Two tables on one pool, one given to the call, the other by `to`; -1 stays -1 although the
    pool's last page is in use."""
    kv, pool = binding.new_cache8(20), binding.new_pages(20)
    tables = [torch.full((2, 2, 3), -1, dtype=torch.int32, device=DEV) for _ in range(2)]
    gone = torch.full((1, 2, 3), -1, dtype=torch.int32, device=DEV)
    for t, n in ((tables[0], [128, 64]), (gone, [150]), (tables[1], [64, 190])):
        assert (binding.vsa_pages_reserve(pool, t, i32([0] * len(n)), i32(n)) == 0).all()
    assert tables[1].max().item() == 19 and (tables[1] == -1).any()
    for t in tables:
        for b in range(2):
            for page in t[b][t[b] >= 0].tolist():
                kv.k[page].view(torch.uint8).fill_(page)
    was = [t.clone() for t in tables]
    binding.vsa_pages_free(pool, gone)
    to, n_used = binding.vsa_cache_compact(kv, pool, tables[0])
    t = tables[1]
    tables[1] = torch.where(t >= 0, to[t.clamp(min=0)], t)
    assert n_used.item() == 14
    for t, w in zip(tables, was):
        assert torch.equal(t >= 0, w >= 0) and t.max().item() < 14
        for page, before in zip(t[t >= 0].tolist(), w[w >= 0].tolist()):
            assert (kv.k[page].view(torch.uint8) == before).all()
    named = torch.cat([t[t >= 0] for t in tables])
    assert torch.equal(torch.bincount(named.long(), minlength=20).int(), pool.refs)

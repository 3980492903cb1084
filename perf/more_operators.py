"""Attention over whole prompts with its gradient, and the pages of the 8-bit cache, measured.

`run` is one pass: through the library's entry points where `own` is true, otherwise the
plain form of the same operator in elementary torch operations (32 bits).  `exact` is the
operator in 64 bits, written apart from the plain form; page operators give whole numbers and
copies, which have no such value.

Prompts.  Sequence b has nq queries and nk keys; query i attends keys j < nk, with `causal`
those with j <= i + nk - nq.  "packed" holds the sequences one behind the other, [tokens,
heads, 128], with their starts; "padded" is a batch [B, heads, S, 128] with lengths, whose
rows behind a length get 0 (lse: the value of a row that attends nothing).

Pages.  A pool has `pages` pages of `block` tokens each: refs[p] counts the table entries that
name page p, bit p % 32 of free[p // 32] says that none does.  The lowest free page is taken
first.  table[b, h, j] is the page of block j of sequence b and key/value head h, -1 where
there is none; lens[b] counts the tokens held.
"""
import math
import random

import torch

own = False

D = 128
LOG2E = 1.4426950408889634
LSE_EMPTY = -3.4028234663852886e38


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # four short prompts that arrive together (one of a single token)
        dict(name="prompt_small", op="fwd", form="packed", B=4, Hq=32, Hkv=8, lo=1, hi=157,
             held_lo=0, held_hi=0, short=0, causal=True),
        # the next 2,000 tokens or less of four prompts behind what is held of them
        dict(name="prompt_chunk", op="fwd", form="padded", B=4, Hq=64, Hkv=8, lo=701, hi=2000,
             held_lo=4001, held_hi=16411, short=0, causal=True),
        # a batch of ragged prompts up to 32,768 tokens, 24 heads
        dict(name="prompt_long", op="fwd", form="packed", B=4, Hq=24, Hkv=24, lo=1001, hi=32768,
             held_lo=0, held_hi=0, short=0, causal=True),
        # a training step on short packed samples
        dict(name="train_small", op="train", form="packed", B=5, Hq=12, Hkv=12, lo=33, hi=411,
             held_lo=0, held_hi=0, short=0, causal=True),
        # a training step on clips of ragged lengths, every token attending every other
        dict(name="train_clip", op="train", form="padded", B=3, Hq=12, Hkv=12, lo=2001, hi=5000,
             held_lo=0, held_hi=0, short=0, causal=False),
        # a training step on packed documents up to 12,345 tokens with grouped heads
        dict(name="train_long", op="train", form="packed", B=3, Hq=32, Hkv=8, lo=501, hi=12345,
             held_lo=0, held_hi=0, short=0, causal=True),
        # room for one more token of every sequence of a serving batch
        dict(name="reserve_token", op="reserve", B=64, Hkv=8, lo=1, hi=8191, n_lo=1, n_hi=1,
             block=64, spare=4096),
        # room for long prompts, most of it behind nothing yet
        dict(name="reserve_prompts", op="reserve", B=16, Hkv=8, lo=1, hi=64, n_lo=1001,
             n_hi=98304, block=64, spare=3000),
        # four samples continued from each of eight stems
        dict(name="fork_samples", op="fork", B=8, N=32, Hkv=8, lo=1, hi=8191, block=64,
             spare=2048),
        # one long video's context shared by eight continuations
        dict(name="fork_long", op="fork", B=1, N=8, Hkv=24, lo=98272, hi=98272, block=64,
             spare=1024),
        # a small pool with a third of its pages free, closed up
        dict(name="compact_small", op="compact", B=4, Hkv=8, lo=100, hi=2000, block=64, hole=50),
        # a pool that held a serving batch, after half of it left
        dict(name="compact_large", op="compact", B=16, Hkv=8, lo=1001, hi=16384, block=64,
             hole=100),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "train", "train", "reserve", "fork", "compact"])
    block = rng.choice([64, 64, 128])
    if op in ("fwd", "train"):
        hi = _log(rng, 1, 16384 if op == "fwd" else 8192)
        b = _log(rng, 1, max(1, min(16, 32768 // hi)))
        hkv = rng.choice([1, 2, 3, 4, 8, 12])
        causal = rng.random() < 0.7
        held = _log(rng, 1, 16384) if rng.random() < 0.3 else 0
        most = 32 if hi * (hi + held) * b < 1 << 28 else 24
        form = rng.choice(["packed", "padded"])
        return dict(op=op, form=form, B=b, Hq=hkv * _log(rng, 1, max(1, most // hkv)), Hkv=hkv,
                    lo=rng.randint(1, hi), hi=hi, held_lo=rng.randint(0, held), held_hi=held,
                    short=0 if held or rng.random() < 0.8 else rng.randint(1, hi), causal=causal)
    hkv = _log(rng, 1, 8)
    hi = _log(rng, 1, 16384)
    if op == "reserve":
        n_hi = _log(rng, 1, 98304)
        return dict(op=op, B=_log(rng, 1, max(1, min(64, (1 << 20) // (hi + n_hi)))), Hkv=hkv,
                    lo=rng.randint(0, hi), hi=hi, n_lo=rng.randint(0, n_hi), n_hi=n_hi,
                    block=block, spare=_log(rng, 1, 4096))
    if op == "fork":
        b = _log(rng, 1, max(1, min(16, (1 << 17) // hi)))
        return dict(op=op, B=b, N=_log(rng, 1, 24), Hkv=hkv, lo=rng.randint(0, hi), hi=hi,
                    block=block, spare=_log(rng, 1, 2048))
    b = _log(rng, 1, max(1, min(16, (1 << 17) // hi)))
    return dict(op=op, B=b, Hkv=hkv, lo=rng.randint(1, hi), hi=hi, block=block,
                hole=rng.randint(0, 100))


def _spread(B, lo, hi):
    """One length per sequence in [lo, hi], the first the longest."""
    r = random.Random(B * 1000003 + lo * 101 + hi)
    return [hi] + [r.randint(lo, hi) for _ in range(B - 1)]


def _lengths(c):
    """Queries and keys of each sequence."""
    nq = _spread(c["B"], c["lo"], c["hi"])
    held = _spread(c["B"], c["held_lo"], c["held_hi"])
    return nq, [max(0, n + h - c["short"]) for n, h in zip(nq, held)]


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _bf16(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lens):
    r = [0]
    for n in lens:
        r.append(r[-1] + n)
    return r


def _free_words(refs):
    """The bitmap of pages without a reference."""
    n = refs.numel()
    bit = torch.nn.functional.pad((refs == 0).long(), (0, -n % 32)).view(-1, 32)
    word = (bit << torch.arange(32, device=refs.device)).sum(-1)
    return torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)


def _pool(c, g, lens, mb, pages):
    """A table with a page for every block held, in shuffled order, and the pool's counts; all
    in one tensor, so that a state can be put back at once."""
    B, H, block = c["B"], c["Hkv"], c["block"]
    need = [-(-n // block) for n in lens]
    words = -(-pages // 32)
    ints = torch.zeros(B * H * mb + pages + words, dtype=torch.int32, device="cuda")
    table = ints[:B * H * mb].view(B, H, mb)
    refs = ints[B * H * mb:B * H * mb + pages]
    free = ints[B * H * mb + pages:]
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table.fill_(-1)
    at = 0
    for b in range(B):
        table[b, :, :need[b]] = perm[at:at + H * need[b]].view(H, need[b])
        at += H * need[b]
    refs[perm[:at].long()] = 1
    free.copy_(_free_words(refs))
    return {"ints": ints, "table": table, "refs": refs, "free": free}


def _codes(c, g, pages):
    """A filled cache: codes of normal values, scales around 2^-7, means of the keys."""
    r = {}
    for t in ("k", "v"):
        x = torch.randn((pages, c["block"], D), generator=g, device="cuda")
        r[t] = (x * 90.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
        e = torch.randint(-8, -5, (pages,), generator=g, device="cuda")
        r[t + "_scale"] = torch.exp2(e.float())
    r["k_mean"] = _bf16((pages, D), g)
    return r


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    st = {"case": dict(c)}
    if op in ("fwd", "train"):
        nq, nk = _lengths(c)
        Hq, Hkv = c["Hq"], c["Hkv"]
        if c["form"] == "packed":
            tq, tk = sum(nq), sum(nk)
            st["q_seq"], st["k_seq"] = _ints(_starts(nq)), _ints(_starts(nk))
            if tq == tk and nq == nk:  # slices of one projection's output
                x = _bf16((tq, Hq + 2 * Hkv, D), g)
                st["q"], st["k"], st["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
            else:
                st["q"] = _bf16((tq, Hq, D), g)
                st["k"], st["v"] = _bf16((tk, Hkv, D), g), _bf16((tk, Hkv, D), g)
            st["dout"] = _bf16((tq, Hq, D), g) if op == "train" else None
        else:
            B = c["B"]
            st["q_seq"], st["k_seq"] = _ints(nq), _ints(nk)
            st["q"] = _bf16((B, Hq, max(nq), D), g)
            st["k"] = _bf16((B, Hkv, max(max(nk), 1), D), g)
            st["v"] = _bf16((B, Hkv, max(max(nk), 1), D), g)
            st["dout"] = _bf16((B, Hq, max(nq), D), g) if op == "train" else None
        return st
    block = c["block"]
    lens = _spread(c["B"], c["lo"], c["hi"])
    held = c["Hkv"] * sum(-(-n // block) for n in lens)
    st["lens"] = _ints(lens)
    if op == "reserve":
        n_new = _spread(c["B"], c["n_lo"], c["n_hi"])
        more = c["Hkv"] * sum(-(-(n + m) // block) - -(-n // block)
                              for n, m in zip(lens, n_new))
        mb = max(-(-(n + m) // block) for n, m in zip(lens, n_new))
        st.update(_pool(c, g, lens, max(mb, 1), held + more + c["spare"]))
        st["n_new"] = _ints(n_new)
    elif op == "fork":
        pages = held + c["N"] * c["Hkv"] + c["spare"]
        st.update(_pool(c, g, lens, max(-(-n // block) for n in lens) + 1, pages))
        st.update(_codes(c, g, pages))
        st["parent"] = _ints([i * c["B"] // c["N"] for i in range(c["N"])])
        st["child"] = torch.full((c["N"],) + tuple(st["table"].shape[1:]), -1,
                                 dtype=torch.int32, device="cuda")
    else:
        pages = held + held * c["hole"] // 100
        st.update(_pool(c, g, lens, max(-(-n // block) for n in lens), pages))
        st.update(_codes(c, g, pages))
        st["before"] = st["ints"].clone()
    if own:
        from block_sparse_attention_vsa_gb300 import binding
        st["pool"] = binding.Pages(st["refs"], st["free"])
        if op != "reserve":
            st["cache"] = binding.Cache8(st["k"], st["v"], st["k_scale"], st["v_scale"],
                                         st["k_mean"])
    return st


# ------------------------------------------------------------------------------ one pass
CACHE = ("k", "v", "k_scale", "v_scale", "k_mean")


def run(st):
    c = st["case"]
    if own:
        return _run_own(c, st)
    return {"fwd": _fwd, "train": _train, "reserve": _reserve, "fork": _fork,
            "compact": _compact}[c["op"]](c, st)


def _run_own(c, st):
    from block_sparse_attention_vsa_gb300 import binding
    op = c["op"]
    if op in ("fwd", "train"):
        out, lse = binding.vsa_fwd_prompt(st["q"], st["k"], st["v"], st["q_seq"], st["k_seq"],
                                          causal=c["causal"])
        if op == "fwd":
            return {"out": out, "lse": lse}
        dq, dk, dv = binding.vsa_bwd_prompt(st["q"], st["k"], st["v"], out, st["dout"], lse,
                                            st["q_seq"], st["k_seq"], causal=c["causal"])
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if op == "reserve":  # what was mapped ahead goes, then room for the tokens to come
        binding.vsa_pages_free(st["pool"], st["table"], st["lens"], block=c["block"])
        lacking = binding.vsa_pages_reserve(st["pool"], st["table"], st["lens"], st["n_new"],
                                            block=c["block"])
        return {"table": st["table"], "refs": st["refs"], "free": st["free"],
                "lacking": lacking}
    if op == "fork":  # the last round's children go, new ones are forked
        binding.vsa_pages_free(st["pool"], st["child"])
        table, lens, lacking = binding.vsa_cache_fork(st["cache"], st["pool"], st["table"],
                                                      st["lens"], st["parent"],
                                                      table_out=st["child"])
        r = {"table": table, "lens": lens, "lacking": lacking, "refs": st["refs"],
             "free": st["free"]}
    else:
        st["ints"].copy_(st["before"])
        to, n_used = binding.vsa_cache_compact(st["cache"], st["pool"], st["table"])
        r = {"to": to, "n_used": n_used, "table": st["table"], "refs": st["refs"],
             "free": st["free"]}
    r.update({t: st[t] for t in CACHE})
    return r


# ------------------------------------------------------------------------ plain forms
def _parts(c, st):
    """For each sequence: its rows of a tensor of queries and of one of keys, as functions that
    give [heads, n, 128] views."""
    nq, nk = _lengths(c)
    if c["form"] == "packed":
        aq, ak = _starts(nq), _starts(nk)
        for b in range(c["B"]):
            yield (nq[b], nk[b], lambda x, b=b: x[aq[b]:aq[b + 1]].transpose(0, 1),
                   lambda x, b=b: x[ak[b]:ak[b + 1]].transpose(0, 1),
                   lambda x, b=b: x[:, aq[b]:aq[b + 1]])
    else:
        for b in range(c["B"]):
            yield (nq[b], nk[b], lambda x, b=b: x[b, :, :nq[b]],
                   lambda x, b=b: x[b, :, :nk[b]], lambda x, b=b: x[b, :, :nq[b]])


ROWS = 8192  # query rows at a time
SCORES = 1 << 29  # scores at a time, so that they fit


def _scores(q, k, i0, off, causal):
    """Base-2 scores of rows i0.. against all keys, masked; the row's maximum, 0 if none."""
    s = (q @ k.transpose(-1, -2)) * (LOG2E / math.sqrt(D))
    if causal:
        i = torch.arange(i0, i0 + q.shape[-2], device=q.device)[:, None] + off
        s.masked_fill_(torch.arange(k.shape[-2], device=q.device) > i, -math.inf)
    m = s.amax(-1, keepdim=True)
    return s, torch.where(m == -math.inf, 0.0, m)


def _attend(c, st, grads):
    q_, k_, v_ = st["q"], st["k"], st["v"]
    out = torch.zeros(q_.shape, dtype=torch.bfloat16, device=q_.device)
    packed = c["form"] == "packed"
    lse = torch.full((c["Hq"], q_.shape[0]) if packed else q_.shape[:3], LSE_EMPTY,
                     device=q_.device)
    r = {"out": out, "lse": lse}
    if grads:
        r["dq"], r["dk"], r["dv"] = (torch.zeros(x.shape, dtype=torch.bfloat16, device=x.device)
                                     for x in (q_, k_, v_))
    G, scale = c["Hq"] // c["Hkv"], 1.0 / math.sqrt(D)
    for nq, nk, at_q, at_k, at_lse in _parts(c, st):
        if nq == 0 or nk == 0:
            continue
        n_rows = min(nq, ROWS)
        step = min(c["Hkv"], max(1, SCORES // (G * n_rows * nk)))  # key/value heads at a time
        for h0 in range(0, c["Hkv"], step):
            kv = slice(h0, min(c["Hkv"], h0 + step))
            heads = slice(kv.start * G, kv.stop * G)
            k, v = (at_k(x)[kv].float()[:, None] for x in (k_, v_))
            if grads:
                dk, dv = torch.zeros_like(k[:, 0]), torch.zeros_like(v[:, 0])
            for i0 in range(0, nq, ROWS):
                rows = slice(i0, min(nq, i0 + ROWS))
                n = nk if not c["causal"] else max(0, min(nk, rows.stop + nk - nq))
                if n == 0:
                    continue
                q = at_q(q_)[heads, rows].float().unflatten(0, (-1, G))
                p, m = _scores(q, k[:, :, :n], i0, nk - nq, c["causal"])
                p = p.sub_(m).exp2_()
                total = p.sum(-1, keepdim=True)
                some = total > 0
                p /= torch.where(some, total, 1.0)
                o = p @ v[:, :, :n]
                at_q(out)[heads, rows] = o.flatten(0, 1).to(torch.bfloat16)
                at_lse(lse)[heads, rows] = torch.where(some, m + torch.log2(total),
                                                       LSE_EMPTY)[..., 0].flatten(0, 1)
                if grads:
                    do = at_q(st["dout"])[heads, rows].float().unflatten(0, (-1, G))
                    dv[:, :n] += (p.transpose(-1, -2) @ do).sum(1)
                    ds = do @ v[:, :, :n].transpose(-1, -2)
                    ds -= (do * o).sum(-1, keepdim=True)
                    ds *= p
                    del p
                    ds *= scale
                    at_q(r["dq"])[heads, rows] = (ds @ k[:, :, :n]).flatten(0, 1).to(
                        torch.bfloat16)
                    dk[:, :n] += (ds.transpose(-1, -2) @ q).sum(1)
                    del ds
            if grads:
                at_k(r["dk"])[kv] = dk.to(torch.bfloat16)
                at_k(r["dv"])[kv] = dv.to(torch.bfloat16)
    return r


def _fwd(c, st):
    return _attend(c, st, False)


def _train(c, st):
    return _attend(c, st, True)


def _let_go(refs, free, pages):
    """One reference less for every page named."""
    pages = pages[(pages >= 0) & (pages < refs.numel())].long()
    refs -= torch.bincount(pages, minlength=refs.numel()).to(torch.int32)
    refs.clamp_(min=0)
    free.copy_(_free_words(refs))


def _take(refs, want):
    """The lowest free pages for the places marked in `want`, in their order, -1 where there
    are no more; each gets its first reference."""
    spare = torch.nonzero(refs == 0)[:, 0]
    rank = want.flatten().long().cumsum(0).view(want.shape) - 1
    got = want & (rank < spare.numel())
    page = torch.full(want.shape, -1, dtype=torch.int32, device=refs.device)
    page[got] = spare[rank[got]].to(torch.int32)
    refs[page[got].long()] = 1
    return page


def _reserve(c, st):
    """Pages for the blocks that tokens lens .. lens + n_new - 1 fall in and have none."""
    table, refs, free, lens = st["table"], st["refs"], st["free"], st["lens"]
    pages, mb = refs.numel(), table.shape[-1]
    j = torch.arange(mb, device=table.device)
    held = -(-lens // c["block"])
    ahead = (j >= held[:, None, None]).expand(table.shape)
    _let_go(refs, free, table[ahead])
    table.masked_fill_(ahead, -1)
    first, last = lens // c["block"], -(-(lens + st["n_new"]) // c["block"])
    want = (j >= first[:, None, None]) & (j < last[:, None, None])
    want = want & ((table < 0) | (table >= pages))
    page = _take(refs, want)
    table[want] = page[want]
    free.copy_(_free_words(refs))
    return {"table": table, "refs": refs, "free": free,
            "lacking": (want & (page < 0)).sum((1, 2)).to(torch.int32)}


def _fork(c, st):
    """Children share their parents' full pages; a part-full last one is copied."""
    refs, free, child, block = st["refs"], st["free"], st["child"], c["block"]
    _let_go(refs, free, child)
    parent = st["parent"].long()
    lens = st["lens"][parent]
    table = st["table"][parent]
    j = torch.arange(table.shape[-1], device=table.device)
    full, part = lens // block, lens % block
    shared = torch.where(j < full[:, None, None], table, -1)
    named = shared[shared >= 0].long()
    refs += torch.bincount(named, minlength=refs.numel()).to(torch.int32)
    want = (j == full[:, None, None]) & (part > 0)[:, None, None] & (table >= 0)
    page = _take(refs, want)
    child.copy_(torch.where(want, page, shared))
    got = want & (page >= 0)
    src, dst = table[got].long(), page[got].long()
    n = part[:, None, None].expand(table.shape)[got]
    held = (torch.arange(block, device=table.device) < n[:, None])[..., None]
    for t in ("k", "v"):
        codes = st[t].view(torch.uint8)
        codes[dst] = torch.where(held, codes[src], codes[dst])
        st[t + "_scale"][dst] = st[t + "_scale"][src]
    st["k_mean"][dst] = st["k_mean"][src]
    free.copy_(_free_words(refs))
    r = {"table": child, "lens": lens, "lacking": (want & ~got).sum((1, 2)).to(torch.int32),
         "refs": refs, "free": free}
    r.update({t: st[t] for t in CACHE})
    return r


def _compact(c, st):
    """With U pages in use, those from U on move to the free ones below it."""
    st["ints"].copy_(st["before"])
    refs, free, table = st["refs"], st["free"], st["table"]
    used = refs > 0
    n_used = used.sum()
    p = torch.arange(refs.numel(), device=refs.device)
    src = torch.nonzero(used & (p >= n_used))[:, 0]
    dst = torch.nonzero(~used & (p < n_used))[:, 0]
    to = torch.where(used, p, -1)
    to[src] = dst
    for t in ("k", "v"):
        codes = st[t].view(torch.uint8)
        codes[dst] = codes[src]
        st[t + "_scale"][dst] = st[t + "_scale"][src]
    st["k_mean"][dst] = st["k_mean"][src]
    refs[dst] = refs[src]
    refs[src] = 0
    free.copy_(_free_words(refs))
    ok = (table >= 0) & (table < refs.numel())
    table.copy_(torch.where(ok, to[table.clamp(0, refs.numel() - 1).long()], table))
    r = {"to": to.to(torch.int32), "n_used": n_used.view(1).to(torch.int32), "table": table,
         "refs": refs, "free": free}
    r.update({t: st[t] for t in CACHE})
    return r


# ------------------------------------------------------------------------------ work
def work(case):
    c = case
    op = c["op"]
    if op in ("fwd", "train"):
        nq, nk = _lengths(c)
        pairs = 0
        for a, b in zip(nq, nk):
            if not c["causal"]:
                pairs += a * b
            else:  # row i attends min(b, max(0, i + b - a + 1)) keys
                first = max(0, a - b)  # rows before it attend nothing
                n, low = a - first, max(0, b - a) + 1
                pairs += n * low + n * (n - 1) // 2
        rows_q, rows_k = c["Hq"] * sum(nq), c["Hkv"] * sum(nk)
        if op == "fwd":
            return {"bytes": 2 * D * (2 * rows_q + 2 * rows_k) + 4 * rows_q,
                    "flops": 4.0 * D * pairs * c["Hq"]}
        return {"bytes": 2 * D * (4 * rows_q + 4 * rows_k) + 4 * rows_q,
                "flops": 14.0 * D * pairs * c["Hq"]}
    block, H = c["block"], c["Hkv"]
    lens = _spread(c["B"], c["lo"], c["hi"])
    page = 2 * block * D + 8 + 2 * D
    if op == "reserve":
        n_new = _spread(c["B"], c["n_lo"], c["n_hi"])
        new = H * sum(-(-(n + m) // block) - -(-n // block) for n, m in zip(lens, n_new))
        # let go and taken again: the entry, its count, and the bits
        return {"bytes": new * 4 * 6 + c["B"] * 12, "flops": float(2 * new)}
    if op == "fork":
        n = [lens[i * c["B"] // c["N"]] for i in range(c["N"])]
        entries = H * sum(-(-x // block) for x in n)
        copied = H * sum((x % block) * 2 * D + (8 + 2 * D) * (x % block > 0) for x in n)
        return {"bytes": 2 * copied + entries * 4 * 6 + c["N"] * 12, "flops": float(2 * entries)}
    held = H * sum(-(-n // block) for n in lens)
    pages = held + held * c["hole"] // 100
    moved = held * (pages - held) // pages  # in a shuffled pool
    return {"bytes": moved * 2 * page + held * 8 + pages * 16, "flops": float(pages)}


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """Attention and its gradients in 64 bits, a block of rows at a time."""
    c = case
    if c["op"] not in ("fwd", "train"):
        return None
    if work(c)["flops"] > 1.5e13:  # more than the 64-bit units do in 20 seconds
        return None
    st = prepare(case, seed)
    q, k, v = st["q"], st["k"], st["v"]
    f8 = dict(dtype=torch.float64, device="cuda")
    packed = c["form"] == "packed"
    nq, nk = _lengths(c)
    if packed:  # [heads, tokens, 128] of everything
        q, k, v = (x.transpose(0, 1) for x in (q, k, v))
    dout = st["dout"]
    if dout is not None and packed:
        dout = dout.transpose(0, 1)
    out, lse = torch.zeros(q.shape, **f8), torch.full(q.shape[:-1], LSE_EMPTY, **f8)
    grads = [torch.zeros(x.shape, **f8) for x in (q, k, v)] if c["op"] == "train" else None
    G = c["Hq"] // c["Hkv"]
    for b in range(c["B"]):
        if packed:
            rq = (slice(None), slice(sum(nq[:b]), sum(nq[:b + 1])))
            rk = (slice(None), slice(sum(nk[:b]), sum(nk[:b + 1])))
        else:
            rq, rk = (b, slice(None), slice(0, nq[b])), (b, slice(None), slice(0, nk[b]))
        for h in range(c["Hq"]):
            kk, vv = k[rk][h // G].double(), v[rk][h // G].double()
            for a in range(0, nq[b], 4096):
                e = min(nq[b], a + 4096)
                allowed = torch.full((e - a,), nk[b], device="cuda")
                if c["causal"]:
                    allowed = (torch.arange(a, e, device="cuda") + 1 + nk[b] - nq[b]).clamp(
                        0, nk[b])
                n = int(allowed.max())
                if n == 0:
                    continue
                mask = torch.arange(n, device="cuda")[None] < allowed[:, None]
                x = q[rq][h, a:e].double()
                z = x @ kk[:n].T / math.sqrt(D)
                z = torch.where(mask, z, -math.inf)
                norm = torch.logsumexp(z, -1, keepdim=True)
                w = torch.where(mask, torch.exp(z - norm), 0.0)
                del z
                row = allowed > 0
                o = w @ vv[:n]
                out[rq][h, a:e] = o
                lse[rq][h, a:e] = torch.where(row, norm[:, 0] / math.log(2.0), LSE_EMPTY)
                if grads is not None:
                    g = dout[rq][h, a:e].double()
                    grads[2][rk][h // G, :n] += w.T @ g
                    t = w * (g @ vv[:n].T - (g * o).sum(-1, keepdim=True)) / math.sqrt(D)
                    grads[0][rq][h, a:e] = t @ kk[:n]
                    grads[1][rk][h // G, :n] += t.T @ x
                    del t
    if packed:
        out = out.transpose(0, 1)
        if grads is not None:
            grads = [x.transpose(0, 1) for x in grads]
    r = {"out": out, "lse": lse}
    if grads is not None:
        r.update(zip(("dq", "dk", "dv"), grads))
    return r

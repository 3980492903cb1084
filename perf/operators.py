"""The serving operators around block-sparse attention, measured: block means, the choice
of blocks by a cheap score (a whole prompt's rows, and single tokens over a cache), the
8-bit key/value cache (writing, attention for single tokens) and eviction from it.

`run` is one pass: through the library's entry points where `own` is true, otherwise the
plain form of the same operator in elementary torch operations (32 bits; 64 bits for the
scores that choose blocks, whose order decides whole numbers).  `exact` is the operator in
64 bits, written apart from the plain form.

All tensors have head size 128.  A cache is a pool of pages, one page holding `block`
tokens of one sequence and key/value head: e4m3 codes [pages, block, 128] for keys and
values, one power-of-two scale per page and tensor, and the bf16 mean of the page's keys.
`table[b, h, j]` is the page of block j; `lens[b]` counts the tokens held.
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
        # block means of the keys of a 16,384-token clip (12 heads) and of a 98,304-token
        # video whose last block is half full (24 heads)
        dict(name="mean_mid", op="mean", B=1, H=12, S=16384, block=64, tail=64),
        dict(name="mean_long_video", op="mean", B=1, H=24, S=98304, block=64, tail=32),
        # the blocks each query block attends: a quarter of 256, and 128 of 1,536
        dict(name="select_mid", op="select", B=1, Hq=12, Hkv=12, nq=256, nk=256, topk=64,
             causal=False, n_first=0, n_near=1, tail=64),
        dict(name="select_long_video", op="select", B=1, Hq=24, Hkv=24, nq=1536, nk=1536,
             topk=128, causal=False, n_first=0, n_near=1, tail=32),
        # the same choice made by one new token per sequence, over a cache of ragged lengths
        dict(name="token_batch", op="token", B=16, Hq=32, Hkv=8, lo=1, hi=98304, block=64,
             topk=128, n_first=1, n_near=2),
        # prompts of ragged lengths written behind what is there already
        dict(name="write_prompt", op="write", B=2, Hkv=8, T=16383, n_lo=9001, lo=37, hi=37,
             block=64),
        # one decoded token per sequence appended to the cache
        dict(name="write_token", op="write", B=32, Hkv=8, T=1, n_lo=1, lo=1, hi=8191,
             block=64),
        # one sequence, one token, 128 chosen blocks of a long video's 1,536
        dict(name="attend_one", op="attend", B=1, Hq=24, Hkv=24, lo=98272, hi=98272, block=64,
             topk=128, weights=False),
        # a serving batch of ragged lengths with grouped heads, attending all it holds and
        # recording each block's weight
        dict(name="attend_batch", op="attend", B=32, Hq=32, Hkv=8, lo=1, hi=16384, block=64,
             topk=0, weights=True),
        # a few long contexts
        dict(name="attend_long", op="attend", B=8, Hq=64, Hkv=8, lo=49152, hi=98304, block=128,
             topk=0, weights=False),
        # one sequence over its budget by half, and a batch cut to a third
        dict(name="evict_one", op="evict", B=1, Hkv=8, lo=16300, hi=16300, block=64, budget=128,
             n_first=1, n_last=4),
        dict(name="evict_batch", op="evict", B=64, Hkv=8, lo=1, hi=98304, block=64, budget=512,
             n_first=1, n_last=4),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["mean", "select", "token", "write", "attend", "attend", "evict"])
    block = rng.choice([64, 64, 128])
    if op == "mean":
        return dict(op=op, B=rng.randint(1, 2), H=_log(rng, 1, 12), S=_log(rng, 1, 98304),
                    block=block, tail=rng.randint(1, block))
    if op == "select":
        nk, nq = _log(rng, 1, 1536), _log(rng, 1, 1536)
        hkv = _log(rng, 1, 8)
        return dict(op=op, B=1, Hq=hkv * rng.randint(1, 3), Hkv=hkv, nq=nq, nk=nk,
                    topk=_log(rng, 1, min(nk, 256)), causal=rng.random() < 0.3,
                    n_first=rng.randint(0, 1), n_near=rng.randint(0, 2),
                    tail=rng.randint(1, block))
    if op == "token":
        hkv = _log(rng, 1, 8)
        hi = _log(rng, block, 98304)
        return dict(op=op, B=_log(rng, 1, 16), Hq=hkv * _log(rng, 1, 8), Hkv=hkv,
                    lo=rng.randint(1, hi), hi=hi, block=block,
                    topk=_log(rng, 1, -(-hi // block)), n_first=rng.randint(0, 2),
                    n_near=rng.randint(0, 3))
    if op == "write":
        T = _log(rng, 1, 16000)
        b = _log(rng, 1, max(1, min(32, 32000 // T)))
        return dict(op=op, B=b, Hkv=_log(rng, 1, 8), T=T, n_lo=rng.randint(1, T), lo=0,
                    hi=_log(rng, 1, 8191), block=block)
    if op == "attend":
        hi = _log(rng, 1, 98304)
        b = _log(rng, 1, max(1, min(64, 500000 // hi)))
        hkv = _log(rng, 1, 8)
        nb = -(-hi // block)
        return dict(op=op, B=b, Hq=hkv * _log(rng, 1, 8), Hkv=hkv, lo=rng.randint(1, hi),
                    hi=hi, block=block, topk=0 if rng.random() < 0.5 else _log(rng, 1, nb),
                    weights=rng.random() < 0.4)
    hi = _log(rng, block, 98304)
    nb = -(-hi // block)
    n_first, n_last = rng.randint(0, 2), rng.randint(1, 4)
    return dict(op=op, B=_log(rng, 1, 64), Hkv=_log(rng, 1, 8), lo=rng.randint(1, hi), hi=hi,
                block=block, budget=max(n_first + n_last, _log(rng, 1, nb)), n_first=n_first,
                n_last=n_last)


def _spread(B, lo, hi):
    """One length per sequence in [lo, hi], the first the longest."""
    r = random.Random(B * 1000003 + lo * 101 + hi)
    return [hi] + [r.randint(lo, hi) for _ in range(B - 1)]


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(shape, g, mul=1.0):
    return torch.randn(shape, generator=g, device="cuda") * mul


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(c, g, lens, spare=0):
    """A page for every block of every sequence and head, in shuffled order; -1 behind."""
    B, H, block = c["B"], c["Hkv"], c["block"]
    need = [-(-n // block) for n in lens]
    mb = max(max(need) + spare, 1)
    total = H * sum(need) + H * B * spare
    perm = torch.randperm(max(total, 1), generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, H, mb), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        n = need[b] + spare
        table[b, :, :n] = perm[at:at + H * n].view(H, n)
        at += H * n
    return table, max(total, 1)


def _cache(c, g, pages, codes=True):
    """A filled cache: codes of normal values, scales around 2^-7, means of the keys."""
    block = c["block"]
    r = {}
    for t in ("k", "v"):
        if codes:
            r[t] = (_randn((pages, block, D), g) * 90.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
        r[t + "_scale"] = torch.exp2(
            torch.randint(-8, -5, (pages,), generator=g, device="cuda").float())
    return r


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    st = {"case": dict(c)}
    if op == "mean":
        nb = -(-c["S"] // c["block"])
        drift = _randn((c["B"], c["H"], nb, 1, D), g, 0.5)
        x = _randn((c["B"], c["H"], nb, c["block"], D), g).add_(drift)
        st["x"] = x.view(c["B"], c["H"], nb * c["block"], D)[:, :, :c["S"]].to(
            torch.bfloat16).contiguous()
        st["sizes"] = _ints([c["block"]] * (nb - 1) + [c["tail"]])
    elif op == "select":
        st["q_mean"] = _randn((c["B"], c["Hq"], c["nq"], D), g, 0.5).to(torch.bfloat16)
        st["k_mean"] = _randn((c["B"], c["Hkv"], c["nk"], D), g, 0.5).to(torch.bfloat16)
        st["sizes"] = _ints([64] * (c["nk"] - 1) + [c["tail"]])
    elif op in ("token", "attend", "evict", "write"):
        lens = _spread(c["B"], c["lo"], c["hi"])
        spare = c["T"] // c["block"] + 2 if op == "write" else 0
        st["table"], pages = _pages(c, g, lens, spare)
        st["lens"] = _ints(lens)
        if op == "token":
            st["q"] = _randn((c["B"], c["Hq"], 1, D), g).to(torch.bfloat16)
            st["k_mean"] = _randn((pages, D), g, 0.5).to(torch.bfloat16)
        elif op == "evict":
            st["weight"] = torch.rand(st["table"].shape, generator=g, device="cuda") ** 4
        else:
            st.update(_cache(c, g, pages))
            if op == "write":
                st["k_mean"] = torch.zeros((pages, D), dtype=torch.bfloat16, device="cuda")
                shape = (c["B"], c["Hkv"], c["T"], D)
                st["k_new"] = _randn(shape, g).to(torch.bfloat16)
                st["v_new"] = _randn(shape, g).to(torch.bfloat16)
                st["n_new"] = _ints(_spread(c["B"], c["n_lo"], c["T"]))
            else:
                st["q"] = _randn((c["B"], c["Hq"], 1, D), g).to(torch.bfloat16)
                if c["topk"]:
                    nb = st["table"].shape[-1]
                    need = (st["lens"] + c["block"] - 1) // c["block"]
                    at = torch.arange(nb, device="cuda")
                    r = torch.rand((c["B"], c["Hkv"], nb), generator=g, device="cuda")
                    r = torch.where(at < need[:, None, None], r, 2.0)
                    num = need.clamp(max=c["topk"])[:, None].expand(c["B"], c["Hkv"])
                    idx = r.argsort(-1)[..., :c["topk"]]
                    slot = torch.arange(idx.shape[-1], device="cuda")
                    idx = torch.where(slot < num[..., None], idx, nb).sort(-1).values
                    st["idx"] = torch.where(idx == nb, -1, idx).to(torch.int32).contiguous()
                    st["num"] = num.to(torch.int32).contiguous()
                if c["weights"]:
                    st["weight"] = torch.zeros(st["table"].shape, device="cuda")
    if own:
        _handles(st)
    return st


def _handles(st):
    """What a user's program keeps beside its tensors: the cache object, a workspace."""
    from block_sparse_attention_vsa_gb300 import binding
    c = st["case"]
    if c["op"] in ("write", "attend"):
        pages = st["k_scale"].shape[0]
        if "k_mean" not in st:
            st["k_mean"] = torch.zeros((pages, D), dtype=torch.bfloat16, device="cuda")
        st["cache"] = binding.Cache8(st["k"], st["v"], st["k_scale"], st["v_scale"],
                                     st["k_mean"])
    if c["op"] == "attend":
        st["workspace"] = binding.new_cache_workspace(
            c["B"], c["Hq"], c["Hkv"], st["table"].shape[-1], weights=c["weights"])


# ------------------------------------------------------------------------------ one pass
def run(st):
    c = st["case"]
    if own:
        return _run_own(c, st)
    return {"mean": _mean, "select": _select, "token": _token, "write": _write,
            "attend": _attend, "evict": _evict}[c["op"]](c, st)


def _run_own(c, st):
    from block_sparse_attention_vsa_gb300 import binding
    op = c["op"]
    if op == "mean":
        return binding.vsa_block_mean(st["x"], st["sizes"], block=c["block"])
    if op == "select":
        return binding.vsa_select_blocks(st["q_mean"], st["k_mean"], c["topk"],
                                         sizes=st["sizes"], causal=c["causal"],
                                         n_first=c["n_first"], n_near=c["n_near"])
    if op == "token":
        return binding.vsa_cache_select(st["q"], st["k_mean"], st["table"], st["lens"],
                                        c["topk"], block=c["block"], n_first=c["n_first"],
                                        n_near=c["n_near"])
    if op == "write":
        binding.vsa_cache_write(st["cache"], st["k_new"], st["v_new"], st["table"], st["lens"],
                                st["n_new"])
        return {t: st[t] for t in ("k", "v", "k_scale", "v_scale", "k_mean")}
    if op == "attend":
        out, lse = binding.vsa_fwd_cache(st["q"], st["cache"], st["table"], st["lens"],
                                         idx=st.get("idx"), num=st.get("num"),
                                         weight=st.get("weight"), keep=0.0,
                                         workspace=st["workspace"])
        r = {"out": out, "lse": lse}
        if c["weights"]:
            r["weight"] = st["weight"]
        return r
    return binding.vsa_cache_evict(st["weight"], st["table"], st["lens"], block=c["block"],
                                   budget=c["budget"], n_first=c["n_first"],
                                   n_last=c["n_last"])


# ------------------------------------------------------------------------ plain forms
def _mean(c, st):
    """The mean of the first `sizes[j]` tokens of block j, 0 where there is none."""
    x, block = st["x"], c["block"]
    B, H, S, _ = x.shape
    nb = -(-S // block)
    x = torch.nn.functional.pad(x, (0, 0, 0, nb * block - S)).view(B, H, nb, block, D).float()
    at = torch.arange(block, device=x.device)
    start = torch.arange(nb, device=x.device) * block
    n = torch.minimum(st["sizes"].clamp(0, block), (S - start).clamp(max=block))
    x = torch.where((at < n[:, None])[..., None], x, 0.0)
    return (x.sum(-2) / n.clamp(min=1)[:, None]).to(torch.bfloat16)


def _best(score, eligible, forced, topk):
    """The `topk` highest of each row's eligible entries, forced ones first and ties to the
    lowest index, ascending with -1 behind; and how many there are."""
    n = score.shape[-1]
    key = torch.where(eligible, torch.where(forced, math.inf, score), -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :topk]
    num = eligible.sum(-1).clamp(max=topk)
    slot = torch.arange(order.shape[-1], device=score.device)
    order = torch.where(slot < num[..., None], order, n).sort(-1).values
    idx = torch.where(order == n, -1, order).to(torch.int32)
    idx = torch.nn.functional.pad(idx, (0, topk - idx.shape[-1]), value=-1)
    return idx, num.to(torch.int32)


def _select(c, st):
    """Row (b, h, i): the blocks j of the highest q_mean_i . k_mean_j."""
    q, k = st["q_mean"].double(), st["k_mean"].double()
    B, Hq, nq, _ = q.shape
    Hkv, nk = k.shape[1:3]
    score = (q.view(B, Hkv, Hq // Hkv, nq, D) @ k[:, :, None].transpose(-1, -2)).view(
        B, Hq, nq, nk)
    i = torch.arange(nq, device=q.device)[:, None] + (nk - nq)
    j = torch.arange(nk, device=q.device)
    eligible = (st["sizes"] > 0) & ((j <= i) if c["causal"] else (j >= 0))
    forced = (j < c["n_first"]) | ((j - i).abs() < c["n_near"])
    return _best(score, (eligible & ~score.isnan()) | (eligible & forced), forced, c["topk"])


def _token(c, st):
    """Per sequence and key/value head: a block's score is the highest of its query heads'
    q . mean of the block's keys."""
    q, table, lens = st["q"].double(), st["table"], st["lens"]
    B, Hkv, mb = table.shape
    mean = st["k_mean"][table.clamp(min=0).long()].double()
    score = (q.view(B, Hkv, -1, D) @ mean.transpose(-1, -2)).amax(-2)
    need = ((lens + c["block"] - 1) // c["block"])[:, None, None]
    j = torch.arange(mb, device=q.device)
    eligible = (j < need) & (table >= 0)
    forced = (j < c["n_first"]) | ((j - need + 1).abs() < c["n_near"])
    return _best(score, eligible, forced, c["topk"])


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, and -100 at least."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, e, -100).clamp(min=-100)


def _write(c, st):
    """Tokens lens .. lens + n_new - 1 of each sequence into their pages: a page's scale
    grows to hold its largest value, what the page held is put on the new scale."""
    table, lens, n_new, block = st["table"], st["lens"], st["n_new"], c["block"]
    B, H, T, _ = st["k_new"].shape
    W = T // block + 2
    slot = (lens // block)[:, None] + torch.arange(W, device=table.device)
    pos = slot[..., None] * block + torch.arange(block, device=table.device)  # [B, W, block]
    first, last = lens[:, None, None], (lens + n_new)[:, None, None]
    new = (pos >= first) & (pos < last)
    old = (pos < first) & new.any(-1, keepdim=True)
    page = torch.gather(table.long(), 2, slot[:, None].expand(B, H, W).long())
    touched = new.any(-1)[:, None].expand(B, H, W)
    src = (pos - first).clamp(0, T - 1).view(B, 1, W * block, 1).expand(B, H, W * block, D)
    is_new, is_old = new[:, None, ..., None], old[:, None, ..., None]
    for t in ("k", "v"):
        x = torch.gather(st[t + "_new"], 2, src).view(B, H, W, block, D).float()
        held, s_old = st[t][page], st[t + "_scale"][page]
        fine = is_new & x.isfinite()
        amax = torch.where(fine, x.abs(), 0.0).amax((-1, -2))
        s = torch.exp2(_exponent(amax).float())
        s = torch.where(old.any(-1)[:, None], torch.maximum(s, s_old), s)[..., None, None]
        moved = held.float() * (s_old[..., None, None] / s)
        code = torch.where(is_new, (x / s).clamp(-448, 448),
                           torch.where(is_old, moved, held.float()))
        code = code.to(torch.float8_e4m3fn)
        st[t][page] = code
        st[t + "_scale"][page] = torch.where(touched, s[..., 0, 0], s_old)
        if t == "k":
            n = (new | old).sum(-1)[:, None]
            mean = torch.where(is_new | is_old, code.float(), 0.0).sum(-2)
            mean = mean / n.clamp(min=1)[..., None] * s[..., 0]
            st["k_mean"][page] = torch.where(touched[..., None], mean.to(torch.bfloat16),
                                             st["k_mean"][page])
    return {t: st[t] for t in ("k", "v", "k_scale", "v_scale", "k_mean")}


def _attend(c, st):
    """Softmax attention of one token per sequence over the blocks of its cache, all of
    them or those listed; each block's share of the weights, summed over its heads."""
    q, table, lens, block = st["q"], st["table"], st["lens"], c["block"]
    B, Hkv, mb = table.shape
    if c["topk"]:
        slot = torch.arange(st["idx"].shape[-1], device=q.device)
        on = slot < st["num"][..., None]
        blk = torch.where(on, st["idx"], 0).long()
    else:
        blk = torch.arange(mb, device=q.device).expand(B, Hkv, mb)
        on = blk * block < lens[:, None, None]
    page = torch.gather(table.long(), 2, blk).clamp(min=0)
    k = (st["k"][page].float() * st["k_scale"][page][..., None, None]).view(B, Hkv, -1, D)
    pos = blk[..., None] * block + torch.arange(block, device=q.device)
    valid = (on[..., None] & (pos < lens[:, None, None, None])).view(B, Hkv, 1, -1)
    s = (q.float().view(B, Hkv, -1, D) @ k.transpose(-1, -2)) * (LOG2E / math.sqrt(D))
    del k
    s = torch.where(valid, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp2(s - m)
    l = p.sum(-1, keepdim=True)
    v = (st["v"][page].float() * st["v_scale"][page][..., None, None]).view(B, Hkv, -1, D)
    p = p / torch.where(l > 0, l, 1.0)
    out = (p @ v).view(B, -1, 1, D).to(torch.bfloat16)
    lse = torch.where(l > 0, m + torch.log2(l), LSE_EMPTY).view(B, -1, 1)
    r = {"out": out, "lse": lse}
    if c["weights"]:
        share = p.view(B, Hkv, p.shape[2], -1, block).sum((-1, -3))
        r["weight"] = torch.zeros(table.shape, device=q.device).scatter_add_(2, blk, share)
    return r


def _evict(c, st):
    """Each row's blocks cut to `budget`: the first and last ones stay, of the rest those of
    the highest weight (ties to the lowest index), in their order; the pages let go."""
    w, table, lens = st["weight"], st["table"], st["lens"]
    B, H, mb = table.shape
    need = ((lens + c["block"] - 1) // c["block"]).clamp(max=mb)[:, None, None]
    j = torch.arange(mb, device=w.device)
    held = j < need
    sure = held & ((j < c["n_first"]) | (j >= need - c["n_last"]))
    key = torch.where(held, torch.where(sure, math.inf, w), -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, j.expand_as(order).contiguous())
    kept = held & (rank < c["budget"])
    gone = held & ~kept
    nowhere = torch.full((B, H, mb + 1), -1, dtype=torch.int32, device=w.device)
    put = torch.where(kept, kept.cumsum(-1) - 1, mb)
    table_out = nowhere.scatter(2, put, table)[..., :mb].contiguous()
    weight_out = torch.zeros((B, H, mb + 1), device=w.device).scatter_(2, put, w)
    weight_out = weight_out[..., :mb].contiguous()
    freed = nowhere.scatter(2, torch.where(gone, gone.cumsum(-1) - 1, mb), table)
    n_freed = (need - c["budget"]).clamp(min=0)[:, 0, 0]
    lens_out = (lens - n_freed * c["block"]).to(torch.int32)
    return table_out, weight_out, lens_out, freed[..., :mb].contiguous(), n_freed.to(torch.int32)


# ------------------------------------------------------------------------------ work
def work(case):
    c = case
    op = c["op"]
    if op == "mean":
        nb = -(-c["S"] // c["block"])
        rows = min(c["S"], (nb - 1) * c["block"] + c["tail"])
        return {"bytes": c["B"] * c["H"] * (rows + nb) * D * 2 + nb * 4,
                "flops": c["B"] * c["H"] * rows * D}
    if op == "select":
        rows = c["B"] * c["Hq"] * c["nq"]
        return {"bytes": 2 * D * (rows + c["B"] * c["Hkv"] * c["nk"])
                + 4 * (rows * (c["topk"] + 1) + c["nk"]),
                "flops": 2.0 * rows * c["nk"] * D}
    lens = _spread(c["B"], c["lo"], c["hi"])
    block, hkv = c["block"], c["Hkv"]
    need = [-(-n // block) for n in lens]
    if op == "token":
        return {"bytes": hkv * sum(need) * (2 * D + 4) + c["B"] * (c["Hq"] * 2 * D + 4)
                + c["B"] * hkv * 4 * (c["topk"] + 1),
                "flops": 2.0 * c["Hq"] * sum(need) * D}
    if op == "write":
        n_new = _spread(c["B"], c["n_lo"], c["T"])
        new = hkv * sum(n_new)
        held = hkv * sum(n % block for n in lens)  # the keys a touched page's mean reads
        pages = hkv * sum(-(-(a + n) // block) - a // block for a, n in zip(lens, n_new))
        return {"bytes": new * 2 * (2 * D + D) + held * D + pages * (4 + 8 + 2 * D),
                "flops": 4.0 * new * D}
    if op == "attend":
        tokens = sum(min(n, c["topk"] * block) if c["topk"] else n for n in lens)
        blocks = sum(min(n, c["topk"]) if c["topk"] else n for n in need)
        return {"bytes": hkv * (tokens * 2 * D + blocks * (4 + 8 + 4 * bool(c["topk"])))
                + c["B"] * c["Hq"] * (4 * D + 4)
                + (4 * c["B"] * hkv * max(need) if c["weights"] else 0),
                "flops": 4.0 * c["Hq"] * tokens * D}
    rows = c["B"] * hkv
    return {"bytes": hkv * sum(need) * 8 + rows * max(need) * 12 + c["B"] * 12,
            "flops": hkv * float(sum(need))}


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """Outputs that are computed numbers, in 64 bits (whole numbers have no such value)."""
    c = case
    if c["op"] in ("select", "token"):
        return None
    st = prepare(case, seed)
    return {"mean": _exact_mean, "write": _exact_write, "attend": _exact_attend,
            "evict": _exact_evict}[c["op"]](c, st)


def _exact_mean(c, st):
    x = st["x"]
    B, H, S, _ = x.shape
    nb = -(-S // c["block"])
    token = torch.arange(S, device=x.device)
    sizes = st["sizes"][token // c["block"]]
    token = token[token % c["block"] < sizes]
    of = token // c["block"]
    total = torch.zeros((B, H, nb, D), dtype=torch.float64, device=x.device)
    for h in range(H):
        total[:, h].index_add_(1, of, x[:, h, token].double())
    count = torch.zeros(nb, dtype=torch.float64, device=x.device).index_add_(
        0, of, torch.ones_like(of, dtype=torch.float64))
    return total / count.clamp(min=1.0).view(nb, 1)


def _e4m3(x):
    """The nearest e4m3 value, ties to even."""
    step = torch.exp2((torch.frexp(x).exponent - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def _exact_write(c, st):
    r = {t: st[t].double() for t in ("k", "v", "k_scale", "v_scale", "k_mean")}
    lens, n_new, table = st["lens"].tolist(), st["n_new"].tolist(), st["table"].tolist()
    block = c["block"]
    for b in range(c["B"]):
        for j in range(lens[b] // block, -(-(lens[b] + n_new[b]) // block)):
            a, e = max(j * block, lens[b]), min((j + 1) * block, lens[b] + n_new[b])
            pages = torch.tensor([table[b][h][j] for h in range(c["Hkv"])], device="cuda")
            n_old, n = a - j * block, e - j * block
            for t in ("k", "v"):
                x = st[t + "_new"][b, :, a - lens[b]:e - lens[b]].double()
                top = x.abs().amax((1, 2))
                s = torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(min=-100.0))
                s_old = r[t + "_scale"][pages]
                if n_old:
                    s = torch.maximum(s, s_old)
                    r[t][pages, :n_old] = _e4m3(r[t][pages, :n_old] * (s_old / s)[:, None, None])
                r[t][pages, n_old:n] = _e4m3(x / s[:, None, None])
                r[t + "_scale"][pages] = s
                if t == "k":
                    r["k_mean"][pages] = r[t][pages, :n].sum(1) * s[:, None] / n
    return r


def _exact_attend(c, st):
    table, lens, block = st["table"], st["lens"].tolist(), c["block"]
    B, Hkv, mb = table.shape
    G = c["Hq"] // Hkv
    out = torch.zeros((B, c["Hq"], 1, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, c["Hq"], 1), LSE_EMPTY, dtype=torch.float64, device="cuda")
    weight = torch.zeros((B, Hkv, mb), dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(Hkv):
            if c["topk"]:
                blocks = st["idx"][b, h, :int(st["num"][b, h])].long()
            else:
                blocks = torch.arange(-(-lens[b] // block), device="cuda")
            token = (blocks[:, None] * block + torch.arange(block, device="cuda")).view(-1)
            there = token < lens[b]
            page = table[b, h, blocks].long()
            k = st["k"][page].double() * st["k_scale"][page].double()[:, None, None]
            v = st["v"][page].double() * st["v_scale"][page].double()[:, None, None]
            k, v = k.view(-1, D)[there], v.view(-1, D)[there]
            heads = slice(h * G, (h + 1) * G)
            s = st["q"][b, heads, 0].double() @ k.T / math.sqrt(D)
            z = torch.logsumexp(s, -1, keepdim=True)
            p = torch.exp(s - z)
            out[b, heads, 0] = p @ v
            lse[b, heads] = z / math.log(2.0)
            weight[b, h].index_add_(0, token[there] // block, p.sum(0))
    r = {"out": out, "lse": lse}
    if c["weights"]:
        r["weight"] = weight
    return r


def _exact_evict(c, st):
    """The weights that stay (the other outputs are whole numbers)."""
    w, lens = st["weight"].double().cpu(), st["lens"].tolist()
    kept = torch.zeros_like(w)
    for b in range(c["B"]):
        n = -(-lens[b] // c["block"])
        for h in range(c["Hkv"]):
            row = w[b, h, :n].tolist()
            stay = set(range(n))
            if n > c["budget"]:
                stay = set(range(c["n_first"])) | set(range(n - c["n_last"], n))
                rest = sorted((j for j in range(n) if j not in stay), key=lambda j: (-row[j], j))
                stay |= set(rest[:c["budget"] - len(stay)])
            for at, j in enumerate(sorted(stay)):
                kept[b, h, at] = row[j]
    return None, kept.cuda(), None, None, None

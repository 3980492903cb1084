"""Plain 64-bit forms of the attention over whole prompts, its gradient and the pages of the
8-bit cache, written from their definitions in include/vsa.h, a sequence and head at a time;
for each output of the attention with a bound on what bf16 products and outputs may be off by."""
import math

import torch

D = 128
LSE_EMPTY = -3.4028234663852886e38
HALF = 2.0 ** -8      # a rounding to bf16, relative
SMALL = 2.0 ** -15    # sums of fp32 and exp2 of them, relative to the terms' magnitude
FLUSH = 2.0 ** -126   # a weight below the least normal fp32 becomes 0: off by that, absolutely


def head(q, k, v, causal, scale, dout=None):
    """One sequence and head: (values, bounds) of out, lse, dq, dk, dv.

    P is rounded to bf16 (each weight by HALF at most) for the product with v, and out to bf16:
    out is off by HALF * sum p |v| before its own rounding, and by HALF * |out| more if the weights
    were normalised by what they were rounded to.  dS is rounded to bf16, and carries the error of D = dout .
    out, which is bounded by |dout| . (out's bound)."""
    nq, nk = q.shape[0], k.shape[0]
    z = q @ k.T * scale
    mask = torch.ones(nq, nk, dtype=torch.bool, device=q.device)
    if causal:
        i = torch.arange(nq, device=q.device)[:, None] + nk - nq
        mask = torch.arange(nk, device=q.device) <= i
    some = mask.any(1)
    z = torch.where(mask, z, -math.inf)
    norm = torch.where(some, torch.logsumexp(z, 1), 0.0)
    p = torch.where(mask, torch.exp(z - norm[:, None]), 0.0)
    out = p @ v
    lse = torch.where(some, norm / math.log(2.0), LSE_EMPTY)
    weigh = p @ v.abs()
    # scores are off by fp32 sums of |q||k|, which every weight carries
    sums = (q.abs() @ k.abs().T) * scale
    fine = SMALL * (1.0 + torch.where(mask, sums, 0.0).amax(1, keepdim=True)) if nk else SMALL
    b_out = HALF * (2 * out.abs() + weigh) * (1 + HALF) + fine * (weigh + out.abs())
    b_out = b_out + (mask * FLUSH).to(v.dtype) @ v.abs()
    b_lse = torch.where(some, (fine[:, 0] if nk else SMALL) + 2.0 ** -22 * lse.abs(), 0.0)
    r, b = {"out": out, "lse": lse}, {"out": b_out, "lse": b_lse}
    if dout is None:
        return r, b
    dp = dout @ v.T
    ds = p * (dp - (dout * out).sum(1, keepdim=True))
    off_d = (dout.abs() * b_out).sum(1, keepdim=True)
    mag = dout.abs() @ v.abs().T + (dout * out).abs().sum(1, keepdim=True)
    off = HALF * ds.abs() + p * (1 + HALF) * (off_d + fine * mag) + mask * FLUSH * mag
    for name, value, near in (("dq", scale * (ds @ k), scale * (off @ k.abs())),
                              ("dk", scale * (ds.T @ q), scale * (off.T @ q.abs())),
                              ("dv", p.T @ dout,
                               (HALF * p + fine * p + mask * FLUSH).T @ dout.abs())):
        r[name], b[name] = value, near * (1 + HALF) + HALF * value.abs() * (1 + HALF)
    return r, b


def attend(q, k, v, nq, nk, aq, ak, causal=True, scale=None, dout=None):
    """q [heads, rows, 128] of any type, sequence b at rows aq[b] .. + nq[b]; the same for keys.
    Returns (values, bounds), NaN where no sequence is."""
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    dout = None if dout is None else dout.double()
    shape = {"out": q, "lse": q[..., 0], "dq": q, "dk": k, "dv": v}
    names = ("out", "lse") if dout is None else tuple(shape)
    r = {n: torch.full_like(shape[n], math.nan) for n in names}
    b = {n: torch.zeros_like(shape[n]) for n in names}
    G = q.shape[0] // k.shape[0]
    for s in range(len(nq)):
        rq, rk = slice(aq[s], aq[s] + nq[s]), slice(ak[s], ak[s] + nk[s])
        for n in ("dk", "dv"):
            if n in r:
                r[n][:, rk] = 0.0
        for h in range(q.shape[0]):
            x, e = head(q[h, rq], k[h // G, rk], v[h // G, rk], causal, scale,
                        None if dout is None else dout[h, rq])
            for n in names:
                if n in ("dk", "dv"):
                    r[n][h // G, rk] += x[n]
                    b[n][h // G, rk] += e[n]
                else:
                    r[n][h, rq], b[n][h, rq] = x[n], e[n]
    return r, b


# ---------------------------------------------------------------------------------- pages
def bits(refs):
    """The bitmap of pages without a reference, as whole numbers."""
    words = [0] * (-(-len(refs) // 32))
    for p, n in enumerate(refs):
        if n == 0:
            words[p // 32] |= 1 << (p % 32)
    return words


def take(refs):
    """The lowest free page, or -1."""
    for p, n in enumerate(refs):
        if n == 0:
            refs[p] = 1
            return p
    return -1


def free(refs, table, lens, block):
    for b, rows in enumerate(table):
        first = 0 if lens is None else -(-max(0, lens[b]) // block)
        for row in rows:
            for j in range(first, len(row)):
                if 0 <= row[j] < len(refs):
                    refs[row[j]] = max(0, refs[row[j]] - 1)
                row[j] = -1


def reserve(refs, table, lens, n_new, block):
    lacking = []
    for b, rows in enumerate(table):
        none, n = 0, max(0, lens[b])
        more = 1 if n_new is None else max(0, n_new[b])
        for row in rows:
            for j in range(n // block, min(len(row), -(-(n + more) // block))):
                if not 0 <= row[j] < len(refs):
                    row[j] = take(refs)
                    none += row[j] < 0
        lacking.append(none)
    return lacking


def fork(refs, table, lens, parent, block, mb):
    """(children's table, lens, lacking, [(src page, dst page, tokens)])."""
    H = len(table[0])
    out, n_out, lacking, copies = [], [], [], []
    for p in parent:
        there = 0 <= p < len(table)
        n = max(0, min(lens[p], mb * block)) if there else 0
        rows, none = [], 0
        for h in range(H):
            row = [-1] * mb
            for j in range(n // block):
                page = table[p][h][j]
                if 0 <= page < len(refs):
                    row[j] = page
                    refs[page] += 1
            if n % block and 0 <= table[p][h][n // block] < len(refs):
                row[n // block] = dst = take(refs)
                none += dst < 0
                if dst >= 0:
                    copies.append((table[p][h][n // block], dst, n % block))
            rows.append(row)
        out.append(rows)
        n_out.append(n)
        lacking.append(none)
    return out, n_out, lacking, copies


def compact(refs, table):
    """(to, pages in use); refs and table changed."""
    used = sum(n > 0 for n in refs)
    low = [p for p in range(used) if refs[p] == 0]
    to = [-1] * len(refs)
    for p, n in enumerate(list(refs)):
        if n > 0:
            to[p] = p if p < used else low.pop(0)
            if to[p] != p:
                refs[to[p]], refs[p] = n, 0
    for rows in table:
        for row in rows:
            for j, p in enumerate(row):
                if 0 <= p < len(refs):
                    row[j] = to[p]
    return to, used

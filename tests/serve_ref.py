"""Plain 64-bit forms of the operators around the attention, on the CPU: block means, the
choice of blocks, the 8-bit cache (writing, attention of one token) and eviction.  Written
from their definitions in include/vsa.h, one row at a time."""
import math

import torch

D = 128
LSE_EMPTY = -3.4028234663852886e38


def block_mean(x, sizes, block):
    """(means, sum of |x| / n per mean) in fp64."""
    x = x.double()
    B, H, S, _ = x.shape
    nb = -(-S // block)
    mean = torch.zeros(B, H, nb, D, dtype=torch.float64)
    mag = torch.zeros_like(mean)
    for j in range(nb):
        n = min(block, S - j * block)
        if sizes is not None:
            n = max(0, min(n, int(sizes[j])))
        if n:
            part = x[:, :, j * block:j * block + n]
            mean[:, :, j] = part.sum(2) / n
            mag[:, :, j] = part.abs().sum(2) / n
    return mean, mag


def choose(score, allowed, forced, topk):
    """Ascending indices of the topk best: forced ones first, then by score, ties to the
    lowest index; a NaN score is out unless forced."""
    got = []
    for j, s in enumerate(score):
        if allowed(j) and (forced(j) or s == s):
            got.append((0, 0.0, j) if forced(j) else (1, -s, j))
    got.sort()
    return sorted(j for _, _, j in got[:topk])


def _lists(rows, topk, shape):
    idx = torch.full((len(rows), topk), -1, dtype=torch.int32)
    for r, row in enumerate(rows):
        idx[r, :len(row)] = torch.tensor(row, dtype=torch.int32)
    num = torch.tensor([len(r) for r in rows], dtype=torch.int32)
    return idx.view(*shape, topk), num.view(shape)


def select_blocks(q, k, topk, sizes=None, causal=False, n_first=0, n_near=0):
    q, k = q.double(), k.double()
    B, Hq, nq, _ = q.shape
    Hkv, nk = k.shape[1:3]
    on = [True] * nk if sizes is None else [s > 0 for s in sizes.tolist()]
    rows = []
    for b in range(B):
        for h in range(Hq):
            s = q[b, h] @ k[b, h // (Hq // Hkv)].T
            for i in range(nq):
                d = i + nk - nq
                rows.append(choose(s[i].tolist(), lambda j: on[j] and (not causal or j <= d),
                                   lambda j: j < n_first or abs(j - d) < n_near, topk))
    return _lists(rows, topk, (B, Hq, nq))


def cache_select(q, k_mean, table, lens, topk, block, n_first=0, n_near=1):
    q, k_mean = q.double(), k_mean.double()
    B, Hkv, mb = table.shape
    G = q.shape[1] // Hkv
    rows = []
    for b in range(B):
        n = min(mb, -(-max(0, int(lens[b])) // block))
        for h in range(Hkv):
            pages = table[b, h, :n].tolist()
            fine = [0 <= p < k_mean.shape[0] for p in pages]
            mean = k_mean[torch.tensor([p if f else 0 for p, f in zip(pages, fine)],
                                       dtype=torch.long)]
            s = q[b, h * G:(h + 1) * G, 0] @ mean.T
            s = torch.where(s.isnan().any(0), math.nan, s.amax(0))
            rows.append(choose(s.tolist(), lambda j: fine[j],
                               lambda j: j < n_first or n - 1 - j < n_near, topk))
    return _lists(rows, topk, (B, Hkv))


def e4m3(x):
    """The nearest e4m3 value in fp64, ties to even, saturating; NaN stays."""
    x = x.double().clamp(-448.0, 448.0)
    step = torch.exp2((torch.frexp(x).exponent - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def cache_write(state, k, v, table, lens, n_new, block):
    """`state`: dict of fp64 k, v [pages, block, 128], k_scale, v_scale, k_mean; changed."""
    pages = state["k"].shape[0]
    B, H, T, _ = k.shape
    mb = table.shape[2]
    for b in range(B):
        n = T if n_new is None else max(0, min(T, int(n_new[b])))
        at = max(0, int(lens[b]))
        for j in range(at // block, min(mb, -(-(at + n) // block))):
            first, last = max(at, j * block), min(at + n, (j + 1) * block)
            if first >= last:
                continue
            a, e = first - j * block, last - j * block
            for h in range(H):
                p = int(table[b, h, j])
                if not 0 <= p < pages:
                    continue
                for t, x in (("k", k), ("v", v)):
                    x = x[b, h, first - at:last - at].double()
                    top = torch.where(x.isfinite(), x.abs(), 0.0).max().item()
                    s = 2.0 ** -100
                    while top > 448.0 * s:
                        s *= 2.0
                    if a:
                        old = state[t + "_scale"][p].item()
                        s = max(s, old)
                        state[t][p, :a] = e4m3(state[t][p, :a] * (old / s))
                    state[t][p, a:e] = e4m3(x / s)
                    state[t + "_scale"][p] = s
                state["k_mean"][p] = state["k"][p, :e].sum(0) * state["k_scale"][p] / e


def attend(q, state, table, lens, block, idx=None, num=None, scale=None):
    """out, lse, block weights, and per row the magnitudes that error bounds go by: the sum
    of p|v|, the largest sum of |q||k| in score units, the tokens and the largest |v|."""
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    B, Hq = q.shape[:2]
    Hkv, mb = table.shape[1:]
    G = Hq // Hkv
    pages = state["k"].shape[0]
    out = torch.zeros(B, Hq, 1, D, dtype=torch.float64)
    mag = torch.zeros(B, Hq, 1, D, dtype=torch.float64)
    lse = torch.full((B, Hq, 1), LSE_EMPTY, dtype=torch.float64)
    qk = torch.zeros(B, Hq, 1, dtype=torch.float64)
    count = torch.zeros(B, Hq, 1, dtype=torch.float64)
    vmax = torch.zeros(B, Hq, 1, dtype=torch.float64)
    weight = torch.zeros(B, Hkv, mb, dtype=torch.float64)
    for b in range(B):
        n = min(mb, -(-max(0, int(lens[b])) // block))
        for h in range(Hkv):
            if idx is None:
                blocks = range(n)
            else:
                c = max(0, min(idx.shape[2], int(num[b, h])))
                blocks = sorted(set(j for j in idx[b, h, :c].tolist() if 0 <= j < n))
            ks, vs, of = [], [], []
            for j in blocks:
                p = int(table[b, h, j])
                m = min(block, int(lens[b]) - j * block)
                if 0 <= p < pages:
                    ks.append(state["k"][p, :m] * state["k_scale"][p])
                    vs.append(state["v"][p, :m] * state["v_scale"][p])
                    of += [j] * m
            if not of:
                continue
            K, V = torch.cat(ks), torch.cat(vs)
            hs = slice(h * G, (h + 1) * G)
            qq = q[b, hs, 0].double()
            s = qq @ K.T * scale
            z = torch.logsumexp(s, -1, keepdim=True)
            pr = torch.exp(s - z)
            out[b, hs, 0] = pr @ V
            mag[b, hs, 0] = pr @ V.abs()
            lse[b, hs] = z / math.log(2.0)
            qk[b, hs] = (qq.abs() @ K.abs().T * scale).amax(-1, keepdim=True)
            count[b, hs] = float(len(of))
            vmax[b, hs] = V.abs().max()
            weight[b, h].index_add_(0, torch.tensor(of), pr.sum(0))
    return dict(out=out, lse=lse, weight=weight, mag=mag, qk=qk, count=count, vmax=vmax)


def evict(weight, table, lens, budget, block, n_first, n_last):
    B, H, mb = table.shape
    t_out = torch.full_like(table, -1)
    w_out = torch.zeros_like(weight)
    freed = torch.full_like(table, -1)
    lens_out, n_freed = lens.clone(), torch.zeros_like(lens)
    for b in range(B):
        n = min(mb, -(-max(0, int(lens[b])) // block))
        gone = max(0, n - budget)
        lens_out[b] = max(0, int(lens[b])) - gone * block
        n_freed[b] = gone
        for h in range(H):
            w = weight[b, h, :n].tolist()
            sure = set(j for j in range(n) if j < n_first or j >= n - n_last)
            rest = sorted((j for j in range(n) if j not in sure),
                          key=lambda j: (w[j] != w[j], -w[j] if w[j] == w[j] else 0.0, j))
            stay = set(range(n)) if not gone else sure | set(rest[:n - gone - len(sure)])
            for at, j in enumerate(sorted(stay)):
                t_out[b, h, at] = table[b, h, j]
                w_out[b, h, at] = weight[b, h, j]
            for at, j in enumerate(j for j in range(n) if j not in stay):
                freed[b, h, at] = table[b, h, j]
    return t_out, w_out, lens_out, freed, n_freed

"""Gradients behind a choice of blocks, held so that a wrong one cannot pass: every element to
a bound derived from the kernel's roundings, and the derivative along the gradient itself to
differences of the 64-bit forward.

The backward takes q, k, v, dout, out (bf16) and lse.  Its roundings, by the formulas
p = 2^(s log2 e - lse), dS = p (dout.v - D), D = dout.out:
  p     fp32, off by ds = 2^-15 max sum |q||k| scale (fp32 sums of exact products) + 2^-18
        (exp2, the subtraction), relative; rounded to bf16 (2^-8) for dv alone
  dout.v, D   fp32 sums: 2^-15 sum |dout||v|, 128 * 2^-24 sum |dout||out|
  dS    rounded to bf16: 2^-8
  dq, dk, dv  fp32 sums of those: 2^-15 of the sum of magnitudes; rounded to bf16: 2^-8
Each bound adds these up over the sums they enter, with a fiftieth more for their products."""
import math

import pytest
import torch

import serve_ref as ref
from block_sparse_attention_vsa_gb300 import binding

D = 128
DEV = "cuda:0"
HALF = 2.0 ** -8  # half a bf16 step


def case(block, seed=91):
    g = torch.Generator().manual_seed(seed)
    B, Hq, Hkv, nb = 1, 4, 2, 9
    sizes = torch.full((nb,), block, dtype=torch.int32)
    sizes[-1] = 17

    def bf16(H):
        return torch.randn((B, H, nb * block, D), generator=g).to(torch.bfloat16)

    return bf16(Hq), bf16(Hkv), bf16(Hkv), bf16(Hq), sizes


def chosen_keys(idx, sizes, block):
    """Which keys each query attends [Hq, S, S]."""
    Hq, nb = idx.shape[1:3]
    mask = torch.zeros(Hq, nb * block, nb * block, dtype=torch.bool)
    for h in range(Hq):
        for i in range(nb):
            for j in idx[0, h, i].tolist():
                if j >= 0:
                    mask[h, i * block:(i + 1) * block, j * block:j * block + int(sizes[j])] = True
    return mask


def attention(q, k, v, mask):
    G = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = (q @ k.transpose(-1, -2) / math.sqrt(D)).masked_fill(~mask, -math.inf)
    return torch.softmax(s, -1) @ v, torch.logsumexp(s, -1) / math.log(2.0)


def gradients(q, k, v, dout, out, lse, mask):
    """((dq, dk, dv) by the formula from this out and lse, their bounds), in fp64."""
    q, k, v, dout, out = (t.double()[0] for t in (q, k, v, dout, out))
    lse = lse.double()[0][..., None]
    Hq, Hkv = q.shape[0], k.shape[0]
    G, scale = Hq // Hkv, 1.0 / math.sqrt(D)
    kk, vv = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
    p = torch.where(mask, torch.exp2(q @ kk.transpose(-1, -2) * (scale / math.log(2.0)) - lse), 0.0)
    ds = 2.0 ** -15 * (q.abs() @ kk.abs().transpose(-1, -2)).amax().item() * scale + 2.0 ** -18
    dp = dout @ vv.transpose(-1, -2)
    delta = (dout * out).sum(-1, keepdim=True)
    dS = p * (dp - delta)
    dS_off = (HALF + ds) * dS.abs() + p * (
        2.0 ** -15 * (dout.abs() @ vv.abs().transpose(-1, -2))
        + 128 * 2.0 ** -24 * (dout * out).abs().sum(-1, keepdim=True))

    def heads(t):  # the sum over each key/value head's query heads
        return t.view(Hkv, G, *t.shape[1:]).sum(1)

    dq, dk, dv = scale * dS @ kk, heads(scale * dS.mT @ q), heads(p.mT @ dout)
    sums = 2.0 ** -15
    off = (scale * (dS_off + sums * dS.abs()) @ kk.abs(),
           heads(scale * (dS_off + sums * dS.abs()).mT @ q.abs()),
           heads((HALF + ds + sums) * p.mT @ dout.abs()))
    grads = (dq, dk, dv)
    return grads, tuple(1.02 * o + HALF * t.abs() for o, t in zip(off, grads))


def check(got, q, k, v, dout, out, lse, mask):
    grads, bounds = gradients(q, k, v, dout, out, lse, mask)
    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    exact = torch.autograd.grad(attention(*leaves, mask)[0], leaves, dout.double())
    for n, (x, want, bound, w) in enumerate(zip(got, grads, bounds, exact)):
        x = x.cpu().double()[0]
        assert ((x - want).abs() <= bound).all(), n
        # along the exact gradient u = w / |w|: the derivative is |w|, and x.u may be off by the
        # bound's length, and by what the rounding of `out` and `lse` moves the formula's values
        u = w / w.norm()
        args = [t.detach() for t in leaves]

        def slope(e):
            hi, lo = list(args), list(args)
            hi[n], lo[n] = args[n] + e * u, args[n] - e * u
            return (((attention(*hi, mask)[0] - attention(*lo, mask)[0]) * dout.double()).sum()
                    / (2 * e)).item()

        with torch.no_grad():
            near, far = slope(1e-2), slope(2e-2)
        # differences are off by a multiple of e^2: a third of what doubling e changes
        off = bound.norm() + (want - w[0]).norm() + abs(far - near)
        assert abs((x * u[0]).sum().item() - near) <= off, n
        assert off <= 0.3 * near, (n, off, near)  # no gradient of zeros, or 1.3 times as large


@pytest.mark.parametrize("wrong", ["zeros", "scaled", "swapped heads", "right"])
def test_the_check_tells_a_wrong_gradient(wrong):
    """On the CPU, with the formula's own gradients, rounded, in place of the kernel's."""
    q, k, v, dout, sizes = case(64)
    qm, km = (ref.block_mean(t, s, 64)[0].to(torch.bfloat16) for t, s in ((q, None), (k, sizes)))
    idx, _ = ref.select_blocks(qm, km, 4, sizes, n_near=1)
    mask = chosen_keys(idx, sizes, 64)
    out, lse = attention(q.double(), k.double(), v.double(), mask)
    out, lse = out.to(torch.bfloat16), lse.float()
    grads = [t[None] for t in gradients(q, k, v, dout, out, lse, mask)[0]]
    got = [t.to(torch.bfloat16) for t in grads]
    if wrong == "right":
        return check(got, q, k, v, dout, out, lse, mask)
    for n in range(3):
        bad = list(got)
        bad[n] = (torch.zeros_like(got[n]) if wrong == "zeros" else
                  (grads[n] * 1.3).to(torch.bfloat16) if wrong == "scaled" else got[n].flip(1))
        with pytest.raises(AssertionError):
            check(bad, q, k, v, dout, out, lse, mask)


@pytest.mark.gpu
@pytest.mark.parametrize("block", [64, 128])
def test_gradients_behind_a_choice(block):
    import __graft_entry__
    __graft_entry__.build()
    q, k, v, dout, sizes = case(block)
    qd, kd, vd, sd = q.to(DEV), k.to(DEV), v.to(DEV), sizes.to(DEV)
    qm, km = binding.vsa_block_mean(qd, block=block), binding.vsa_block_mean(kd, sd, block=block)
    idx, num = binding.vsa_select_blocks(qm, km, 4, sizes=sd, n_near=1)
    out, lse = binding.vsa_fwd_gqa(qd, kd, vd, idx, num, sd, block=block)
    got = binding.vsa_bwd(qd, kd, vd, out, dout.to(DEV), lse, idx, num, sd, block=block)
    check(got, q, k, v, dout, out.cpu(), lse.cpu(), chosen_keys(idx.cpu(), sizes, block))

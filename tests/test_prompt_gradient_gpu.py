"""The gradient of the attention over whole prompts where its kernels' single parts show: one
step a tile, what lies around a sequence, and copies that come late."""
import math

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


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(shape, g, mul=1.0):
    return (torch.randn(shape, generator=g) * mul).to(torch.bfloat16).to(DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def ok():
    torch.cuda.synchronize()
    code, detail = binding.vsa_device_status()
    assert code == binding.VSA_OK, hex(detail)


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (16, 4)], ids=str)
def test_sequences_of_one_step_with_anything_behind_them(Hq, Hkv, causal):
    """Every key tile sees one query tile, whose rows behind the sequence hold NaN; dout is fetched
    from memory each time, so that its copy lands last."""
    g = gen(60)
    B, S = 64, 200
    most = 128 * Hkv // Hq  # tokens of a query tile
    n = [1 + (b * 37) % (most - 1) for b in range(B)]
    q, k, v, dout = (randn((B, h, S, D), g) for h in (Hq, Hkv, Hkv, Hq))
    for b in range(B):
        for t in (q, k, v, dout):
            t[b, :, n[b]:] = math.nan
    out, lse = binding.vsa_fwd_prompt(q, k, v, i32(n), causal=causal)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    first = None
    for _ in range(20):
        flush.zero_()
        for t in (q, k, v):
            t.add_(0)
        grads = binding.vsa_bwd_prompt(q, k, v, out, dout, lse, i32(n), causal=causal)
        first = first or grads
        for x, y in zip(first, grads):
            assert torch.equal(x, y)
    ok()
    for b in range(0, B, 9):
        want, bound = ref.attend(q[b], k[b], v[b], [n[b]], [n[b]], [0], [0], causal, None, dout[b])
        for x, name in zip(first, ("dq", "dk", "dv")):
            there = slice(0, n[b])
            err = (x[b, :, there].double() - want[name][:, there]).abs()
            assert (err <= bound[name][:, there]).all(), (name, b)
            assert (x[b, :, n[b]:] == 0).all(), (name, b)


@pytest.mark.parametrize("nq,nk,Hq,Hkv", [
    ([200, 130], [3, 129], 4, 2), ([300], [40], 2, 2), ([513], [257], 1, 1), ([90, 1], [0, 1], 6, 2),
    ([1100], [90], 6, 1), ([700, 260], [330, 130], 16, 1)], ids=str)
@pytest.mark.parametrize("bad", [math.nan, math.inf], ids=["nan", "inf"])
def test_rows_that_attend_nothing_reach_nothing(nq, nk, Hq, Hkv, bad):
    """More queries than keys, causal: the first queries' q and dout may hold anything."""
    g = gen(61)
    aq, ak = [0], [0]
    for x, y in zip(nq, nk):
        aq.append(aq[-1] + x)
        ak.append(ak[-1] + y)
    q, k, v, dout = (randn((n, h, D), g)
                     for n, h in ((aq[-1], Hq), (ak[-1], Hkv), (ak[-1], Hkv), (aq[-1], Hq)))

    def run():
        out, lse = binding.vsa_fwd_prompt(q, k, v, i32(aq), i32(ak))
        grads = binding.vsa_bwd_prompt(q, k, v, out, dout, lse, i32(aq), i32(ak))
        ok()
        return dict(out=out, lse=lse.T, dq=grads[0], dk=grads[1], dv=grads[2])

    none = torch.zeros(aq[-1], dtype=torch.bool, device=DEV)
    for a, x, y in zip(aq, nq, nk):
        none[a:a + max(0, x - y)] = True
    q[none], dout[none] = 0.0, 0.0
    want = run()
    q[none], dout[none] = bad, bad
    dout[none, :, ::2] = -bad
    got = run()
    for name in want:
        assert torch.equal(got[name], want[name]), name
    assert (got["dq"][none] == 0).all()


def near(got, want, what, tol=0.005):
    """Off by `tol` of its norm at most, each head for itself.  Roundings to bf16 on the way to an
    element -- its own, that of P or dS, that of out -- are each spread over half a step, 2^-8 of a
    value at most and 2^-8 / sqrt(3) = 0.00226 in the mean square; three, independent, make
    0.0039."""
    err, size = (got.double() - want).norm(dim=(-2, -1)), want.norm(dim=(-2, -1))
    assert (err <= tol * size).all(), (what, (err / size).max().item())


@pytest.mark.parametrize("nq,cut,nk,Hq,Hkv,causal,less", [
    (300, 100, 300, 4, 4, False, 0), (130, 700, 1000, 8, 2, False, 0), (257, 384, 641, 2, 2, True, 0),
    (40, 2000, 2040, 4, 1, True, 0), (513, 64, 2500, 12, 2, False, 0), (100, 64, 192, 4, 4, False, 8),
    (100, 64, 128, 4, 4, False, 11), (300, 64, 564, 4, 2, False, 8), (300, 64, 564, 4, 2, False, 20)],
    ids=str)
def test_keys_in_two_parts(nq, cut, nk, Hq, Hkv, causal, less):
    """out and lse over all keys, the gradient over a part of them at a time, against 64 bits with
    this out and lse: dk and dv are the parts', dq adds up.  (The later keys are the causal ones;
    the earlier ones may weigh 2^-less of what they would.)"""
    g = gen(62)
    q, k, v, dout = (randn((1, h, n, D), g)
                     for n, h in ((nq, Hq), (nk, Hkv), (nk, Hkv), (nq, Hq)))
    if less:
        q[..., 0], k[..., 0] = 4.0, 0.0
        k[:, :, :cut, 0] = -less * math.log(2.0) * math.sqrt(D) / 4.0
    out, lse = binding.vsa_fwd_prompt(q, k, v, causal=causal)
    parts = [binding.vsa_bwd_prompt(q, k[:, :, a:b], v[:, :, a:b], out, dout, lse, causal=c)
             for a, b, c in ((0, cut, False), (cut, nk, causal))]
    ok()
    scale, G = 1.0 / math.sqrt(D), Hq // Hkv
    x, y, z, d, o = (t[0].double() for t in (q, k, v, dout, out))
    y, z = y.repeat_interleave(G, 0), z.repeat_interleave(G, 0)
    s = x @ y.transpose(1, 2) * scale
    if causal:
        s = s.masked_fill(torch.ones(nq, nk, dtype=torch.bool, device=DEV).triu(nk - nq + 1),
                          -math.inf)
    p = torch.exp(s - lse[0].double()[..., None] * math.log(2.0))
    ds = p * (d @ z.transpose(1, 2) - (d * o).sum(-1, keepdim=True))
    dk = (scale * ds.transpose(1, 2) @ x).unflatten(0, (Hkv, G)).sum(1)
    dv = (p.transpose(1, 2) @ d).unflatten(0, (Hkv, G)).sum(1)
    for (a, b), (dq_p, dk_p, dv_p) in zip(((0, cut), (cut, nk)), parts):
        near(dq_p[0], scale * ds[:, :, a:b] @ y[:, a:b], "dq")
        near(dk_p[0], dk[:, a:b], "dk")
        near(dv_p[0], dv[:, a:b], "dv")
    near(parts[0][0][0].double() + parts[1][0][0].double(), scale * ds @ y, "dq of both", 0.0071)

"""The gradient of the attention over whole prompts where its kernels' single parts show: one
step a tile, what lies around a sequence, and copies that come late."""
import math

import pytest
import torch

import prompt_ref as ref
from block_sparse_attention_vsa_gb300 import binding
from prompt_norm import NORM, off

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


def near(got, want, what, tol=NORM):
    assert off(got, want) <= tol, (what, off(got, want))


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
    near(parts[0][0][0].double() + parts[1][0][0].double(), scale * ds @ y, "dq of both",
         math.sqrt(2) * NORM)


def plain(q, k, v, dout, nq, nk, causal):
    """The 64-bit values of out, dq, dk, dv for packed sequences, [heads, tokens, 128], a sequence
    and head at a time."""
    r = {n: torch.zeros(x.shape, dtype=torch.float64, device=DEV)
         for n, x in (("out", q), ("dq", q), ("dk", k), ("dv", v))}
    G, scale, aq, ak = q.shape[0] // k.shape[0], 1.0 / math.sqrt(D), 0, 0
    for n, m in zip(nq, nk):
        for h in range(q.shape[0]):
            rq, rk = (h, slice(aq, aq + n)), (h // G, slice(ak, ak + m))
            x, y, z, d = q[rq].double(), k[rk].double(), v[rk].double(), dout[rq].double()
            p = x @ y.T * scale
            if causal:
                p.masked_fill_(torch.ones(n, m, dtype=torch.bool, device=DEV).triu(m - n + 1), -math.inf)
            p = torch.softmax(p, 1).nan_to_num_(0.0)  # (rows that attend nothing)
            r["out"][rq] = out = p @ z
            r["dv"][rk] += p.T @ d
            ds = d @ z.T
            ds -= (d * out).sum(1, keepdim=True)
            ds *= p
            r["dq"][rq] = scale * ds @ y
            r["dk"][rk] += scale * ds.T @ x
        aq, ak = aq + n, ak + m
    return r


NORMS = [  # queries, keys of packed sequences, heads, causal
    ([300, 33, 411], [300, 33, 411], 12, 12, True), ([70], [700], 4, 2, False),
    ([513], [513], 1, 1, False), ([200, 130], [103, 129], 4, 2, True), ([128], [128], 2, 1, True),
    # keys, or steps, cut into ranges
    ([70], [2500], 4, 4, False), ([300, 41], [300, 41], 24, 1, True), ([600], [600], 8, 1, True),
    ([500, 2], [2100, 700], 16, 1, True), ([1100], [90], 6, 1, False), ([3], [2500], 2, 1, True),
    # long walks: rings that go round many times, masks in the last tiles
    ([5000, 3001], [5000, 3001], 2, 1, True), ([4100], [4100], 2, 2, False), ([600], [6001], 3, 1, True),
    ([8192], [8192], 12, 2, True), ([2048], [2048], 12, 12, True),
    # more tiles than SMs, longest first and as they come
    ([700, 1300, 60, 900], [700, 1300, 60, 900], 32, 8, True), ([257] * 40, [257] * 40, 6, 6, True)]


@pytest.mark.parametrize("nq,nk,Hq,Hkv,causal", NORMS, ids=str)
def test_errors_in_norm(nq, nk, Hq, Hkv, causal):
    g = gen(sum(nq) + Hq)
    aq, ak = [0], [0]
    for x, y in zip(nq, nk):
        aq.append(aq[-1] + x)
        ak.append(ak[-1] + y)
    q, k, v, dout = (randn((n, h, D), g)
                     for n, h in ((aq[-1], Hq), (ak[-1], Hkv), (ak[-1], Hkv), (aq[-1], Hq)))
    out, lse = binding.vsa_fwd_prompt(q, k, v, i32(aq), i32(ak), causal=causal)
    grads = binding.vsa_bwd_prompt(q, k, v, out, dout, lse, i32(aq), i32(ak), causal=causal)
    ok()
    want = plain(*(x.transpose(0, 1) for x in (q, k, v, dout)), nq, nk, causal)
    for n, x in zip(("out", "dq", "dk", "dv"), (out, *grads)):
        near(x.transpose(0, 1), want[n], n)


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_differences_along_the_gradient(causal):
    """Along the gradient itself the slope of sum(out * dout) is the gradient's norm: central
    differences in 64 bits, which a gradient of another size, sign or direction does not meet."""
    g = gen(63)
    n = 180
    q, k, v, dout = (randn((1, 2, n, D), g) for _ in range(4))
    out, lse = binding.vsa_fwd_prompt(q, k, v, causal=causal)
    grads = binding.vsa_bwd_prompt(q, k, v, out, dout, lse, causal=causal)
    ok()
    x, h = [t[0].double() for t in (q, k, v)], 1e-4
    for i in range(3):
        got = grads[i][0].double()
        d = got / got.norm()

        def f(t):
            y = [a + t * d if j == i else a for j, a in enumerate(x)]
            s = y[0] @ y[1].transpose(1, 2) / math.sqrt(D)
            if causal:
                s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1), -math.inf)
            return ((torch.softmax(s, -1) @ y[2]) * dout[0].double()).sum().item()

        slope = (f(h) - f(-h)) / (2 * h)
        # (got - true) . d is at most NORM of the norm; the differences are off by h^2 / 6 of a
        # third derivative, 1e-8 here
        assert slope > 1.0 and abs(got.norm().item() - slope) <= (NORM + 1e-6) * slope, i


def test_calls_on_another_stream_do_not_wait():
    """The current stream is held up long behind what the calls take; they end before it does."""
    g = gen(64)
    q, k, v, dout = (randn((500, h, D), g) for h in (4, 2, 2, 4))
    seq = i32([0, 333, 500])
    out, lse = binding.vsa_fwd_prompt(q, k, v, seq)
    want = (out, lse, *binding.vsa_bwd_prompt(q, k, v, out, dout, lse, seq))
    side = torch.cuda.Stream()
    ok()
    busy = torch.ones(8192, 8192, device=DEV, dtype=torch.bfloat16)
    for _ in range(200):  # about 0.1 s
        busy = busy @ busy
    last = torch.cuda.Event()
    last.record()
    out, lse = binding.vsa_fwd_prompt(q, k, v, seq, stream=side)
    grads = binding.vsa_bwd_prompt(q, k, v, out, dout, lse, seq, stream=side)
    side.synchronize()
    assert not last.query()
    for x, y in zip(want, (out, lse, *grads)):
        assert torch.equal(x, y)
    ok()

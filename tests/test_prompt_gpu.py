"""Attention over whole prompts and its gradient against plain 64-bit forms, at the lengths,
masks, layouts and values where they can go wrong."""
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


def starts(lens):
    r = [0]
    for n in lens:
        r.append(r[-1] + n)
    return r


def ok():
    torch.cuda.synchronize()
    code, detail = binding.vsa_device_status()
    assert code == binding.VSA_OK, hex(detail)


def hold(got, want, bound):
    """Every output inside its bound; rows that attend nothing exactly."""
    for n, w in want.items():
        g = got[n].double()
        there = ~w.isnan()
        err = (g - w).abs()[there]
        assert (err <= bound[n][there]).all(), (n, (err - bound[n][there]).max().item(),
                                                err.max().item())
        if n == "lse":
            assert (g[w == ref.LSE_EMPTY] == ref.LSE_EMPTY).all()
        if n == "out":
            none = (want["lse"] == ref.LSE_EMPTY)
            assert (got["out"][none] == 0).all() and not got["out"][none].signbit().any()


def both(q, k, v, dout, **kw):
    out, lse = binding.vsa_fwd_prompt(q, k, v, **kw)
    dq, dk, dv = binding.vsa_bwd_prompt(q, k, v, out, dout, lse, **kw)
    ok()
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)


def check_packed(nq, nk, Hq, Hkv, causal, seed, mul=1.0, scale=None, gap=0):
    g = gen(seed)
    aq, ak = [gap + x for x in starts(nq)], [gap + x for x in starts(nk)]
    q, k, v, dout = (randn((n[-1] + gap, h, D), g, mul)
                     for n, h in ((aq, Hq), (ak, Hkv), (ak, Hkv), (aq, Hq)))
    got = both(q, k, v, dout, q_seq=i32(aq), k_seq=i32(ak), causal=causal, scale=scale)
    flat = {n: t if n == "lse" else t.transpose(0, 1) for n, t in got.items()}
    want, bound = ref.attend(*(x.transpose(0, 1) for x in (q, k, v)), nq, nk, aq[:-1], ak[:-1],
                             causal, scale, dout.transpose(0, 1))
    hold(flat, want, bound)


ONE = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 385, 513]


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("n", ONE)
def test_one_sequence(n, causal):
    check_packed([n], [n], 1, 1, causal, n)


@pytest.mark.parametrize("heads", [(1, 1), (2, 1), (3, 1), (5, 5), (6, 2), (8, 1), (12, 4), (16, 1),
                                   (32, 1), (48, 2)], ids=str)
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
def test_grouped_heads(heads, causal):
    check_packed([150, 1, 37], [150, 1, 37], *heads, causal, heads[0])


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("nq,nk", [
    ([0, 5, 0, 300, 0], [0, 5, 0, 300, 0]),           # sequences of nothing
    ([7, 130, 64], [0, 0, 0]),                        # no keys at all
    ([200, 130], [3, 129]),                           # first queries attend nothing (causal)
    ([1, 1, 1], [1, 500, 128]),                       # single tokens behind a past
    ([20, 300], [1021, 640]),                         # a chunk behind a past
    ([0, 0], [40, 300]),                              # keys that nothing attends
    ([40] * 70, [40] * 70),                           # more sequences than a search step
    ([1] * 1100, [1] * 1100),                         # than two
], ids=["empty", "keyless", "short", "token", "chunk", "queryless", "many", "crowd"])
def test_lengths(nq, nk, causal):
    check_packed(nq, nk, 4, 2, causal, sum(nq) + sum(nk))


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("B,most,Hq,Hkv", [(2, 700, 32, 32), (31, 300, 6, 6), (32, 300, 12, 2),
                                           (33, 300, 6, 6)], ids=str)
def test_more_tiles_than_start_at_once(B, most, Hq, Hkv, causal):
    """Sequences of unlike and of equal lengths, some of nothing, whose tiles come in turn; packed,
    then the same padded, with 0 behind them."""
    g = gen(B)
    nq = torch.randint(0, most, (B,), generator=g).tolist()
    nk = torch.randint(0, most, (B,), generator=g).tolist()
    nq[0] = nk[0] = most
    nq[-1], nk[-1] = nq[B // 2], nk[B // 2] = 129, most
    if B > 2:
        nq[3], nk[5], nq[7], nk[7] = 0, 0, 0, 0
    aq, ak = starts(nq), starts(nk)
    q, k, v, dout = (randn((n + 9, h, D), g)
                     for n, h in ((aq[-1], Hq), (ak[-1], Hkv), (ak[-1], Hkv), (aq[-1], Hq)))
    got = both(q, k, v, dout, q_seq=i32(aq), k_seq=i32(ak), causal=causal)
    flat = {n: t if n == "lse" else t.transpose(0, 1) for n, t in got.items()}
    want, bound = ref.attend(*(x.transpose(0, 1) for x in (q, k, v)), nq, nk, aq[:-1], ak[:-1],
                             causal, None, dout.transpose(0, 1))
    hold(flat, want, bound)

    def pad(x, at, n):
        y = torch.full((B, x.shape[1], most + 3, D), math.nan, dtype=x.dtype, device=DEV)
        for b in range(B):
            y[b, :, :n[b]] = x[at[b]:at[b] + n[b]].transpose(0, 1)
        return y

    pads = both(pad(q, aq, nq), pad(k, ak, nk), pad(v, ak, nk), pad(dout, aq, nq), q_seq=i32(nq),
                k_seq=i32(nk), causal=causal)
    # (not the bits of the packed call: a batch of fewer tiles than SMs is cut into more ranges)
    for b in range(B):
        rows = {"out": (aq, nq), "lse": (aq, nq), "dq": (aq, nq), "dk": (ak, nk), "dv": (ak, nk)}
        at = {n: slice(a[b], a[b] + m[b]) for n, (a, m) in rows.items()}
        hold({n: pads[n][b][:, :rows[n][1][b]] for n in rows},
             {n: want[n][:, at[n]] for n in rows}, {n: bound[n][:, at[n]] for n in rows})
        for n in ("out", "dq", "dk", "dv"):
            assert (pads[n][b][:, rows[n][1][b]:] == 0).all(), (n, b)


def test_rows_of_no_sequence_are_left_alone():
    g = gen(5)
    q, k, v, dout = (randn((300, h, D), g) for h in (4, 2, 2, 4))
    for t in (q, k, v, dout):  # what lies there reaches nothing
        t[:7] = math.nan
        t[150:] = math.inf
    seq = i32([7, 80, 80, 150])
    out = torch.full_like(q, 3.0)
    lse = torch.full((4, 300), 5.0, device=DEV)
    binding.vsa_fwd_prompt(q, k, v, seq, out=out, lse=lse)
    d = [torch.full_like(x, 7.0) for x in (q, k, v)]
    binding.vsa_bwd_prompt(q, k, v, out, dout, lse, seq, dq=d[0], dk=d[1], dv=d[2])
    ok()
    got = dict(out=out, lse=lse, dq=d[0], dk=d[1], dv=d[2])
    for n, mark in (("out", 3.0), ("dq", 7.0), ("dk", 7.0), ("dv", 7.0)):
        assert (got[n][:7] == mark).all() and (got[n][150:] == mark).all()
    assert (lse[:, :7] == 5.0).all() and (lse[:, 150:] == 5.0).all()
    at, n = [7, 80, 80], [73, 0, 70]
    flat = {x: t if x == "lse" else t.transpose(0, 1) for x, t in got.items()}
    hold(flat, *ref.attend(*(x.transpose(0, 1) for x in (q, k, v)), n, n, at, at, True, None,
                           dout.transpose(0, 1)))


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("nq,nk,Sq,Sk", [
    ([130, 0, 77], [130, 0, 77], 130, 130), ([5, 1, 200], [300, 33, 200], 201, 320),
    ([256, 255, 1], [1, 0, 256], 256, 256), (None, None, 100, 190)])
def test_padded(nq, nk, Sq, Sk, causal):
    """Rows behind a length get 0, and what they hold reaches nothing."""
    g = gen(Sq)
    B = 3
    q, dout = randn((B, 4, Sq, D), g), randn((B, 4, Sq, D), g)
    k, v = randn((B, 2, Sk, D), g), randn((B, 2, Sk, D), g)
    mq, mk = nq or [Sq] * B, nk or [Sk] * B
    for b in range(B):
        q[b, :, mq[b]:] = dout[b, :, mq[b]:] = math.nan
        k[b, :, mk[b]:] = v[b, :, mk[b]:] = math.inf
    got = both(q, k, v, dout, q_seq=nq and i32(nq), k_seq=nk and i32(nk), causal=causal)
    for b in range(B):
        one = {n: t[b] for n, t in got.items()}
        hold(one, *ref.attend(q[b], k[b], v[b], [mq[b]], [mk[b]], [0], [0], causal, None, dout[b]))
        for n, rows in (("out", mq), ("dq", mq), ("dk", mk), ("dv", mk)):
            assert (one[n][:, rows[b]:] == 0).all(), n
        assert (one["lse"][:, mq[b]:] == ref.LSE_EMPTY).all()


def test_layouts_agree():
    """Slices of a fused projection, [B,S,H,D] views, outputs as slices of one buffer: the bits
    of the contiguous call."""
    g = gen(9)
    B, S, Hq, Hkv = 2, 300, 8, 2
    x = randn((B, S, Hq + 2 * Hkv, D), g)
    dout = randn((B, S, Hq, D), g)
    seq = i32([0, S, 2 * S])
    sl = (slice(0, Hq), slice(Hq, Hq + Hkv), slice(Hq + Hkv, None))
    plain = [x.flatten(0, 1)[:, s].contiguous() for s in sl]
    want = both(*plain, dout.flatten(0, 1), q_seq=seq)
    # packed, all of them slices
    f = x.flatten(0, 1)
    y = torch.empty_like(f)
    out = torch.empty((2 * S, 2 * Hq, D), dtype=torch.bfloat16, device=DEV)[:, ::2]
    o, lse = binding.vsa_fwd_prompt(f[:, sl[0]], f[:, sl[1]], f[:, sl[2]], seq, out=out)
    assert o is out
    binding.vsa_bwd_prompt(f[:, sl[0]], f[:, sl[1]], f[:, sl[2]], out, dout.flatten(0, 1), lse, seq,
                           dq=y[:, sl[0]], dk=y[:, sl[1]], dv=y[:, sl[2]])
    ok()
    for n, t in (("out", out), ("lse", lse), ("dq", y[:, sl[0]]), ("dk", y[:, sl[1]]),
                 ("dv", y[:, sl[2]])):
        assert torch.equal(t, want[n]), n
    # padded, as views of [B, S, H, D], into views of one buffer
    v4 = [x[:, :, s].transpose(1, 2) for s in sl]
    want = both(*(t.contiguous() for t in v4), dout.transpose(1, 2).contiguous())
    z = torch.empty_like(x)
    z4 = [z[:, :, s].transpose(1, 2) for s in sl]
    o4, l4 = binding.vsa_fwd_prompt(*v4)
    binding.vsa_bwd_prompt(*v4, o4, dout.transpose(1, 2), l4, dq=z4[0], dk=z4[1], dv=z4[2])
    ok()
    assert torch.equal(o4, want["out"]) and torch.equal(l4, want["lse"])
    for t, n in zip(z4, ("dq", "dk", "dv")):
        assert torch.equal(t, want[n]), n


@pytest.mark.parametrize("mul", [0.0, 4.0, 20.0], ids=["flat", "peaky", "one-hot"])
def test_scores_of_any_size(mul):
    check_packed([300, 40], [300, 40], 4, 2, True, 11, mul)


def test_other_scales():
    for scale in (1e-6, 1.0):
        check_packed([200], [260], 2, 1, True, 12, 1.0, scale)


def test_a_sequence_of_one_row_has_no_gradient_of_its_score():
    check_packed([1] * 9, [1] * 9, 2, 2, True, 13, 3.0)


def test_scores_that_are_no_numbers():
    """NaN where the formula gives NaN, and nowhere else."""
    g = gen(14)
    q, k, v = randn((200, 1, D), g), randn((200, 1, D), g), randn((200, 1, D), g)
    q[3] = math.nan                      # one row's scores
    q[9], k[:, :, 0] = 0.0, 1.0
    q[9, 0, 0] = -math.inf               # a row whose scores are all -infinity
    out, lse = binding.vsa_fwd_prompt(q, k, v, i32([0, 200]))
    ok()
    bad = [3, 9]
    assert out[bad].isnan().all() and lse[:, bad].isnan().all()
    good = [i for i in range(200) if i not in bad]
    assert out[good].isfinite().all() and lse[:, good].isfinite().all()


def test_gradient_against_differences():
    """The directional derivative of sum(out * dout) by central differences in 64 bits."""
    g = gen(15)
    n, off = [70, 33], [0, 70]
    q, k, v, dout = (randn((103, 2, D), g) for _ in range(4))
    got = both(q, k, v, dout, q_seq=i32([0, 70, 103]))
    x = [t.double().transpose(0, 1) for t in (q, k, v)]

    def f(t):
        y = [a + t * b for a, b in zip(x, step)]
        r, _ = ref.attend(*y, n, n, off, off)
        return (r["out"] * dout.double().transpose(0, 1)).sum().item()

    for which, name in enumerate(("dq", "dk", "dv")):
        d = torch.randn(x[0].shape, generator=g, dtype=torch.float64).to(DEV)
        step = [d if i == which else torch.zeros_like(d) for i in range(3)]
        slope = (f(1e-4) - f(-1e-4)) / 2e-4
        grad = got[name].double().transpose(0, 1)
        _, bound = ref.attend(*x, n, n, off, off, dout=dout.transpose(0, 1))
        assert abs((grad * d).sum().item() - slope) <= (bound[name] * d.abs()).sum().item() + 1e-4


def test_long_sequences_by_rows():
    """A long ragged pair: sampled rows against 64 bits."""
    g = gen(16)
    n = [9001, 2500]
    q, k, v = (randn((sum(n), h, D), g) for h in (4, 2, 2))
    out, lse = binding.vsa_fwd_prompt(q, k, v, i32(starts(n)))
    ok()
    for a, m in ((0, n[0]), (n[0], n[1])):
        for i in (0, 1, 127, 128, 255, 256, m // 2, m - 129, m - 2, m - 1):
            for h in (0, 3):
                r, b = ref.head(q[a + i:a + i + 1, h].double(), k[a:a + i + 1, h // 2].double(),
                                v[a:a + i + 1, h // 2].double(), True, 1.0 / math.sqrt(D))
                assert ((out[a + i, h].double() - r["out"][0]).abs() <= b["out"][0]).all()
                assert (lse[h, a + i].double() - r["lse"][0]).abs() <= b["lse"][0]


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("nq,nk,Hq,Hkv", [([1], [5000], 1, 1), ([3, 1], [4000, 129], 8, 2),
                                          ([70], [4100], 4, 4), ([300], [40], 2, 2),
                                          ([2, 5, 0], [3700, 0, 300], 6, 1)], ids=str)
def test_few_queries_against_many_keys(nq, nk, Hq, Hkv, causal):
    """Keys cut into ranges: within the bounds, and near the uncut result."""
    g = gen(sum(nk))
    q, k, v = randn((sum(nq), Hq, D), g), randn((sum(nk), Hkv, D), g), randn((sum(nk), Hkv, D), g)
    aq, ak = i32(starts(nq)), i32(starts(nk))
    assert binding.fwd_prompt_workspace_bytes(True, len(nq), Hq, Hkv, sum(nq), sum(nk)) > 0 \
        or nk == [40]
    out, lse = binding.vsa_fwd_prompt(q, k, v, aq, ak, causal=causal)
    ok()
    x = [t.transpose(0, 1) for t in (q, k, v)]
    want, bound = ref.attend(*x, nq, nk, starts(nq), starts(nk), causal)
    hold(dict(out=out.transpose(0, 1), lse=lse), want, bound)
    whole, l2 = binding.vsa_fwd_prompt(q, k, v, aq, ak, causal=causal, workspace=False)
    ok()
    hold(dict(out=whole.transpose(0, 1), lse=l2), want, bound)


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("nq,nk,Hq,Hkv", [([3], [2500], 2, 1), ([70, 1], [2500, 600], 4, 2),
                                          ([600], [600], 8, 1), ([300, 41], [300, 41], 24, 1),
                                          ([1100], [90], 6, 1), ([500, 0, 2], [2100, 700, 0], 16, 1)],
                         ids=str)
def test_gradients_of_few_tiles(nq, nk, Hq, Hkv, causal):
    """dq over ranges of keys, (dk, dv) over ranges of queries and heads."""
    check_packed(nq, nk, Hq, Hkv, causal, sum(nq) * 3 + Hq)


def test_gradients_of_few_tiles_padded():
    g = gen(27)
    q, dout = randn((2, 16, 400, D), g), randn((2, 16, 400, D), g)
    k, v = randn((2, 1, 2100, D), g), randn((2, 1, 2100, D), g)
    nq, nk = [400, 37], [2100, 130]
    got = both(q, k, v, dout, q_seq=i32(nq), k_seq=i32(nk))
    for b in range(2):
        one = {n: t[b] for n, t in got.items()}
        hold(one, *ref.attend(q[b], k[b], v[b], [nq[b]], [nk[b]], [0], [0], True, None, dout[b]))
        for n, rows in (("out", nq), ("dq", nq), ("dk", nk), ("dv", nk)):
            assert (one[n][:, rows[b]:] == 0).all(), n


def test_few_queries_scores_that_are_no_numbers():
    g = gen(26)
    q, k, v = randn((3, 1, D), g), randn((3000, 1, D), g), randn((3000, 1, D), g)
    k[100] = math.nan                  # every query sees it
    out, lse = binding.vsa_fwd_prompt(q, k, v, i32([0, 3]), i32([0, 3000]))
    assert out.isnan().all() and lse.isnan().all()
    k[100] = 0.0
    k[:, :, 0] = 1.0
    q[1], q[1, 0, 0] = 0.0, -math.inf  # all of one row's scores are -infinity
    out, lse = binding.vsa_fwd_prompt(q, k, v, i32([0, 3]), i32([0, 3000]))
    ok()
    assert out[1].isnan().all() and lse[0, 1].isnan()
    assert out[[0, 2]].isfinite().all() and lse[0, [0, 2]].isfinite().all()


def test_results_do_not_depend_on_timing():
    g = gen(17)
    n = [1500, 3, 700]
    q, k, v, dout = (randn((sum(n), h, D), g) for h in (8, 2, 2, 8))
    seq = i32(starts(n))
    first = both(q, k, v, dout, q_seq=seq)
    side = torch.cuda.Stream()
    for i in range(4):
        busy = torch.randn(2000, 2000, device=DEV)
        with torch.cuda.stream(side):
            for _ in range(i):
                busy = busy @ busy
        again = both(q, k, v, dout, q_seq=seq)
        for x in first:
            assert torch.equal(first[x], again[x]), x


def test_captured_and_replayed_with_other_lengths():
    """A graph of the step replays with other starts, behind eager calls that live on."""
    g = gen(18)
    q, k, v, dout = (randn((400, h, D), g) for h in (4, 2, 2, 4))
    seq = i32([0, 400, 400])
    eager = both(q, k, v, dout, q_seq=seq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = binding.vsa_fwd_prompt(q, k, v, seq)
        grads = binding.vsa_bwd_prompt(q, k, v, out, dout, lse, seq)
    for lens in ([400, 0], [130, 270], [399, 1]):
        seq.copy_(i32([0, lens[0], 400]))
        graph.replay()
        ok()
        want = both(q, k, v, dout, q_seq=seq)
        for x, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
            assert torch.equal(t, want[x]), x
    assert torch.equal(eager["out"][:1], out[:1])


def test_another_stream():
    g = gen(19)
    q, k, v, dout = (randn((500, h, D), g) for h in (4, 2, 2, 4))
    seq = i32([0, 333, 500])
    want = both(q, k, v, dout, q_seq=seq)
    side = torch.cuda.Stream()
    busy = torch.randn(4000, 4000, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        busy = busy @ busy  # the current stream is held up; the calls below must not wait
    out, lse = binding.vsa_fwd_prompt(q, k, v, seq, stream=side)
    grads = binding.vsa_bwd_prompt(q, k, v, out, dout, lse, seq, stream=side)
    side.synchronize()
    for x, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        assert torch.equal(t, want[x]), x


def test_starts_outside_the_tensor_are_clamped():
    g = gen(20)
    q, k, v = (randn((100, h, D), g) for h in (2, 1, 1))
    out, _ = binding.vsa_fwd_prompt(q, k, v, i32([-5, 60, 1 << 30]))
    want, _ = binding.vsa_fwd_prompt(q, k, v, i32([0, 60, 100]))
    ok()
    assert torch.equal(out, want)
    x = [t.transpose(0, 1)[None] for t in (q, k, v)]
    out, _ = binding.vsa_fwd_prompt(*x, i32([1 << 30]), i32([1000]))
    want, _ = binding.vsa_fwd_prompt(*x)
    ok()
    assert torch.equal(out, want)
    # starts that do not ascend: nothing outside is touched, the call ends
    binding.vsa_fwd_prompt(q, k, v, i32([90, 10, 50, 0, 70]))
    ok()


def test_far_rows_pass_32_bit_offsets():
    """Rows whose elements lie more than 2^32 bytes into the tensors."""
    g = gen(21)
    H, T = 40, 460_000  # 4.7 GB a tensor
    x = torch.zeros((T, H, D), dtype=torch.bfloat16, device=DEV)
    x[-300:] = randn((300, H, D), g)
    seq = i32([T - 300, T])
    out = torch.empty_like(x)
    binding.vsa_fwd_prompt(x, x, x, seq, out=out)
    near = x[-300:].clone()
    want, lse = binding.vsa_fwd_prompt(near, near, near, i32([0, 300]))
    ok()
    assert torch.equal(out[-300:], want)
    lse_far = torch.zeros((H, T), device=DEV)
    lse_far[:, -300:] = lse
    d = [torch.empty_like(x) for _ in range(3)]
    binding.vsa_bwd_prompt(x, x, x, out, x, lse_far, seq, dq=d[0], dk=d[1], dv=d[2])
    for a, b in zip(d, binding.vsa_bwd_prompt(near, near, near, want, near, lse, i32([0, 300]))):
        assert torch.equal(a[-300:], b)
    ok()


def test_agrees_with_the_block_sparse_forward_over_all_blocks():
    g = gen(22)
    q, k, v = (randn((1, h, 512, D), g) for h in (4, 2, 2))
    idx = torch.arange(8, dtype=torch.int32, device=DEV).expand(1, 4, 8, 8).contiguous()
    num = torch.full((1, 4, 8), 8, dtype=torch.int32, device=DEV)
    a, la = binding.vsa_fwd_gqa(q, k, v, idx, num, None, block=64)
    b, lb = binding.vsa_fwd_prompt(q, k, v, causal=False)
    ok()
    _, bound = ref.attend(q[0], k[0], v[0], [512], [512], [0], [0], False)
    assert ((a[0].double() - b[0].double()).abs() <= 2 * bound["out"]).all()
    assert ((la[0].double() - lb[0].double()).abs() <= 2 * bound["lse"]).all()


def test_launches_and_no_lse():
    g = gen(23)
    q, k, v = (randn((64, h, D), g) for h in (2, 1, 1))
    out, lse = binding.vsa_fwd_prompt(q, k, v, i32([0, 64]))
    assert binding.vsa_last_launch_count() == 1
    o2, l2 = binding.vsa_fwd_prompt(q, k, v, i32([0, 64]), lse=False)
    assert l2 is None and torch.equal(out, o2)
    binding.vsa_bwd_prompt(q, k, v, out, out, lse, i32([0, 64]))
    assert binding.vsa_last_launch_count() == 2
    empty = q[:0]
    o3, _ = binding.vsa_fwd_prompt(empty, k, v, i32([0, 0]), i32([0, 64]))
    assert o3.shape == (0, 2, D)
    _, dk, dv = binding.vsa_bwd_prompt(empty, k, v, o3, empty, lse[:, :0].contiguous(), i32([0, 0]),
                                       i32([0, 64]))
    ok()
    assert (dk == 0).all() and (dv == 0).all()


@pytest.mark.parametrize("shape", [(1, 2, 300, 300), (2, 8, 40, 2500)], ids=str)
def test_a_wait_that_runs_out_is_reported(shape):
    """The test hook holds the MMA warps on a barrier that nothing completes: every role ends, the
    status says so, and the next calls are right again."""
    B, H, Sq, Sk = shape
    g = gen(28)
    q, k, v = randn((B, H, Sq, D), g), randn((B, 1, Sk, D), g), randn((B, 1, Sk, D), g)
    want, lse = binding.vsa_fwd_prompt(q, k, v)
    grads = binding.vsa_bwd_prompt(q, k, v, want, q, lse)
    ok()
    try:
        binding.vsa_set_wait_limit_ns(2_000_000)
        binding.vsa_set_stall_test(True)
        binding.vsa_fwd_prompt(q, k, v)
        code, detail = binding.vsa_device_status()
        assert code == binding.VSA_ERR_DEVICE_TIMEOUT and detail & 0x100
        binding.vsa_bwd_prompt(q, k, v, want, q, lse)
        code, detail = binding.vsa_device_status()
        assert code == binding.VSA_ERR_DEVICE_TIMEOUT and detail & 0x100
    finally:
        binding.vsa_set_stall_test(False)
        binding.vsa_set_wait_limit_ns(0)
    out, l2 = binding.vsa_fwd_prompt(q, k, v)
    again = binding.vsa_bwd_prompt(q, k, v, out, q, l2)
    ok()
    assert torch.equal(out, want) and torch.equal(l2, lse)
    for x, y in zip(again, grads):
        assert torch.equal(x, y)


def test_keys_are_as_long_as_queries_unless_said_otherwise():
    g = gen(29)
    q, k, v = randn((2, 2, 90, D), g), randn((2, 1, 90, D), g), randn((2, 1, 90, D), g)
    n = i32([50, 90])
    for causal in (True, False):
        a, la = binding.vsa_fwd_prompt(q, k, v, n, causal=causal)
        b, lb = binding.vsa_fwd_prompt(q, k, v, n, n, causal=causal)
        assert torch.equal(a, b) and torch.equal(la, lb)
    with pytest.raises(ValueError):
        binding.vsa_fwd_prompt(q, k[:, :, :80], v[:, :, :80], n)
    ok()


def test_refusals():
    g = gen(24)
    q, k, v = (randn((64, h, D), g) for h in (4, 2, 2))
    seq = i32([0, 64])
    fwd = binding.vsa_fwd_prompt
    out, lse = fwd(q, k, v, seq)
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(k=k[:, :, :64]), dict(v=v[:, :1]),
                dict(q_seq=None), dict(q_seq=seq.long()), dict(k_seq=i32([0, 1, 2])),
                dict(q=q[0]), dict(q=q.transpose(1, 2)), dict(q="q"),
                dict(out=out[:63]), dict(lse=lse[:1])):
        with pytest.raises((ValueError, TypeError)):
            fwd(**{**dict(q=q, k=k, v=v, q_seq=seq), **bad})
    for bad in (dict(k=k.expand(64, 2, D)[:, :1].expand(64, 3, D), v=v[:, :1].expand(64, 3, D)),
                dict(scale=0.0), dict(scale=math.nan), dict(out=q),
                dict(q=q[:, :1].expand(64, 4, D))):  # broadcast heads: copy them first
        with pytest.raises(binding.VsaError):
            fwd(**{**dict(q=q, k=k, v=v, q_seq=seq), **bad})
    with pytest.raises(binding.VsaError):
        binding.vsa_bwd_prompt(q, k, v, out, out, lse, seq, dk=k)
    with pytest.raises(binding.VsaError):
        binding.vsa_bwd_prompt(q, k, v, out, out, lse, seq,
                               workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    d = torch.empty((64, 4, D), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(binding.VsaError):  # two gradients that share rows
        binding.vsa_bwd_prompt(q, k, v, out, out, lse, seq, dq=d, dk=d[:, 1:3])
    with pytest.raises(binding.VsaError):  # a result whose own rows overlap
        fwd(q, k, v, seq, out=d.as_strided((64, 4, D), (D, D, 1)))
    ok()


def test_short_and_long_way_agree(monkeypatch):
    g = gen(25)
    q, k, v, dout = (randn((150, h, D), g) for h in (4, 2, 2, 4))
    seq = i32([0, 100, 150])
    a = both(q, k, v, dout, q_seq=seq)
    monkeypatch.setattr(binding, "_fast", False)
    b = both(q, k, v, dout, q_seq=seq)
    for n in a:
        assert torch.equal(a[n], b[n])
    x = [t.transpose(0, 1)[None] for t in (q, k, v, dout)]
    c = both(*x, q_seq=i32([100]), k_seq=i32([77]), causal=False)
    monkeypatch.undo()
    d = both(*x, q_seq=i32([100]), k_seq=i32([77]), causal=False)
    for n in c:
        assert torch.equal(c[n], d[n])

"""The operators around the attention start up while their predecessor in the stream ends, so
what that one writes has to be read by ordinary loads behind the wait for it.  On the CPU the
kernels' sources are held to that; on the GPU a server's step and a training step's choice
run behind a busy stream with nothing between the calls, on buffers that hold other (valid)
contents beforehand, and are compared with the plain forms once at the end."""
import os
import re

import pytest
import torch

import serve_ref as ref
from block_sparse_attention_vsa_gb300 import binding
from block_sparse_attention_vsa_gb300 import build as libbuild

DEV = "cuda:0"
D = 128


@pytest.mark.parametrize("name", ["vsa_select_kernel.cuh", "vsa_cache_kernel.cuh",
                                  "vsa_warp_ptx.cuh"])
def test_no_read_only_loads_in_kernels_that_start_early(name):
    with open(os.path.join(libbuild.CSRC, name)) as f:
        code = re.sub(r"//.*", "", f.read())
    for word in ("__ldg", "__restrict__", "ld.global.nc", ".nc."):
        assert word not in code, word
    # nothing but L2 prefetches and indices comes before the wait
    for body in code.split("__global__")[1:]:
        head = body[:body.index("after_predecessor();")]
        assert "read_global" not in head


def chain_case(seed):
    """Three sequences on three heads, tokens to write, and a second set of contents."""
    g = torch.Generator().manual_seed(seed)
    block, Hkv, T = 64, 3, 200
    lens = [700, 64 * 30, 0]
    n_new = [T, 37, T]
    mb, spare = 40, 4
    need = [-(-n // block) + spare for n in lens]
    pages = Hkv * sum(need) + 5
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((3, Hkv, mb), -1, dtype=torch.int32)
    at = 0
    for b in range(3):
        for h in range(Hkv):
            table[b, h, :need[b]] = perm[at:at + need[b]]
            at += need[b]

    def bf16(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16)

    state = {t: ref.e4m3(torch.randn((pages, block, D), generator=g) * 60) for t in "kv"}
    for t in ("k_scale", "v_scale"):
        state[t] = torch.exp2(torch.randint(-9, -4, (pages,), generator=g).double())
    state["k_mean"] = bf16(pages, D).double()
    return dict(block=block, table=table, lens=torch.tensor(lens, dtype=torch.int32),
                n_new=torch.tensor(n_new, dtype=torch.int32), state=state,
                k=bf16(3, Hkv, T, D), v=bf16(3, Hkv, T, D), q=bf16(3, Hkv * 4, 1, D),
                weight=torch.rand((3, Hkv, mb), generator=g))


def to_cache(state):
    return binding.Cache8(*(state[t].float().to(torch.float8_e4m3fn).to(DEV) for t in "kv"),
                          state["k_scale"].float().to(DEV), state["v_scale"].float().to(DEV),
                          state["k_mean"].to(torch.bfloat16).to(DEV))


def expected(c, mean):
    """The step's outcome by the plain forms; the choice on the means that the cache holds."""
    state = {t: x.clone() for t, x in c["state"].items()}
    ref.cache_write(state, c["k"], c["v"], c["table"], c["lens"], c["n_new"], c["block"])
    held = c["lens"] + c["n_new"]
    idx, num = ref.cache_select(c["q"], mean, c["table"], held, 6, c["block"], 1, 2)
    r = ref.attend(c["q"], state, c["table"], held, c["block"], idx, num)
    return state, idx, num, r


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True], ids=["eager", "graph"])
def test_a_step_behind_a_busy_stream(captured):
    """write -> select -> attend -> evict, each reading what the one before wrote.  The buffers
    hold another case's contents until the moment they are written."""
    import __graft_entry__
    __graft_entry__.build()
    c, other = chain_case(71), chain_case(72)
    assert c["table"].shape == other["table"].shape
    cache, start, stale = to_cache(c["state"]), to_cache(c["state"]), to_cache(other["state"])
    k, v, q = c["k"].to(DEV), c["v"].to(DEV), c["q"].to(DEV)
    table, lens, n_new = c["table"].to(DEV), c["lens"].to(DEV), c["n_new"].to(DEV)
    held = lens + n_new
    weight, past = c["weight"].to(DEV), c["weight"].to(DEV)
    stale_w = other["weight"].to(DEV)
    ws = binding.new_cache_workspace(3, q.shape[1], k.shape[1], table.shape[2], True, DEV)

    def step():
        binding.vsa_cache_write(cache, k, v, table, lens, n_new)
        idx, num = binding.vsa_cache_select(q, cache.k_mean, table, held, 6, n_first=1, n_near=2)
        out, lse = binding.vsa_fwd_cache(q, cache, table, held, idx=idx, num=num, weight=weight,
                                         keep=0.5, workspace=ws)
        gone = binding.vsa_cache_evict(weight, table, held, 8, n_first=1, n_last=2)
        # evicted, then attended without what went
        out2, lse2 = binding.vsa_fwd_cache(q, cache, gone.table, gone.lens, workspace=ws)
        return idx, num, out, lse, gone, out2, lse2

    def fill(src, w):
        for a, b in zip(cache, src):
            a.view(torch.uint8).copy_(b.view(torch.uint8))
        weight.copy_(w)

    fill(start, past)
    first = step()                       # launches, allocations
    torch.cuda.synchronize()
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
    busy = torch.ones(4096, 4096, device=DEV, dtype=torch.bfloat16)
    runs = []
    for _ in range(20):
        fill(stale, stale_w)
        torch.cuda.synchronize()
        for _ in range(3):
            busy = busy @ busy
        fill(start, past)
        if graph is None:
            got = step()
        else:
            graph.replay()
        runs.append([t.clone() for t in
                     (*cache[2:], got[0], got[1], got[2], got[3], *got[4], got[5], got[6], weight)])
    torch.cuda.synchronize()
    for run in runs[1:]:
        for a, b in zip(run, runs[0]):
            assert torch.equal(a, b)
    # once against the plain forms
    state, idx, num, r = expected(c, cache.k_mean.cpu())
    # exact code sums; one division, one rounding to fp32 and one to bf16
    assert ((cache.k_mean.cpu().double() - state["k_mean"]).abs()
            <= (2.0 ** -8 + 2.0 ** -22) * state["k_mean"].abs()).all()
    for t in "kv":
        assert torch.equal(getattr(cache, t).cpu().double(), state[t])
        assert torch.equal(getattr(cache, t + "_scale").cpu().double(), state[t + "_scale"])
    assert torch.equal(got[0].cpu(), idx) and torch.equal(got[1].cpu(), num)
    from test_serve_gpu import check_attend
    check_attend(r, got[2], got[3], weight, c["weight"], 0.5)
    want = ref.evict(weight.cpu(), c["table"], held.cpu(), 8, c["block"], 1, 2)
    for a, b in zip(got[4], want):
        assert torch.equal(a.cpu(), b)
    assert int(got[4].n_freed.max()) > 0
    check_attend(ref.attend(c["q"], state, want[0], want[2], c["block"]), got[5], got[6])
    assert all(torch.equal(a, b) for a, b in zip(first[:4], got[:4]))


@pytest.mark.gpu
def test_means_then_choice_then_attention_behind_a_busy_stream():
    import __graft_entry__
    __graft_entry__.build()
    g = torch.Generator().manual_seed(73)
    x = [torch.randn((1, 4, 64 * 20, D), generator=g).to(torch.bfloat16) for _ in range(3)]
    q, k, v = (t.to(DEV) for t in x)
    sizes = torch.full((20,), 64, dtype=torch.int32, device=DEV)
    qm, km = (torch.zeros((1, 4, 20, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    busy = torch.ones(4096, 4096, device=DEV, dtype=torch.bfloat16)
    runs = []
    for _ in range(20):
        qm.normal_()
        km.normal_()
        torch.cuda.synchronize()
        for _ in range(3):
            busy = busy @ busy
        binding.vsa_block_mean(q, out=qm)
        binding.vsa_block_mean(k, out=km)
        idx, num = binding.vsa_select_blocks(qm, km, 5, n_near=1)
        out, lse = binding.vsa_fwd(q, k, v, idx, num, sizes)
        runs.append([t.clone() for t in (qm, km, idx, num, out, lse)])
    torch.cuda.synchronize()
    for run in runs[1:]:
        for a, b in zip(run, runs[0]):
            assert torch.equal(a, b)
    want = ref.select_blocks(qm.cpu(), km.cpu(), 5, n_near=1)
    assert torch.equal(idx.cpu(), want[0]) and torch.equal(num.cpu(), want[1])
    for t, m in ((x[0], qm), (x[1], km)):
        mean, mag = ref.block_mean(t, None, 64)
        # one bf16 rounding, an fp32 sum of 64 terms
        assert ((m.cpu().double() - mean).abs() <= 2.0 ** -8 * mean.abs()
                + 64 * 2.0 ** -24 * mag).all()

"""Host-side argument checks of the attention over whole prompts and of the cache's pages: bad
calls get the documented status before the GPU is touched (no GPU needed); and the plain 64-bit
forms the GPU tests compare with, pinned to torch's autograd and to hand-made pools."""
import ctypes
import math
import os
import re

import pytest
import torch

import prompt_ref as ref
from block_sparse_attention_vsa_gb300 import binding
from block_sparse_attention_vsa_gb300 import build as libbuild

OK, INVALID, UNSUPPORTED = (binding.VSA_OK, binding.VSA_ERR_INVALID_ARG,
                            binding.VSA_ERR_UNSUPPORTED)
P = ctypes.c_void_p
MB = 1 << 20
D = 128


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return binding.load()


def p(v):
    return P(v) if v else None


def rows(heads):  # (batch, head, token) strides of a packed tensor
    return [0, D, heads * D]


def strides(values):
    return None if values is None else (ctypes.c_int64 * len(values))(*values)


def fwd(lib, **kw):
    a = dict(q=64 * MB, k=96 * MB, v=128 * MB, s=rows(4) + 2 * rows(2) + rows(4), qs=1 * MB,
             ks=2 * MB, packed=1, B=2, Hq=4, Hkv=2, Sq=200, Sk=300, D=D, causal=1, scale=0.1,
             out=160 * MB, lse=3 * MB, ws=0, n=0)
    a.update(kw)
    return lib.vsa_fwd_prompt(p(a["q"]), p(a["k"]), p(a["v"]), strides(a["s"]), p(a["qs"]),
                              p(a["ks"]), a["packed"], a["B"], a["Hq"], a["Hkv"], a["Sq"], a["Sk"],
                              a["D"], a["causal"], a["scale"], p(a["out"]), p(a["lse"]), p(a["ws"]),
                              a["n"], None)


def with_strides(i, values, base=rows(4) + 2 * rows(2) + rows(4)):
    s = list(base)
    s[3 * i:3 * i + 3] = values
    return s


@pytest.mark.parametrize("kw,code", [
    (dict(D=64), UNSUPPORTED), (dict(B=-1), INVALID), (dict(Hkv=3), INVALID),
    (dict(Hkv=0), INVALID), (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(q=0), INVALID), (dict(k=0), INVALID),
    (dict(out=0), INVALID), (dict(s=None), INVALID), (dict(qs=0), INVALID), (dict(ks=0), INVALID),
    (dict(qs=1 * MB + 2), INVALID), (dict(lse=3 * MB + 1), INVALID), (dict(q=64 * MB + 8), INVALID),
    (dict(s=with_strides(0, [0, D, 4 * D + 4])), INVALID),    # not 16 bytes apart
    (dict(s=with_strides(1, [0, D, 0])), INVALID),            # broadcast
    (dict(s=with_strides(2, [0, 64, 256])), INVALID),         # rows that overlap
    (dict(s=with_strides(3, [0, D, -4 * D])), INVALID),
    (dict(s=with_strides(3, [0, D, 2 * D])), INVALID),        # a result over itself
    (dict(s=with_strides(3, [0, 150 * D, D])), INVALID),
    (dict(s=with_strides(0, [0, 1 << 39, 4 * D])), INVALID),  # more than a copy's stride holds
    (dict(out=64 * MB), INVALID), (dict(out=96 * MB), INVALID), (dict(out=128 * MB + 256), INVALID),
    (dict(lse=160 * MB), INVALID), (dict(lse=1 * MB), INVALID), (dict(lse=64 * MB), INVALID), (dict(out=1 * MB), INVALID),
    (dict(Sq=(1 << 31) - 1), UNSUPPORTED), (dict(B=0), OK), (dict(Sq=0), OK), (dict(Hq=0), OK),
    (dict(packed=0, k=0), INVALID), (dict(ws=4 * MB, n=1000, Sk=5000), INVALID),
    (dict(ws=4 * MB + 8, n=1 << 30), INVALID), (dict(ws=64 * MB, n=1 << 30, Sk=5000), INVALID),
    (dict(ws=4 * MB, n=1 << 30, Sk=5000, lse=4 * MB + 64), INVALID),
    (dict(ws=4 * MB, n=1 << 30, Sk=5000, qs=4 * MB + 64), INVALID),
    (dict(Sq=1 << 30, s=with_strides(0, [0, D, 1 << 37])), INVALID),  # beyond any address
    (dict(packed=0, B=1 << 30, Hq=1 << 30, Hkv=1 << 30, Sq=1 << 30), UNSUPPORTED),
    (dict(B=(1 << 31) - 1, Hq=1 << 30, Hkv=1 << 30), UNSUPPORTED),
])
def test_fwd_prompt_checks(lib, kw, code):
    assert fwd(lib, **kw) == code


def test_slices_of_one_buffer_are_told_from_shared_rows(lib):
    """q, k, v and out as neighbouring heads of one token's row do not meet; a head further do."""
    if torch.cuda.is_available():
        pytest.skip("a call that passes would run on addresses that are not there")
    row = 12 * D
    s = [0, D, row] * 4

    def at(head):
        return 64 * MB + 2 * D * head

    apart = dict(q=at(0), k=at(4), v=at(6), s=s)
    good = fwd(lib, **apart, out=at(8))
    assert good == binding.VSA_ERR_CUDA  # past the checks, and no device
    for head in (1, 3, 5, 7, 9, 11):  # over q, k, v, or round into the next token's q
        assert fwd(lib, **apart, out=at(head)) == INVALID
    # a padded batch of [B, S, heads, D]
    s4 = [200 * row, D, row] * 4
    kw = dict(apart, s=s4, packed=0, Sk=200, ks=0, qs=0)
    assert fwd(lib, **kw, out=at(9)) == INVALID
    assert fwd(lib, **kw, out=at(8)) == good


def bwd(lib, **kw):
    a = dict(q=64 * MB, k=96 * MB, v=128 * MB, o=160 * MB, g=192 * MB, lse=3 * MB,
             s=rows(4) + 2 * rows(2) + 3 * rows(4) + 2 * rows(2), qs=1 * MB, ks=2 * MB, packed=1,
             B=2, Hq=4, Hkv=2, Sq=200, Sk=300, D=D, causal=1, scale=0.1, dq=224 * MB, dk=256 * MB,
             dv=288 * MB, ws=4 * MB, n=1 << 20)
    a.update(kw)
    return lib.vsa_bwd_prompt(p(a["q"]), p(a["k"]), p(a["v"]), p(a["o"]), p(a["g"]), p(a["lse"]),
                              strides(a["s"]), p(a["qs"]), p(a["ks"]), a["packed"], a["B"], a["Hq"],
                              a["Hkv"], a["Sq"], a["Sk"], a["D"], a["causal"], a["scale"],
                              p(a["dq"]), p(a["dk"]), p(a["dv"]), p(a["ws"]), a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), UNSUPPORTED), (dict(Hkv=3), INVALID), (dict(scale=-1.0), INVALID),
    (dict(o=0), INVALID), (dict(g=0), INVALID), (dict(lse=0), INVALID), (dict(dq=0), INVALID),
    (dict(dk=0), INVALID), (dict(dv=0), INVALID), (dict(ws=0), INVALID), (dict(n=1000), INVALID),
    (dict(ws=4 * MB + 8), INVALID), (dict(dq=64 * MB), INVALID), (dict(dk=96 * MB), INVALID),
    (dict(dv=256 * MB), INVALID), (dict(dq=192 * MB + 1024), INVALID), (dict(dk=4 * MB), INVALID),
    (dict(dv=3 * MB), INVALID), (dict(ws=160 * MB), INVALID), (dict(ws=1 * MB), INVALID),
    (dict(ws=3 * MB), INVALID),
    (dict(qs=0), INVALID), (dict(s=None), INVALID), (dict(B=0), OK), (dict(Sq=0, Sk=0), OK),
])
def test_bwd_prompt_checks(lib, kw, code):
    assert bwd(lib, **kw) == code


def test_workspaces_of_more_rows_than_memory(lib):
    big = (0, 1 << 30, 1 << 30, 1 << 30, 1 << 30, 1 << 30)
    assert lib.vsa_fwd_prompt_workspace_bytes(*big) == 0
    assert lib.vsa_bwd_prompt_workspace_bytes(*big) == 0


def test_fwd_prompt_workspace(lib):
    f = lib.vsa_fwd_prompt_workspace_bytes
    unit = (256 * 128 + 512) * 4
    # 2 heads of 128 tokens an item: (200 // 128 + 2) * 2 items, 25 of 152 SMs each; 40 key
    # tiles, 8 a range
    assert f(1, 2, 4, 2, 200, 5000) == 6 * 5 * unit
    assert f(1, 2, 4, 2, 200, 2048) == 6 * 2 * unit
    assert f(1, 2, 4, 2, 200, 1900) == 0 and f(1, 2, 4, 2, 20000, 20000) == 0
    assert f(0, 1, 1, 1, 1, 1 << 20) == 32 * unit
    assert f(1, 2, 5, 2, 200, 2500) == 0 and f(1, 0, 4, 2, 200, 2500) == 0


def test_bwd_prompt_workspace(lib):
    f = lib.vsa_bwd_prompt_workspace_bytes
    # a tile of 128 rows -- 2 heads of 64 tokens -- 1 KB each; 200 // 64 + 2 tiles a pair of heads
    assert f(1, 2, 4, 2, 200, 200) == 5 * 2 * 1024
    assert f(0, 2, 4, 2, 200, 200) == 2 * 4 * 2 * 1024
    # dq of 10 tiles in 5 ranges of 8 key tiles; (dk, dv) of 82 in one
    assert f(1, 2, 4, 2, 200, 5120) == 10 * 1024 + 10 * 5 * (128 * 128 + 128) * 4
    # (dk, dv) of 8 tiles -- 300 // 128 + 2 for 2 heads -- in 4 ranges of its 38 steps
    assert f(1, 2, 32, 2, 300, 300) == (37 + 2) * 2 * 1024 + 8 * 4 * 2 * 128 * 128 * 4
    # of 130 tiles in 2 ranges of its 384 steps (tiles of 2 heads and 64 tokens)
    assert f(1, 1, 12, 2, 8192, 8192) == 129 * 6 * 1024 + 130 * 2 * 2 * 128 * 128 * 4
    assert f(1, 2, 5, 2, 200, 200) == 0 and f(1, 0, 4, 2, 200, 200) == 0
    assert f(1, 2, 4, 0, 200, 200) == 0


def free(lib, **kw):
    a = dict(t=1 * MB, n=2 * MB, B=2, H=3, mb=5, block=64, pages=40, refs=3 * MB, bits=4 * MB)
    a.update(kw)
    return lib.vsa_pages_free(p(a["t"]), p(a["n"]), a["B"], a["H"], a["mb"], a["block"], a["pages"],
                              p(a["refs"]), p(a["bits"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(block=32), UNSUPPORTED), (dict(B=-1), INVALID), (dict(pages=-1), INVALID),
    (dict(t=0), INVALID), (dict(refs=0), INVALID), (dict(bits=0), INVALID),
    (dict(t=1 * MB + 2), INVALID), (dict(n=2 * MB + 1), INVALID), (dict(refs=1 * MB + 8), INVALID),
    (dict(bits=3 * MB), INVALID), (dict(n=1 * MB), INVALID), (dict(B=1 << 16, H=1 << 16), UNSUPPORTED),
    (dict(B=0), OK), (dict(mb=0, t=0), OK),
])
def test_pages_free_checks(lib, kw, code):
    assert free(lib, **kw) == code


def reserve(lib, **kw):
    a = dict(t=1 * MB, n=2 * MB, new=5 * MB, B=2, H=3, mb=5, block=64, pages=40, refs=3 * MB,
             bits=4 * MB, lack=6 * MB)
    a.update(kw)
    return lib.vsa_pages_reserve(p(a["t"]), p(a["n"]), p(a["new"]), a["B"], a["H"], a["mb"],
                                 a["block"], a["pages"], p(a["refs"]), p(a["bits"]), p(a["lack"]),
                                 None)


@pytest.mark.parametrize("kw,code", [
    (dict(block=100), UNSUPPORTED), (dict(H=-1), INVALID), (dict(t=0), INVALID), (dict(n=0), INVALID),
    (dict(lack=0), INVALID), (dict(refs=0), INVALID), (dict(lack=2 * MB), INVALID),
    (dict(lack=5 * MB + 4), INVALID), (dict(new=1 * MB), INVALID), (dict(bits=4 * MB + 2), INVALID),
    (dict(B=1 << 20, H=1 << 10, mb=2), UNSUPPORTED), (dict(B=0), OK),
])
def test_pages_reserve_checks(lib, kw, code):
    assert reserve(lib, **kw) == code


def fork(lib, **kw):
    a = dict(t=1 * MB, n=2 * MB, par=5 * MB, B=2, N=4, H=3, D=D, mb=5, block=64, pages=40, kc=64 * MB,
             vc=96 * MB, ks=7 * MB, vs=8 * MB, km=9 * MB, refs=3 * MB, bits=4 * MB, to=10 * MB,
             no=11 * MB, lack=6 * MB)
    a.update(kw)
    return lib.vsa_cache_fork(p(a["t"]), p(a["n"]), p(a["par"]), a["B"], a["N"], a["H"], a["D"],
                              a["mb"], a["block"], a["pages"], p(a["kc"]), p(a["vc"]), p(a["ks"]),
                              p(a["vs"]), p(a["km"]), p(a["refs"]), p(a["bits"]), p(a["to"]),
                              p(a["no"]), p(a["lack"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=64), UNSUPPORTED), (dict(block=16), UNSUPPORTED), (dict(N=-1), INVALID),
    (dict(par=0), INVALID), (dict(n=0), INVALID), (dict(t=0), INVALID), (dict(to=0), INVALID),
    (dict(no=0), INVALID), (dict(lack=0), INVALID), (dict(kc=0), INVALID), (dict(vs=0), INVALID),
    (dict(refs=0), INVALID), (dict(kc=64 * MB + 8), INVALID), (dict(km=9 * MB + 4), INVALID),
    (dict(to=1 * MB), INVALID), (dict(to=64 * MB), INVALID), (dict(no=5 * MB), INVALID),
    (dict(lack=11 * MB), INVALID), (dict(refs=1 * MB), INVALID), (dict(vc=64 * MB), INVALID),
    (dict(N=1 << 28), UNSUPPORTED), (dict(N=0), OK),
])
def test_cache_fork_checks(lib, kw, code):
    assert fork(lib, **kw) == code


def compact(lib, **kw):
    a = dict(t=1 * MB, B=2, H=3, D=D, mb=5, block=64, pages=40, kc=64 * MB, vc=96 * MB, ks=7 * MB,
             vs=8 * MB, km=9 * MB, refs=3 * MB, bits=4 * MB, to=10 * MB, used=11 * MB)
    a.update(kw)
    return lib.vsa_cache_compact(p(a["t"]), a["B"], a["H"], a["D"], a["mb"], a["block"], a["pages"],
                                 p(a["kc"]), p(a["vc"]), p(a["ks"]), p(a["vs"]), p(a["km"]),
                                 p(a["refs"]), p(a["bits"]), p(a["to"]), p(a["used"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=256), UNSUPPORTED), (dict(block=65), UNSUPPORTED), (dict(mb=-1), INVALID),
    (dict(t=0), INVALID), (dict(to=0), INVALID), (dict(used=0), INVALID), (dict(kc=0), INVALID),
    (dict(ks=7 * MB + 1), INVALID), (dict(to=1 * MB), INVALID), (dict(used=10 * MB), INVALID),
    (dict(km=96 * MB), INVALID), (dict(B=1 << 15, H=1 << 15, mb=2), UNSUPPORTED),
])
def test_cache_compact_checks(lib, kw, code):
    assert compact(lib, **kw) == code


@pytest.mark.parametrize("call", [free, reserve, fork, compact])
def test_entries_that_pass_64_bits(lib, call):
    assert call(lib, B=1 << 30, H=1 << 30, mb=16) == UNSUPPORTED


@pytest.mark.parametrize("name", ["vsa_prompt_common.cuh", "vsa_prompt_fwd_kernel.cuh",
                                  "vsa_prompt_bwd_kernel.cuh", "vsa_pages_kernel.cuh"])
def test_no_read_only_loads_in_kernels_that_start_early(name):
    """They start up while their predecessor ends: what it may have written is read by ordinary
    loads behind the wait for it."""
    with open(os.path.join(libbuild.CSRC, name)) as f:
        code = re.sub(r"//.*", "", f.read())
    for word in ("__ldg", "__restrict__", "ld.global.nc", ".nc."):
        assert word not in code, word
    for body in code.split("__global__")[1:]:
        wait = min(x for x in (body.find("after_predecessor();"), body.find("wait_predecessor();"))
                   if x >= 0)
        assert "read_global" not in body[:wait] and "load_seq" not in body[:wait]


# ------------------------------------------------------------------- the plain forms' pins
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk", [(5, 5), (3, 9), (9, 4)])
def test_plain_attention_is_that_of_autograd(nq, nk, causal):
    g = torch.Generator().manual_seed(nq * 10 + nk)
    q, k, v, do = (torch.randn(n, D, generator=g, dtype=torch.float64) for n in (nq, nk, nk, nq))
    r, b = ref.head(q, k, v, causal, 0.3, do)
    for t in (q, k, v):
        t.requires_grad_()
    first = max(0, nq - nk) if causal else 0  # rows before it attend nothing
    z = torch.stack([torch.cat([(q[i] * k[j]).sum().view(1) * 0.3 for j in range(nk)])
                     for i in range(nq)])
    for i in range(nq):
        for j in range(nk):
            if causal and j > i + nk - nq:
                z = z.masked_fill(((torch.arange(nq) == i)[:, None] & (torch.arange(nk) == j)),
                                  -math.inf)
    out = torch.softmax(z[first:], -1) @ v
    (out * do[first:]).sum().backward()
    assert torch.allclose(r["out"][first:], out) and (r["out"][:first] == 0).all()
    assert torch.allclose(r["lse"][first:], torch.logsumexp(z[first:], -1) / math.log(2))
    assert (r["lse"][:first] == ref.LSE_EMPTY).all()
    for n, t in (("dq", q), ("dk", k), ("dv", v)):
        assert torch.allclose(r[n], t.grad)
    assert all((x >= 0).all() for x in b.values())


def test_plain_pages():
    refs = [1, 0, 2, 0, 1]
    assert ref.bits(refs) == [0b01010]
    table = [[[2, 0, -1]], [[2, 4, 9]]]
    assert ref.reserve(refs, table, [130, 100], [1, 29], 64) == [0, 0]  # block 2; blocks 1, 2
    assert table == [[[2, 0, 1]], [[2, 4, 3]]] and refs == [1, 1, 2, 1, 1]
    assert ref.reserve(refs, table, [192, 0], [1, 0], 64) == [0, 0]     # past the table; nothing
    table[0][0][1] = -1
    assert ref.reserve(refs, table, [64, 0], [1, 0], 64) == [1, 0]      # no page left
    refs, table = [1, 0, 2, 0, 1], [[[2, 0, -1]], [[2, 4, -1]]]
    out, n, lacking, copies = ref.fork(refs, table, [100, 128], [0, 0, 1, 7], 64, 3)
    assert out == [[[2, 1, -1]], [[2, 3, -1]], [[2, 4, -1]], [[-1, -1, -1]]]
    assert n == [100, 100, 128, 0] and lacking == [0, 0, 0, 0]
    assert copies == [(0, 1, 36), (0, 3, 36)] and refs == [1, 1, 5, 1, 2]
    ref.free(refs, out, None, 64)
    assert refs == [1, 0, 2, 0, 1] and out[2] == [[-1, -1, -1]]
    to, used = ref.compact(refs, table)
    assert to == [0, -1, 2, -1, 1] and used == 3 and refs == [1, 1, 2, 0, 0]
    assert table == [[[2, 0, -1]], [[2, 1, -1]]]

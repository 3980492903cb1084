"""Host-side argument checks of the operators around the attention: bad calls get the
documented status before the GPU is touched (no GPU needed), and the plain 64-bit forms the
GPU tests compare with are pinned to hand-made values."""
import ctypes
import math

import pytest
import torch

import serve_ref as ref
from block_sparse_attention_vsa_gb300 import binding
from block_sparse_attention_vsa_gb300 import build as libbuild

OK, INVALID, UNSUPPORTED = (binding.VSA_OK, binding.VSA_ERR_INVALID_ARG,
                            binding.VSA_ERR_UNSUPPORTED)
P = ctypes.c_void_p
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return binding.load()


def p(v):
    return P(v) if v else None


def mean(lib, **kw):
    a = dict(x=16 * MB, sizes=1 * MB, B=1, H=2, S=200, D=128, block=64, mean=64 * MB)
    a.update(kw)
    return lib.vsa_block_mean(p(a["x"]), p(a["sizes"]), a["B"], a["H"], a["S"], a["D"], a["block"],
                              p(a["mean"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=64), UNSUPPORTED), (dict(block=32), UNSUPPORTED), (dict(B=-1), INVALID),
    (dict(x=0), INVALID), (dict(mean=0), INVALID), (dict(x=16 * MB + 8), INVALID),
    (dict(mean=64 * MB + 2), INVALID), (dict(mean=16 * MB + 1024), INVALID),
    (dict(mean=1 * MB), INVALID), (dict(sizes=1 * MB + 2), INVALID), (dict(S=0), OK),
    (dict(B=0, x=0), OK), (dict(B=1 << 20, H=1 << 20), UNSUPPORTED),
    (dict(B=1 << 15, H=1 << 10, S=64 * 64), UNSUPPORTED),
])
def test_block_mean_checks(lib, kw, code):
    assert mean(lib, **kw) == code


def select(lib, **kw):
    a = dict(q=16 * MB, k=32 * MB, sizes=1 * MB, B=1, Hq=4, Hkv=2, nq=10, nk=20, D=128, topk=3,
             causal=0, n_first=0, n_near=0, idx=64 * MB, num=96 * MB)
    a.update(kw)
    return lib.vsa_select_blocks(p(a["q"]), p(a["k"]), p(a["sizes"]), a["B"], a["Hq"], a["Hkv"],
                                 a["nq"], a["nk"], a["D"], a["topk"], a["causal"], a["n_first"],
                                 a["n_near"], p(a["idx"]), p(a["num"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=64), UNSUPPORTED), (dict(nk=2049), UNSUPPORTED), (dict(topk=0), INVALID),
    (dict(n_first=-1), INVALID), (dict(n_near=-1), INVALID), (dict(Hkv=3), INVALID),
    (dict(Hkv=0), INVALID), (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(idx=0), INVALID),
    (dict(num=0), INVALID), (dict(q=16 * MB + 4), INVALID), (dict(idx=64 * MB + 1), INVALID),
    (dict(num=64 * MB), INVALID), (dict(idx=32 * MB), INVALID), (dict(nq=0), OK), (dict(B=0), OK),
    (dict(topk=1 << 25), UNSUPPORTED),
])
def test_select_blocks_checks(lib, kw, code):
    assert select(lib, **kw) == code


def cselect(lib, **kw):
    a = dict(q=16 * MB, m=32 * MB, table=1 * MB, lens=2 * MB, B=2, Hq=4, Hkv=2, D=128, pages=9,
             mb=7, block=64, topk=3, n_first=0, n_near=1, idx=64 * MB, num=96 * MB)
    a.update(kw)
    return lib.vsa_cache_select(p(a["q"]), p(a["m"]), p(a["table"]), p(a["lens"]), a["B"], a["Hq"],
                                a["Hkv"], a["D"], a["pages"], a["mb"], a["block"], a["topk"],
                                a["n_first"], a["n_near"], p(a["idx"]), p(a["num"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), UNSUPPORTED), (dict(block=16), UNSUPPORTED), (dict(mb=2049), UNSUPPORTED),
    (dict(topk=0), INVALID), (dict(Hq=5), INVALID), (dict(Hq=0), INVALID), (dict(pages=-1), INVALID),
    (dict(lens=0), INVALID), (dict(table=0), INVALID), (dict(m=0), INVALID),
    (dict(idx=32 * MB), INVALID), (dict(lens=2 * MB + 2), INVALID), (dict(B=0), OK),
])
def test_cache_select_checks(lib, kw, code):
    assert cselect(lib, **kw) == code


def write(lib, **kw):
    a = dict(k=16 * MB, v=32 * MB, table=1 * MB, lens=2 * MB, n=3 * MB, B=2, Hkv=2, T=5, D=128,
             pages=9, mb=7, block=64, kc=64 * MB, vc=96 * MB, ks=4 * MB, vs=5 * MB, km=6 * MB)
    a.update(kw)
    return lib.vsa_cache_write(p(a["k"]), p(a["v"]), p(a["table"]), p(a["lens"]), p(a["n"]), a["B"],
                               a["Hkv"], a["T"], a["D"], a["pages"], a["mb"], a["block"],
                               p(a["kc"]), p(a["vc"]), p(a["ks"]), p(a["vs"]), p(a["km"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=64), UNSUPPORTED), (dict(block=100), UNSUPPORTED), (dict(mb=4000), UNSUPPORTED),
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(lens=0), INVALID), (dict(ks=0), INVALID),
    (dict(k=16 * MB + 2), INVALID), (dict(kc=64 * MB + 8), INVALID), (dict(ks=4 * MB + 1), INVALID),
    (dict(vc=64 * MB), INVALID), (dict(kc=16 * MB), INVALID), (dict(km=64 * MB), INVALID),
    (dict(vs=1 * MB), INVALID), (dict(T=0), OK), (dict(B=0), OK), (dict(pages=0), OK),
])
def test_cache_write_checks(lib, kw, code):
    assert write(lib, **kw) == code


def fwd(lib, **kw):
    a = dict(q=16 * MB, kc=64 * MB, vc=96 * MB, ks=4 * MB, vs=5 * MB, table=1 * MB, lens=2 * MB,
             idx=0, num=0, ms=0, B=2, Hq=4, Hkv=2, D=128, pages=9, mb=7, block=64, scale=0.1,
             keep=1.0, out=32 * MB, lse=7 * MB, w=0, ws=128 * MB, n=MB * 64)
    a.update(kw)
    return lib.vsa_fwd_cache(p(a["q"]), p(a["kc"]), p(a["vc"]), p(a["ks"]), p(a["vs"]),
                             p(a["table"]), p(a["lens"]), p(a["idx"]), p(a["num"]), a["ms"],
                             a["B"], a["Hq"], a["Hkv"], a["D"], a["pages"], a["mb"], a["block"],
                             a["scale"], a["keep"], p(a["out"]), p(a["lse"]), p(a["w"]),
                             p(a["ws"]), a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=64), UNSUPPORTED), (dict(block=32), UNSUPPORTED), (dict(mb=2049), UNSUPPORTED),
    (dict(Hq=5), INVALID), (dict(Hkv=0), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=math.inf), INVALID), (dict(w=8 * MB, keep=math.nan), INVALID),
    (dict(idx=9 * MB), INVALID), (dict(idx=9 * MB, num=10 * MB, ms=0), INVALID),
    (dict(ws=0), INVALID), (dict(n=1000), INVALID), (dict(ws=128 * MB + 4), INVALID),
    (dict(q=0), INVALID), (dict(kc=0), INVALID), (dict(table=0), INVALID), (dict(out=0), INVALID),
    (dict(out=16 * MB), INVALID), (dict(lse=32 * MB), INVALID), (dict(w=1 * MB), INVALID),
    (dict(ws=64 * MB), INVALID), (dict(out=32 * MB + 8), INVALID), (dict(lse=7 * MB + 2), INVALID),
    (dict(B=5000, Hq=64, Hkv=8, n=1 << 40, ws=1 << 50), UNSUPPORTED),
    (dict(B=0), OK), (dict(Hq=0), OK),
])
def test_fwd_cache_checks(lib, kw, code):
    assert fwd(lib, **kw) == code


def test_cache_workspace_bytes(lib):
    n = lib.vsa_cache_workspace_bytes(2, 4, 2, 7, 0)
    assert n > 256 * 1024
    # the log-sum-exps, and a weight and maximum per block and head of a chunk
    assert lib.vsa_cache_workspace_bytes(2, 4, 2, 7, 1) == n + 256 + 2 * 2 * 7 * 8 * 8
    assert lib.vsa_cache_workspace_bytes(2, 5, 2, 7, 0) == 0
    assert lib.vsa_cache_workspace_bytes(2, 4, 2, 2049, 0) == 0
    assert lib.vsa_cache_workspace_bytes(-1, 4, 2, 7, 0) == 0


def evict(lib, **kw):
    a = dict(w=16 * MB, table=1 * MB, lens=2 * MB, B=2, Hkv=2, mb=7, block=64, budget=3, nf=1, nl=1,
             to=3 * MB, wo=4 * MB, lo=5 * MB, f=6 * MB, nfr=7 * MB)
    a.update(kw)
    return lib.vsa_cache_evict(p(a["w"]), p(a["table"]), p(a["lens"]), a["B"], a["Hkv"], a["mb"],
                               a["block"], a["budget"], a["nf"], a["nl"], p(a["to"]), p(a["wo"]),
                               p(a["lo"]), p(a["f"]), p(a["nfr"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(block=63), UNSUPPORTED), (dict(mb=2049), UNSUPPORTED), (dict(budget=0), INVALID),
    (dict(nl=0), INVALID), (dict(nf=-1), INVALID), (dict(nf=3), INVALID),
    (dict(nf=2 ** 31 - 1), INVALID), (dict(w=0), INVALID), (dict(lo=0), INVALID),
    (dict(to=1 * MB), INVALID), (dict(wo=16 * MB), INVALID), (dict(lo=2 * MB), INVALID),
    (dict(f=3 * MB), INVALID), (dict(f=6 * MB + 1), INVALID), (dict(B=0), OK),
])
def test_cache_evict_checks(lib, kw, code):
    assert evict(lib, **kw) == code


# ------------------------------------------------------------------ the plain forms' pins
@pytest.mark.parametrize("big", [2**31, 2**32 + 64, -2**31 - 1, 1.5])
def test_arguments_beyond_32_bits(lib, big):
    """The binding refuses what a 32-bit argument would wrap round."""
    x, t = torch.zeros(1, 1, 1, 128, dtype=torch.bfloat16), torch.zeros(1, 1, 1, dtype=torch.int32)
    calls = [(binding.vsa_block_mean, (x,), {"block": big})]
    calls += [(binding.vsa_select_blocks, (x, x), {"topk": 1, name: big})
              for name in ("topk", "n_first", "n_near")]
    calls += [(binding.vsa_cache_select, (x, x[0, 0], t, t[0, 0]), {"topk": 1, name: big})
              for name in ("topk", "block", "n_first", "n_near")]
    calls += [(binding.vsa_cache_evict, (t.float(), t, t[0, 0]), {"budget": 1, name: big})
              for name in ("budget", "block", "n_first", "n_last")]
    calls += [(binding.cache_workspace_bytes, tuple(big if i == at else 1 for i in range(4)), {})
              for at in range(4)]
    for call, args, names in calls:
        with pytest.raises(ValueError, match="32-bit"):
            call(*args, **names)


def test_plain_e4m3_values():
    x = torch.tensor([0.0, 1.0, 17.0, 18.0, 19.0, 447.0, 500.0, math.inf, -math.inf, 2.0 ** -9,
                      2.0 ** -10, 3 * 2.0 ** -10, 1.0625, 1.1875, -0.3])
    want = [0.0, 1.0, 16.0, 18.0, 20.0, 448.0, 448.0, 448.0, -448.0, 2.0 ** -9, 0.0, 2.0 ** -8,
            1.0, 1.25, -0.3125]
    assert ref.e4m3(x).tolist() == want
    # every code is its own nearest value
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    fine = codes[~codes.isnan()]
    assert torch.equal(ref.e4m3(fine), fine)


def test_plain_choice():
    nan = math.nan
    got = ref.choose([1.0, 5.0, nan, 5.0, 5.0, -1.0], lambda j: j != 1, lambda j: j == 5, 3)
    assert got == [3, 4, 5]
    assert ref.choose([nan, nan], lambda j: True, lambda j: j == 1, 2) == [1]


def test_plain_attention_of_equal_keys():
    """Equal scores: out is the mean of the values, lse = log2 n + s log2 e, and each block's
    weight its share of the tokens."""
    state = {"k": torch.ones(3, 64, 128).double(), "v": torch.randn(3, 64, 128).double(),
             "k_scale": torch.ones(3).double(), "v_scale": torch.full((3,), 2.0).double()}
    q = torch.full((1, 1, 1, 128), 0.5)
    table = torch.tensor([[[2, 0]]], dtype=torch.int32)
    r = ref.attend(q, state, table, torch.tensor([80]), 64)
    mean = (state["v"][2].sum(0) + state["v"][0, :16].sum(0)) * 2.0 / 80
    assert torch.allclose(r["out"][0, 0, 0], mean, rtol=1e-12, atol=1e-12)
    s = 64.0 / math.sqrt(128)
    assert abs(r["lse"].item() - (math.log2(80) + s * math.log2(math.e))) < 1e-9
    assert torch.allclose(r["weight"][0, 0], torch.tensor([0.8, 0.2]).double())

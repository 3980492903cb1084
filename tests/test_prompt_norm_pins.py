"""On the CPU: wrong gradients that the limit in norm has to reject, and right ones, rounded as the
kernels round, that it has to let pass."""
import math

import pytest
import torch

import prompt_ref as ref
from prompt_norm import NORM, off

D = 128
SHAPES = [(300, 300, True), (300, 300, False), (70, 700, False), (40, 41, True), (2, 2, False)]


def inputs(nq, nk):
    g = torch.Generator().manual_seed(nq + nk)
    return [torch.randn(n, D, generator=g).bfloat16().double() for n in (nq, nk, nk, nq)]


def weights(q, k, causal):
    z = q @ k.T / math.sqrt(D)
    if causal:
        z = z.masked_fill(torch.ones_like(z, dtype=torch.bool).triu(k.shape[0] - q.shape[0] + 1),
                          -math.inf)
    return torch.softmax(z, 1)


def rounded(x):
    return x.bfloat16().double()


def grads(q, k, v, dout, causal, bad=None):
    """From the formula, rounded where the kernels round, or with a mistake planted."""
    p = weights(q, k, causal)
    out = rounded(rounded(p) @ v)
    dp, d = dout @ v.T, (dout * out).sum(1, keepdim=True)
    d = {"no D": 0 * d, "D x 1.1": 1.1 * d, "D x 0.9": 0.9 * d, "D of the next row": d.roll(1, 0),
         "-D": -d}.get(bad, d)
    ds = p * (dp - d)
    if bad is None or bad == "less D's rounding":
        ds = ds - p * ds.sum(1, keepdim=True) if bad else ds
        ds, p = rounded(ds), rounded(p)
    scale = 1.0 / math.sqrt(D)
    r = {"out": out, "dq": scale * ds @ k, "dk": scale * ds.T @ q, "dv": p.T @ dout}
    if bad in ("x 1.05", "x 0.95", "x -1", "x 0"):
        r = {n: float(bad[2:]) * x for n, x in r.items()}
    return {n: rounded(x) for n, x in r.items()}


@pytest.mark.parametrize("nq,nk,causal", SHAPES)
@pytest.mark.parametrize("how", [None, "less D's rounding"])
def test_rounded_gradients_pass(nq, nk, causal, how):
    x = inputs(nq, nk)
    want, _ = ref.head(*x[:3], causal, 1.0 / math.sqrt(D), x[3])
    for n, got in grads(*x, causal, how).items():
        assert off(got, want[n]) <= NORM, n


@pytest.mark.parametrize("nq,nk,causal", SHAPES)
@pytest.mark.parametrize("bad", ["x 1.05", "x 0.95", "x -1", "x 0"])
def test_scaled_gradients_fail(nq, nk, causal, bad):
    x = inputs(nq, nk)
    want, _ = ref.head(*x[:3], causal, 1.0 / math.sqrt(D), x[3])
    for n, got in grads(*x, causal, bad).items():
        assert off(got, want[n]) > NORM, n


@pytest.mark.parametrize("nq,nk,causal", SHAPES)
@pytest.mark.parametrize("bad", ["no D", "-D", "D of the next row"])
def test_gradients_without_their_D_fail(nq, nk, causal, bad):
    x = inputs(nq, nk)
    want, _ = ref.head(*x[:3], causal, 1.0 / math.sqrt(D), x[3])
    got = grads(*x, causal, bad)
    assert off(got["dq"], want["dq"]) > NORM and off(got["dk"], want["dk"]) > NORM


@pytest.mark.parametrize("nq,nk,causal", [s for s in SHAPES if s[2] or s[1] < 300])
@pytest.mark.parametrize("bad", ["D x 1.1", "D x 0.9"])
def test_gradients_of_a_D_off_by_a_tenth_fail(nq, nk, causal, bad):
    """(Where many keys count alike D is small beside dP, and a tenth of it is lost in roundings.)"""
    x = inputs(nq, nk)
    want, _ = ref.head(*x[:3], causal, 1.0 / math.sqrt(D), x[3])
    got = grads(*x, causal, bad)
    assert off(got["dq"], want["dq"]) > NORM and off(got["dk"], want["dk"]) > NORM

"""The order in which the gradient's warps touch a tile in shared memory, on the CPU: who waits
for whom is written down as it stands in the kernels (each wait with the piece of source that it
is), and whatever follows from it has to put every product behind the copy and the zeroing of the
tiles that it reads, and every copy behind the last product that reads what it overwrites.  Tiles
in time by luck are not enough: a copy may land as late as it likes."""
import os
import re

import pytest

from block_sparse_attention_vsa_gb300 import build as libbuild


def source():
    with open(os.path.join(libbuild.CSRC, "vsa_prompt_bwd_kernel.cuh")) as f:
        code = re.sub(r"//.*", "", f.read())
    code = re.sub(r"\s+", " ", code)
    at = code.index("namespace dq {")
    return {"dkv": code[:at], "dq": code[at:]}


# Every entry: the wait (or arrival) and the source that it is.  What the source does not hold is
# not there in the model either.
DKV = {
    "mma q": "x ? g_in(0) : q_in(0)",
    "mma next": "(!more || (x ? g_in(g + 1) : q_in(g + 1)))",
    "mma own dO": "(x || g_in(g))",
    "mma weights": "wait_warp(ready, g & 1, w, 0x2d)",
    "mma turn": "((x == 0 && g == 0) || wait_warp(&ctl->turn[x], (x ? g : g - 1) & 1, w, 0x32))",
    "grad copy": "!wait_warp(&ctl->g_full[st], (g >> 1) & 1, w, 0x20)",
    "grad s": "!wait_warp(&ctl->s_full, g & 1, w, 0x21)",
    "grad dp": "!wait_warp(&ctl->dp_full, g & 1, w, 0x22)",
    "clean q": "if (!wait_warp(&ctl->q_full[qs], (g / kQStages) & 1, w, 0x30)) break; "
               "if (clean) zero_tokens(smem + kOffQ + qs * kTile, from, to, T); "
               "if (lane == 0) mbar_arrive(&ctl->q_ready[qs]);",
    "clean g": "if (!wait_warp(&ctl->g_full[gs], (g / kGStages) & 1, w, 0x31)) break; "
               "if (clean) zero_tokens(smem + kOffG + gs * kTile, from, to, T); "
               "if (lane == 0) mbar_arrive(&ctl->g_ready[gs]);",
    "load q": "!wait(&ctl->q_empty[qs], (g / kQStages + 1) & 1, w, 0x24)",
    "load g": "!wait(&ctl->g_empty[gs], (g / kGStages + 1) & 1, w, 0x25)",
    "empty by commit": "warp_mma_commit(x ? &ctl->q_empty[st] : &ctl->g_empty[st]);",
    "empty by grad": "mbar_arrive(&ctl->ds_full); mbar_arrive(&ctl->g_empty[st]);",
}
DQ = {
    "mma k": "wait_warp(&ctl->k_ready[ks], (g / kKStages) & 1, w, 0x49)",
    "mma v": "wait_warp(&ctl->v_full[vs], (g / kVStages) & 1, w, 0x4b)",
    "mma ds": "!wait_warp(&ctl->ds_full[g & 1], (g >> 1) & 1, w, 0x4d)",
    "grad s": "!wait_warp(&ctl->s_full, g & 1, w, 0x40)",
    "clean k": "if (!wait_warp(&ctl->k_full[ks], (g / kKStages) & 1, w, 0x4f)) break; "
               "if (nk - 128 * g < 128) zero_rows(smem + kOffK + ks * kTile, nk - 128 * g); "
               "if (lane == 0) mbar_arrive(&ctl->k_ready[ks]);",
    "load k": "!wait(&ctl->k_empty[ks], (g / kKStages + 1) & 1, w, 0x43)",
    "load v": "!wait(&ctl->v_empty[vs], (g / kVStages + 1) & 1, w, 0x44)",
    "empty": "warp_mma_commit(&ctl->ds_empty[g & 1]); warp_mma_commit(&ctl->k_empty[ks]);",
}


class Order:
    """Events of threads, each thread's in a row, and what waits add."""

    def __init__(self):
        self.after = {}  # event -> those it comes directly behind

    def thread(self, events):
        for a, b in zip([None] + events, events):
            self.after.setdefault(b, set())
            if a is not None:
                self.after[b].add(a)

    def behind(self, event, *others):
        self.after[event].update(o for o in others if o in self.after)

    def follows(self, event, other):
        seen, todo = set(), [event]
        while todo:
            for e in self.after[todo.pop()]:
                if e == other:
                    return True
                if e not in seen:
                    seen.add(e)
                    todo.append(e)
        return False


def dkv(n, has):
    """A CTA of n steps."""
    o = Order()
    steps = range(n)
    # a copy in flight lands when it likes: its issue and its landing are different threads
    o.thread([("issue", t, g) for g in steps for t in "QG"])
    for g in steps:
        for t in "QG":
            o.thread([("landed", t, g)])
            o.behind(("landed", t, g), ("issue", t, g))
    o.thread([e for g in steps for e in (("clean", "Q", g), ("clean", "G", g))])
    for x, (score, grad) in enumerate((("S", "dV"), ("dP", "dK"))):
        o.thread([("wait", x, -1), (score, 0)] + [
            e for g in steps for e in (("wait", x, g), (grad, g)) +
            (((score, g + 1),) if g + 1 < n else ()) + (("turn", x, g),)])
    o.thread([e for g in steps for e in (("s read", g), ("P", g), ("dp read", g), ("dS", g))])
    for g in steps:
        # warp 11, the copies, the gradient warps
        if "clean q" in has:
            o.behind(("clean", "Q", g), ("landed", "Q", g))
        if "clean g" in has:
            o.behind(("clean", "G", g), ("landed", "G", g))
        if "load q" in has and "empty by commit" in has:
            o.behind(("issue", "Q", g), ("dK", g - 3))
        if "load g" in has and "empty by commit" in has:
            o.behind(("issue", "G", g), ("dV", g - 2))
        if "load g" in has and "empty by grad" in has:
            o.behind(("issue", "G", g), ("dS", g - 2))
        if "grad copy" in has:
            o.behind(("s read", g), ("landed", "G", g))
        if "grad s" in has:
            o.behind(("s read", g), ("S", g))
        if "grad dp" in has:
            o.behind(("dp read", g), ("dP", g))
        # the issuers
        for x, tile in enumerate("QG"):
            if "mma next" in has:
                o.behind(("wait", x, g), ("clean", tile, g + 1))
            if "mma weights" in has:
                o.behind(("wait", x, g), ("dS" if x else "P", g))
            if "mma turn" in has:
                o.behind(("wait", x, g), ("turn", 1 - x, g if x else g - 1))
        if "mma own dO" in has:
            o.behind(("wait", 0, g), ("clean", "G", g))
    if "mma q" in has:
        o.behind(("wait", 0, -1), ("clean", "Q", 0))
        o.behind(("wait", 1, -1), ("clean", "G", 0))
    wrong = [(p, g) for g in steps for p, *needs in (
        ("S", ("clean", "Q", g)), ("dP", ("clean", "G", g)), ("P", ("S", g)), ("dS", ("dP", g)),
        ("dV", ("P", g), ("clean", "G", g)), ("dK", ("dS", g), ("clean", "Q", g)))
        if not all(o.follows((p, g), e) for e in needs)]
    wrong += [("clean", t, g) for g in steps for t in "QG"
              if not o.follows(("clean", t, g), ("landed", t, g))]
    for g in steps:  # what a copy overwrites has been read
        for t, ring, by in (("Q", 3, ("S", "dK")), ("G", 2, ("dP", "dV", "dS"))):
            wrong += [("copy", t, g) for p in by if g >= ring
                      and not o.follows(("issue", t, g), (p, g - ring))]
    return wrong


def dq(n, has):
    o = Order()
    steps = range(n)
    o.thread([("issue", t, g) for g in steps for t in "KV"])
    for g in steps:
        for t in "KV":
            o.thread([("landed", t, g)])
            o.behind(("landed", t, g), ("issue", t, g))
    o.thread([("clean", g) for g in steps])
    o.thread([e for g in steps for e in (("S", g), ("dP", g))])
    o.thread([("dQ", g) for g in steps])
    o.thread([("dS", g) for g in steps])
    for g in steps:
        for event, key, other in (
                (("clean", g), "clean k", ("landed", "K", g)), (("S", g), "mma k", ("clean", g)),
                (("dP", g), "mma v", ("landed", "V", g)), (("dQ", g), "mma ds", ("dS", g)),
                (("dS", g), "grad s", ("S", g))):
            if key in has:
                o.behind(event, other)
        if "load k" in has and "empty" in has:
            o.behind(("issue", "K", g), ("dQ", g - 3))
        if "load v" in has:
            o.behind(("issue", "V", g), ("dP", g - 2))
    wrong = [(p, g) for g in steps for p, e in (
        ("clean", ("landed", "K", g)), ("S", ("clean", g)), ("dS", ("S", g)), ("dQ", ("dS", g)),
        ("dQ", ("clean", g)), ("dP", ("landed", "V", g))) if not o.follows((p, g), e)]
    for g in steps:
        for t, ring, by in (("K", 3, ("S", "dQ")), ("V", 2, ("dP",))):
            wrong += [("copy", t, g) for p in by if g >= ring
                      and not o.follows(("issue", t, g), (p, g - ring))]
    return wrong


def held(kernel, table):
    code = source()[kernel]
    return {name for name, text in table.items() if text in code}


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 6, 9])
def test_products_come_behind_what_they_read(n):
    assert dkv(n, held("dkv", DKV)) == []
    assert dq(n, held("dq", DQ)) == []


def test_the_model_sees_what_is_missing():
    """Each wait left out leaves something unordered, but for those that others imply."""
    whole = set(DKV)
    assert dkv(1, whole - {"mma own dO"}) == [("dV", 0)]   # a single step has no later Q to wait for
    for n in (2, 3, 6):
        assert dkv(n, whole - {"mma own dO"}) == []
    implied = {"mma own dO", "mma turn", "grad copy"}
    for name in whole - implied:
        assert dkv(6, whole - {name}), name
    for name in DQ:
        assert dq(6, set(DQ) - {name}), name

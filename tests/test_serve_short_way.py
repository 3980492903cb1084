"""The short way from torch tensors (the extension built beside the library) only saves host
time: without it every entry point still loads and serves."""
import io
import os
import subprocess
import sys

import pytest
import torch

from block_sparse_attention_vsa_gb300 import binding
from block_sparse_attention_vsa_gb300 import build as libbuild

DEV = "cuda:0"

HIDDEN = """
import warnings
import torch
from block_sparse_attention_vsa_gb300 import binding, build
build.torch_lib = lambda version: "/nowhere/_vsa_torch.so"
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    assert binding.load() is binding.load()
    assert binding.workspace_bytes() > 0
assert [w.category for w in said] == [RuntimeWarning], said
for call in (lambda: binding.vsa_block_mean(torch.zeros(1, 1, 64, 128)),
             lambda: binding.vsa_block_mean(torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16),
                                            block=2**32)):
    try:
        call()
    except (TypeError, ValueError):
        continue
    raise AssertionError("not refused")
print("served")
"""


def test_everything_loads_without_the_short_way():
    libbuild.build()
    got = subprocess.run([sys.executable, "-c", HIDDEN], cwd=libbuild.ROOT, capture_output=True,
                         text=True, env=dict(os.environ, PYTHONPATH=libbuild.ROOT))
    assert got.returncode == 0 and "served" in got.stdout, got.stdout + got.stderr


@pytest.mark.gpu
def test_calls_without_the_short_way(monkeypatch):
    libbuild.build()
    g = torch.Generator().manual_seed(5)

    def bf16(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV)

    x, q = bf16(1, 2, 500, 128), bf16(1, 4, 1, 128)
    k, v = bf16(1, 2, 300, 128), bf16(1, 2, 300, 128)
    table = torch.arange(12, dtype=torch.int32, device=DEV).view(1, 2, 6)
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = none + 300
    ws = binding.new_cache_workspace(1, 4, 2, 6, True, DEV)

    def calls():
        m = binding.vsa_block_mean(x)
        cache = binding.new_cache8(12, 64, DEV)
        binding.vsa_cache_write(cache, k, v, table, none)
        idx, num = binding.vsa_cache_select(q, cache.k_mean, table, lens, 3)
        weight = torch.zeros(table.shape, device=DEV)
        out = binding.vsa_fwd_cache(q, cache, table, lens, idx=idx, num=num, weight=weight,
                                    workspace=ws)
        return (m, *binding.vsa_select_blocks(m, m, 3), idx, num, *out, weight,
                *(t.view(torch.uint8) for t in cache),
                *binding.vsa_cache_evict(weight, table, lens, 3))

    binding.load()
    short = calls()
    monkeypatch.setattr(binding, "_fast", False)
    for a, b in zip(calls(), short):
        assert a.dtype == b.dtype and torch.equal(a, b)


@pytest.mark.gpu
def test_evicted_tensors_stand_alone():
    """What an eviction returns can be saved together, and what is kept does not hold
    the memory of the rest."""
    libbuild.build()
    g = torch.Generator().manual_seed(6)
    weight = torch.rand((2, 3, 10), generator=g).to(DEV)
    table = torch.arange(60, dtype=torch.int32, device=DEV).view(2, 3, 10)
    lens = torch.tensor([640, 100], dtype=torch.int32, device=DEV)
    for stream in (None, torch.cuda.current_stream()):  # the short way, the long way
        got = binding.vsa_cache_evict(weight, table, lens, 4, stream=stream)
        kept = io.BytesIO()
        torch.save(got._asdict(), kept)
        kept.seek(0)
        for name, t in torch.load(kept).items():
            assert torch.equal(t, getattr(got, name))
        # at most one number a sequence more
        for t in (got.table, got.weight, got.freed):
            assert t.untyped_storage().nbytes() <= t.numel() * t.element_size() + 2 * 4
        apart = {t.untyped_storage().data_ptr() for t in (got.table, got.weight, got.freed)}
        assert len(apart) == 3
        assert got.lens.untyped_storage().data_ptr() != got.freed.untyped_storage().data_ptr()

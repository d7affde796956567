"""The sliding-window attention with sinks without a GPU: what its entry points
refuse (every check precedes the first CUDA call), the workspace queries, and
the oracle pinned to the windowed decode's and to sums written out."""

import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle
from relative_bias_gqa_b200 import build as build_mod
from relative_bias_gqa_b200 import workloads as W

OK = 1 << 20                                      # an aligned address that is never read


@pytest.fixture(scope="module")
def ra():
    build_mod.build()
    from relative_bias_gqa_b200 import rel_attn
    return rel_attn


def invoke(ra, *, e4m3=False, prefill=False, window=128, sinks=4, splits=0, nbytes=1 << 40, shape=None, **kw):
    base = dict(batch=2, q_tokens=1, num_q_heads=12, num_kv_heads=2, num_pages=50, max_pages_per_seq=10, num_buckets=1280)
    base.update(shape or {})
    s = ra.make_shape(**base)
    a = dict(q=OK, k=OK, v=OK, ks=OK, vs=OK, table=OK, lens=OK, rel=OK, out=OK, lse=OK, ws=OK)
    a.update(kw)
    fn = getattr(ra.lib, f"rel_attn_sink_{'prefill' if prefill else 'decode'}{'_e4m3' if e4m3 else ''}")
    return fn(ctypes.byref(s), a["q"], a["k"], a["v"], *([a["ks"], a["vs"]] if e4m3 else []), a["table"], a["lens"], a["rel"],
              window, sinks, *([] if prefill else [splits]), a["out"], a["lse"], a["ws"], nbytes, None)


ENTRIES = [(e, p) for e in (False, True) for p in (False, True)]


@pytest.mark.parametrize("e4m3,prefill", ENTRIES)
def test_bad_arguments_are_refused(ra, e4m3, prefill):
    bad = lambda **kw: invoke(ra, e4m3=e4m3, prefill=prefill, **kw) == ra.REL_ATTN_ERR_INVALID_ARG  # noqa: E731
    assert bad(window=0) and bad(window=-5) and bad(sinks=-1)
    for name in ("q", "k", "v", "table", "lens", "rel", "out", "ws") + (("ks", "vs") if e4m3 else ()):
        assert bad(**{name: None}), name
    for name, to in (("q", 8), ("k", 8), ("v", 4), ("rel", 2), ("out", 8), ("ws", 128), ("table", 2), ("lens", 1), ("lse", 2)):
        assert bad(**{name: OK + to}), name
    if e4m3:
        assert bad(ks=OK + 2) and bad(vs=OK + 1)
    for kw in (dict(batch=0), dict(batch=65536), dict(q_tokens=0), dict(num_q_heads=13), dict(num_q_heads=10), dict(head_dim=64),
               dict(page_size=32), dict(num_pages=0), dict(max_pages_per_seq=0), dict(max_pages_per_seq=1 << 25),
               dict(num_pages=1 << 24), dict(num_buckets=0), dict(exact_buckets=0), dict(max_seq_len=-1),
               dict(q_tokens=(1 << 20) + 1 if prefill else 10)):
        assert bad(shape=kw), kw
    if not prefill:
        assert bad(splits=257) and bad(shape=dict(q_tokens=9, num_q_heads=16))
    assert invoke(ra, e4m3=e4m3, prefill=prefill, nbytes=255) == ra.REL_ATTN_ERR_WORKSPACE_TOO_SMALL


def test_null_shape_is_refused(ra):
    assert ra.lib.rel_attn_sink_decode(None, OK, OK, OK, OK, OK, OK, 5, 0, 0, OK, OK, OK, 1 << 30, None) == ra.REL_ATTN_ERR_INVALID_ARG
    assert ra.lib.rel_attn_sink_workspace_bytes(None, 5, 0, 0) == 0
    assert ra.lib.rel_attn_sink_prefill_workspace_bytes(None, 5, 0) == 0


def test_workspace_queries(ra):
    one = ctypes.byref(ra.make_shape(batch=2, q_tokens=1, num_q_heads=12, num_kv_heads=2, num_pages=50, max_pages_per_seq=1000, num_buckets=1280))
    four = ctypes.byref(ra.make_shape(batch=2, q_tokens=4, num_q_heads=12, num_kv_heads=2, num_pages=50, max_pages_per_seq=1000, num_buckets=1280))
    need = ra.lib.rel_attn_sink_workspace_bytes
    assert need(one, 0, 4, 0) == need(one, 5, -1, 0) == need(one, 5, 0, 257) == 0
    assert need(one, 500, 4, 1) == need(one, 500, 4, 8) == need(four, 500, 4, 1) == 256
    rows = 2 * 12
    assert need(one, 500, 4, 9) >= 256 + 9 * rows * (4 + 512)
    assert need(four, 500, 4, 2) >= 256 + 2 * 4 * rows * (4 + 512)
    assert need(one, 500, 4, 0) >= 256 and ra.lib.rel_attn_sink_prefill_workspace_bytes(four, 500, 4) >= 256


def test_tensors_are_checked(ra):
    q = torch.zeros(1, 1, 6, 128, dtype=torch.bfloat16)
    kv = torch.zeros(3, 1, 64, 128, dtype=torch.bfloat16)
    table, lens, rel = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):               # not on a GPU
        ra.rel_attn_sink_decode(q, kv, kv, table, lens, rel, 5)
    for kw in (dict(window=2 ** 32 + 5), dict(window=5, num_sinks=2 ** 31), dict(window=5, num_splits=-2 ** 31 - 1)):
        with pytest.raises(ValueError, match="32 bits"):
            ra.SinkPrepared(q, kv, kv, table, lens, rel, **kw)
    with pytest.raises(ValueError):               # one scale of two
        ra.SinkPrepared(q, kv, kv, table, lens, rel, 5, k_scale=torch.ones(1))
    with pytest.raises(ValueError):
        ra.rel_attn_sink_prefill(q[0], kv, kv, table, lens, rel, 5)


def test_head_dims_that_differ_are_refused(ra):
    """A cache of another head dim than the queries' would be read past its end:
    refused where every call makes its shape."""
    q = torch.zeros(1, 1, 6, 128, dtype=torch.bfloat16)
    table, kv, rel = (torch.zeros(*s) for s in ((1, 2), (3, 1, 64, 128), (1, 8, 128)))
    assert ra.shape_of(q, kv, table, rel).head_dim == 128
    with pytest.raises(ValueError, match="head dims"):
        ra.shape_of(q, kv[..., :64], table, rel)
    with pytest.raises(ValueError, match="head dims"):
        ra.shape_of(q, kv, table, rel[..., :64])


def test_memory_that_kernels_cannot_write_is_refused(ra):
    from relative_bias_gqa_b200.rel_attn import _check_written
    cuda, here = torch.device("cuda", 0), torch.zeros(4)
    for host in (False, True):
        with pytest.raises(ValueError, match="out is on cpu"):
            _check_written("out", here, cuda, host=host)
        with pytest.raises(ValueError, match="out is on meta"):
            _check_written("out", here.to("meta"), cuda, host=host)


# ------------------------------------------------------------------ oracle
def case(lens, T, **kw):
    return W.make_case(seq_lens=lens, q_tokens=T, num_q_heads=4, num_kv_heads=1, rel_std=0.5, **kw)


def run(c, window, sinks):
    return oracle.rel_attn_sink_ref(c.q, c.k_cache, c.v_cache, c.block_table, c.seq_lens, c.rel_table, window, sinks,
                                    exact_buckets=c.exact_buckets, max_distance=c.max_distance)


@pytest.mark.parametrize("lens,T,window", [([200, 70], 1, 64), ([150], 5, 1), ([300], 3, 500)])
def test_oracle_without_sinks_is_the_windowed_decode(lens, T, window):
    c = case(lens, T, num_buckets=40, exact_buckets=16, max_distance=400, seed=1)
    a = run(c, window, 0)
    b = oracle.rel_attn_decode_ref(c.q, c.k_cache, c.v_cache, c.block_table, c.seq_lens, c.rel_table, window,
                                   exact_buckets=c.exact_buckets, max_distance=c.max_distance)
    assert np.abs(a[0] - b[0]).max() < 1e-12 and np.abs(a[1] - b[1]).max() < 1e-12


def test_oracle_with_sinks_everywhere_is_the_full_context():
    c = case([200, 70], 2, num_buckets=40, exact_buckets=16, max_distance=400, seed=2)
    a = run(c, 3, 1000)
    b = oracle.rel_attn_decode_ref(c.q, c.k_cache, c.v_cache, c.block_table, c.seq_lens, c.rel_table, 0,
                                   exact_buckets=c.exact_buckets, max_distance=c.max_distance)
    assert np.abs(a[0] - b[0]).max() < 1e-12 and np.abs(a[1] - b[1]).max() < 1e-12


def test_oracle_is_the_formula_written_out():
    c = case([9, 0], 2, num_buckets=6, exact_buckets=3, max_distance=9, seed=3)
    c.seq_lens[1] = 0
    out, lse = run(c, 3, 2)
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all()
    bucket = lambda d: int(oracle.bucket_of_distance(np.array([d]), 6, 3, 9)[0])  # noqa: E731
    for t, sees in ((0, (0, 1, 5, 6, 7)), (1, (0, 1, 6, 7, 8))):
        p, page = 7 + t, int(c.block_table[0, 0])
        for h in range(4):
            q = c.q[0, t, h].double().numpy()
            w = [math.exp((q @ c.k_cache[page, 0, j].double().numpy() + q @ c.rel_table[0, bucket(p - j)].double().numpy()) / math.sqrt(128))
                 for j in sees]
            o = sum(x * c.v_cache[page, 0, j].double().numpy() for x, j in zip(w, sees)) / sum(w)
            assert np.abs(out[0, t, h] - o).max() < 1e-12 and abs(lse[0, t, h] - math.log(sum(w))) < 1e-12


THREADS = r"""
#include <atomic>
#include <chrono>
#include <thread>
#include <vector>
#include "rel_attn.h"
// 32 threads, a dense bucket table each: its steps go to the tiles, whose two
// splits need room, whatever tables the other threads ask for meanwhile.
int main() {
  std::vector<std::thread> threads;
  std::atomic<int> wrong{0};
  const auto end = std::chrono::steady_clock::now() + std::chrono::seconds(5);
  for (int i = 0; i < 32; ++i)
    threads.emplace_back([&, i] {
      const rel_attn_shape dense = {2, 1, 12, 2, 128, 64, 50, 1000, 90 + i, 1, 60, 0, 0};
      while (std::chrono::steady_clock::now() < end)
        wrong += rel_attn_sink_workspace_bytes(&dense, 500, 4, 2) <= 256;
    });
  for (auto& t : threads) t.join();
  return wrong != 0;
}
"""


def test_bucket_spans_while_other_threads_use_other_tables(ra, tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("needs g++")
    (tmp_path / "threads.cc").write_text(THREADS)
    exe, where = tmp_path / "threads", os.path.dirname(build_mod.LIB_PATH)
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", build_mod.INCLUDE, str(tmp_path / "threads.cc"), "-o", str(exe), "-L", where,
                    "-lrel_attn", f"-Wl,-rpath,{where}", "-lpthread"], check=True)
    assert subprocess.run([str(exe)]).returncode == 0

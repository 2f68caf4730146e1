"""Window and shared-prefix decode past the sizes of their kernels' tables: more tasks than a CTA
has threads, more pieces on one worker than the ring of bad-page marks holds, rows on either side
of a tile's edge.  Against the fp64 oracle; tolerances: test_gpu_window."""
import numpy as np
import pytest
import torch

import mla_latent_kv_22_b200 as M
from test_gpu_shared import Shared
from test_gpu_window import KNOBS, assert_rounded, ref, run, window_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def knobs():
    yield
    for k in KNOBS:
        M.mla_set_knob(k, 0)


def but(res, skip, n):
    keep = [b for b in range(n) if b not in skip]
    return [r[keep] for r in res], keep


def spoilt(out, lse, rows):
    return all(torch.isnan(out[b]).all() and torch.isnan(lse[b]).all() for b in rows)


# 384 threads: the schedule takes the tasks in passes above that.  With more workers than tasks
# each runs whole.
@pytest.mark.parametrize("B", [384, 385, 1000])
@pytest.mark.parametrize("tile,workers,policy", [(16, 0, 0), (32, 0, 1), (128, 0, 0), (16, 1024, 2), (128, 7, 0)])
def test_windows_of_more_sequences_than_threads(B, tile, workers, policy):
    lens = [int(x) for x in np.random.default_rng(B).integers(0, 260, B)]
    lens[0], lens[B - 1] = 0, 259
    M.mla_set_knob("row_tile", tile)
    M.mla_set_knob("num_workers", workers)
    M.mla_set_knob("split_policy", policy)
    c, q = window_case(lens, 1, 2, 130, 4, seed=910)
    good = ref(c, q, 130, 4)
    out, lse, err = run(c, q, 130, 4)
    assert err == 0
    assert_rounded(out, lse, good)
    bad = (5, B // 2, B - 1)
    for b, T in zip(bad, (-1, 64 * c.block_table.shape[1] + 1, 1 << 30)):
        c.cache_seqlens[b] = T
    out, lse, err = run(c, q, 130, 4)
    assert err == 5 and spoilt(out, lse, bad)
    want, keep = but(good, bad, B)
    assert_rounded(out[keep], lse[keep], want)


@pytest.mark.parametrize("B,H,tile,workers,policy", [
    (400, 16, 16, 0, 0),        # 400 tiles of one sequence each
    (430, 15, 16, 0, 1),        # 404 tiles that cross sequences
    (800, 16, 32, 0, 0),
    (385, 128, 128, 0, 0),
    (400, 16, 16, 512, 2),
    (700, 2, 128, 0, 0),        # few tiles of many sequences
])
def test_shared_prefix_of_more_tiles_than_threads(B, H, tile, workers, policy):
    lens = [int(x) for x in np.random.default_rng(B).integers(0, 140, B)]
    M.mla_set_knob("row_tile", tile)
    M.mla_set_knob("num_workers", workers)
    M.mla_set_knob("split_policy", policy)
    c = Shared(100, lens, 1, H, seed=911)
    good = c.ref()
    out, lse, err = c.run()
    assert err == 0
    assert_rounded(out, lse, good)
    bad = (0, B // 2, B - 1)
    for b, T in zip(bad, (-1, 64 * c.table.shape[1] + 1, 1 << 30)):
        c.lens[b] = T
    out, lse, err = c.run()
    assert err == 5 and spoilt(out, lse, bad)
    want, keep = but(good, bad, B)
    assert_rounded(out[keep], lse[keep], want)
    c.P = -1
    out, lse, err = c.run()
    assert err == 5 and spoilt(out, lse, range(B))


# The marks are a ring of 16 pieces: a mark that outlived its piece would spoil a sequence 16 or
# 32 further on.
@pytest.mark.parametrize("tile,H", [(16, 16), (32, 32), (128, 128), (128, 100)])
def test_marks_of_bad_pages_end_with_their_piece(tile, H):
    B, bad = 52, (0, 3, 15, 37)
    rng = np.random.default_rng(H)
    lens = [int(x) for x in rng.integers(1, 200, B)]
    for b in bad:
        lens[b] = 130
    M.mla_set_knob("row_tile", tile)
    M.mla_set_knob("num_workers", 1)
    d, q = window_case(lens, 1, H, 100, 3, seed=920)
    good = ref(d, q, 100, 3)
    for b in bad:
        d.block_table[b, 1] = -7 if b % 2 else d.kv_cache.shape[0]
    out, lse, err = run(d, q, 100, 3)
    assert err == 5 and spoilt(out, lse, bad)
    want, keep = but(good, bad, B)
    assert_rounded(out[keep], lse[keep], want)
    c = Shared(70, lens, 1, H, seed=921)
    good = c.ref()
    for b in bad:
        c.table[b, 2] = -7 if b % 2 else c.kv.shape[0]
    out, lse, err = c.run()
    assert err == 5 and spoilt(out, lse, bad)
    want, keep = but(good, bad, B)
    assert_rounded(out[keep], lse[keep], want)


@pytest.mark.parametrize("tile", [0, 16, 32, 128])
@pytest.mark.parametrize("s_q,H", [(1, 15), (1, 31), (11, 3), (1, 127), (3, 43), (2, 65), (2, 127), (3, 86)])
def test_rows_beside_a_tiles_edge(tile, s_q, H):
    # 15, 31, 33, 127, 129, 130, 254 and 258 rows a sequence
    M.mla_set_knob("row_tile", tile)
    c, q = window_case([700, 90, 5, 0], s_q, H, 64, 1, seed=930 + H)
    out, lse, err = run(c, q, 64, 1)
    assert err == 0
    assert_rounded(out, lse, ref(c, q, 64, 1))
    d = Shared(200, [130, 1, 0], s_q, H, seed=931 + H)
    out, lse, err = d.run()
    assert err == 0
    assert_rounded(out, lse, d.ref())


@pytest.mark.parametrize("tile", [0, 16, 32, 128])
def test_the_most_rows_of_a_sequence(tile):
    M.mla_set_knob("row_tile", tile)
    c, q = window_case([150, 7], 16, 128, 60, 2, seed=940)   # 2,048 rows
    out, lse, err = run(c, q, 60, 2)
    assert err == 0
    assert_rounded(out, lse, ref(c, q, 60, 2))
    d = Shared(70, [3, 90], 16, 128, seed=941)
    out, lse, err = d.run()
    assert err == 0
    assert_rounded(out, lse, d.ref())


FIRST = """
import torch
import mla_latent_kv_22_b200 as M
bf, i32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.int32, device="cuda")
B, H = 2, 16
x = lambda *s: torch.randn(*s, device="cuda").bfloat16()
kv, table, lens, cos_sin = x(8, 64, 576), torch.arange(8, **i32).view(2, 4), torch.tensor([200, 70], **i32), torch.randn(300, 64, device="cuda")
new, q, w = x(B, 576), x(B, H, 576), x(H, 512, 128)
ptab, plen = torch.tensor([1, 2], **i32), torch.tensor([100], **i32)

def step():
    M.mla_append(new[:, :512], new[:, 512:], kv, table, lens, cos_sin)
    r = [torch.empty(B, H, 512, **bf), torch.empty(B, H, device="cuda"), torch.empty(B, H, 512, **bf), torch.empty(B, H, device="cuda"),
         torch.empty(B, H, 128, device="cuda")]
    M.mla_decode_window(q, kv, table, lens, r[0], r[1], 0.07, 90, 4)
    M.mla_decode_shared(q, kv, ptab, plen, table, lens, r[2], r[3], 0.07)
    M.mla_absorb_o(r[0], w, r[4])
    return r

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    held = step()
g.replay()
want = step()
torch.cuda.synchronize()
assert M.mla_get_device_error() == 0
assert all(torch.equal(a, b) for a, b in zip(held, want)) and all(torch.isfinite(a).all() for a in want)
z = lambda *s, **k: torch.empty(*s, **k)
M.mla_decode_window(z(0, H, 576, **bf), kv, z(0, 4, **i32), z(0, **i32), z(0, H, 512, **bf), z(0, H, device="cuda"), 0.07, 90)   # no sequence
M.mla_decode_shared(z(0, H, 576, **bf), kv, ptab, plen, z(0, 4, **i32), z(0, **i32), z(0, H, 512, **bf), z(0, H, device="cuda"), 0.07)
M.mla_absorb_o(z(0, H, 512, **bf), w, z(0, H, 128, device="cuda"))
M.mla_append(z(0, 512, **bf), z(0, 64, **bf), kv, z(0, 4, **i32), z(0, **i32), cos_sin)
assert M.mla_get_device_error() == 0
del g
print("same")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["same"], r.stderr[-2000:]

"""A wait that runs out makes the outputs that depend on it NaN, as every device error does.
A test hook withholds one load of one worker, so that its waits end at their limit."""
import pytest
import torch

import mla_latent_kv_22_b200 as M
from gpu_helpers import bf16_dev
from test_gpu_shared import Shared
from test_gpu_window import assert_rounded, ref, window_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def knobs():
    M.mla_set_knob("wait_limit", 100)
    yield
    for k in ("wait_limit", "withhold_arrive", "piece_cost", "row_tile", "num_workers", "split_policy"):
        M.mla_set_knob(k, 0)


def check(call, want):
    """`call` fills outputs that held zeros; the withheld one leaves no row that is neither right nor NaN."""
    M.mla_set_knob("withhold_arrive", 1)
    out, lse, err = call()
    M.mla_set_knob("withhold_arrive", 0)
    assert err == 6
    spoilt = torch.isnan(lse)
    assert spoilt.any() and torch.equal(spoilt, torch.isnan(out).any(-1)) and torch.equal(spoilt, torch.isnan(out).all(-1))
    keep = ~spoilt
    k = keep.cpu().numpy()
    if keep.any():
        assert_rounded(out[keep], lse[keep], [w[k] for w in want])
    out, lse, err = call()
    assert err == 0
    assert_rounded(out, lse, want)


@pytest.mark.parametrize("tile", [16, 32, 128])
@pytest.mark.parametrize("policy", [1, 2])   # pieces merged by the second grid; rows written where they are made
def test_window_rows_of_a_worker_that_gave_up_are_nan(tile, policy):
    M.mla_set_knob("row_tile", tile)
    M.mla_set_knob("split_policy", policy)
    M.mla_set_knob("piece_cost", 1)
    c, q = window_case([900, 300, 0, 2000], 2, 20, 700, 4, seed=900)
    check(lambda: window(c, q, 700, 4), ref(c, q, 700, 4))


def window(c, q, w, sinks):
    out = torch.zeros(q.shape[:3] + (512,), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(q.shape[:3], device="cuda")
    M.mla_decode_window(bf16_dev(q), bf16_dev(c.kv_cache), torch.from_numpy(c.block_table).cuda(),
                        torch.from_numpy(c.cache_seqlens).cuda(), out, lse, c.softmax_scale, w, sinks)
    return out, lse, M.mla_get_device_error()


def shared(d):
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    out = torch.zeros(d.q.shape[:3] + (512,), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(d.q.shape[:3], device="cuda")
    M.mla_decode_shared(bf16_dev(d.q), bf16_dev(d.kv), i32(d.ptab), i32([d.P]), i32(d.table), i32(d.lens), out, lse, d.scale)
    return out, lse, M.mla_get_device_error()


def test_rows_of_a_short_call_that_gave_up_are_nan():
    c, q = window_case([900, 300], 1, 16, 500, 4, seed=901)   # clusters that merge their own pieces
    check(lambda: window(c, q, 500, 4), ref(c, q, 500, 4))


@pytest.mark.parametrize("tile", [16, 32, 128])
@pytest.mark.parametrize("policy", [1, 2])
def test_shared_rows_of_a_worker_that_gave_up_are_nan(tile, policy):
    M.mla_set_knob("row_tile", tile)
    M.mla_set_knob("split_policy", policy)
    M.mla_set_knob("piece_cost", 1)
    d = Shared(900, [30, 70, 0, 5, 64] * 3, 1, 20, seed=902)
    check(lambda: shared(d), d.ref())

"""GPU parity of mla_decode_window against the fp64 oracle.

Tolerances, from the roundings the kernel makes.  Half a bf16 step is 2^-8 relative: the
output is rounded once (2^-8 |out|) and each softmax weight once, which moves an output
by at most 2^-8 sum_t p_t |v_t| =: 2^-8 A.  A score is a sum of 576 products in fp32,
off by at most 577 x 2^-23 |scale| sum |q k| =: d (2^-23: the accumulation may truncate);
the scaling and the exponential's argument add 4 roundings of the score, which the same
sum bounds.  d moves the lse by at most d and every weight by a factor e^(2d).
The fp32 sums that remain are below 2^-16 of A, and 2^-16 covers the exponentials.
"""
import numpy as np
import pytest
import torch

import mla_latent_kv_22_b200 as M
import mla_synth as S
import oracle as O
from gpu_helpers import bf16_dev

pytestmark = pytest.mark.gpu

KNOBS = ("num_workers", "min_pages", "split_policy", "piece_cost", "wait_limit", "withhold_arrive", "row_tile")


@pytest.fixture(autouse=True, params=[0, 16, 32, 128], ids=["auto", "tile16", "tile32", "tile128"])
def _knobs(request):
    M.mla_set_knob("row_tile", request.param)
    yield
    for k in KNOBS:
        M.mla_set_knob(k, 0)


def assert_rounded(out, lse, ref, what=""):
    ro, rl, mag, smax = ref
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert o.shape == ro.shape and l.shape == rl.shape, what
    fin = np.isfinite(rl)
    assert np.array_equal(l[~fin], rl[~fin]) and (o[~fin] == 0).all(), f"{what}: empty rows"
    d = 581 * 2.0 ** -23 * smax
    off = np.abs(l[fin] - rl[fin]) - (d[fin] + 2.0 ** -16 * (1 + np.abs(rl[fin])))
    assert (off <= 0).all(), f"{what}: lse off by {off.max():.2e} more than allowed"
    tol = 2.0 ** -8 * np.abs(ro) + mag * (2.0 ** -8 + 2.0 ** -16 + 2.1 * d[..., None])
    off = np.abs(o - ro) - tol * (1 + 2.0 ** -7)
    assert (off <= 0).all(), f"{what}: {(off > 0).sum()} outputs off by up to {off.max():.2e} more than allowed"


def window_case(lens, s_q, H, window, sinks, seed, paged=True, **kw):
    """A case whose rows that no query sees are NaN and whose unneeded table entries are no page."""
    c = S.make_decode_case(len(lens), s_q * H, lens, seed=seed, poison=True, paged=paged, **kw)
    for b, T in enumerate(lens):
        lo = max(0, T - s_q - window + 1)
        for t in range(min(sinks, T), lo):
            if paged:
                c.kv_cache[c.block_table[b, t // 64], t % 64] = S.BF16_NAN
            else:
                c.kv_cache[b, t] = S.BF16_NAN
        if paged:
            for p in range(c.block_table.shape[1]):
                seen = [t for t in range(64 * p, min(64 * p + 64, T)) if t < sinks or t >= lo]
                if not seen:
                    c.block_table[b, p] = -1 if p % 2 else 1 << 30
    return c, c.q.reshape(len(lens), s_q, H, -1)


def run(c, q, window, sinks, scale=None, **kw):
    dq, kv = bf16_dev(q), bf16_dev(c.kv_cache)
    bt = None if c.block_table is None else torch.from_numpy(c.block_table).cuda()
    sl = torch.from_numpy(c.cache_seqlens).cuda()
    out = torch.full(q.shape[:3] + (512,), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    M.mla_decode_window(dq, kv, bt, sl, out, lse, c.softmax_scale if scale is None else scale, window, sinks, **kw)
    return out, lse, M.mla_get_device_error()


def ref(c, q, window, sinks, scale=None):
    return O.mla_decode_window_ref(q, c.kv_cache, c.block_table, c.cache_seqlens,
                                   c.softmax_scale if scale is None else scale, window, sinks)


@pytest.mark.parametrize("lens,s_q,H,window,sinks", [
    ([1], 1, 1, 1, 0),                        # one token, one head
    ([0, 1, 2, 63, 64, 65], 1, 16, 64, 4),    # empty and page-edge lengths
    ([300, 1000, 127], 1, 16, 100, 4),        # sink page, window and last page all ragged
    ([300, 1000, 70], 1, 17, 1, 0),           # a window of the token itself
    ([400, 200], 1, 5, 128, 130),             # sinks over two pages
    ([130, 129, 128], 1, 16, 10, 100),        # window inside the sinks' page, hole within one page
    ([700, 90], 1, 32, 200, 0),               # 32 rows
    ([700, 90, 5], 1, 33, 64, 1),             # 33 rows: the 64-row tile with dead rows
    ([700, 90, 0, 1], 1, 64, 300, 64),
    ([1030, 257], 1, 100, 257, 3),            # two row groups of 64, one ragged
    ([1030, 257, 3], 1, 128, 300, 5),
    ([5, 500, 1, 64], 2, 8, 70, 4),           # several queries, T < s_q
    ([3, 300], 4, 20, 65, 10),                # 80 rows over two groups, queries split across them
    ([200, 1000], 3, 128, 129, 0),            # six groups
    ([66, 400], 7, 1, 1, 2),                  # windows of one token, seven queries
])
def test_window_matches_oracle(lens, s_q, H, window, sinks):
    c, q = window_case(lens, s_q, H, window, sinks, seed=500 + H)
    out, lse, err = run(c, q, window, sinks)
    assert err == 0
    assert_rounded(out, lse, ref(c, q, window, sinks))


@pytest.mark.parametrize("H", [16, 32, 64, 128])
@pytest.mark.parametrize("workers", [1, 3, 40, 148])
def test_forced_splits(H, workers):
    M.mla_set_knob("num_workers", workers)
    M.mla_set_knob("min_pages", 1)
    c, q = window_case([2000, 0, 65, 900], 1, H, 777, 70, seed=520)
    out, lse, err = run(c, q, 777, 70)
    assert err == 0
    assert_rounded(out, lse, ref(c, q, 777, 70), f"{workers} workers")


@pytest.mark.parametrize("policy,cost", [(1, 0), (2, 0), (0, 1), (0, 30)])
def test_schedule_policies(policy, cost):
    M.mla_set_knob("split_policy", policy)
    M.mla_set_knob("piece_cost", cost)
    c, q = window_case([1500] * 5 + [3], 1, 24, 1200, 4, seed=521)
    out, lse, err = run(c, q, 1200, 4)
    assert err == 0
    assert_rounded(out, lse, ref(c, q, 1200, 4))


def test_many_short_sequences_and_more_sequences_than_workers():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 400, 331)]
    c, q = window_case(lens, 1, 3, 130, 4, seed=522)
    out, lse, err = run(c, q, 130, 4)
    assert err == 0
    assert_rounded(out, lse, ref(c, q, 130, 4))


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_scales(scale):
    # Scale 1 gives scores of standard deviation 24: one token takes nearly all the weight
    # and the reference maximum moves along the sequence.
    c, q = window_case([900, 64], 1, 16, 500, 4, seed=523)
    out, lse, err = run(c, q, 500, 4, scale=scale)
    assert err == 0
    assert_rounded(out, lse, ref(c, q, 500, 4, scale))


@pytest.mark.parametrize("H", [16, 64])
def test_growing_scores_move_the_reference_maximum(H):
    c, q = window_case([1000], 1, H, 1000, 0, seed=524)
    lat = S.bf16_bits_to_f32(c.kv_cache)
    for p, page in enumerate(c.block_table[0]):  # rope dims grow with the position
        if page >= 0:
            lat[page, :, 512:] *= (1 + p) * 0.5
    c.kv_cache[:] = S.f32_to_bf16_bits(lat)
    tail = 1000 % 64
    c.kv_cache[c.block_table[0, -1], tail:] = S.BF16_NAN
    out, lse, err = run(c, q, 1000, 0)
    assert err == 0
    assert_rounded(out, lse, ref(c, q, 1000, 0))


def test_a_window_beyond_the_sequence_is_the_causal_decode():
    c, q = window_case([700, 65], 2, 16, 10 ** 9, 0, seed=525)
    out, lse, err = run(c, q, (1 << 31) - 1, 0)
    assert err == 0
    assert_rounded(out, lse, ref(c, q, 10 ** 9, 0))
    for big in (2 ** 32 + 1, 2 ** 63 - 1, np.int64(2 ** 40)):  # integers of more than 32 bits
        o2, l2, err = run(c, q, big, 0)
        assert err == 0 and torch.equal(o2, out) and torch.equal(l2, lse)
    for bad in (-2 ** 32 + 5, -2 ** 40):
        with pytest.raises(M.MlaError):
            run(c, q, bad, 0)


@pytest.mark.parametrize("H", [16, 128])
def test_paged_equals_contiguous_and_runs_repeat(H):
    lens = [200, 3, 1000, 640]
    a, qa = window_case(lens, 1, H, 300, 4, seed=526)
    b, qb = window_case(lens, 1, H, 300, 4, seed=526, paged=False)
    oa, la, ea = run(a, qa, 300, 4)
    ob, lb, eb = run(b, qb, 300, 4)
    oc, lc, _ = run(a, qa, 300, 4)
    assert ea == 0 and eb == 0
    assert torch.equal(oa, ob) and torch.equal(la, lb)
    assert torch.equal(oa, oc) and torch.equal(la, lc)


def test_a_bad_page_or_length_spoils_its_sequence_alone():
    lens = [700, 300, 500]
    c, q = window_case(lens, 1, 16, 200, 4, seed=527)
    good = ref(c, q, 200, 4)
    c.block_table[1, 4] = c.kv_cache.shape[0]   # in sequence 1's window
    out, lse, err = run(c, q, 200, 4)
    assert err == 5 and torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    sub = [0, 2]
    assert_rounded(out[sub], lse[sub], [g[sub] for g in good])
    c.block_table[1, 4] = 0
    c.cache_seqlens[1] = c.block_table.shape[1] * 64 + 1
    out, lse, err = run(c, q, 200, 4)
    assert err == 5 and torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert_rounded(out[sub], lse[sub], [g[sub] for g in good])


def test_a_withheld_load_times_out_and_the_context_survives():
    c, q = window_case([700, 300], 1, 16, 500, 4, seed=528)
    M.mla_set_knob("wait_limit", 200)
    M.mla_set_knob("withhold_arrive", 1)
    M.mla_set_knob("piece_cost", 1)  # no fixed cost: the first worker has pages
    _, _, err = run(c, q, 500, 4)
    assert err == 6
    M.mla_set_knob("withhold_arrive", 0)
    out, lse, err = run(c, q, 500, 4)
    assert err == 0
    assert_rounded(out, lse, ref(c, q, 500, 4))


def test_own_workspaces_on_two_streams_at_once():
    cases = [window_case([4000, 100], 1, 16, 3000, 4, seed=529), window_case([900, 2500], 1, 64, 2000, 0, seed=530)]
    args = [(3000, 4), (2000, 0)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    dev, outs = [], []
    for (c, q), _ in zip(cases, args):
        dev.append((bf16_dev(q), bf16_dev(c.kv_cache), torch.from_numpy(c.block_table).cuda(), torch.from_numpy(c.cache_seqlens).cuda()))
        n = M.mla_decode_window_workspace_size(*q.shape[:3])
        outs.append((torch.empty(q.shape[:3] + (512,), dtype=torch.bfloat16, device="cuda"), torch.empty(q.shape[:3], device="cuda"),
                     torch.full((n,), 255, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for (c, _), (w, s), d, (o, l, ws), st in zip(cases, args, dev, outs, streams):
            M.mla_decode_window(*d, o, l, c.softmax_scale, w, s, workspace=ws, stream=st)
    torch.cuda.synchronize()
    assert M.mla_get_device_error() == 0
    for (c, q), (w, s), (o, l, _) in zip(cases, args, outs):
        assert_rounded(o, l, ref(c, q, w, s))


def test_two_captured_graphs_replay_on_new_inputs():
    # Each graph holds its own workspace (from the graph's pool); replayed in turn and
    # with eager calls in between.
    c, q = window_case([900, 64, 3000], 1, 16, 700, 4, seed=531)
    c2, q2 = window_case([900, 64, 3000], 1, 16, 700, 4, seed=532)
    dq, kv = bf16_dev(q), bf16_dev(c.kv_cache)
    bt, sl = torch.from_numpy(c.block_table).cuda(), torch.from_numpy(c.cache_seqlens).cuda()
    outs = [(torch.empty(3, 1, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 1, 16, device="cuda")) for _ in range(3)]
    call = lambda o, w: M.mla_decode_window(dq, kv, bt, sl, o[0], o[1], c.softmax_scale, w, 4)
    call(outs[2], 700)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g, o, w in zip(graphs, outs, (700, 100)):
        with torch.cuda.graph(g):
            call(o, w)
    dq.copy_(bf16_dev(q2))
    for _ in range(3):
        graphs[0].replay()
        call(outs[2], 300)
        graphs[1].replay()
    torch.cuda.synchronize()
    assert M.mla_get_device_error() == 0
    for o, w in zip(outs, (700, 100, 300)):
        assert_rounded(o[0], o[1], ref(c, q2, w, 4), f"window {w}")
    del graphs


def test_refusals():
    c, q = window_case([100], 1, 4, 10, 0, seed=533)
    for w, s in ((0, 0), (-1, 0), (10, -1)):
        with pytest.raises(M.MlaError) as ei:
            run(c, q, w, s)
        assert ei.value.name == "MLA_ERR_INVALID_ARG"
    with pytest.raises(M.MlaError) as ei:
        run(c, q, 10, 0, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert ei.value.name == "MLA_ERR_WORKSPACE"
    dq, kv = bf16_dev(q), bf16_dev(c.kv_cache)
    bt, sl = torch.from_numpy(c.block_table).cuda(), torch.from_numpy(c.cache_seqlens).cuda()
    with pytest.raises(TypeError):  # out is bf16
        M.mla_decode_window(dq, kv, bt, sl, torch.empty(1, 1, 4, 512, device="cuda"), torch.empty(1, 1, 4, device="cuda"), 0.1, 5)
    big = torch.zeros(1, 17, 128, 576, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(M.MlaError) as ei:
        M.mla_decode_window(big, kv, bt, sl, torch.empty(1, 17, 128, 512, dtype=torch.bfloat16, device="cuda"),
                            torch.empty(1, 17, 128, device="cuda"), 0.1, 5)
    assert ei.value.name in ("MLA_ERR_UNSUPPORTED", "MLA_ERR_WORKSPACE")

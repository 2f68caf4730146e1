"""Row tiles of the window and shared-prefix decode where they can go wrong: every tile width,
tiles that hold many sequences or a part of one, values that are not finite in tokens that
some rows of a tile do not see, bad pages among many pieces, waits that run out.  Against the
fp64 oracle; tolerances: test_gpu_window."""
import numpy as np
import pytest
import torch

import mla_latent_kv_22_b200 as M
import mla_synth as S
from test_gpu_shared import Shared
from test_gpu_window import _knobs, assert_rounded, ref, run, window_case  # noqa: F401

pytestmark = pytest.mark.gpu

NAN, INF = S.BF16_NAN, 0x7F80


def but(res, skip, n):
    keep = [b for b in range(n) if b not in skip]
    return [r[keep] for r in res], keep


# Rows per sequence and sequences: 16-, 32-, 64- and 128-row tiles; up to 128 sequences in a tile.
@pytest.mark.parametrize("B,H,P,most", [
    (16, 1, 70, 130), (40, 1, 200, 300), (64, 1, 1, 64), (150, 1, 129, 200), (43, 3, 65, 90), (9, 16, 2100, 600),
    (5, 96, 100, 200), (2, 65, 64, 64),
])
def test_shared_tiles_of_many_sequences(B, H, P, most):
    lens = [int(x) for x in np.random.default_rng(B + H).integers(0, most + 1, B)]
    c = Shared(P, lens, 1, H, seed=700 + B)
    out, lse, err = c.run()
    assert err == 0
    assert_rounded(out, lse, c.ref())


@pytest.mark.parametrize("workers", [1, 5, 74])
def test_shared_pieces_cut_anywhere(workers):
    M.mla_set_knob("num_workers", workers)
    M.mla_set_knob("min_pages", 1)
    M.mla_set_knob("piece_cost", 1)
    c = Shared(700, [300, 0, 1, 64, 65, 500, 7, 128, 90, 30], 1, 20, seed=720)
    out, lse, err = c.run()
    assert err == 0
    assert_rounded(out, lse, c.ref())


# Pieces of one step in front: the next one's loads find free slots before its turn.
@pytest.mark.parametrize("workers", [1, 3])
@pytest.mark.parametrize("lens", [[1] * 12, [128, 64, 1, 129, 300, 90], [257, 1, 700, 2, 2, 640], [0, 100, 0, 64, 500]])
def test_first_pieces_of_one_step(lens, workers):
    M.mla_set_knob("num_workers", workers)
    c, q = window_case(lens, 1, 128, 1024, 0, seed=760 + len(lens))
    want = ref(c, q, 1024, 0)
    for _ in range(20):
        out, lse, err = run(c, q, 1024, 0)
        assert err == 0
    assert_rounded(out, lse, want)


@pytest.mark.parametrize("shared", [False, True])
def test_growing_scores_rescale_a_pair(shared):
    # The rope dims grow along the tokens, so the reference maximum moves many times.
    if shared:
        c = Shared(900, [200, 130], 1, 128, seed=730)
        tables, at = [c.ptab[:15]] + [c.table[b, :-(-n // 64)] for b, n in enumerate(c.lens)], 0
        lat = S.bf16_bits_to_f32(c.kv)
        for i, tab in enumerate(tables):
            for p, page in enumerate(tab):
                lat[page, :, 512:] *= (1 + p + (15 if i else 0)) * 0.5
        c.kv[:] = S.f32_to_bf16_bits(lat)
        for tab, n in zip(tables, [900, 200, 130]):
            if n % 64:
                c.kv[tab[-1], n % 64:] = NAN
        out, lse, err = c.run()
        want = c.ref()
    else:
        c, q = window_case([1000], 1, 128, 1000, 0, seed=731)
        lat = S.bf16_bits_to_f32(c.kv_cache)
        for p, page in enumerate(c.block_table[0]):
            lat[page, :, 512:] *= (1 + p) * 0.5
        c.kv_cache[:] = S.f32_to_bf16_bits(lat)
        c.kv_cache[c.block_table[0, -1], 1000 % 64:] = NAN
        out, lse, err = run(c, q, 1000, 0)
        want = ref(c, q, 1000, 0)
    assert err == 0
    assert_rounded(out, lse, want)


@pytest.mark.parametrize("H", [4, 8, 16, 40, 128])
def test_a_sequence_with_nan_tokens_spoils_itself_alone(H):
    c = Shared(100, [70, 30, 200, 5], 1, H, seed=740)
    good = c.ref()
    c.kv[c.table[1, 0], 3, 7] = NAN
    c.kv[c.table[1, 0], 10, 100] = INF
    c.kv[c.table[3, 0], 4, 570] = NAN      # a rope dim of its last token
    out, lse, err = c.run()
    assert err == 0
    want, keep = but(good, (1, 3), 4)
    assert_rounded(out[keep], lse[keep], want)
    for b in (1, 3):
        assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()
    c.kv[c.table[1, 0], 3, 7] = c.kv[c.table[1, 0], 2, 7]
    c.kv[c.table[3, 0], 4, 570] = 0
    out, lse, _ = c.run()                  # an infinity alone: scores of either sign, the others as before
    want, keep = but(good, (1, 3), 4)
    assert_rounded(out[keep], lse[keep], want)
    c.q[2] = NAN                           # and a query that is not finite
    out, lse, _ = c.run()
    want, keep = but(good, (1, 2, 3), 4)
    assert_rounded(out[keep], lse[keep], want)
    assert torch.isnan(out[2]).all() and torch.isnan(lse[2]).all()


# Both queries in one tile (16, 32, 64 and 128 rows), tiles that hold a part of them, a tile each.
@pytest.mark.parametrize("H", [8, 16, 30, 64, 100, 128])
def test_a_token_a_query_does_not_see_may_be_nan(H):
    c, q = window_case([300, 64, 2], 2, H, 100, 4, seed=750)
    good = ref(c, q, 100, 4)
    for b, T in enumerate((300, 64, 2)):   # the last query's own token
        c.kv_cache[c.block_table[b, (T - 1) // 64], (T - 1) % 64] = NAN
    out, lse, err = run(c, q, 100, 4)
    assert err == 0
    assert_rounded(out[:, :1], lse[:, :1], [g[:, :1] for g in good])
    assert torch.isnan(out[:, 1]).all() and torch.isnan(lse[:, 1]).all()
    q[1, 0, 0] = NAN                       # one head's query: no other row's tokens are dropped for it
    out, lse, err = run(c, q, 100, 4)
    keep = [(b, h) for b in range(3) for h in range(H) if (b, h) != (1, 0)]
    bi, hi = [k[0] for k in keep], [k[1] for k in keep]
    assert_rounded(out[bi, 0, hi], lse[bi, 0, hi], [g[bi, 0, hi] for g in good])
    assert torch.isnan(out[1, 0, 0]).all()
    d = Shared(100, [70, 1, 0], 2, H, seed=751)
    good = d.ref()
    d.kv[d.table[0, 1], 5] = NAN
    d.kv[d.table[1, 0], 0] = NAN
    d.kv[d.ptab[1], 35] = NAN              # the prefix's last token is the last query's own where there is no other
    out, lse, err = d.run()
    assert err == 0
    assert_rounded(out[2:, :1], lse[2:, :1], [g[2:, :1] for g in good])   # the other two see all of the prefix
    assert torch.isnan(out[:2]).all() and torch.isnan(out[2, 1]).all()


@pytest.mark.parametrize("H", [2, 20, 128])
def test_bad_pages_spoil_their_rows_in_whichever_piece(H):
    # More pieces on the one worker than the marks' ring is deep.
    M.mla_set_knob("num_workers", 1)
    lens = [70, 1, 65, 130, 64, 200, 3, 90, 10, 128, 66, 5, 77, 64]
    c = Shared(130, lens, 1, H, seed=760)
    good = c.ref()
    bad = (0, 3, 12)
    c.table[0, 1], c.table[3, 0], c.table[12, 1] = -7, c.kv.shape[0], 1 << 30
    out, lse, err = c.run()
    assert err == 5
    want, keep = but(good, bad, len(lens))
    assert_rounded(out[keep], lse[keep], want)
    for b in bad:
        assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()
    d, q = window_case(lens, 1, H, 64, 3, seed=761)
    good = ref(d, q, 64, 3)
    d.block_table[3, 2] = -7
    d.block_table[12, 0] = d.kv_cache.shape[0]
    out, lse, err = run(d, q, 64, 3)
    assert err == 5
    want, keep = but(good, (3, 12), len(lens))
    assert_rounded(out[keep], lse[keep], want)
    for b in (3, 12):
        assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()


def test_bad_lengths_in_a_tile_of_many():
    c = Shared(100, [30] * 40, 1, 8, seed=770)
    good = c.ref()
    bad = (0, 17, 39)
    c.lens[0], c.lens[17], c.lens[39] = -1, 64 * c.table.shape[1] + 1, 1 << 30
    out, lse, err = c.run()
    assert err == 5
    want, keep = but(good, bad, 40)
    assert_rounded(out[keep], lse[keep], want)
    for b in bad:
        assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()


@pytest.mark.parametrize("H", [64, 128])
def test_withheld_loads_time_out_and_the_context_survives(H):
    c, q = window_case([900, 300], 1, H, 700, 4, seed=780)
    d = Shared(900, [30, 70], 1, H, seed=781)
    for call, want in ((lambda: run(c, q, 700, 4), lambda: ref(c, q, 700, 4)), (d.run, d.ref)):
        M.mla_set_knob("wait_limit", 200)
        M.mla_set_knob("withhold_arrive", 1)
        M.mla_set_knob("piece_cost", 1)  # no fixed cost: the first worker has pages
        assert call()[2] == 6
        M.mla_set_knob("withhold_arrive", 0)
        out, lse, err = call()
        assert err == 0
        assert_rounded(out, lse, want())


def test_pairs_on_two_streams_and_in_a_graph():
    cases = [window_case([4000, 100, 900], 1, 128, 3000, 4, seed=790), window_case([900, 2500], 1, 100, 2000, 0, seed=791)]
    args = [(3000, 4), (2000, 0)]
    calls, outs = [], []
    for (c, q), (w, s) in zip(cases, args):
        from gpu_helpers import bf16_dev
        dev = (bf16_dev(q), bf16_dev(c.kv_cache), torch.from_numpy(c.block_table).cuda(), torch.from_numpy(c.cache_seqlens).cuda())
        o, l = torch.empty(q.shape[:3] + (512,), dtype=torch.bfloat16, device="cuda"), torch.empty(q.shape[:3], device="cuda")
        outs.append((o, l))
        calls.append(lambda st=None, dev=dev, o=o, l=l, c=c, w=w, s=s: M.mla_decode_window(*dev, o, l, c.softmax_scale, w, s, stream=st))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for call, st in zip(calls, streams):
            call(st)
    torch.cuda.synchronize()
    eager = [(o.clone(), l.clone()) for o, l in outs]
    for (c, q), (w, s), (o, l) in zip(cases, args, outs):
        assert_rounded(o, l, ref(c, q, w, s))
        o.fill_(float("nan"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in calls:
            call()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert M.mla_get_device_error() == 0
    for (o, l), (eo, el) in zip(outs, eager):
        assert torch.equal(o, eo) and torch.equal(l, el)
    del g


# Short calls: clusters that merge their own pieces, up to as many as run at once and above.
@pytest.mark.parametrize("B", [1, 2, 6, 7, 8, 14, 16])
@pytest.mark.parametrize("H,s_q,window,sinks", [(16, 1, 60, 0), (16, 1, 400, 5), (9, 3, 700, 64), (64, 1, 500, 4)])
def test_short_windows(B, H, s_q, window, sinks):
    lens = [(900, 0, 1, 64, 65, 3000, 129, 450)[i % 8] for i in range(B)]
    c, q = window_case(lens, s_q, H, window, sinks, seed=800 + B)
    good = ref(c, q, window, sinks)
    out, lse, err = run(c, q, window, sinks)
    assert err == 0
    assert_rounded(out, lse, good)
    o2, l2, _ = run(c, q, window, sinks)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    c.block_table[0, 899 // 64] = c.kv_cache.shape[0]
    skip = (0,) if B < 4 else (0, 3)
    if B > 3:
        c.cache_seqlens[3] = -5
    out, lse, err = run(c, q, window, sinks)
    assert err == 5
    want, keep = but(good, skip, B)
    if keep:
        assert_rounded(out[keep], lse[keep], want)
    for b in skip:
        assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()


@pytest.mark.parametrize("B,H,P,most", [(1, 16, 400, 60), (7, 16, 700, 250), (14, 16, 130, 64), (16, 8, 300, 200), (9, 5, 200, 100)])
def test_short_shared_prefixes(B, H, P, most):
    lens = [int(x) for x in np.random.default_rng(B).integers(0, most + 1, B)]
    c = Shared(P, lens, 1, H, seed=820 + B)
    good = c.ref()
    out, lse, err = c.run()
    assert err == 0
    assert_rounded(out, lse, good)
    c.lens[B - 1] = 64 * c.table.shape[1] + 1
    out, lse, err = c.run()
    assert err == 5 and torch.isnan(out[B - 1]).all() and torch.isnan(lse[B - 1]).all()
    want, keep = but(good, (B - 1,), B)
    if keep:
        assert_rounded(out[keep], lse[keep], want)
    c.lens[B - 1], c.P = lens[B - 1], -1
    out, lse, err = c.run()
    assert err == 5 and torch.isnan(out).all() and torch.isnan(lse).all()


def test_a_short_call_times_out_and_the_context_survives():
    c, q = window_case([900, 300], 1, 16, 500, 4, seed=840)
    M.mla_set_knob("wait_limit", 200)
    M.mla_set_knob("withhold_arrive", 1)
    assert run(c, q, 500, 4)[2] == 6
    M.mla_set_knob("withhold_arrive", 0)
    out, lse, err = run(c, q, 500, 4)
    assert err == 0
    assert_rounded(out, lse, ref(c, q, 500, 4))


def test_short_calls_on_streams_and_replayed_with_other_lengths():
    # Three at a time, each with up to 14 clusters: more than run at once.
    from gpu_helpers import bf16_dev
    T = [900, 64, 3000, 5, 400, 1, 777, 300, 500, 128, 129, 640, 33, 1000]
    c, q = window_case(T, 1, 16, 10 ** 6, 0, seed=841)
    dq, kv, bt = bf16_dev(q), bf16_dev(c.kv_cache), torch.from_numpy(c.block_table).cuda()
    sl = torch.from_numpy(c.cache_seqlens).cuda()
    windows, streams = (100, 500, 640), [torch.cuda.Stream() for _ in range(3)]
    outs = [(torch.empty(14, 1, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(14, 1, 16, device="cuda")) for _ in windows]
    call = lambda i, st=None: M.mla_decode_window(dq, kv, bt, sl, *outs[i], c.softmax_scale, windows[i], 2, stream=st)
    torch.cuda.synchronize()
    for _ in range(30):
        for i, st in enumerate(streams):
            call(i, st)
    torch.cuda.synchronize()
    for w, o in zip(windows, outs):
        assert_rounded(*o, ref(c, q, w, 2), f"window {w}")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in (0, 1, 2, 1):
            call(i)
    c.cache_seqlens[:] = [max(0, t - 70 * (i % 3)) for i, t in enumerate(T)]
    sl.copy_(torch.from_numpy(c.cache_seqlens))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert M.mla_get_device_error() == 0
    for w, o in zip(windows, outs):
        assert_rounded(*o, ref(c, q, w, 2), f"window {w}, replayed")
    del g

"""Pins of the serving operators' oracle (CPU): identities with the decode oracle and
small brute forces written with the conditions spelt out."""
import math

import numpy as np
import pytest

import mla_synth as S
import oracle as O


def _case(lens, s_q, H, seed):
    c = S.make_decode_case(len(lens), s_q * H, lens, seed=seed, poison=True)
    return c, c.q.reshape(len(lens), s_q, H, -1)


def test_a_window_of_the_whole_sequence_is_the_causal_decode():
    c, q = _case([1, 70, 200], 2, 3, 11)
    want = O.mla_decode_multi_ref(q, c.kv_cache, c.block_table, c.cache_seqlens, c.softmax_scale)
    for window, sinks in ((200, 0), (10 ** 6, 7), (1, 200)):
        got = O.mla_decode_window_ref(q, c.kv_cache, c.block_table, c.cache_seqlens, c.softmax_scale, window, sinks)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_a_window_of_one_without_sinks_returns_the_token_itself():
    c, q = _case([5, 130], 2, 2, 12)
    out, lse, _, _ = O.mla_decode_window_ref(q, c.kv_cache, c.block_table, c.cache_seqlens, c.softmax_scale, 1)
    for b, T in enumerate((5, 130)):
        rows = O.gather_rows(c.kv_cache, c.block_table, b, T)
        for i in range(2):
            assert np.allclose(out[b, i], rows[T - 2 + i, :512], rtol=1e-13)
            assert np.allclose(lse[b, i], c.softmax_scale * O.bf16_to_f64(q[b, i]) @ rows[T - 2 + i], rtol=1e-13)


@pytest.mark.parametrize("window,sinks", [(3, 0), (4, 2), (64, 65), (100, 1)])
def test_window_against_a_loop(window, sinks):
    c, q = _case([6, 150], 3, 1, 13)
    out, lse, mag, _ = O.mla_decode_window_ref(q, c.kv_cache, c.block_table, c.cache_seqlens, c.softmax_scale, window, sinks)
    for b, T in enumerate((6, 150)):
        rows = O.gather_rows(c.kv_cache, c.block_table, b, T)
        for i in range(3):
            at, ws = T - 3 + i, {}
            for t in range(T):
                if t <= at and (t < sinks or at - t < window):
                    ws[t] = math.exp(c.softmax_scale * math.fsum(O.bf16_to_f64(q[b, i, 0]) * rows[t]))
            total = math.fsum(ws.values())
            assert abs(lse[b, i, 0] - math.log(total)) < 1e-12
            for j in (0, 7, 511):
                assert abs(out[b, i, 0, j] - math.fsum(w * rows[t, j] for t, w in ws.items()) / total) < 1e-12
                assert abs(mag[b, i, 0, j] - math.fsum(w * abs(rows[t, j]) for t, w in ws.items()) / total) < 1e-12


def test_shared_is_the_decode_of_the_joined_cache():
    rng = np.random.default_rng(5)
    P, own = 70, [0, 3, 64]
    flat = [S.f32_to_bf16_bits(rng.standard_normal((P + t, 576)).astype(np.float32)) for t in own]
    for f in flat[1:]:
        f[:P] = flat[0][:P]
    cache = np.full((6, 64, 576), S.BF16_NAN, dtype=np.uint16)
    cache[4], cache[1, :6] = flat[0][:64], flat[0][64:]
    table = np.array([[0], [5], [2]], dtype=np.int32)
    cache[5, :3], cache[2] = flat[1][P:], flat[2][P:]
    q = S.f32_to_bf16_bits(rng.standard_normal((3, 2, 2, 576)).astype(np.float32))
    out, lse, _, _ = O.mla_decode_shared_ref(q, cache, [4, 1], P, table, own, 0.07)
    for b in range(3):
        want = O.mla_decode_multi_ref(q[b:b + 1], flat[b][None], None, [P + own[b]], 0.07)
        assert np.allclose(out[b], want[0][0], rtol=1e-12, atol=1e-14) and np.allclose(lse[b], want[1][0], rtol=1e-13)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_preserves_pairs_and_relative_positions(interleaved):
    rng = np.random.default_rng(6)
    ang = rng.uniform(0, 6, 32)
    table = lambda p: np.concatenate([np.cos(p * ang), np.sin(p * ang)])
    x, y = rng.standard_normal((2, 64))
    a = O.rotate_ref(x, table(3), interleaved) @ O.rotate_ref(y, table(10), interleaved)
    b = O.rotate_ref(x, table(20), interleaved) @ O.rotate_ref(y, table(27), interleaved)
    assert abs(a - b) < 1e-12
    i, j = (4, 5) if interleaved else (2, 34)
    r = O.rotate_ref(x, table(1), interleaved)
    assert np.allclose([r[i], r[j]], [x[i] * math.cos(ang[2]) - x[j] * math.sin(ang[2]), x[i] * math.sin(ang[2]) + x[j] * math.cos(ang[2])])


def test_append_places_the_last_tokens():
    c = S.f32_to_bf16_bits(np.arange(4 * 512, dtype=np.float32).reshape(4, 512) % 97)
    k = S.f32_to_bf16_bits(np.ones((4, 64), dtype=np.float32))
    cos_sin = np.concatenate([np.ones((200, 32)), np.zeros((200, 32))], 1)
    writes, q_out = O.mla_append_ref(c, k, None, cos_sin, [0, 1, 1, 3], [65, 9, 2], None, [[7, 3], [0, 0], [5, 0]], True)
    assert [w[:3] for w in writes] == [(3, 0, 0), (5, 0, 1), (5, 1, 2)] and q_out is None
    assert np.array_equal(writes[1][3][:512], O.bf16_to_f64(c[1])) and (writes[1][3][512:] == 1).all()

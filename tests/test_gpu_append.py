"""GPU parity of mla_append against the fp64 oracle.

Latent values are copied: they must be equal.  A rotated value is computed in fp32 from
bf16 values and fp32 cosines (three roundings of at most 2^-24 of |x c| + |y s| each) and
rounded once to bf16, half a step of which is 2^-8 relative.
"""
import numpy as np
import pytest
import torch

import mla_latent_kv_22_b200 as M
import mla_synth as S
import oracle as O
from gpu_helpers import bf16_dev

pytestmark = pytest.mark.gpu

FILL = 0x4321  # a finite bf16 pattern marking rows that must stay as they were


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def table_of(max_pos, seed):
    ang = np.random.default_rng(seed).uniform(0, 2 * np.pi, (max_pos, 32))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


class Append:
    def __init__(self, new, old, H, seed, inter=True, pad=0, offset=None, paged=True, with_q=True):
        rng = np.random.default_rng(seed)
        bf = lambda *s: S.f32_to_bf16_bits(rng.standard_normal(s).astype(np.float32))
        self.new, self.T = np.asarray(new), np.asarray(new) + np.asarray(old)
        self.B, self.inter, n = len(new), inter, int(np.sum(new)) + pad
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.c, self.k, self.q = bf(n, 512), bf(n, 64), bf(n, H, 64) if with_q else None
        blocks = [-(-int(t) // 64) for t in self.T]
        self.offset = None if offset is None else np.asarray(offset, dtype=np.int32)
        top = int(np.max(self.T + (0 if offset is None else self.offset)))
        self.cos_sin = table_of(max(1, top), seed)
        w = max(1, max(blocks))
        if paged:
            order, at = rng.permutation(sum(blocks)), 0
            self.table = np.full((self.B, w), -1, dtype=np.int32)
            for b, m in enumerate(blocks):
                self.table[b, :m] = order[at:at + m]
                at += m
            self.kv = np.full((sum(blocks) + 1, 64, 576), FILL, dtype=np.uint16)
        else:
            self.table = None
            self.kv = np.full((self.B, 64 * w, 576), FILL, dtype=np.uint16)

    def dev(self):
        t = lambda a: None if a is None else torch.from_numpy(np.asarray(a)).cuda()
        return dict(c_kv=bf16_dev(self.c), k_rope=bf16_dev(self.k), kv_cache=bf16_dev(self.kv), block_table=t(self.table),
                    cache_seqlens=t(self.T.astype(np.int32)), cos_sin=t(self.cos_sin), cu_tokens=t(self.cu),
                    q_rope=None if self.q is None else bf16_dev(self.q),
                    q_out=None if self.q is None else bf16_dev(np.full(self.q.shape, FILL, dtype=np.uint16)),
                    pos_offset=t(self.offset), interleaved=self.inter)

    def check(self, kv, q_out, skip=()):
        writes, qr = O.mla_append_ref(self.c, self.k, self.q, self.cos_sin, self.cu, self.T, self.offset, self.table, self.inter)
        got, want = bits(kv), self.kv.copy()
        mags = O.bf16_to_f64(self.k)
        for a, r, n, row in writes:
            if n in skip:
                continue
            assert np.array_equal(got[a, r, :512], self.c[n]), f"token {n}: latent"
            self._near(got[a, r, 512:], row[512:], mags[n], n)
            want[a, r] = got[a, r]
        assert np.array_equal(got, want), "a row that no token belongs to changed"
        if self.q is None:
            return
        g = bits(q_out)
        for n in range(len(self.c)):
            if n in skip:
                assert np.isnan(O.bf16_to_f64(g[n])).all()
            elif n >= self.cu[-1]:
                assert (g[n] == FILL).all(), "padding was written"
            else:
                self._near(g[n], qr[n], O.bf16_to_f64(self.q[n]), n)

    def _near(self, got, want, x, n):
        x = np.abs(x)
        pair = (x.reshape(x.shape[:-1] + (32, 2)).sum(-1).repeat(2, -1) if self.inter
                else np.concatenate([x[..., :32] + x[..., 32:]] * 2, -1))
        off = np.abs(O.bf16_to_f64(got) - want) - (2.0 ** -8 * np.abs(want) + 4 * 2.0 ** -24 * pair)
        assert (off <= 0).all(), f"token {n}: rotation off by {off.max():.2e} more than allowed"


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("new,old,H,kw", [
    ([1], [0], 1, {}),
    ([1], [64], 16, {}),
    ([1] * 9, [0, 1, 62, 63, 64, 65, 127, 128, 1000], 128, {}),
    ([0, 5, 0, 0, 130, 1, 0], [3, 60, 0, 64, 63, 0, 9], 33, dict(pad=3)),   # empty sequences and padding
    ([1] * 300, [3] * 300, 2, {}),                                         # more sequences than a block's threads
    ([7, 64], [0, 1], 100, dict(offset=[1000, 5])),
    ([70, 1], [0, 200], 7, dict(paged=False)),
    ([70, 1], [0, 200], 7, dict(with_q=False)),
])
def test_append_matches_oracle(inter, new, old, H, kw):
    c = Append(new, old, H, seed=700 + H, inter=inter, **kw)
    d = c.dev()
    M.mla_append(**d)
    assert M.mla_get_device_error() == 0
    c.check(d["kv_cache"], d["q_out"])


def test_equal_counts_need_no_cu_tokens():
    c = Append([3] * 5, [10, 0, 63, 64, 1], 8, seed=720)
    d = c.dev()
    d["cu_tokens"] = None
    M.mla_append(**d)
    assert M.mla_get_device_error() == 0
    c.check(d["kv_cache"], d["q_out"])


@pytest.mark.parametrize("inter", [True, False])
def test_views_and_rotation_in_place(inter):
    # The usual projections: [c_kv | k_rope] in one 576-wide buffer, q_rope the last 64 of
    # each head's 192, rotated where it lies.
    c = Append([3, 40], [5, 30], 12, seed=721, inter=inter)
    d = c.dev()
    both = torch.cat([d["c_kv"], d["k_rope"]], 1)
    q = torch.zeros(43, 12, 192, dtype=torch.bfloat16, device="cuda")
    q[..., 128:] = d["q_rope"]
    d.update(c_kv=both[:, :512], k_rope=both[:, 512:], q_rope=q[..., 128:], q_out=q[..., 128:])
    M.mla_append(**d)
    assert M.mla_get_device_error() == 0
    c.check(d["kv_cache"], q[..., 128:])
    assert (q[..., :128] == 0).all()


def test_a_single_token_or_head_of_any_stride():
    c = Append([1], [70], 1, seed=760)
    d = c.dev()
    odd = lambda t, *st: t.as_strided(t.shape, st)
    d.update(c_kv=odd(d["c_kv"], 577, 1), k_rope=odd(d["k_rope"], 3, 1), q_rope=odd(d["q_rope"], 129, 67, 1),
             q_out=odd(d["q_out"], 65, 65, 1))
    M.mla_append(**d)
    assert M.mla_get_device_error() == 0
    c.check(d["kv_cache"], d["q_out"])


def test_bad_tokens_write_nothing():
    c = Append([1, 2, 1, 1], [10, 70, 5, 6], 4, seed=722)
    c.table[1, 1] = c.kv.shape[0]            # sequence 1's new rows lie there
    d = c.dev()
    M.mla_append(**d)
    assert M.mla_get_device_error() == 5
    c.table[1, 1] = 0                        # (for the oracle, which skips those tokens)
    c.check(d["kv_cache"], d["q_out"], skip=(1, 2))

    c = Append([1, 2, 1], [10, 70, 5], 4, seed=723)
    d = c.dev()
    d["cos_sin"] = d["cos_sin"][:71].contiguous()   # token 2 (position 71) is beyond it
    M.mla_append(**d)
    assert M.mla_get_device_error() == 7
    c.check(d["kv_cache"], d["q_out"], skip=(2,))

    c = Append([1, 2, 1], [10, 70, 5], 4, seed=724)
    d = c.dev()
    d["cache_seqlens"][1] = 1                # two new tokens in a sequence of one: the first has no row
    d["cache_seqlens"][2] = 64 * c.table.shape[1] + 1
    M.mla_append(**d)
    assert M.mla_get_device_error() == 5
    c.T[1] = 1
    writes_at_row0 = bits(d["kv_cache"])[c.table[1, 0], 0]
    assert np.array_equal(writes_at_row0[:512], c.c[2])
    assert np.isnan(O.bf16_to_f64(bits(d["q_out"])[[1, 3]])).all()


def test_no_tokens_is_a_no_op():
    c = Append([0, 0], [3, 4], 4, seed=725)
    d = c.dev()
    M.mla_append(**d)
    assert M.mla_get_device_error() == 0 and np.array_equal(bits(d["kv_cache"]), c.kv)


def test_rows_beyond_32_bit_offsets():
    # A pool of 59,000 pages holds 2.17e9 values: the last pages lie past 2^31 elements.
    if torch.cuda.mem_get_info()[0] < 6 << 30:
        pytest.skip("needs 4.4 GB")
    kv = torch.zeros(59000, 64, 576, dtype=torch.bfloat16, device="cuda")
    c = Append([2], [62], 1, seed=726)
    d = c.dev()
    d["kv_cache"] = kv
    d["block_table"] = torch.tensor([[58999]], dtype=torch.int32, device="cuda")
    M.mla_append(**d)
    assert M.mla_get_device_error() == 0
    assert np.array_equal(bits(kv[58999, 62:, :512]), c.c) and not kv[58999, :62].any()
    # and the window decode reads them back: one visible token returns its latent
    q = torch.ones(1, 1, 576, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty(1, 1, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 1, device="cuda")
    M.mla_decode_window(q, kv, d["block_table"], d["cache_seqlens"], out, lse, 0.01, window=1)
    assert M.mla_get_device_error() == 0
    assert np.array_equal(bits(out)[0, 0], c.c[1])
    del kv


def test_refusals():
    c = Append([3], [10], 4, seed=727)
    d = c.dev()
    bad = [("c_kv", d["c_kv"].t().contiguous().t(), ValueError), ("k_rope", d["k_rope"].float(), TypeError),
           ("q_out", None, ValueError), ("cos_sin", d["cos_sin"][:, :32].contiguous(), ValueError),
           ("cu_tokens", d["cu_tokens"].long(), TypeError), ("cu_tokens", d["cu_tokens"][:1], ValueError),
           ("k_rope", d["k_rope"][:2], ValueError), ("pos_offset", torch.zeros(2, dtype=torch.int32, device="cuda"), ValueError)]
    for name, v, exc in bad:
        with pytest.raises(exc):
            M.mla_append(**{**d, name: v})
    wide = torch.zeros(3, 516, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(M.MlaError):   # rows that are not 16-byte aligned
        M.mla_append(**{**d, "c_kv": wide[:, :512]})
    with pytest.raises(M.MlaError):   # three tokens, two sequences, no cu_tokens
        M.mla_append(**{**d, "cu_tokens": None, "cache_seqlens": torch.tensor([13, 1], dtype=torch.int32, device="cuda"),
                        "block_table": d["block_table"].expand(2, -1).contiguous()})
    assert M.mla_get_device_error() == 0

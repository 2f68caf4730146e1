"""GPU parity of mla_decode_shared against the fp64 oracle (tolerances: test_gpu_window)."""
import numpy as np
import pytest
import torch

import mla_latent_kv_22_b200 as M
import mla_synth as S
import oracle as O
from gpu_helpers import bf16_dev
from test_gpu_window import _knobs, assert_rounded  # noqa: F401  (the knob-resetting fixture)

pytestmark = pytest.mark.gpu


class Shared:
    """A seeded case: prefix and own tokens in one shuffled pool, NaN in every other row."""

    def __init__(self, P, lens, s_q, H, seed, prefix_blocks=None, max_blocks=None):
        rng = np.random.default_rng(seed)
        self.B, self.P, self.lens, self.scale = len(lens), P, np.asarray(lens, dtype=np.int32), 192 ** -0.5
        blocks = lambda n: -(-n // 64)
        live = [P] + list(lens)
        order = rng.permutation(sum(blocks(n) for n in live))
        self.kv = np.full((len(order) + 1, 64, 576), S.BF16_NAN, dtype=np.uint16)
        self.ptab = np.full(prefix_blocks or max(1, blocks(P)), 1 << 30, dtype=np.int32)
        self.table = np.full((self.B, max_blocks or max(1, max(blocks(n) for n in lens))), -1, dtype=np.int32)
        at = 0
        for k, n in enumerate(live):
            ids = order[at:at + blocks(n)]
            at += blocks(n)
            (self.ptab if k == 0 else self.table[k - 1])[:len(ids)] = ids
            rows = S.f32_to_bf16_bits(rng.standard_normal((n, 576)).astype(np.float32))
            for i, pg in enumerate(ids):
                part = rows[64 * i:64 * i + 64]
                self.kv[pg, :len(part)] = part
        self.q = S.f32_to_bf16_bits(rng.standard_normal((self.B, s_q, H, 576)).astype(np.float32))

    def run(self, **kw):
        i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()
        q = bf16_dev(self.q)
        out = torch.full(self.q.shape[:3] + (512,), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full(self.q.shape[:3], float("nan"), device="cuda")
        M.mla_decode_shared(q, bf16_dev(self.kv), i32(self.ptab), i32([self.P]), i32(self.table), i32(self.lens), out, lse,
                            self.scale, **kw)
        return out, lse, M.mla_get_device_error()

    def ref(self):
        return O.mla_decode_shared_ref(self.q, self.kv, self.ptab, self.P, self.table, self.lens, self.scale)


@pytest.mark.parametrize("P,lens,s_q,H", [
    (1, [0], 1, 1),                      # one token, one row
    (64, [1, 0, 64], 1, 4),              # 12 rows, a sequence that is the prefix alone
    (100, [1, 300, 65, 7, 64, 0, 12], 1, 16),
    (1000, [130, 5], 1, 16),             # 32 rows
    (333, [40, 0, 1], 1, 20),            # 60 rows: one 64-row tile across three sequences
    (500, [7, 70], 1, 128),
    (200, [3, 1, 0], 1, 100),            # tiles that cross sequence borders, two own groups
    (130, [5, 64, 1], 2, 33),            # several queries
    (65, [0, 1, 2, 100], 3, 40),         # T < s_q: queries end inside the prefix
    (2, [0, 1], 5, 3),                   # P + T < s_q: queries that see nothing
    (0, [0, 5, 100], 1, 16),             # no prefix; one sequence with nothing at all
    (4097, [1] * 9, 1, 16),
    (700, [50] * 70, 1, 3),              # 210 rows of 70 sequences
])
def test_shared_matches_oracle(P, lens, s_q, H):
    c = Shared(P, lens, s_q, H, seed=600 + P)
    out, lse, err = c.run()
    assert err == 0
    assert_rounded(out, lse, c.ref())


@pytest.mark.parametrize("H", [4, 8, 64])
@pytest.mark.parametrize("workers", [1, 2, 7, 148])
def test_forced_splits(H, workers):
    M.mla_set_knob("num_workers", workers)
    M.mla_set_knob("min_pages", 1)
    c = Shared(1500, [300, 0, 65], 1, H, seed=620)
    out, lse, err = c.run()
    assert err == 0
    assert_rounded(out, lse, c.ref(), f"{workers} workers")


@pytest.mark.parametrize("policy", [1, 2])
def test_schedule_policies(policy):
    M.mla_set_knob("split_policy", policy)
    c = Shared(600, [90, 300, 64], 1, 16, seed=621)
    out, lse, err = c.run()
    assert err == 0
    assert_rounded(out, lse, c.ref())


def test_wider_tables_than_needed_and_equal_runs():
    c = Shared(300, [90, 0, 64], 1, 16, seed=622, prefix_blocks=9, max_blocks=7)
    a, b = c.run(), c.run()
    assert a[2] == 0
    assert_rounded(a[0], a[1], c.ref())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bad_pages_and_lengths():
    c = Shared(300, [90, 30, 64], 1, 16, seed=623)
    good = c.ref()
    keep = c.table[1, 0]
    c.table[1, 0] = -5
    out, lse, err = c.run()
    assert err == 5 and torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert_rounded(out[[0, 2]], lse[[0, 2]], [g[[0, 2]] for g in good])
    c.table[1, 0] = keep
    c.lens[1] = -1
    out, lse, err = c.run()
    assert err == 5 and torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert_rounded(out[[0, 2]], lse[[0, 2]], [g[[0, 2]] for g in good])
    c.lens[1] = 30
    c.P = 64 * len(c.ptab) + 1   # every sequence sees the prefix
    out, lse, err = c.run()
    assert err == 5 and torch.isnan(out).all() and torch.isnan(lse).all()
    c.P = 300
    c.ptab[2] = c.kv.shape[0]
    out, lse, err = c.run()
    assert err == 5 and torch.isnan(out).all() and torch.isnan(lse).all()
    c.ptab[2] = 0
    assert c.run()[2] == 0


def test_captured_and_replayed():
    c, d = Shared(500, [70, 3, 200], 1, 16, seed=624), Shared(500, [70, 3, 200], 1, 16, seed=624)
    d.q = S.f32_to_bf16_bits(np.random.default_rng(9).standard_normal(d.q.shape).astype(np.float32))
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()
    q, kv, pt, pl, bt, sl = bf16_dev(c.q), bf16_dev(c.kv), i32(c.ptab), i32([c.P]), i32(c.table), i32(c.lens)
    out = torch.empty(3, 1, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 1, 16, device="cuda")
    call = lambda: M.mla_decode_shared(q, kv, pt, pl, bt, sl, out, lse, c.scale)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    q.copy_(bf16_dev(d.q))
    sl.copy_(i32([1, 0, 130]))   # lengths are read on the device: a replay follows them
    d.lens[:] = [1, 0, 130]
    out.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert M.mla_get_device_error() == 0
    # rows past the shorter lengths are still finite, so the case needs no new poison
    assert_rounded(out, lse, d.ref())
    del g


def test_refusals():
    c = Shared(100, [10], 1, 4, seed=625)
    with pytest.raises(M.MlaError) as ei:
        c.run(workspace=torch.empty(512, dtype=torch.uint8, device="cuda"))
    assert ei.value.name == "MLA_ERR_WORKSPACE"
    t = lambda *s, **k: torch.zeros(*s, device="cuda", **k)
    bf = dict(dtype=torch.bfloat16)
    ii = dict(dtype=torch.int32)
    ok = dict(q=t(1, 4, 576, **bf), kv_cache=t(2, 64, 576, **bf), prefix_table=t(1, **ii), prefix_len=t(1, **ii),
              block_table=t(1, 1, **ii), cache_seqlens=t(1, **ii), out=t(1, 4, 512, **bf), lse=t(1, 4), softmax_scale=0.1)
    M.mla_decode_shared(**ok)
    for name, bad in (("block_table", None), ("prefix_len", t(2, **ii)), ("prefix_table", t(1, 1, **ii)),
                      ("cache_seqlens", t(2, **ii)), ("lse", t(1, 5)), ("kv_cache", t(2, 32, 576, **bf))):
        with pytest.raises(ValueError):
            M.mla_decode_shared(**{**ok, name: bad})
    with pytest.raises(TypeError):
        M.mla_decode_shared(**{**ok, "out": t(1, 4, 512)})
    assert M.mla_get_device_error() == 0

"""mla_absorb_o on a bf16 latent, and the serving operators run together as a step does:
append, key absorption, decode over the window or the shared prefix, value absorption."""
import numpy as np
import pytest
import torch

import mla_latent_kv_22_b200 as M
import mla_synth as S
import oracle as O
from gpu_helpers import bf16_dev
from test_gpu_window import _knobs, assert_rounded  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H", [(1, 1), (5, 16), (16, 3), (17, 74), (32, 75), (33, 128), (64, 20), (70, 2), (130, 128), (300, 40)])
def test_absorb_o_of_a_bf16_latent(B, H):
    rng = np.random.default_rng(B * H)
    x = S.f32_to_bf16_bits(rng.standard_normal((B, H, 512)).astype(np.float32))
    w = S.f32_to_bf16_bits((rng.standard_normal((H, 512, 128)) / 16).astype(np.float32))
    out = torch.full((B, H, 128), float("nan"), device="cuda")
    M.mla_absorb_o(bf16_dev(x), bf16_dev(w), out)
    assert M.mla_get_device_error() == 0
    xf, wf = torch.from_numpy(O.bf16_to_f64(x)), torch.from_numpy(O.bf16_to_f64(w))
    ref = torch.bmm(xf.transpose(0, 1), wf).transpose(0, 1)
    mag = torch.bmm(xf.abs().transpose(0, 1), wf.abs()).transpose(0, 1)
    # 512 products summed in fp32, each addition off by at most 2^-23 of the running magnitude
    assert ((out.double().cpu() - ref).abs() <= 512 * 2.0 ** -23 * mag).all()


def test_absorb_o_rounds_an_fp32_latent_to_the_same_result():
    x = torch.randn(9, 30, 512, device="cuda").bfloat16()
    w = torch.randn(30, 512, 128, device="cuda").bfloat16()
    a, b = torch.empty(9, 30, 128, device="cuda"), torch.empty(9, 30, 128, device="cuda")
    M.mla_absorb_o(x, w, a)
    M.mla_absorb_o(x.float(), w, b)
    assert M.mla_get_device_error() == 0
    mag = torch.bmm(x.float().abs().transpose(0, 1), w.float().abs()).transpose(0, 1)
    assert ((a - b).abs() <= 2 * 512 * 2.0 ** -23 * mag).all()


class Step:
    """A serving step of B sequences with H heads: the projections' outputs and the layer's
    weights; sequences grow by one token a step."""

    def __init__(self, B, H, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()
        self.B, self.H, self.n = B, H, n
        self.w_uk, self.w_uv = n(H, 128, 512, std=512 ** -0.5), n(H, 512, 128, std=512 ** -0.5)
        ang = torch.arange(4096, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float64) / 32)
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()

    def token(self):
        B, H = self.B, self.H
        return dict(kv=self.n(B, 576), q=self.n(B, H, 192))

    def attend(self, t, kv, table, lens, decode, pos_offset=None):
        B, H = self.B, self.H
        M.mla_append(t["kv"][:, :512], t["kv"][:, 512:], kv, table, lens, self.cos_sin, q_rope=t["q"][..., 128:],
                     q_out=t["q"][..., 128:], pos_offset=pos_offset)
        q = torch.empty(B, H, 576, dtype=torch.bfloat16, device="cuda")
        M.mla_absorb_q(t["q"][..., :128].contiguous(), t["q"][..., 128:].contiguous(), self.w_uk, q)
        lat = torch.empty(B, H, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(B, H, device="cuda")
        decode(q, lat, lse)
        out = torch.empty(B, H, 128, device="cuda")
        M.mla_absorb_o(lat, self.w_uv, out)
        return q, lat, lse, out


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("H", [16, 128])
def test_window_steps(H):
    B, W, K = 3, 70, 4
    s = Step(B, H, seed=40 + H)
    kv = torch.full((16, 64, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[9, 3, 1, -1], [0, 7, -1, -1], [5, 2, 11, 14]], dtype=torch.int32, device="cuda")
    start = [126, 0, 190]
    for b, T in enumerate(start):   # the prompts, already cached
        for p in range(-(-T // 64)):
            kv[table[b, p].item(), :min(64, T - 64 * p)] = s.n(min(64, T - 64 * p), 576)
    lens = torch.tensor(start, dtype=torch.int32, device="cuda")
    for _ in range(5):
        lens += 1
        t = s.token()
        raw = t["kv"].clone(), t["q"].clone()
        q, lat, lse, out = s.attend(t, kv, table, lens, lambda q, o, l: M.mla_decode_window(q, kv, table, lens, o, l, 192 ** -0.5, W, K))
        assert M.mla_get_device_error() == 0
        ref = O.mla_decode_window_ref(bits(q)[:, None], bits(kv), table.cpu().numpy(), lens.cpu().numpy(), 192 ** -0.5, W, K)
        assert_rounded(lat[:, None], lse[:, None], ref)
        for b in range(B):   # the token's row in the cache, and the query's rotated part
            T = lens[b].item() - 1
            row = kv[table[b, T // 64].item(), T % 64]
            assert torch.equal(row[:512], raw[0][b, :512])
            cs = s.cos_sin[T].cpu().numpy()
            for got, x in ((row[512:], raw[0][b, 512:]), (q[b, :, 512:], raw[1][b, :, 128:])):
                want = torch.from_numpy(O.rotate_ref(bits(x), cs, True))
                assert torch.allclose(got.double().cpu(), want, rtol=2.0 ** -8, atol=2.0 ** -20)
        up = torch.bmm(lat.double().transpose(0, 1), s.w_uv.double()).transpose(0, 1)
        assert torch.allclose(out.double(), up, rtol=1e-4, atol=1e-4)


def test_shared_prefix_steps():
    B, H, P = 5, 16, 150
    s = Step(B, H, seed=50)
    kv = torch.full((12, 64, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    ptab = torch.tensor([4, 0, 8], dtype=torch.int32, device="cuda")
    for p in range(3):
        kv[ptab[p].item(), :min(64, P - 64 * p)] = s.n(min(64, P - 64 * p), 576)
    plen = torch.tensor([P], dtype=torch.int32, device="cuda")
    table = torch.tensor([[1], [2], [3], [5], [6]], dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    offset = torch.full((B,), P, dtype=torch.int32, device="cuda")
    for _ in range(4):
        lens += 1
        q, lat, lse, _ = s.attend(s.token(), kv, table, lens, lambda q, o, l: M.mla_decode_shared(
            q, kv, ptab, plen, table, lens, o, l, 192 ** -0.5), pos_offset=offset)
        assert M.mla_get_device_error() == 0
        ref = O.mla_decode_shared_ref(bits(q)[:, None], bits(kv), ptab.cpu().numpy(), P, table.cpu().numpy(), lens.cpu().numpy(), 192 ** -0.5)
        assert_rounded(lat[:, None], lse[:, None], ref)


def test_a_step_captured_and_replayed():
    B, H = 4, 16
    s = Step(B, H, seed=60)
    kv = s.n(20, 64, 576)
    table = torch.arange(20, device="cuda", dtype=torch.int32).view(4, 5)
    lens = torch.tensor([100, 1, 64, 300], dtype=torch.int32, device="cuda")
    t, src = s.token(), s.token()
    call = lambda: s.attend(t, kv, table, lens, lambda q, o, l: M.mla_decode_window(q, kv, table, lens, o, l, 192 ** -0.5, 90, 4))
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = call()
    for k in range(3):   # each replay appends the next token
        lens += 1
        for key in t:
            t[key].copy_(src[key])
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in held]
        for key in t:
            t[key].copy_(src[key])
        want = call()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert M.mla_get_device_error() == 0
    del g

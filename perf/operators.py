"""Cases of the paged latent cache's append, sliding-window and shared-prefix operators.

Four operators are covered, each through its public entry point and in a plain form
made of elementary torch operations in fp32:

* ``append``: new tokens' rows ``[c_kv | rotated k_rope]`` into the paged cache, and the
  rotation of the same tokens' query parts (``mla_append``);
* ``window``: decode over a sliding window and a few first tokens that stay visible
  (``mla_decode_window``);
* ``shared``: decode of a batch whose sequences share one cached prefix
  (``mla_decode_shared``);
* ``lift``: value absorption of a bf16 latent output (``mla_absorb_o``).

A case's lengths follow from its sizes alone, so ``work`` knows them; contents and page
order come from the seed.
"""
import math

import numpy as np
import torch

own = False

PAGE, D_C, D_R, D_ROW, D_V = 64, 512, 64, 576, 128
SCALE = 192 ** -0.5


def listed():
    return [
        # One new token for one sequence on a shard of 16 heads: latency alone.
        dict(name="append 1 token h16", op="append", batch=1, heads=16, new_lo=1, new_hi=1, len_hi=257, inter=True),
        # The append of a decode step of 64 sequences with all 128 heads.
        dict(name="append 64 tokens h128", op="append", batch=64, heads=128, new_lo=1, new_hi=1, len_hi=1024, inter=True),
        # A chunk of ragged prompts, 13 sequences with 0 to 1,259 new tokens each, half-split rotation.
        dict(name="append ragged prompts h128", op="append", batch=13, heads=128, new_lo=0, new_hi=1259, len_hi=2048,
             inter=False),
        # One short conversation on a shard of 16 heads: the smallest decode call.
        dict(name="window b1 h16 w512", op="window", batch=1, heads=16, s_q=1, len_lo=4096, len_hi=4096, window=512,
             sinks=4),
        # A large serving batch on a shard, ragged and odd: window and sinks end inside pages, some sequences are short.
        dict(name="window b256 h16 w1021", op="window", batch=256, heads=16, s_q=1, len_lo=1, len_hi=8192, window=1021,
             sinks=5),
        # All 128 heads over a long window.
        dict(name="window b64 h128 w4096", op="window", batch=64, heads=128, s_q=1, len_lo=8192, len_hi=8192,
             window=4096, sinks=64),
        # Two new tokens for each sequence (a verified draft) at 128K tokens, pages outside the window given back.
        dict(name="window b16 h64 two queries", op="window", batch=16, heads=64, s_q=2, len_lo=100000, len_hi=131072,
             window=4096, sinks=4),
        # A few users behind one system prompt on a shard.
        dict(name="shared b7 h16 p1000", op="shared", batch=7, heads=16, s_q=1, prefix=1000, len_lo=1, len_hi=300),
        # Many users behind one long document on a shard: the prefix would be read 64 times without sharing.
        dict(name="shared b64 h16 p32768", op="shared", batch=64, heads=16, s_q=1, prefix=32768, len_lo=0, len_hi=1024),
        # The same with all 128 heads: bound by the matrix products.
        dict(name="shared b64 h128 p8192", op="shared", batch=64, heads=128, s_q=1, prefix=8192, len_lo=1, len_hi=1024),
        # The value absorption that follows a decode, on a shard and with all heads.
        dict(name="lift b5 h16", op="lift", batch=5, heads=16),
        dict(name="lift b64 h128", op="lift", batch=64, heads=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "window", "window", "shared", "shared", "lift"))
    if op == "append":
        b = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, 8192 // b))
        return dict(op=op, batch=b, heads=_log(rng, 1, 128), new_lo=rng.choice((0, 1)) if hi > 1 else 1, new_hi=hi,
                    len_hi=hi + _log(rng, 1, 512), inter=rng.random() < 0.5)
    if op == "window":
        b, s_q = _log(rng, 1, 256), rng.choice((1, 1, 1, 2, 3))
        w = _log(rng, 64, min(4096, 262144 // b))
        lo = _log(rng, 1, 8192)
        return dict(op=op, batch=b, heads=_log(rng, 1, 128 // s_q), s_q=s_q, len_lo=lo, len_hi=lo + _log(rng, 1, 32768),
                    window=w, sinks=rng.choice((0, 1, 4, 16, 64, 100)))
    if op == "shared":
        b = _log(rng, 2, 128)
        h = _log(rng, 1, min(128, 8192 // b))
        p = _log(rng, 64, min(65536, (8192 * 8192) // (b * h)))
        return dict(op=op, batch=b, heads=h, s_q=rng.choice((1, 1, 2)) if b * h <= 4096 else 1, prefix=p,
                    len_lo=rng.choice((0, 1)), len_hi=_log(rng, 1, 512))
    return dict(op=op, batch=_log(rng, 1, 64), heads=_log(rng, 1, 128))


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], spread by the golden ratio: the ends' neighbourhood is met from the first few on."""
    if n == 1:
        return np.array([hi], dtype=np.int64)
    x = (np.arange(n) * 0.6180339887498949) % 1.0
    return lo + np.minimum(np.floor(x * (hi - lo + 1)).astype(np.int64), hi - lo)


def _append_lens(case):
    new = _spread(case["new_lo"], case["new_hi"], case["batch"])
    old = _spread(0, case["len_hi"] - case["new_hi"], case["batch"])[::-1]
    return new, old + new


def _window_spans(case):
    """Lengths, and the first token that any query's window reaches."""
    T = _spread(case["len_lo"], case["len_hi"], case["batch"])
    return T, np.maximum(0, T - case["s_q"] - case["window"] + 1)


def _normal(gen, *shape, std=1.0):
    """bf16 normals made a part at a time, so that fp32 copies of a large cache are never whole."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        part = flat[i:i + (1 << 26)]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda").mul_(std))
    return out


def _table(live, order, width):
    """A block table [B, width]: the pages listed for each sequence numbered by `order`, -1 elsewhere."""
    t, at = np.full((len(live), max(1, width)), -1, dtype=np.int32), 0
    for b, pages in enumerate(live):
        t[b, pages] = order[at:at + len(pages)]
        at += len(pages)
    return torch.from_numpy(t).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, B, H = case["op"], case["batch"], case["heads"]
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()
    if op == "lift":
        return dict(op=op, x=_normal(gen, B, H, D_C, std=0.25), w=_normal(gen, H, D_C, D_V, std=D_C ** -0.5),
                    out=torch.empty(B, H, D_V, device="cuda"))
    if op == "append":
        new, T = _append_lens(case)
        n = int(new.sum())
        pages = [np.arange(-(-int(t) // PAGE)) for t in T]
        used = sum(len(p) for p in pages)
        pos = np.arange(int(T.max()))[:, None] * 10000.0 ** (-np.arange(D_R // 2) / (D_R // 2))[None]
        cos_sin = np.concatenate([np.cos(pos), np.sin(pos)], 1).astype(np.float32)
        return dict(op=op, inter=case["inter"], c_kv=_normal(gen, n, D_C), k_rope=_normal(gen, n, D_R),
                    q_rope=_normal(gen, n, H, D_R), q_out=torch.zeros(n, H, D_R, dtype=torch.bfloat16, device="cuda"),
                    cos_sin=torch.from_numpy(cos_sin).cuda(), kv=_normal(gen, used + 1, PAGE, D_ROW),
                    table=_table(pages, rng.permutation(used), max(len(p) for p in pages)), lens=i32(T),
                    cu=i32(np.concatenate([[0], np.cumsum(new)])))
    s_q = case["s_q"]
    q = _normal(gen, B, s_q, H, D_ROW)
    out = torch.empty(B, s_q, H, D_C, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, s_q, H, device="cuda")
    if op == "window":
        T, first = _window_spans(case)
        pages = []
        for t, f in zip(T, first):
            n, s = -(-int(t) // PAGE), -(-min(int(t), case["sinks"]) // PAGE)
            pages.append(np.unique(np.concatenate([np.arange(s), np.arange(int(f) // PAGE, n)])).astype(np.int64))
        used = sum(len(p) for p in pages)
        return dict(op=op, q=q, out=out, lse=lse, kv=_normal(gen, used + 1, PAGE, D_ROW), lens=i32(T),
                    table=_table(pages, rng.permutation(used), -(-int(T.max()) // PAGE)), window=case["window"],
                    sinks=case["sinks"])
    T = _spread(case["len_lo"], case["len_hi"], B)
    pages = [np.arange(-(-case["prefix"] // PAGE))] + [np.arange(-(-int(t) // PAGE)) for t in T]
    used = sum(len(p) for p in pages)
    order = rng.permutation(used)
    np_ = len(pages[0])
    return dict(op=op, q=q, out=out, lse=lse, kv=_normal(gen, used + 1, PAGE, D_ROW), lens=i32(T),
                prefix_table=i32(order[:np_]), prefix_len=i32([case["prefix"]]),
                table=_table(pages[1:], order[np_:], max(1, max(len(p) for p in pages[1:]))),
                sizes=(case["prefix"], int(T.max())))


def _rotated(x, cs, inter):
    """x [..., 64] turned by the angles whose cosines and sines cs [..., 64] holds, in fp32."""
    x, c, s = x.float(), cs[..., :32], cs[..., 32:]
    if inter:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _softmax_rows(scores, rows):
    """Softmax over the last axis with an empty row giving zeros and -inf; its product with rows, and the lse."""
    m = scores.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(scores - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows) / torch.where(l > 0, l, torch.ones_like(l))
    return o, (torch.log(l) + m).squeeze(-1)


def _plain(s):
    if s["op"] == "lift":
        s["out"].copy_(torch.einsum("bhd,hdv->bhv", s["x"].float(), s["w"].float()))
        return [s["out"]]
    if s["op"] == "append":
        n = s["c_kv"].shape[0]
        cu, lens = s["cu"].long(), s["lens"].long()
        i = torch.arange(n, device="cuda")
        b = torch.searchsorted(cu, i, right=True) - 1
        pos = lens[b] - cu[b + 1] + i
        cs = s["cos_sin"][pos]
        row = torch.cat([s["c_kv"].float(), _rotated(s["k_rope"], cs, s["inter"])], 1).bfloat16()
        s["kv"][s["table"].long()[b, pos // PAGE], pos % PAGE] = row
        s["q_out"].copy_(_rotated(s["q_rope"], cs[:, None], s["inter"]))
        return [s["kv"], s["q_out"]]
    B, s_q, H, _ = s["q"].shape
    q = s["q"].float() * SCALE
    T = s["lens"].long()
    table = s["table"].long().clamp_min(0)
    flat = s["kv"].view(-1, D_ROW)
    i = torch.arange(s_q, device="cuda")
    if s["op"] == "window":
        W, S = s["window"], s["sinks"]
        first = (T - s_q - W + 1).clamp_min(0)[:, None]
        sink = torch.arange(S, device="cuda").expand(B, S)
        near = first + torch.arange(W + s_q - 1, device="cuda")
        t = torch.cat([sink, near], 1)
        once = torch.cat([torch.ones_like(sink, dtype=torch.bool), near >= S], 1)
        at = (T[:, None] - s_q + i)[:, :, None]
        seen = once[:, None] & (t[:, None] <= at) & ((t[:, None] < S) | (t[:, None] > at - W))
        page = torch.gather(table, 1, (t // PAGE).clamp_max(table.shape[1] - 1))
        rows = flat[page * PAGE + t % PAGE].float()
        scores = torch.matmul(q.view(B, s_q * H, D_ROW), rows.transpose(1, 2)).view(B, s_q, H, -1)
        scores = scores.masked_fill(~seen[:, :, None], -math.inf).view(B, s_q * H, -1)
        o, lse = _softmax_rows(scores, rows[..., :D_C])
    else:
        P, most = s["sizes"]
        t = torch.arange(P, device="cuda")
        pre = flat[s["prefix_table"].long()[t // PAGE] * PAGE + t % PAGE].float()
        u = torch.arange(most, device="cuda")
        mine = flat[table[:, u // PAGE] * PAGE + u % PAGE].float()
        # Query i of s_q sees the first P + T - s_q + 1 + i of the prefix and the sequence's own tokens.
        end = (P + T[:, None] - s_q + 1 + i)[:, :, None, None]
        sp = torch.matmul(q, pre.t()).masked_fill(t >= end, -math.inf)
        so = torch.matmul(q.view(B, s_q * H, D_ROW), mine.transpose(1, 2)).view(B, s_q, H, most)
        so = so.masked_fill(P + u >= end, -math.inf)
        m = torch.cat([sp.amax(-1), so.amax(-1) if most else sp.amax(-1)], 0).view(2, B, s_q, H).amax(0)
        m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))[..., None]
        pp, po = torch.exp(sp - m), torch.exp(so - m)
        l = pp.sum(-1, keepdim=True) + po.sum(-1, keepdim=True)
        o = torch.matmul(pp, pre[:, :D_C])
        o += torch.matmul(po.view(B, s_q * H, most), mine[..., :D_C]).view(B, s_q, H, D_C)
        o /= torch.where(l > 0, l, torch.ones_like(l))
        lse = (torch.log(l) + m).squeeze(-1)
    s["out"].copy_(o.view(B, s_q, H, D_C))
    s["lse"].copy_(lse.view(B, s_q, H))
    return [s["out"], s["lse"]]


def run(state):
    if not own:
        return _plain(state)
    import mla_latent_kv_22_b200 as M
    s = state
    if s["op"] == "lift":
        M.mla_absorb_o(s["x"], s["w"], s["out"])
        return [s["out"]]
    if s["op"] == "append":
        M.mla_append(s["c_kv"], s["k_rope"], s["kv"], s["table"], s["lens"], s["cos_sin"], cu_tokens=s["cu"],
                     q_rope=s["q_rope"], q_out=s["q_out"], interleaved=s["inter"])
        return [s["kv"], s["q_out"]]
    if s["op"] == "window":
        M.mla_decode_window(s["q"], s["kv"], s["table"], s["lens"], s["out"], s["lse"], SCALE, s["window"],
                            sinks=s["sinks"])
    else:
        M.mla_decode_shared(s["q"], s["kv"], s["prefix_table"], s["prefix_len"], s["table"], s["lens"], s["out"],
                            s["lse"], SCALE)
    return [s["out"], s["lse"]]


def work(case):
    op, B, H = case["op"], case["batch"], case["heads"]
    if op == "lift":
        return dict(bytes=2 * B * H * D_C + 2 * H * D_C * D_V + 4 * B * H * D_V, flops=2 * B * H * D_C * D_V)
    if op == "append":
        new, T = _append_lens(case)
        n = int(new.sum())
        return dict(bytes=n * (4 * D_ROW + 4 * H * D_R) + 4 * D_R * min(n, int(T.max())) + 8 * B + 4,
                    flops=n * 3 * D_R * (H + 1))
    s_q = case["s_q"]
    io = B * s_q * H * (2 * D_ROW + 2 * D_C + 4)
    if op == "window":
        T, first = _window_spans(case)
        tokens = int((T - first).sum() + np.minimum(first, case["sinks"]).sum())
        at = T[:, None] - s_q + np.arange(s_q)
        seen = np.minimum(at + 1, case["window"]) + np.clip(at + 1 - case["window"], 0, case["sinks"])
        return dict(bytes=io + 2 * D_ROW * tokens, flops=2 * H * (D_ROW + D_C) * int(np.maximum(seen, 0).sum()))
    T = _spread(case["len_lo"], case["len_hi"], B)
    seen = case["prefix"] + T[:, None] - s_q + 1 + np.arange(s_q)
    return dict(bytes=io + 2 * D_ROW * (case["prefix"] + int(T.sum())),
                flops=2 * H * (D_ROW + D_C) * int(np.maximum(seen, 0).sum()))


def exact(case, seed):
    """The operators from their definitions in fp64, one sequence at a time."""
    s = prepare(case, seed)
    if s["op"] == "lift":
        return [torch.bmm(s["x"].double().transpose(0, 1), s["w"].double()).transpose(0, 1)]
    if s["op"] == "append":
        kv, q_out, cs = s["kv"].double(), torch.empty(s["q_rope"].shape, dtype=torch.float64, device="cuda"), s["cos_sin"].double()
        turn = torch.complex(cs[:, :32], cs[:, 32:])

        def rotated(x, z):
            x = x.double()
            v = torch.view_as_complex(x.reshape(*x.shape[:-1], 32, 2).contiguous()) if s["inter"] else torch.complex(x[..., :32].contiguous(), x[..., 32:].contiguous())
            v = torch.view_as_real(v * z)
            return v.flatten(-2) if s["inter"] else torch.cat([v[..., 0], v[..., 1]], -1)

        cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].cpu()
        for b, T in enumerate(lens):
            lo, hi = cu[b], cu[b + 1]
            if lo == hi:
                continue
            pos = torch.arange(T - (hi - lo), T)
            z = turn[pos.cuda()]
            rows = torch.cat([s["c_kv"][lo:hi].double(), rotated(s["k_rope"][lo:hi], z)], 1)
            kv[table[b][pos // PAGE].long().cuda(), (pos % PAGE).cuda()] = rows
            q_out[lo:hi] = rotated(s["q_rope"][lo:hi], z[:, None])
        return [kv, q_out]
    B, s_q, H, _ = s["q"].shape
    out = torch.zeros(B, s_q, H, D_C, dtype=torch.float64, device="cuda")
    lse = torch.full((B, s_q, H), -math.inf, dtype=torch.float64, device="cuda")
    lens, table = s["lens"].tolist(), s["table"].cpu().long()
    shared = s["op"] == "shared"
    pre = s["kv"][s["prefix_table"].long()].double().reshape(-1, D_ROW)[:s["sizes"][0]] if shared else None
    for b, T in enumerate(lens):
        n = -(-T // PAGE)
        if shared:
            rows = torch.cat([pre, s["kv"][table[b, :n].cuda()].double().reshape(-1, D_ROW)[:T]])
            where = torch.arange(rows.shape[0], device="cuda")
        else:
            keep = torch.nonzero(table[b, :n] >= 0).squeeze(1)
            rows = s["kv"][table[b, keep].cuda()].double().reshape(-1, D_ROW)
            where = (keep[:, None] * PAGE + torch.arange(PAGE)).reshape(-1).cuda()
        total = (s["sizes"][0] if shared else 0) + T
        for i in range(s_q):
            at = total - s_q + i
            see = where <= at
            if not shared:
                see &= (where < s["sinks"]) | (where > at - s["window"])
            if at < 0 or not bool(see.any()):
                continue
            keys = rows[see]
            y = s["q"][b, i].double() @ keys.t() * SCALE
            lse[b, i] = torch.logsumexp(y, -1)
            out[b, i] = torch.exp(y - lse[b, i][:, None]) @ keys[:, :D_C]
    return [out, lse]

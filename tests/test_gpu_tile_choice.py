"""The row tile of a shared-prefix decode does not follow the spare columns of a block table: a
server's table is as wide as its longest allowed sequence, its sequences are not.  The choice
shows in the bits (each tile width sums in an order of its own), and at these sizes no width
lets the call's row tiles be merged by clusters, so equal bits mean the same tile."""
import numpy as np
import pytest
import torch

import mla_latent_kv_22_b200 as M

pytestmark = pytest.mark.gpu


def shared_call(B, H, prefix, most, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = np.random.default_rng(seed).integers(1, most + 1, B)
    own, first = -(-lens // 64), -(-prefix // 64)
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()
    kv = torch.randn(first + int(own.sum()), 64, 576, generator=g, device="cuda").bfloat16()
    q = torch.randn(B, H, 576, generator=g, device="cuda").bfloat16()
    at = first + np.concatenate([[0], np.cumsum(own)])

    def call(columns):
        table = np.full((B, columns), -1)
        for b in range(B):
            table[b, :own[b]] = np.arange(at[b], at[b + 1])
        out, lse = torch.empty(B, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(B, H, device="cuda")
        M.mla_decode_shared(q, kv, i32(np.arange(first)), i32([prefix]), i32(table), i32(lens), out, lse, 192 ** -0.5)
        assert M.mla_get_device_error() == 0
        return out, lse

    return call, int(own.max())


@pytest.mark.parametrize("B,H,prefix,most", [(32, 16, 4000, 300), (64, 16, 4096, 200), (43, 16, 9000, 90)])
def test_spare_table_columns_do_not_change_the_tile(B, H, prefix, most):
    call, columns = shared_call(B, H, prefix, most, seed=B)
    exact = call(columns)
    bits = {}
    for tile in (16, 32, 128):
        M.mla_set_knob("row_tile", tile)
        try:
            bits[tile] = call(columns)[1]
        finally:
            M.mla_set_knob("row_tile", 0)
    assert sum(torch.equal(b, exact[1]) for b in bits.values()) == 1   # the bits tell the tiles apart
    for wide in (512, 2048):
        got = call(wide)
        assert torch.equal(got[0], exact[0]) and torch.equal(got[1], exact[1]), f"{wide} columns"

"""mla_append reads vectors that share memory (broadcast inputs), and refuses to write any that do.
CPU only: the refusals come before anything is launched."""
import pytest

import mla_latent_kv_22_b200 as M
from test_abi import _append


@pytest.mark.parametrize("token,head,N,H", [(0, 64, 4, 16), (1024, 0, 4, 16), (56, 1024, 2, 2), (1024, 32, 1, 2), (-56, 64, 2, 1),
                                            (0, 0, 3, 1)])
def test_overlapping_query_outputs_are_refused(token, head, N, H):
    assert _append(st=(512, 64, 1024, 64, token, head), N=N, H=H) == 1
    assert b"overlap" in M.lib.mla_last_error_message()


# What is in order gets as far as the next check, of alignment.
@pytest.mark.parametrize("st,N,H", [
    ((512, 64, 1024, 64, 1024, 64), 4, 16), ((512, 64, 1024, 64, 64, 256), 4, 16),   # heads outside tokens
    ((512, 64, 0, 0, 1024, 64), 4, 16), ((0, 0, 1024, 64, 1024, 64), 4, 16),         # broadcast inputs
    ((512, 64, 1024, 64, 0, 64), 1, 16), ((512, 64, 1024, 64, 64, 0), 4, 1),         # the stride of a single one
])
def test_other_strides_are_not(st, N, H):
    assert _append(st=st, N=N, H=H, kv=24) == 1
    assert b"16-byte aligned" in M.lib.mla_last_error_message()

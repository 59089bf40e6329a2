"""Softmax scales that float32 cannot hold once the key scale has joined them are
refused (a zero factor would make NaN of masked scores). Host checks only."""
import ctypes

import pytest

import paged_kv_gqa_row_gb300 as lnk
from paged_kv_gqa_row_gb300.binding import raw_status

LNK_OK, LNK_EINVAL, LNK_ERANGE = 0, 1, 2


def status(**kw):
    """What a call of no tokens makes of the descriptor."""
    desc = lnk.attn_desc(8, 2, 128, 4, 1, 4, **kw)
    rope = lnk.rope_desc(1e4)
    return raw_status("lnk_paged_append_rope", ctypes.byref(desc), ctypes.byref(rope), *[None] * 9, 0.0, *[None] * 3, 0, None,
                      None)


@pytest.mark.parametrize("kv", [lnk.KV_E4M3, lnk.KV_E2M1])
@pytest.mark.parametrize("scale,k_scale,want", [(0.0, 1e-45, LNK_ERANGE), (1e-30, 1e-20, LNK_ERANGE), (1e30, 1e20, LNK_ERANGE),
                                                (0.0, 1e-36, LNK_OK), (1e-30, 1e-6, LNK_OK), (1e30, 1e6, LNK_OK),
                                                (0.0, 1.0, LNK_OK), (0.0, 0.0, LNK_EINVAL)])
def test_scales_of_quantized_pools(kv, scale, k_scale, want):
    assert status(kv_dtype=kv, scale=scale, k_scale=k_scale) == want


@pytest.mark.parametrize("scale,want", [(0.0, LNK_OK), (1e-37, LNK_OK), (1e38, LNK_OK), (3.4e38, LNK_ERANGE),
                                        (float("inf"), LNK_ERANGE), (float("nan"), LNK_EINVAL), (-1.0, LNK_EINVAL)])
def test_scales_of_bf16_pools(scale, want):
    assert status(scale=scale, k_scale=0.0) == want

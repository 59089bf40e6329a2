"""Attention over 4-bit pools where what matters has small softmax weights: one key
takes nearly all of the weight and its value is zero, so that the output is what the
other keys, whose weights are 2^-LEVEL of it, add up to.

Tolerance: the output is rounded to bf16 (half a step, 2^-8 of it), a weight to 11
bits (2^-11 of it; all values here have one sign), the exponents are float32 (levels
of up to 26: 2^-19) and so are the sums of up to 1000 equal terms (2^-14): 2^-8 +
2^-10."""
import numpy as np
import pytest

from harness import to_bits
from oracle import bf16 as obf16
from oracle import fp4 as ofp4
from test_gpu_fp4 import d8, d16, d32

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def pool_of(ones, d):
    """Pool bytes of one kv head: ones in the elements of `ones` [slots, d], else zeros
    (code 2 stands for 1, and the scale code 0x38 too)."""
    n = ones.shape[0]
    codes = np.where(ones, 2, 0).astype(np.uint8).reshape(1, n, d)
    return ofp4.pack_pool(codes, np.full((1, n, d // 16), 0x38, dtype=np.uint8))


def problem(n, d, level, heavy):
    """n keys, all zero but one at `heavy`, with a query that scores it `level` in
    log2 units; the values are ones, zero at `heavy`."""
    pages = -(-n // 64)
    keys, values = np.zeros((pages * 64, d), dtype=bool), np.zeros((pages * 64, d), dtype=bool)
    keys[heavy, 0] = True
    values[:n] = True
    values[heavy] = False
    q = np.zeros((1, d))
    q[0, 0] = 1.0
    scale = np.float32(level * np.log(2.0))  # the score of the heavy key
    want = np.exp(-float(scale)) * (n - 1) / (1.0 + np.exp(-float(scale)) * (n - 1))
    return pages, keys, values, obf16.from_f64(q), float(scale), want


def check(got_bits, want, what):
    got = obf16.to_f64(got_bits)
    assert np.abs(got / want - 1.0).max() <= 2.0 ** -8 + 2.0 ** -10, f"{what}: {got.flat[0]:.6g} for {want:.6g}"


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("n,heavy,level", [(64, 0, 26.3), (64, 63, 20.6), (1000, 3, 25.7), (1000, 700, 17.2)])
def test_decode_adds_up_small_weights(d, n, heavy, level):
    import paged_kv_gqa_row_gb300 as lnk
    pages, keys, values, q, scale, want = problem(n, d, level, heavy)
    kp, vp = (d8(pool_of(x, d)) for x in (keys, values))
    # (enough rows that a warp takes about 16 pages, all of a row, on end)
    rows = 1700 if n > 64 else 3
    desc = lnk.attn_desc(1, 1, d, pages, rows, pages, scale=scale, kv_dtype=lnk.KV_E2M1)
    ws_bytes = lnk.lnk_paged_workspace_size(desc, rows)
    ws = torch.zeros(ws_bytes, dtype=torch.uint8, device="cuda")
    out = torch.zeros((rows, 1, d), dtype=torch.int16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lnk.lnk_paged_decode_attn(desc, d16(np.repeat(q[None], rows, 0)), d32([n - 1] * rows), d32([np.arange(pages)] * rows), kp,
                              vp, out, rows, ws, ws_bytes, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    check(to_bits(out), want, f"{n} keys at 2^-{level}")


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("n,heavy,level", [(64, 0, 20.6), (200, 3, 19.7), (1000, 130, 20.6), (1000, 900, 18.4),
                                           (300, 290, 7.95)])
def test_chunks_add_up_small_weights(d, n, heavy, level):
    import paged_kv_gqa_row_gb300 as lnk
    pages, keys, values, q, scale, want = problem(n, d, level, heavy)
    kp, vp = (d8(pool_of(x, d)) for x in (keys, values))
    desc = lnk.attn_desc(1, 1, d, pages, 1, pages, scale=scale, kv_dtype=lnk.KV_E2M1)
    out = torch.zeros((3, 1, d), dtype=torch.int16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lnk.lnk_paged_step_attn(desc, d16(np.repeat(q[None], 3, 0)), d32([0] * 3), d32([n - 1] * 3), None, None,
                            d32([np.arange(pages)]), kp, vp, out, None, None, 3, 0, 0, None, 0, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    check(to_bits(out), want, f"{n} keys at 2^-{level}")

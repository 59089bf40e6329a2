"""QK-norm of heads of very small and very large magnitude, with norm_eps = 0 (with
an epsilon of the usual size small heads meet no such sums of squares)."""
import numpy as np
import pytest

import synth
from harness import assert_ulp_close, to_bits
from oracle import bf16 as obf16
from oracle import fp4 as ofp4
from oracle import rope as orope
from test_gpu_fp4 import d8, d16, d32, u8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def heads_of_magnitudes(seed, tokens, heads, d, low, high):
    """Normal rows scaled by 2^low .. 2^high, one power a head."""
    x = obf16.to_f64(synth.tensor_bf16(seed, 0, (tokens, heads, d)))
    powers = np.random.RandomState(seed).randint(low, high + 1, (tokens, heads, 1))
    return obf16.from_f64(x * np.exp2(powers.astype(np.float64)))


def append(q, k, positions, pools, gamma, size, kind="KV_E2M1"):
    """Appends `size` tokens a call, token t to slot t; returns q_out's bits."""
    import paged_kv_gqa_row_gb300 as lnk
    tokens, hq, d = q.shape
    hkv = k.shape[1]
    pages = tokens // 64 + 1
    desc = lnk.attn_desc(hq, hkv, d, pages, 1, 1, kv_dtype=getattr(lnk, kind), k_scale=0.25, v_scale=0.25)
    got = []
    for a in range(0, tokens, size):
        z = min(tokens, a + size)
        q_out = torch.full((z - a, hq, d), 0x55, dtype=torch.int16, device="cuda")
        lnk.lnk_paged_append_rope(desc, lnk.rope_desc(1e4), d16(q[a:z]), d16(k[a:z]), d16(k[a:z]), d32(positions[a:z]), None,
                                  d32(np.arange(a, z)), None, d16(gamma), d16(gamma), 0.0, pools[0], pools[1], q_out, z - a)
        torch.cuda.synchronize()
        got.append(to_bits(q_out))
    return np.concatenate(got)


@pytest.mark.parametrize("low,high", [(-100, -40), (-75, -45), (55, 64), (-100, 120)])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (6, 6, 96), (5, 5, 64)])
def test_large_and_small_launches_agree_at_any_magnitude(hq, hkv, d, low, high):
    tokens = 400
    q = heads_of_magnitudes(1000 + d + low, tokens, hq, d, low, high)
    k = heads_of_magnitudes(2000 + d + high, tokens, hkv, d, low, high)
    q[5, 1] = 0
    k[7, 0] = 0
    positions = np.arange(tokens) * 7
    gamma = obf16.from_f64(1 + 0.1 * np.random.RandomState(d).standard_normal(d))
    results = []
    for size in (tokens, 50):
        pools = [d8(np.zeros((hkv, tokens // 64 + 1, 36 * d))) for _ in range(2)]
        results.append((append(q, k, positions, pools, gamma, size), u8(pools[0])))
    for large, small in zip(*results):
        assert np.array_equal(large, small), f"{int(np.sum(large != small))} of {large.size} differ"


@pytest.mark.parametrize("size", [400, 50])
@pytest.mark.parametrize("kind", ["KV_E2M1", "KV_BF16"])
def test_heads_in_the_stated_range_match_the_oracle(kind, size):
    """Mean squares of 2^-96 to 2^120."""
    tokens, hq, hkv, d = 400, 8, 2, 128
    q, k = (heads_of_magnitudes(s, tokens, h, d, -46, 58) for s, h in ((1, hq), (2, hkv)))
    positions = np.arange(tokens) * 7
    gamma = obf16.from_f64(1 + 0.1 * np.random.RandomState(3).standard_normal(d))
    inv = orope.inv_freq(1e4, d)
    want = [np.stack([orope.rotate(orope.qk_norm(obf16.to_f64(x[t]), obf16.to_f64(gamma), 0.0), orope.angles(int(p), inv))
                      for t, p in enumerate(positions)]) for x in (q, k)]
    four = kind == "KV_E2M1"
    pages = tokens // 64 + 1
    pools = [d8(np.zeros((hkv, pages, 36 * d))) if four else d16(np.zeros((hkv, pages * 64, d), dtype=np.uint16))
             for _ in range(2)]
    got = append(q, k, positions, pools, gamma, size, kind)
    assert_ulp_close(got, obf16.from_f64(want[0]), "q_out")
    if four:
        codes, scales = ofp4.quantize(obf16.from_f64(want[1]), 0.25)
        page = np.zeros((hkv, pages, 36 * d), dtype=np.uint8)
        for t in range(tokens):
            for h in range(hkv):
                ofp4.write_row(page[h, t // 64], t % 64, codes[t, h], scales[t, h])
        assert np.array_equal(u8(pools[0]), page)
    else:
        assert_ulp_close(to_bits(pools[0])[:, :tokens].transpose(1, 0, 2), obf16.from_f64(want[1]), "keys")

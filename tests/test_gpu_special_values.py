"""Queries and keys that hold NaN or infinities (a broken activation) through the
append, in every pool type and launch form: such an element shows in what is
stored and returned, and touches nothing but its own pair of elements (with
QK-norm: its own head).

The expectation is the rotation's expression in float64, with IEEE's rules for
infinities and NaN; finite results beyond bf16's range are infinite."""
import numpy as np
import pytest

import synth
from harness import assert_ulp_close, to_bits
from oracle import bf16 as obf16
from oracle import fp4 as ofp4
from oracle import fp8 as ofp8
from oracle import rope as orope
from test_gpu_fp4 import d8, d16, d32, u8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

THETA = 1e4
BF16_OVERFLOW = (2.0 - 2.0 ** -8) * 2.0 ** 127  # rounds to infinity from here on
SPECIALS = np.array([0x7FC0, 0xFFC1, 0x7F81, 0x7F80, 0xFF80, 0x7F7F, 0xFF7F], dtype=np.uint16)
NANS = 3  # of SPECIALS; then +-infinity and the largest finite values


def rotated(bits, positions, inv, gamma=None, eps=1e-6):
    """float64 results [T, H, D]; with QK-norm a head that is not finite, or whose sum
    of squares is beyond float32, is NaN."""
    x = obf16.to_f64(bits)
    out = np.empty_like(x)
    with np.errstate(all="ignore"):
        for t, p in enumerate(positions):
            xt = x[t]
            if gamma is not None:
                broken = ~((xt * xt).sum(-1) < 2.0 ** 128)
                xt = np.where(broken[:, None], np.nan, orope.qk_norm(np.where(broken[:, None], 1.0, xt), gamma, eps))
            out[t] = orope.rotate(xt, orope.angles(int(p), inv))
    return out


def want_bits(values):
    """bf16 bits of float64 values (NaN as 0x7FC0)."""
    finite = np.abs(values) < BF16_OVERFLOW
    bits = obf16.from_f64(np.where(finite, values, 0.0))
    special = np.where(np.isnan(values), 0x7FC0, np.where(values > 0, 0x7F80, 0xFF80)).astype(np.uint16)
    return np.where(finite, bits, special)


def check_bits(got, values, what):
    want = want_bits(values)
    finite = np.abs(values) < BF16_OVERFLOW
    nan = np.isnan(values)
    assert np.array_equal(np.isnan(obf16.to_f64(got)), nan), f"{what}: NaN where it should not be, or the reverse"
    inf = ~finite & ~nan
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities"
    assert_ulp_close(np.where(finite, got, 0), np.where(finite, want, 0), what)


def poison(bits, rng, specials, tokens):
    """A special value in one element of one head of each of `tokens`."""
    _, heads, d = bits.shape
    for i, t in enumerate(tokens):
        bits[t, rng.randint(heads), rng.randint(d)] = specials[i % len(specials)]


def inputs(seed, tokens, hq, hkv, d, specials, every, first_position=1):
    rng = np.random.RandomState(seed)
    q, k, v = (synth.tensor_bf16(seed, i, (tokens, h, d)) for i, h in enumerate((hq, hkv, hkv)))
    where = range(0, tokens, every)
    poison(q, rng, specials, where)
    poison(k, rng, specials, where)
    positions = rng.randint(first_position, 5000, tokens)
    positions[0] = first_position
    if first_position == 0:  # every other poisoned token: sines of zero
        positions[::2 * every] = 0
    return q, k, v, positions, rng


def append(kind, q, k, v, positions, slots, pages, gamma, pools, scales):
    """Returns q_out's bits; the pools are written."""
    import paged_kv_gqa_row_gb300 as lnk
    t, hq, d = q.shape
    hkv = k.shape[1]
    dtype = {"bf16": lnk.KV_BF16, "e4m3": lnk.KV_E4M3, "e2m1": lnk.KV_E2M1}[kind]
    desc = lnk.attn_desc(hq, hkv, d, pages, 1, 1, kv_dtype=dtype, k_scale=scales[0], v_scale=scales[1])
    q_out = torch.full((t, hq, d), 0x55, dtype=torch.int16, device="cuda")
    gq, gk = (None, None) if gamma is None else (d16(g) for g in gamma)
    lnk.lnk_paged_append_rope(desc, lnk.rope_desc(THETA), d16(q), d16(k), d16(v), d32(positions), None, d32(slots), None,
                              gq, gk, 1e-6, pools[0], pools[1], q_out, t)
    torch.cuda.synchronize()
    return to_bits(q_out)


def check_append(kind, tokens, hq, hkv, d, norm, specials, every, seed, scales=(0.25, 0.5), first_position=1):
    q, k, v, positions, rng = inputs(seed, tokens, hq, hkv, d, specials, every, first_position)
    inv = orope.inv_freq(THETA, d)
    gamma = [obf16.from_f64(1 + 0.1 * rng.standard_normal(d)) for _ in range(2)] if norm else None
    g64 = (None, None) if gamma is None else [obf16.to_f64(g) for g in gamma]
    pages = tokens // 64 + 1
    slots = rng.permutation(pages * 64)[:tokens]
    shape, dtype = {"bf16": ((hkv, pages * 64, d), np.uint16), "e4m3": ((hkv, pages * 64, d), np.uint8),
                    "e2m1": ((hkv, pages, 36 * d), np.uint8)}[kind]
    blank = np.zeros(shape, dtype=dtype)
    pools = [d16(blank) if kind == "bf16" else d8(blank) for _ in range(2)]
    got_q = append(kind, q, k, v, positions, slots, pages, gamma, pools, scales)
    check_bits(got_q, rotated(q, positions, inv, g64[0]), "q_out")
    values = rotated(k, positions, inv, g64[1])
    assert np.isnan(values).any()
    if kind == "bf16":
        check_bits(to_bits(pools[0])[:, slots].transpose(1, 0, 2), values, "stored keys")
    elif kind == "e4m3":
        got = u8(pools[0])[:, slots].transpose(1, 0, 2)
        nan = np.isnan(values)
        assert np.array_equal((got & 0x7F) == 0x7F, nan), "NaN codes"
        with np.errstate(all="ignore"):
            u = obf16.to_f64(want_bits(np.where(nan, 0.0, values))).astype(np.float32) / np.float32(scales[0])
        assert np.array_equal(got[~nan], ofp8.encode(u.astype(np.float64))[~nan]), "codes"
    else:
        want = blank.copy()
        codes, scale_codes = ofp4.quantize(want_bits(values), scales[0])
        for t in range(tokens):
            for h in range(hkv):
                ofp4.write_row(want[h, slots[t] // 64], slots[t] % 64, codes[t, h], scale_codes[t, h])
        assert np.isin(0x7F, scale_codes)
        got = u8(pools[0])
        assert np.array_equal(got, want), f"K bytes: {int(np.sum(got != want))} differ"


# launches of few tokens (heads split over CTAs), one CTA a token, and wide ones
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("tokens,hq,hkv,d", [(9, 8, 2, 128), (60, 6, 6, 96), (200, 8, 2, 64), (1500, 4, 1, 128)])
def test_special_queries_and_keys_in_the_append(kind, tokens, hq, hkv, d, norm):
    specials = SPECIALS[:NANS] if kind == "e2m1" and tokens > 70 else SPECIALS
    check_append(kind, tokens, hq, hkv, d, norm, specials, 3, 5000 + tokens + d)


@pytest.mark.parametrize("norm", [False, True])
def test_special_keys_with_a_pool_scale_that_is_no_power_of_two(norm):
    check_append("e2m1", 300, 8, 4, 128, norm, SPECIALS[:NANS], 2, 77, scales=(0.37, 1.9))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("norm", [False, True])
def test_the_one_kernel_decode_step_keeps_special_values(kv, norm):
    """Bit for bit the append's queries and keys, NaN and infinities among them."""
    import paged_kv_gqa_row_gb300 as lnk
    rows, hq, hkv, d = 16, 16, 8, 128
    q, k, v, positions, rng = inputs(88, rows, hq, hkv, d, SPECIALS, 2)
    positions = positions % 60 + 1
    table = np.arange(rows)[:, None]
    dtype = lnk.KV_BF16 if kv == "bf16" else lnk.KV_E4M3
    desc = lnk.attn_desc(hq, hkv, d, rows, rows, 1, kv_dtype=dtype)
    assert lnk.lnk_paged_decode_step_launches(desc, rows) == 1
    gq, gk = (d16(obf16.from_f64(1 + 0.1 * rng.standard_normal(d))) for _ in range(2)) if norm else (None, None)
    ws_bytes = lnk.lnk_paged_workspace_size(desc, rows)
    ws = torch.zeros(ws_bytes, dtype=torch.uint8, device="cuda")
    results = []
    for fused in (True, False):
        pools = [torch.zeros((hkv, rows * 64, d), dtype=torch.int16 if kv == "bf16" else torch.uint8, device="cuda")
                 for _ in range(2)]
        q_out, out = (torch.zeros((rows, hq, d), dtype=torch.int16, device="cuda") for _ in range(2))
        args = (d16(q), d16(k), d16(v), d32(positions))
        if fused:
            lnk.lnk_paged_decode_step(desc, lnk.rope_desc(THETA), *args, d32(table), gq, gk, 1e-6, *pools, q_out, out, rows,
                                      ws, ws_bytes)
        else:
            lnk.lnk_paged_append_rope(desc, lnk.rope_desc(THETA), *args, None, None, d32(table), gq, gk, 1e-6, *pools, q_out,
                                      rows)
        torch.cuda.synchronize()
        results.append((q_out, *pools))
    for one, two in zip(*results):
        assert torch.equal(one, two)
    gamma = None if gq is None else obf16.to_f64(to_bits(gq))
    check_bits(to_bits(results[0][0]), rotated(q, positions, orope.inv_freq(THETA, d), gamma), "q_out")


@pytest.mark.parametrize("scales", [(0.25, 0.5), (0.37, 1.9)])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("tokens,hq,hkv,d", [(80, 6, 6, 96), (400, 8, 2, 64), (1500, 4, 1, 128)])
def test_infinities_in_large_launches_over_4_bit_pools(tokens, hq, hkv, d, norm, scales):
    """Position 0 among them, where an infinity meets coefficients that are exactly zero."""
    check_append("e2m1", tokens, hq, hkv, d, norm, SPECIALS, 3, 6000 + tokens + d, scales, first_position=0)


@pytest.mark.parametrize("norm", [False, True])
def test_large_and_small_launches_store_the_same_special_heads(norm):
    """Special values among heads of which a few in a hundred are near a rounding
    border: the same bytes whichever form the launch takes."""
    tokens, hq, hkv, d = 600, 8, 4, 128
    q, k, v, positions, rng = inputs(91, tokens, hq, hkv, d, SPECIALS, 1, first_position=0)
    gamma = [obf16.from_f64(1 + 0.1 * rng.standard_normal(d)) for _ in range(2)] if norm else None
    pages = 10
    slots = rng.permutation(pages * 64)[:tokens]
    results = []
    for size in (tokens, 40):
        pools = [d8(np.zeros((hkv, pages, 36 * d))) for _ in range(2)]
        got = [append("e2m1", q[a:a + size], k[a:a + size], v[a:a + size], positions[a:a + size], slots[a:a + size], pages,
                      gamma, pools, (0.25, 0.5)) for a in range(0, tokens, size)]
        results.append((np.concatenate(got), u8(pools[0]), u8(pools[1])))
    for large, small in zip(*results):
        assert np.array_equal(large, small)

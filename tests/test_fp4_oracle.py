"""The oracle's 4-bit pools (oracle/fp4.py) pinned to facts that do not come
from it, and the library's host-side answers about such pools (no GPU)."""
import numpy as np
import pytest

from oracle import bf16, fp4, fp8


def test_the_sixteen_codes():
    want = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert fp4.decode(np.arange(16)).tolist() == want + [-x for x in want]
    assert np.signbit(fp4.decode(8))


def test_every_code_and_every_border_round_to_nearest_even():
    values = fp4.decode(np.arange(8))
    assert fp4.encode(values).tolist() == list(range(8))
    assert fp4.encode(-values).tolist() == [8 + c for c in range(8)]
    for c in range(7):
        middle = (values[c] + values[c + 1]) / 2
        assert fp4.encode(middle) == (c if c % 2 == 0 else c + 1)
        assert fp4.encode(middle - 1e-9) == c and fp4.encode(middle + 1e-9) == c + 1
    assert fp4.encode(np.array([6.1, 1e30, np.inf, -np.inf])).tolist() == [7, 7, 7, 15]


def test_a_block_by_hand():
    # the largest magnitude 12 gives the scale 2 exactly; elements divide by 2
    x = np.array([12, -12, 6, 5, 1, 0.5, 0.4, 0, 3, 3.5, 7, -2.5, 9, 10, 11, -1])
    codes, scales = fp4.quantize(bf16.from_f64(x), 1.0)
    assert fp8.decode(scales).tolist() == [2.0]
    # 2.5 -> 2 (even), 0.25 -> 0 (even), 0.2 -> 0, 1.75 -> 2 (even), 3.5 -> 4 (even), -1.25 -> -1 (even),
    # 4.5 -> 4, 5 -> 4 (even), 5.5 -> 6
    want = [6, -6, 3, 2, 0.5, 0, 0, 0, 1.5, 2, 4, -1, 4, 4, 6, -0.5]
    assert fp4.decode(codes).tolist() == want
    assert fp4.row_values(codes, scales, 1.0).tolist() == [2 * w for w in want]


def test_scales_saturate_vanish_and_carry_nan():
    x = np.zeros(32)
    x[0], x[16] = 1e6, 1e-6
    codes, scales = fp4.quantize(bf16.from_f64(x), 1.0)
    assert scales.tolist() == [0x7E, 0] and codes[0] == 7 and not codes[1:].any()
    bits = bf16.from_f64(np.ones(32))
    bits[3] = 0x7FC0
    codes, scales = fp4.quantize(bits, 1.0)
    assert scales[0] == fp4.NAN_SCALE and np.isnan(fp4.row_values(codes, scales, 1.0)[:16]).all()
    assert np.isfinite(fp4.row_values(codes, scales, 1.0)[16:]).all()


def test_an_element_is_off_by_half_a_step_of_its_block():
    # half a step of E2M1 is at most 1 (between 4 and 6) times the scale, and a scale
    # that was rounded down by half a step of E4M3 (1/16 relative) saturates the largest
    # element by at most 6/16 of it
    rng = np.random.RandomState(5)
    x = bf16.to_f64(bf16.from_f64(rng.standard_normal((200, 64))))
    codes, scales = fp4.quantize(bf16.from_f64(x), 0.5)
    got = fp4.row_values(codes, scales, 0.5)
    step = np.repeat(fp8.decode(scales), 16, axis=-1) * 0.5
    assert np.all(np.abs(got - x) <= step * (1 + 1e-6))
    assert np.linalg.norm(got - x) / np.linalg.norm(x) < 0.12


@pytest.mark.parametrize("d", [64, 96, 128])
def test_rows_of_a_page_are_written_and_read_in_their_own_bytes(d):
    rng = np.random.RandomState(d)
    page = np.full(36 * d, 0xA5, dtype=np.uint8)
    rows = [(rng.randint(0, 16, d).astype(np.uint8), rng.randint(0, 127, d // 16).astype(np.uint8)) for _ in range(64)]
    for j in rng.permutation(64):
        fp4.write_row(page, j, *rows[j])
    for j in range(64):
        codes, scales = fp4.read_row(page, j)
        assert np.array_equal(codes, rows[j][0]) and np.array_equal(scales, rows[j][1])
    # 64 rows fill all of the page's bytes
    codes, scales = np.stack([r[0] for r in rows])[None], np.stack([r[1] for r in rows])[None]
    assert np.array_equal(fp4.pack_pool(codes, scales)[0, 0], page)
    assert np.array_equal(fp4.pool_values(page[None, None], 0.25)[0], fp4.row_values(codes[0], scales[0], 0.25))


def test_page_bytes_and_descriptor_checks():
    lnk = pytest.importorskip("paged_kv_gqa_row_gb300")
    for d in (64, 96, 128):
        for dtype, want in ((lnk.KV_BF16, 128 * d), (lnk.KV_E4M3, 64 * d), (lnk.KV_E2M1, 36 * d)):
            assert lnk.lnk_paged_page_bytes(lnk.attn_desc(4, 2, d, 6, 1, 6, kv_dtype=dtype)) == want
    for bad in (dict(kv_dtype=2), dict(kv_dtype=3), dict(kv_dtype=5), dict(k_scale=0.0), dict(v_scale=-1.0),
                dict(k_scale=float("nan")), dict(v_scale=float("inf"))):
        args = dict(kv_dtype=lnk.KV_E2M1)
        args.update(bad)
        assert lnk.lnk_paged_page_bytes(lnk.attn_desc(4, 2, 96, 6, 1, 6, **args)) == 0


def test_read_tokens_refuses_bad_arguments_without_a_launch():
    lnk = pytest.importorskip("paged_kv_gqa_row_gb300")
    d = lnk.attn_desc(4, 2, 96, 6, 3, 6, kv_dtype=lnk.KV_E2M1)

    def status(*args):
        try:
            lnk.lnk_paged_read_tokens(*args, stream=0)
        except lnk.LnkError as e:
            return e.status
        return 0

    good = [d, 16, 16, 16, 16, None, 16, 16, 16, 0]
    assert status(*good) == 0  # no tokens: nothing is enqueued
    einval, eunsupported = 1, 4

    def changed(**kw):
        names = ["desc", "k_pool", "v_pool", "positions", "rows", "slots", "table", "k_out", "v_out", "T"]
        args = dict(zip(names, good), T=2)
        args.update(kw)
        return [args[n] for n in names]

    for kw in (dict(T=-1), dict(positions=None), dict(table=None), dict(k_out=None, v_out=None), dict(k_pool=None),
               dict(v_pool=None), dict(k_pool=8), dict(v_out=8), dict(rows=None, T=4)):
        assert status(*changed(**kw)) == einval, kw
    bad = lnk.attn_desc(4, 2, 80, 6, 3, 6, kv_dtype=lnk.KV_E2M1)
    assert status(*changed(desc=bad)) == eunsupported


def test_a_step_with_chunks_refuses_outputs_off_16_bytes_without_a_launch():
    lnk = pytest.importorskip("paged_kv_gqa_row_gb300")
    einval, eworkspace = 1, 5
    for kind in (lnk.KV_BF16, lnk.KV_E2M1):
        d = lnk.attn_desc(4, 2, 96, 6, 3, 6, kv_dtype=kind)

        def status(out, P, B, **kw):
            args = dict(q=16, k_pool=16, v_pool=16)
            args.update(kw)
            try:
                lnk.lnk_paged_step_attn(d, args["q"], 16, 16, None, 16, 16, args["k_pool"], args["v_pool"], out, None, None,
                                        P, B, 0, None, 0, None, 0)
            except lnk.LnkError as e:
                return e.status
            return 0

        assert status(24, 1, 0) == einval  # the chunks' rows are stored 16 bytes at a time
        assert status(24, 0, 1) == eworkspace  # decode rows alone: 8 bytes are enough, the workspace is missing
        assert status(20, 0, 1) == einval
        assert status(16, 1, 1) == eworkspace
        assert status(16, 1, 0, q=24) == einval and status(16, 1, 0, v_pool=8) == einval

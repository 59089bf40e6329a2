"""Attention over 4-bit (E2M1) pools against exact attention of the values that
the pool holds (oracle/fp4.py).

Tolerance, per output element, from the roundings on the way (all of them
relative to exact arithmetic on the same pool):
  * the result is rounded to bf16: 2^-8 |out|;
  * the probabilities are rounded to f16 on their way into the product with V:
    2^-11 of A = sum p |v| / sum p;
  * an f16 probability below 2^-14 of the largest is subnormal: at most 2^-25
    each, n keys of at most max|v|;
  * scores and sums are float32 (products of 8 and 5 significant bits are exact
    in it), the exponentials are good to 2^-22: together well below 2^-12 of A
    for scores of this size, and as much again is allowed.
"""
import zlib

import numpy as np
import pytest

import synth
from harness import assert_ulp_close, to_bits
from oracle import bf16 as obf16
from oracle import fp4 as ofp4
from oracle import paged as opaged
from test_gpu_fp4 import K_SCALE, V_SCALE, F4Step, d8, d32, oracle_append, u8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def check_token(got_bits, q_bits, row, position, table, k_values, v_values, window, what, scale=None):
    """One token's outputs [Hq, D] within the bound above."""
    got = obf16.to_f64(got_bits)
    if position < 0:
        assert not got_bits.any(), f"{what}: an inactive token's output is zero"
        return
    want = ofp4.attention_at(q_bits, row, position, table, k_values, v_values, window, scale)
    spread = ofp4.attention_at(q_bits, row, position, table, k_values, np.abs(v_values), window, scale)
    lo, hi = opaged.visible_range(position, window)
    top = np.abs(v_values[:, opaged.row_slots(table, row, lo, hi)]).max()
    bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * spread + (hi - lo + 1) * 2.0 ** -25 * top
    bad = ~(np.abs(got - want) <= bound + 1e-30)
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, worst {np.abs(got - want).max():.3g} of {bound.max():.3g}"


def decode(dev, stream=None):
    w = dev.w
    dev.lnk.lnk_paged_decode_attn(dev.desc, dev.q_out[w.P:], dev.dec_positions, dev.table, dev.k_pool, dev.v_pool,
                                  dev.out[w.P:], w.B, dev.ws, dev.ws_bytes, dev.status, stream)


def check_decode(w, dev, rows=None, k_scale=K_SCALE, v_scale=V_SCALE, scale=None):
    """The rows' outputs against the pool's own bytes (which the append test pins)."""
    torch.cuda.synchronize()
    assert int(dev.status.item()) == 0
    kv = ofp4.pool_values(u8(dev.k_pool), k_scale)
    vv = ofp4.pool_values(u8(dev.v_pool), v_scale)
    out, q = to_bits(dev.out), to_bits(dev.q_out)
    for b in range(w.B) if rows is None else rows:
        check_token(out[w.P + b], q[w.P + b], b, int(w.dec_positions[b]), w.table, kv, vv, w.window,
                    f"row {b} at {w.dec_positions[b]}", scale)


DECODE_CASES = [
    ("mha64-edges", 4, 4, 64, [1, 2, 63, 64, 65, 130], 0, ()),
    ("gqa4-ragged", 8, 2, 128, [1000, 5, 64, 128, 2000, 777], 0, ()),
    ("gqa8", 16, 2, 128, [3000, 10, 4096], 0, ()),
    ("gqa8-64", 16, 2, 64, [1500, 1, 4097], 0, ()),
    ("gqa2-window2047", 8, 4, 96, [300, 2047, 2048, 2049, 2100, 5000], 2047, ()),
    ("mha96-window100", 6, 6, 96, [50, 129, 700, 101, 100], 100, ()),
    ("window1", 8, 2, 128, [1, 64, 65, 500], 1, ()),
    ("inactive-rows", 8, 2, 128, [100, 1, 257, 64], 0, (1, 3)),
    ("all-inactive", 8, 2, 128, [100, 1], 0, (0, 1)),
    ("one-row-one-key", 1, 1, 96, [1], 0, ()),
    ("one-long-row", 4, 1, 128, [20011], 0, ()),
    ("many-short-rows", 32, 8, 128, [17] * 40 + [65] * 9, 0, ()),
    ("more-pairs-than-ctas", 8, 8, 64, [1 + (37 * i) % 700 for i in range(90)], 0, (7,)),
]


@pytest.mark.parametrize("case", DECODE_CASES, ids=[c[0] for c in DECODE_CASES])
def test_append_and_decode_match_exact_attention(case):
    name, hq, hkv, d, lengths, window, inactive = case
    w = synth.custom(seed=zlib.crc32(("e2m1d" + name).encode()) % 10000, hq=hq, hkv=hkv, head_dim=d, dec_lengths=lengths,
                     window=window, inactive=inactive)
    dev = F4Step(w)
    dev.append()
    decode(dev)
    check_decode(w, dev)
    first = dev.out.clone()
    dev.out.fill_(0x7FC0)
    decode(dev)  # the workspace is as a call leaves it
    check_decode(w, dev, rows=[0])
    assert torch.equal(first, dev.out)  # partial results are merged in one order, whoever arrives last


def test_decode_ignores_what_unread_slots_hold():
    """Every byte of unread slots set, NaN scales among them: all of the last page
    behind the token, the page before the window, and pages of no row."""
    w = synth.custom(seed=78, hq=8, hkv=2, head_dim=128, dec_lengths=[5, 64, 130, 300, 1000], window=200)
    dev = F4Step(w)
    dev.append()
    decode(dev)
    check_decode(w, dev)
    clean = dev.out.clone()
    seen = np.zeros(w.pool_positions, dtype=bool)
    for b, p in enumerate(w.dec_positions):
        lo, hi = opaged.visible_range(int(p), w.window)
        seen[opaged.row_slots(w.table, b, lo, hi)] = True
    for pool in (dev.k_pool, dev.v_pool):
        host = u8(pool)
        for slot in np.nonzero(~seen)[0]:
            for h in range(w.hkv):
                ofp4.write_row(host[h, slot // 64], slot % 64, np.full(128, 15, dtype=np.uint8),
                               np.full(8, [0x7F, 0xFF, 0x7E][slot % 3], dtype=np.uint8))
        pool.copy_(d8(host))
    dev.out.fill_(0x7FC0)
    decode(dev)
    torch.cuda.synchronize()
    assert torch.equal(dev.out, clean)


@pytest.mark.parametrize("hq,hkv,d,window", [(8, 2, 128, 0), (6, 6, 96, 100), (16, 2, 64, 0)])
def test_every_code_with_every_finite_scale(hq, hkv, d, window):
    """Pools drawn from all codes and all finite scale codes, signs of scales among
    them; pool scales that keep the values at unit size."""
    w = synth.custom(seed=41 + d, hq=hq, hkv=hkv, head_dim=d, dec_lengths=[1, 64, 65, 700, 3000], window=window)
    dev = F4Step(w, k_scale=2.0 ** -9, v_scale=2.0 ** -8)
    rng = np.random.RandomState(d)
    finite = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    for pool in (dev.k_pool, dev.v_pool):
        codes = rng.randint(0, 16, (hkv, w.pool_positions, d)).astype(np.uint8)
        scales = rng.choice(finite, (hkv, w.pool_positions, d // 16))
        pool.copy_(d8(ofp4.pack_pool(codes, scales)))
    dev.q_out.copy_(dev.q)
    decode(dev)
    check_decode(w, dev, k_scale=2.0 ** -9, v_scale=2.0 ** -8)


def test_explicit_scale_and_peaked_scores():
    w = synth.custom(seed=3, hq=8, hkv=2, head_dim=128, dec_lengths=[700, 65, 1])
    dev = F4Step(w, scale=0.6)
    dev.append()
    decode(dev)
    check_decode(w, dev, scale=float(np.float32(0.6)))


def test_a_bad_page_is_skipped_and_reported():
    w = synth.custom(seed=6, hq=8, hkv=2, head_dim=96, dec_lengths=[300, 200, 64])
    dev = F4Step(w)
    dev.append()
    table = np.array(w.table)
    table[0, 1], table[1, 0], table[2, 0] = w.num_pages, -1, -5  # (row 2 has no other page)
    dev.table = d32(table)
    decode(dev)
    torch.cuda.synchronize()
    assert int(dev.status.item()) == 0x04
    kv, vv = ofp4.pool_values(u8(dev.k_pool), K_SCALE), ofp4.pool_values(u8(dev.v_pool), V_SCALE)
    out, q = to_bits(dev.out), to_bits(dev.q_out)
    # what is left: keys of the good pages, as rows of their own
    kept = [np.r_[0:64, 128:300], np.r_[64:200]]
    for b, keys in enumerate(kept):
        slots = np.array([int(w.table[b, j // 64]) * 64 + j % 64 for j in keys])
        n = len(slots)
        packed = np.zeros((1, -(-n // 64)), dtype=np.int32)
        packed[0] = np.arange(packed.shape[1])
        kc, vc = (np.zeros((w.hkv, packed.shape[1] * 64, 96)) for _ in range(2))
        kc[:, :n], vc[:, :n] = kv[:, slots], vv[:, slots]
        check_token(out[b], q[b], 0, n - 1, packed, kc, vc, 0, f"row {b}")
    assert not out[2].any()


def test_decode_step_equals_append_then_decode():
    import paged_kv_gqa_row_gb300 as lnk
    w = synth.custom(seed=12, hq=8, hkv=2, head_dim=128, dec_lengths=[100, 1, 64, 65, 900], inactive=(1,))
    one, two = F4Step(w), F4Step(w)
    assert lnk.lnk_paged_decode_step_launches(one.desc, w.B) == 2
    lnk.lnk_paged_decode_step(one.desc, one.rope, one.q, one.k, one.v, one.dec_positions, one.table, None, None, 1e-6,
                              one.k_pool, one.v_pool, one.q_out, one.out, w.B, one.ws, one.ws_bytes, one.status)
    two.append()
    decode(two)
    torch.cuda.synchronize()
    assert torch.equal(one.q_out, two.q_out) and torch.equal(one.k_pool, two.k_pool) and torch.equal(one.v_pool, two.v_pool)
    check_decode(w, one)
    q_want, kp, vp = oracle_append(w, one.k_host, one.v_host)
    assert_ulp_close(to_bits(one.q_out), q_want, "q_out")
    assert np.array_equal(u8(one.k_pool), kp) and np.array_equal(u8(one.v_pool), vp)


def test_static_scratch_and_the_step_call_serve_decode_rows():
    import paged_kv_gqa_row_gb300 as lnk
    w = synth.custom(seed=13, hq=32, hkv=8, head_dim=128, dec_lengths=[4000, 300, 64, 1, 2500])
    dev = F4Step(w)
    dev.append()
    for call in range(2):
        dev.out.fill_(0x7FC0)
        lnk.lnk_paged_decode_attn_static(dev.desc, dev.q_out, dev.dec_positions, dev.table, dev.k_pool, dev.v_pool,
                                         dev.out, w.B, dev.status)
        check_decode(w, dev, rows=[1, 2, 3])
    dev.out.fill_(0x7FC0)
    lnk.lnk_paged_step_attn(dev.desc, dev.q_out, None, None, None, dev.dec_positions, dev.table, dev.k_pool, dev.v_pool,
                            dev.out, None, None, 0, w.B, 0, dev.ws, dev.ws_bytes, dev.status)
    check_decode(w, dev, rows=[1, 3, 4])


def test_a_captured_step_replays_on_new_tokens_and_on_another_stream():
    """Append and decode captured once, replayed after the inputs in the captured
    buffers have changed, beside the same calls on a stream of their own."""
    lengths = [130, 64, 700, 1]
    w = synth.custom(seed=21, hq=8, hkv=2, head_dim=128, dec_lengths=lengths)
    dev, eager = F4Step(w), F4Step(w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dev.append()
        decode(dev)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dev.append()
        decode(dev)
    for turn in range(2):
        fresh = torch.randn(dev.q.shape, device="cuda").to(torch.bfloat16).view(torch.int16)
        for x in (dev, eager):
            x.q.copy_(fresh)
            x.out.fill_(0x7FC0)
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            eager.append(stream=side)
            decode(eager, stream=side)
        check_decode(w, dev)
        check_decode(w, eager)
        assert torch.equal(dev.k_pool, eager.k_pool) and torch.equal(dev.q_out, eager.q_out)


# ---------------------------------------------------------------- chunks ----

def step(dev, segments=True, last=None, last_out=None):
    w = dev.w
    dev.lnk.lnk_paged_step_attn(dev.desc, dev.q_out, d32(w.ch_rows), d32(w.ch_positions),
                                d32(w.ch_segments) if segments else None, dev.dec_positions if w.B else None, dev.table,
                                dev.k_pool, dev.v_pool, dev.out, last, last_out, w.P, w.B, 0 if last is None else len(last),
                                dev.ws, dev.ws_bytes, dev.status)


def check_step(w, dev, tokens=None, scale=None, k_scale=K_SCALE, v_scale=V_SCALE):
    torch.cuda.synchronize()
    assert int(dev.status.item()) == 0
    kv, vv = ofp4.pool_values(u8(dev.k_pool), k_scale), ofp4.pool_values(u8(dev.v_pool), v_scale)
    out, q = to_bits(dev.out), to_bits(dev.q_out)
    rows, positions = w.token_rows(), w.token_positions()
    for t in range(w.T) if tokens is None else tokens:
        check_token(out[t], q[t], int(rows[t]), int(positions[t]), w.table, kv, vv, w.window,
                    f"token {t} of row {rows[t]} at {positions[t]}", scale)


STEP_CASES = [
    # hq, hkv, d, decode lengths, chunks (start, tokens), window, inactive tokens
    ("gqa4-128", 8, 2, 128, [700, 65, 1], [(0, 40), (130, 25)], 0, ()),
    ("one-token-chunk", 8, 2, 128, [], [(0, 1)], 0, ()),
    ("tile-edges", 8, 2, 128, [], [(0, 64), (64, 65), (63, 130)], 0, ()),
    ("mha64", 3, 3, 64, [5], [(0, 257), (1000, 3)], 0, ()),
    ("gqa8-64", 16, 2, 64, [], [(17, 33), (0, 31), (500, 40)], 0, ()),
    ("gqa2-96-window100", 4, 2, 96, [300], [(90, 150), (0, 99), (640, 70)], 100, ()),
    ("mha96-many-steps", 2, 2, 96, [], [(900, 300)], 0, ()),
    ("gqa8-128-window1", 8, 1, 128, [], [(0, 70)], 1, ()),
    ("inactive-tokens", 8, 2, 128, [100, 30], [(0, 50), (200, 20)], 0, (3, 49, 50, 71)),
    ("many-short-chunks", 4, 1, 128, [], [(7 * i, 1 + i % 5) for i in range(40)], 0, ()),
]


@pytest.mark.parametrize("case", STEP_CASES, ids=[c[0] for c in STEP_CASES])
def test_chunks_and_decode_rows_match_exact_attention(case):
    name, hq, hkv, d, lengths, chunks, window, inactive = case
    w = synth.custom(seed=zlib.crc32(("e2m1c" + name).encode()) % 10000, hq=hq, hkv=hkv, head_dim=d, dec_lengths=lengths,
                     chunks=chunks, window=window)
    for t in inactive:
        (w.ch_positions if t < w.P else w.dec_positions)[t if t < w.P else t - w.P] = -1
    dev = F4Step(w)
    dev.append()
    step(dev)
    check_step(w, dev)
    first = dev.out.clone()
    dev.out.fill_(0x7FC0)
    step(dev, segments=False)
    torch.cuda.synchronize()
    assert torch.equal(first, dev.out)


def test_chunks_ignore_what_unread_slots_hold():
    """Slots of the chunks' pages behind their last tokens, and before the window,
    hold NaN scales."""
    w = synth.custom(seed=79, hq=8, hkv=2, head_dim=96, dec_lengths=[], chunks=[(0, 70), (300, 10), (129, 1)], window=150)
    dev = F4Step(w)
    dev.append()
    step(dev)
    check_step(w, dev)
    clean = dev.out.clone()
    seen = np.zeros(w.pool_positions, dtype=bool)
    for r, p in zip(w.token_rows(), w.token_positions()):
        lo, hi = opaged.visible_range(int(p), w.window)
        seen[opaged.row_slots(w.table, int(r), lo, hi)] = True
    for pool in (dev.k_pool, dev.v_pool):
        host = u8(pool)
        for slot in np.nonzero(~seen)[0]:
            for h in range(w.hkv):
                ofp4.write_row(host[h, slot // 64], slot % 64, np.full(96, 15, dtype=np.uint8),
                               np.full(6, [0x7F, 0xFF, 0x7E][slot % 3], dtype=np.uint8))
        pool.copy_(d8(host))
    dev.out.fill_(0x7FC0)
    step(dev)
    torch.cuda.synchronize()
    assert torch.equal(dev.out, clean)


def test_a_chunk_skips_a_bad_page_and_reports_it():
    w = synth.custom(seed=8, hq=8, hkv=2, head_dim=128, dec_lengths=[], chunks=[(200, 30), (0, 20)])
    dev = F4Step(w)
    dev.append()
    table = np.array(w.table)
    row = int(w.ch_rows[0])
    table[row, 1] = w.num_pages + 3
    dev.table = d32(table)
    step(dev)
    torch.cuda.synchronize()
    assert int(dev.status.item()) == 0x04
    kv, vv = ofp4.pool_values(u8(dev.k_pool), K_SCALE), ofp4.pool_values(u8(dev.v_pool), V_SCALE)
    out, q = to_bits(dev.out), to_bits(dev.q_out)
    for t in (0, 17, 29):
        keys = np.r_[0:64, 128:int(w.ch_positions[t]) + 1]
        slots = np.array([int(w.table[row, j // 64]) * 64 + j % 64 for j in keys])
        packed = np.arange(-(-len(keys) // 64), dtype=np.int32)[None]
        kc, vc = (np.zeros((w.hkv, packed.shape[1] * 64, 128)) for _ in range(2))
        kc[:, :len(keys)], vc[:, :len(keys)] = kv[:, slots], vv[:, slots]
        check_token(out[t], q[t], 0, len(keys) - 1, packed, kc, vc, 0, f"token {t}")
    for t in range(30, 50):
        check_token(out[t], q[t], int(w.ch_rows[t]), int(w.ch_positions[t]), w.table, kv, vv, 0, f"token {t}")


def test_a_running_maximum_that_jumps():
    """Keys whose scores climb by more than 2^8 from step to step (the rescaling of
    the accumulated output), and last tokens gathered."""
    w = synth.custom(seed=11, hq=8, hkv=2, head_dim=128, dec_lengths=[], chunks=[(600, 20), (0, 3)])
    dev = F4Step(w, scale=1.5)
    dev.append()
    last = d32([19, 22, 0])
    last_out = torch.zeros((3,) + tuple(dev.out.shape[1:]), dtype=torch.int16, device="cuda")
    step(dev, last=last, last_out=last_out)
    check_step(w, dev, scale=1.5)
    assert torch.equal(last_out, dev.out[[19, 22, 0]])


def test_a_whole_prompt_at_serving_size_sampled():
    w = synth.custom(seed=31, hq=32, hkv=8, head_dim=128, dec_lengths=[2000, 100], chunks=[(0, 700), (3000, 300)])
    dev = F4Step(w)
    dev.append()
    step(dev)
    check_step(w, dev, tokens=[0, 1, 63, 64, 255, 256, 511, 699, 700, 850, 999, 1000, 1001])

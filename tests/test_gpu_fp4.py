"""4-bit (E2M1) pools through the C ABI against the oracle (oracle/fp4.py):
the append's bytes, and the tokens read back out of pools of every type.

Codes and scales are decided by single float32 operations and roundings to
nearest even on both sides, so the pools' bytes must match exactly, the bytes
that no token writes among them."""
import zlib

import numpy as np
import pytest

import synth
from harness import assert_ulp_close, to_bits
from oracle import bf16 as obf16
from oracle import fp4 as ofp4
from oracle import fp8 as ofp8
from oracle import rope as orope

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

K_SCALE, V_SCALE = 0.25, 0.5


def d16(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda()


def d8(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.uint8)).cuda()


def d32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def u8(t):
    return t.detach().cpu().numpy().astype(np.uint8)


def host_pool(w, which, ps):
    """The workload's bf16 pool in 4 bits, as the append would have left it."""
    codes, scales = ofp4.quantize(w.pool(which), ps)
    return ofp4.pack_pool(codes, scales)


class F4Step:
    """Device buffers of one workload step over 4-bit pools."""

    def __init__(self, w, k_scale=K_SCALE, v_scale=V_SCALE, scale=0.0):
        import paged_kv_gqa_row_gb300 as lnk
        self.w, self.lnk = w, lnk
        self.k_host, self.v_host = host_pool(w, "k", k_scale), host_pool(w, "v", v_scale)
        self.k_pool, self.v_pool = d8(self.k_host), d8(self.v_host)
        self.q, self.k, self.v = d16(w.step_q()), d16(w.step_k()), d16(w.step_v())
        self.positions, self.rows, self.table = d32(w.token_positions()), d32(w.token_rows()), d32(w.table)
        gq, gk = w.gamma_q(), w.gamma_k()
        self.gamma_q = None if gq is None else d16(gq)
        self.gamma_k = None if gk is None else d16(gk)
        self.q_out = torch.zeros((w.T, w.hq, w.head_dim), dtype=torch.int16, device="cuda")
        self.out = torch.full_like(self.q_out, 0x7FC0)  # NaN: every output has to be written
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.desc = lnk.attn_desc(w.hq, w.hkv, w.head_dim, w.num_pages, w.num_rows, w.pages_per_row, window=w.window,
                                  scale=scale, kv_dtype=lnk.KV_E2M1, k_scale=k_scale, v_scale=v_scale)
        self.rope = lnk.rope_desc(w.theta, w.llama3)
        self.ws_bytes = max(lnk.lnk_paged_workspace_size(self.desc, max(w.B, 1)), 256)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device="cuda")
        self.dec_positions = d32(w.dec_positions)

    def append(self, slots=None, stream=None):
        w = self.w
        self.lnk.lnk_paged_append_rope(self.desc, self.rope, self.q, self.k, self.v, self.positions, self.rows, slots,
                                       self.table, self.gamma_q, self.gamma_k, w.norm_eps, self.k_pool, self.v_pool,
                                       self.q_out, w.T, self.status, stream)


def oracle_append(w, k_pool, v_pool, k_scale=K_SCALE, v_scale=V_SCALE):
    inv = orope.inv_freq(w.theta, w.head_dim, w.llama3)
    return ofp4.append_rope(w.step_q(), w.step_k(), w.step_v(), w.token_positions(), w.token_rows(), w.table, k_pool,
                            v_pool, inv, k_scale, v_scale, gamma_q=w.gamma_q(), gamma_k=w.gamma_k(), eps=w.norm_eps)


APPEND_CASES = [
    # hq, hkv, d, decode lengths, chunks, inactive rows, K and V scale
    ("gqa4-128", 8, 2, 128, [1, 64, 65, 300, 17], [(0, 70)], (2,), 0.25, 0.5),
    ("mha96", 6, 6, 96, [5, 128, 63], [], (), 1.0, 1.0),
    ("gqa8-64", 16, 2, 64, [700, 2], [(100, 33), (0, 1)], (), 0.003, 7.0),
    ("one-token", 2, 1, 128, [1], [], (), 0.5, 0.25),
    ("many-tokens", 8, 2, 96, [9] * 20, [(3, 700)], (4,), 0.5, 0.25),
]


@pytest.mark.parametrize("case", APPEND_CASES, ids=[c[0] for c in APPEND_CASES])
def test_append_writes_the_oracles_bytes(case):
    name, hq, hkv, d, lengths, chunks, inactive, ks, vs = case
    w = synth.custom(seed=zlib.crc32(("e2m1" + name).encode()) % 10000, hq=hq, hkv=hkv, head_dim=d, dec_lengths=lengths,
                     chunks=chunks, inactive=inactive)
    dev = F4Step(w, k_scale=ks, v_scale=vs)
    dev.append()
    torch.cuda.synchronize()
    q_want, kp, vp = oracle_append(w, dev.k_host, dev.v_host, ks, vs)
    assert_ulp_close(to_bits(dev.q_out), q_want, "q_out")
    kg, vg = u8(dev.k_pool), u8(dev.v_pool)
    assert np.array_equal(vg, vp), f"V bytes: {int(np.sum(vg != vp))} differ"
    assert np.array_equal(kg, kp), f"K bytes: {int(np.sum(kg != kp))} differ"
    assert int(dev.status.item()) == 0


def test_append_with_qk_norm_and_with_slots():
    w = synth.build("qwen3", scale=0.02, rows=17)
    dev = F4Step(w)
    dev.append()
    torch.cuda.synchronize()
    q_want, kp, vp = oracle_append(w, dev.k_host, dev.v_host)
    assert_ulp_close(to_bits(dev.q_out), q_want, "q_out")
    assert np.array_equal(u8(dev.k_pool), kp) and np.array_equal(u8(dev.v_pool), vp)
    # the same tokens by slot, into fresh pools
    again = F4Step(w)
    slots = [int(w.table[r, p // 64]) * 64 + p % 64 if p >= 0 else -1
             for p, r in zip(w.token_positions(), w.token_rows())]
    again.append(slots=d32(slots))
    torch.cuda.synchronize()
    assert torch.equal(again.k_pool, dev.k_pool) and torch.equal(again.v_pool, dev.v_pool)


@pytest.mark.parametrize("hq,hkv,d,tokens,norm", [(8, 2, 128, 400, True), (6, 6, 96, 160, True), (5, 5, 64, 153, False),
                                                  (16, 2, 128, 700, False), (32, 8, 128, 151, True), (3, 3, 96, 1300, True),
                                                  (1, 1, 64, 2000, True)])
def test_prompts_at_any_position_with_and_without_norm(hq, hkv, d, tokens, norm):
    """Launches around and above the size where the many-token form takes over:
    positions of every magnitude (far ones have angles beyond 2^20), inactive
    tokens, bad slots, and heads of zeros, against the oracle's bytes."""
    import paged_kv_gqa_row_gb300 as lnk
    rng = np.random.RandomState(tokens + d)
    pages = tokens // 64 + 2
    q, k, v = (synth.tensor_bf16(tokens + d, i, (tokens, h, d)) for i, h in enumerate((hq, hkv, hkv)))
    q[7, 0] = 0
    positions = (2.0 ** rng.uniform(0, 30, tokens)).astype(np.int64)
    positions[:40] = np.arange(40)
    positions[[3, 50, tokens - 1]] = -1
    slots = rng.permutation(pages * 64)[:tokens]
    gq = gk = None
    if norm:
        gq, gk = (obf16.from_f64(1 + 0.1 * rng.standard_normal(d)) for _ in range(2))
    inv = orope.inv_freq(5e5, d, (8.0, 1.0, 4.0, 8192))
    blank = np.zeros((hkv, pages, 36 * d), dtype=np.uint8)
    q_want, kp, vp = ofp4.append_rope(q, k, v, positions, None, None, blank, blank, inv, K_SCALE, V_SCALE, slots=slots,
                                      gamma_q=gq, gamma_k=gk, eps=1e-6)
    bad = slots.copy()
    bad_tokens = [5, 60]
    bad[bad_tokens] = [pages * 64, -3]
    desc = lnk.attn_desc(hq, hkv, d, pages, 1, 1, kv_dtype=lnk.KV_E2M1, k_scale=K_SCALE, v_scale=V_SCALE)
    rope = lnk.rope_desc(5e5, (8.0, 1.0, 4.0, 8192))
    for use, want_status in ((slots, 0), (bad, 0x08)):
        kd, vd = d8(blank), d8(blank)
        q_out = torch.full((tokens, hq, d), 0x55, dtype=torch.int16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lnk.lnk_paged_append_rope(desc, rope, d16(q), d16(k), d16(v), d32(positions), None, d32(use), None,
                                  None if gq is None else d16(gq), None if gk is None else d16(gk), 1e-6, kd, vd, q_out,
                                  tokens, status)
        torch.cuda.synchronize()
        assert int(status.item()) == want_status
        assert_ulp_close(to_bits(q_out), q_want, "q_out")
        if want_status:  # the bad tokens' slots stay as they were
            for t in bad_tokens:
                for pool in (kp, vp):
                    for h in range(hkv):
                        ofp4.write_row(pool[h, slots[t] // 64], slots[t] % 64, np.zeros(d, np.uint8), np.zeros(d // 16, np.uint8))
        assert np.array_equal(u8(vd), vp), f"V bytes: {int(np.sum(u8(vd) != vp))} differ"
        assert np.array_equal(u8(kd), kp), f"K bytes: {int(np.sum(u8(kd) != kp))} differ"


def test_blocks_of_zeros_extremes_infinities_and_nan():
    """Value rows (stored without rotation) whose blocks are zero, below the least
    scale, saturating, infinite, NaN, and full of ties."""
    import paged_kv_gqa_row_gb300 as lnk
    d, t = 128, 12
    rng = np.random.RandomState(9)
    x = rng.standard_normal((t, 1, d))
    x[0] = 0.0
    x[1] = rng.choice([-0.25, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -5.0], size=(1, d))
    x[2] *= 1e-4
    x[3] *= 1e6
    x[4, 0, ::17] = 448 * 6
    x[5, 0, 16:32] = 0
    bits = obf16.from_f64(x)
    bits[6, 0, 3] = 0x7F80   # +inf
    bits[7, 0, 40] = 0xFF80  # -inf
    bits[8, 0, 0] = 0x7FC0   # NaN
    bits[9, 0, 127] = 0xFFFF
    bits[10, 0, 5] = 0x8000  # -0
    bits[11, 0, :] = 0x0001  # the least subnormal
    codes, scales = ofp4.quantize(bits, 1.0)
    page = np.full((1, 1, 36 * d), 0xEE, dtype=np.uint8)
    for j in range(t):
        ofp4.write_row(page[0, 0], j, codes[j, 0], scales[j, 0])
    desc = lnk.attn_desc(1, 1, d, 1, 1, 1, kv_dtype=lnk.KV_E2M1)
    kp = d8(np.full((1, 1, 36 * d), 0xEE))
    vp = kp.clone()
    q = torch.zeros((t, 1, d), dtype=torch.int16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos, rows, tab = d32(np.arange(t)), d32(np.zeros(t)), d32([[0]])
    lnk.lnk_paged_append_rope(desc, lnk.rope_desc(1e4), q, q, d16(bits), pos, rows, None, tab, None, None, 0.0, kp, vp,
                              torch.empty_like(q), t, status)
    out = torch.full((t, 1, d), 0x1234, dtype=torch.int16, device="cuda")
    lnk.lnk_paged_read_tokens(desc, None, vp, pos, rows, None, tab, None, out, t, status)
    torch.cuda.synchronize()
    assert np.array_equal(u8(vp), page)
    got, want = obf16.to_f64(to_bits(out)), ofp4.row_values(codes, scales, 1.0)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    # the values have at most 5 significant bits here: exact in bf16
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])
    assert np.isnan(got[8, 0, :16]).all() and np.isfinite(got[8, 0, 16:]).all()
    assert int(status.item()) == 0


def _bf16_of_products(values, scale):
    """bf16 bits of fl32(value * scale), rounded to nearest even (torch on the host)."""
    f = torch.from_numpy(np.asarray(values, dtype=np.float32)) * torch.tensor(scale, dtype=torch.float32)
    return f.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 96), (2, 128)])
def test_read_tokens_gives_the_stored_values(kind, hkv, d):
    import paged_kv_gqa_row_gb300 as lnk
    rng = np.random.RandomState(d + hkv)
    n_pages, n_rows, per_row, ks, vs = 9, 4, 3, 0.37, 1.9
    table = np.full((n_rows, per_row), -1, dtype=np.int32)
    table[:3] = rng.permutation(n_pages).reshape(3, per_row)
    table[2, 2] = n_pages  # outside the pool
    if kind == "bf16":
        pools = [rng.randint(0, 1 << 16, (hkv, n_pages * 64, d)).astype(np.uint16) for _ in range(2)]
        dtype, bits, on = lnk.KV_BF16, pools, [d16(p) for p in pools]
    elif kind == "e4m3":
        pools = [rng.choice([c for c in range(256) if c not in ofp8.NAN_CODES], (hkv, n_pages * 64, d)).astype(np.uint8)
                 for _ in range(2)]
        dtype, on = lnk.KV_E4M3, [d8(p) for p in pools]
        bits = [_bf16_of_products(ofp8.decode(p), s) for p, s in zip(pools, (ks, vs))]
    else:
        codes = [rng.randint(0, 16, (hkv, n_pages * 64, d)).astype(np.uint8) for _ in range(2)]
        scales = [rng.randint(0, 127, (hkv, n_pages * 64, d // 16)).astype(np.uint8) for _ in range(2)]
        dtype, on = lnk.KV_E2M1, [d8(ofp4.pack_pool(c, s)) for c, s in zip(codes, scales)]
        bits = [_bf16_of_products(ofp4.row_values(c, s, 1.0), p) for c, s, p in zip(codes, scales, (ks, vs))]
    desc = lnk.attn_desc(hkv, hkv, d, n_pages, n_rows, per_row, kv_dtype=dtype, k_scale=ks, v_scale=vs)
    where = [(0, 0), (0, 63), (1, 64), (0, 191), (2, 70), (1, -1), (0, 63), (1, 130), (2, 127)]
    bad = [(2, 130), (0, 192), (4, 3), (-1, 3), (3, 5)]  # page outside, position outside, row outside (2), unmapped
    for tokens, want_status in ((where, 0), (where + bad, 0x01 | 0x02 | 0x04)):
        t = len(tokens)
        outs = [torch.full((t, hkv, d), 0x55, dtype=torch.int16, device="cuda") for _ in range(2)]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lnk.lnk_paged_read_tokens(desc, on[0], on[1], d32([p for _, p in tokens]), d32([r for r, _ in tokens]), None,
                                  d32(table), outs[0], outs[1], t, status)
        torch.cuda.synchronize()
        assert int(status.item()) == want_status
        for which in range(2):
            got = to_bits(outs[which])
            for i, (r, p) in enumerate(tokens):
                if i < len(where) and p >= 0:
                    want = bits[which][:, int(table[r, p // 64]) * 64 + p % 64]
                else:
                    want = np.zeros((hkv, d), dtype=np.uint16)
                assert np.array_equal(got[i], want), (kind, which, i)
    # by slot, one pool alone, a slot outside among them
    slots = [0, n_pages * 64 - 1, 100, n_pages * 64, -1, 100]
    out = torch.full((6, hkv, d), 0x55, dtype=torch.int16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lnk.lnk_paged_read_tokens(desc, on[0], None, d32([0] * 6), None, d32(slots), None, out, None, 6, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0x08
    got = to_bits(out)
    for i, s in enumerate(slots):
        want = bits[0][:, s] if 0 <= s < n_pages * 64 else np.zeros((hkv, d), dtype=np.uint16)
        assert np.array_equal(got[i], want), i


@pytest.mark.parametrize("ps", [1.0, 0.25, 2.0 ** -20, 2.0 ** 30, 2.0 ** -70, 0.37, 3.0])
@pytest.mark.parametrize("tokens", [12, 300])
def test_values_of_every_bit_pattern(tokens, ps):
    """Value rows of arbitrary bf16 bits (subnormals, infinities and NaN among them),
    of elements that lie on the formats' borders, and of wild ranges, in launches of
    either form and with pool scales that are powers of two or not."""
    import paged_kv_gqa_row_gb300 as lnk
    d, hkv = 128, 3
    rng = np.random.RandomState(tokens + int(abs(np.log2(ps)) * 10))
    bits = rng.randint(0, 1 << 16, (tokens, hkv, d)).astype(np.uint16)
    # blocks of exact borders: multiples of a scale value times the borders' halves
    scale = ofp8.decode(rng.randint(8, 120, (tokens, d // 16)).astype(np.uint8)) * ps
    grid = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 3.0], (tokens, d)) * rng.choice([-1, 1], (tokens, d))
    exact = np.repeat(scale, 16, axis=-1) * grid
    exact[:, ::16] = scale * 6
    small = (np.abs(exact) < 1e37) & (np.abs(exact) > 1e-37)
    bits[:, 0] = obf16.from_f64(np.where(small, exact, 1.0))
    bits[:, 1] = obf16.from_f64(rng.standard_normal((tokens, d)) * ps * 2.0 ** rng.uniform(-12, 14, (tokens, 1)))
    codes, scales = ofp4.quantize(bits, ps)
    pages = tokens // 64 + 1
    want = np.full((hkv, pages, 36 * d), 0xEE, dtype=np.uint8)
    for t in range(tokens):
        for h in range(hkv):
            ofp4.write_row(want[h, t // 64], t % 64, codes[t, h], scales[t, h])
    desc = lnk.attn_desc(hkv, hkv, d, pages, 1, pages, kv_dtype=lnk.KV_E2M1, k_scale=ps, v_scale=ps)
    kp = d8(np.zeros_like(want))
    vp = d8(np.full_like(want, 0xEE))
    q = torch.zeros((tokens, hkv, d), dtype=torch.int16, device="cuda")
    lnk.lnk_paged_append_rope(desc, lnk.rope_desc(1e4), q, q, d16(bits), d32(np.arange(tokens)), d32(np.zeros(tokens)),
                              None, d32([np.arange(pages)]), None, None, 0.0, kp, vp, torch.empty_like(q), tokens)
    torch.cuda.synchronize()
    got = u8(vp)
    assert np.array_equal(got, want), f"{int(np.sum(got != want))} bytes differ"


@pytest.mark.parametrize("hq,hkv,d,tokens,norm", [(1, 1, 64, 80, True), (64, 8, 128, 90, False), (20, 20, 96, 77, True)])
def test_few_prompt_tokens_whose_heads_are_split(hq, hkv, d, tokens, norm):
    """Fewer tokens than SMs: a token's heads, fewer or more than 16, go to two CTAs."""
    test_prompts_at_any_position_with_and_without_norm(hq, hkv, d, tokens, norm)

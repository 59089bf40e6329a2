"""The latent cache on the GPU: append, absorbed decode and step attention against the
oracle in 64 bits (tolerances: latent_harness)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from latent_harness import PAGE, Step, bits, check, d16, d32, normal, tables  # noqa: E402
from oracle import bf16, latent, rope  # noqa: E402

pytestmark = pytest.mark.gpu

DECODE = [
    ("one-key", 1, 128, 32, [1], 0, ()),
    ("small", 4, 128, 64, [1, 2, 63, 64, 65, 130], 0, ()),
    ("heads-3", 3, 256, 32, [77, 640], 0, ()),
    ("heads-24", 24, 256, 64, [1000, 5, 64, 128, 2000, 777], 0, ()),
    ("heads-40", 40, 512, 64, [300, 1, 4097], 0, ()),
    ("heads-64", 64, 512, 64, [129, 500, 64], 0, ()),
    ("heads-65", 65, 384, 64, [200, 64, 7], 0, ()),
    ("heads-128", 128, 512, 32, [700, 65], 0, ()),
    ("heads-160", 160, 512, 64, [333, 3], 0, ()),
    ("window-100", 8, 512, 64, [50, 129, 700, 101, 100], 100, ()),
    ("window-1", 20, 256, 64, [1, 64, 65, 500], 1, ()),
    ("window-64", 20, 128, 64, [63, 64, 65, 129, 900], 64, ()),
    ("idle-rows", 16, 512, 64, [100, 1, 257, 64], 0, (1, 3)),
    ("all-idle", 16, 256, 64, [100, 1], 0, (0, 1)),
    ("one-long-row", 16, 512, 64, [30011], 0, ()),
    ("many-rows", 8, 128, 32, [1 + (37 * i) % 700 for i in range(200)], 0, (7, 199)),
]


@pytest.mark.parametrize("name,heads,c,r,dec,window,idle", DECODE, ids=[x[0] for x in DECODE])
def test_decode(name, heads, c, r, dec, window, idle):
    Step(len(name), heads, c, r, dec=dec, window=window, idle=idle).upload().run().verify()


STEPS = [
    ("one-token", 8, 128, 64, [(1, 0)], [], 0),
    ("pieces", 24, 256, 64, [(17, 70), (83, 35), (150, 0)], [], 0),
    ("one-head", 1, 128, 32, [(150, 3), (65, 64)], [], 0),
    ("three-heads", 3, 256, 64, [(50, 100)], [5, 200], 0),
    ("odd-heads", 20, 384, 32, [(5, 1000), (4, 61), (9, 0)], [300], 0),
    ("with-rows", 64, 512, 64, [(8, 500), (40, 64)], [129, 64, 700], 0),
    ("many-heads", 128, 512, 64, [(5, 300), (3, 64)], [200], 0),
    ("window", 16, 512, 64, [(70, 200), (33, 0)], [500, 3], 65),
    ("window-1", 8, 128, 64, [(70, 100)], [70], 1),
    # enough rows for tiles of 128 on pairs of SMs
    ("pairs", 20, 128, 64, [(700, 30), (330, 5)], [70], 0),
    ("pairs-c256", 48, 256, 32, [(300, 0), (113, 64)], [], 0),
    ("pairs-c384", 30, 384, 64, [(651, 3)], [300, 1], 0),
    ("pairs-window", 64, 512, 64, [(310, 90)], [500], 65),
    ("pairs-one-head", 1, 128, 32, [(19500, 0)], [], 40),
]


@pytest.mark.parametrize("name,heads,c,r,pieces,dec,window", STEPS, ids=[x[0] for x in STEPS])
def test_step(name, heads, c, r, pieces, dec, window):
    s = Step(100 + len(name), heads, c, r, pieces, dec, window).upload().run()
    # (of many tokens: the ends, and every 37th)
    s.verify(None if s.P < 200 else {*range(0, s.P, 37), *range(s.P - 3, s.P + s.B), *range(5)})


def _ulp1(got, want, what):
    """The append rounds once: identical but for one element in a million (a tie that 46 bits do not see)."""
    d = bf16.ulp_distance(got, want)
    assert d.max(initial=0) <= 1 and (d != 0).sum() <= 1 + d.size // 1000000, f"{what}: {int((d != 0).sum())} differ"


APPEND = [
    ("one-token", 1, 128, 32, [7], None, True, 1e4, None),
    ("decode-rows", 64, 512, 64, [4000 + (37 * i) % 61 for i in range(64)], None, True, 1e4, None),
    ("prompt", 5, 512, 64, list(range(60, 460)), 0, True, 5e5, (8.0, 1.0, 4.0, 8192)),
    ("no-norm", 24, 256, 64, [0, 1, 63, 64, 65, 20000], None, False, 1e6, None),
    ("c384", 40, 384, 32, [5, -1, 700, -1, 1], None, True, 1e4, None),
    ("many-tokens", 3, 128, 64, list(range(0, 900)), 0, True, 1e4, None),
]


@pytest.mark.parametrize("name,heads,c,r,positions,row,norm,theta,llama3", APPEND, ids=[x[0] for x in APPEND])
def test_append(name, heads, c, r, positions, row, norm, theta, llama3):
    import paged_kv_gqa_row_gb300 as lnk
    rng = np.random.default_rng(len(name))
    t = len(positions)
    positions = np.array(positions, dtype=np.int32)
    rows = np.arange(t, dtype=np.int32) if row is None else np.full(t, row, dtype=np.int32)
    lengths = [0] * (int(rows.max()) + 1)
    for p, x in zip(positions, rows):
        lengths[x] = max(lengths[x], int(p) + 1)
    table, pages = tables(rng, lengths)
    lead = 2 * r  # projected queries: other numbers before the rotated ones
    q, kv = normal(rng, t, heads, lead + r), normal(rng, t, c + r)
    w = normal(rng, c, scale=0.1) if norm else None
    pool = normal(rng, pages * PAGE, c + r)
    dq, dkv, dpool = d16(q), d16(kv), d16(pool)
    q_out = torch.full((t, heads, c + r), 0x1234, dtype=torch.int16, device="cuda")
    kv_out = torch.full((t, c + r), 0x1234, dtype=torch.int16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    desc = lnk.latent_desc(heads, c, r, pages, table.shape[0], table.shape[1], scale=1.0)
    lnk.lnk_latent_append(desc, lnk.rope_desc(theta, llama3), dq[:, :, lead:], lead + r, dkv, d32(positions),
                          None if row is None else d32(rows), None, d32(table), d16(w) if norm else None, 1e-6, dpool,
                          q_out[:, :, c:], c + r, kv_out, t, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want_q, want_kv, want_pool = latent.append(q[:, :, lead:], kv, positions, rows, table, pool,
                                               rope.inv_freq(theta, r, llama3), c, None, w, float(np.float32(1e-6)))
    got_q = bits(q_out)
    _ulp1(got_q[:, :, c:], want_q, "queries")
    assert (got_q[:, :, :c] == 0x1234).all(), "numbers beside the rotated ones are left as they are"
    _ulp1(bits(kv_out), want_kv, "rows")
    _ulp1(bits(dpool), want_pool, "pool")


def test_append_in_place_by_slots_and_bad_places():
    import paged_kv_gqa_row_gb300 as lnk
    rng = np.random.default_rng(3)
    t, heads, c, r, pages = 6, 10, 256, 64, 4
    q, kv, pool = normal(rng, t, heads, r), normal(rng, t, c + r), normal(rng, pages * PAGE, c + r)
    positions = np.array([0, 5, 64, 700, 9, -1], dtype=np.int32)
    slots = np.array([3, 255, 0, 256, -1, 7], dtype=np.int32)  # 256 and -1: outside the pool
    desc = lnk.latent_desc(heads, c, r, pages, 2, 2, scale=1.0)
    inv = rope.inv_freq(1e4, r)
    dq, dpool, status = d16(q), d16(pool), torch.zeros(1, dtype=torch.int32, device="cuda")
    lnk.lnk_latent_append(desc, lnk.rope_desc(1e4), dq, r, d16(kv), d32(positions), None, d32(slots), None, None, 0.0, dpool,
                          dq, r, None, t, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0x08
    want_q, want_kv, _ = latent.append(q, kv, positions, None, None, np.zeros((t, c + r), np.uint16), inv, c,
                                       slots=np.arange(t))
    _ulp1(bits(dq), want_q, "queries in place")
    want = pool.copy()
    want[[3, 255, 0]] = want_kv[[0, 1, 2]]
    _ulp1(bits(dpool), want, "pool")
    # a row, a position and a page that are not there: nothing is written, each is reported
    dpool.copy_(d16(pool))
    table = np.array([[1, -1], [2, 4]], dtype=np.int32)
    for row, pos, flag in ((2, 0, 0x01), (-1, 0, 0x01), (0, 128, 0x02), (0, 64, 0x04), (1, 127, 0x04)):
        status.zero_()
        lnk.lnk_latent_append(desc, lnk.rope_desc(1e4), d16(q), r, d16(kv), d32([pos]), d32([row]), None, d32(table), None,
                              0.0, dpool, dq, r, None, 1, status)
        torch.cuda.synchronize()
        assert int(status.item()) == flag
        assert (bits(dpool) == pool).all()


def test_copy_pages():
    import paged_kv_gqa_row_gb300 as lnk
    rng = np.random.default_rng(4)
    for c, r, layers, pages, pairs in ((512, 64, 3, 9, [(8, 0), (5, 1), (2, 2)]), (128, 32, 300, 4, [(3, 1), (4, 0), (2, -1)])):
        pools = [torch.randint(-30000, 30000, (pages * PAGE, c + r), dtype=torch.int16, device="cuda") for _ in range(layers)]
        want = [p.clone() for p in pools]
        bad = 0
        for s, d in pairs:
            if 0 <= s < pages and 0 <= d < pages:
                for w in want:
                    w[d * PAGE:(d + 1) * PAGE] = w[s * PAGE:(s + 1) * PAGE].clone()
            else:
                bad = 0x04
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        desc = lnk.latent_desc(1, c, r, pages, 1, 1, scale=1.0)
        src, dst = rng.permutation(len(pairs)), None
        dst = [pairs[i][1] for i in src]
        src = [pairs[i][0] for i in src]
        lnk.lnk_latent_copy_pages(desc, pools, d32(src), d32(dst), len(pairs), status)
        torch.cuda.synchronize()
        assert int(status.item()) == bad
        for a, b in zip(pools, want):
            assert torch.equal(a, b)


def test_bad_rows_positions_and_pages():
    s = Step(5, 16, 256, 64, pieces=[(6, 60), (4, 10)], dec=[200, 130, 64]).upload()
    # a piece token's row, a decode row's position and an entry of a table that are not there
    s.rows[2] = 99
    s.step_positions[1] = s.table.shape[1] * PAGE
    s.d["rows"], s.d["step"] = d32(s.rows), d32(s.step_positions)
    table = s.table.copy()
    table[0, 1] = s.pages
    s.d["table"] = d32(table)
    s.run()
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0x01 | 0x02 | 0x04
    out = bits(s.out)
    assert not out[2].any() and not out[s.P + 1].any()
    # row 0's second page is skipped: the keys of the others remain
    keys = bf16.to_f64(s.pool[np.concatenate([table[0, j] * PAGE + np.arange(PAGE) for j in (0, 2)] + [
        table[0, 3] * PAGE + np.arange(200 - 192)])])
    want, spread, size = latent.attend(bf16.to_f64(s.q[s.P]), keys, keys[:, :s.c], s.scale)
    check(out[s.P], want, spread, size, 200, s.c + s.r, "row 0")
    for t, row, p in list(s.tokens()):
        if t not in (2, s.P, s.P + 1):
            want, spread, size = latent.attention_at(s.q[t], row, p, s.table, s.pool, s.c, s.scale)
            check(out[t], want, spread, size, p + 1, s.c + s.r, f"token {t}")


@pytest.mark.parametrize("scale", [0.3, 2.0])
def test_raises_of_the_reference(scale):
    """Scores that grow by far more than 2^32 from page to page, and sums that must follow."""
    for heads, c, r in ((24, 512, 64), (64, 256, 32), (100, 512, 64), (16, 128, 64)):
        s = Step(6, heads, c, r, pieces=[(9, 300)], dec=[1000, 333], scale=scale)
        grow = np.linspace(0.05, 3.0, s.pages * PAGE)
        for row in range(s.table.shape[0]):
            pages = s.table[row][s.table[row] >= 0]
            slots = (pages[:, None] * PAGE + np.arange(PAGE)).reshape(-1)
            s.pool[slots] = bf16.from_f64(bf16.to_f64(s.pool[slots]) * grow[:len(slots), None] * (s.pages * PAGE / len(slots)) ** 0.25)
        s.upload().run().verify()


def _numbers_where(out, finite_tokens, nan_tokens):
    f = bf16.to_f64(out)
    for t in finite_tokens:
        assert np.isfinite(f[t]).all(), f"token {t}"
    for t in nan_tokens:
        assert np.isnan(f[t]).all(), f"token {t}"


@pytest.mark.parametrize("heads,count", [(12, 12), (40, 500)], ids=["one-sm", "pairs"])
@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80, 0xFF80], ids=["nan", "inf", "-inf"])
def test_values_that_are_not_finite_reach_only_those_who_see_them(bad, heads, count):
    # a piece of tokens, a few a tile, whose 7th token's key is not finite
    s = Step(7, heads, 256, 64, pieces=[(count, 100)], dec=[500, 70])
    slot = s.table[2, 106 // PAGE] * PAGE + 106 % PAGE
    clean = s.pool.copy()
    s.pool[slot] = bad
    # what lies behind each row's last key may be anything as well
    for row, p in ((0, 500), (1, 70), (2, 100 + count)):
        if p % PAGE:
            first = s.table[row, p // PAGE] * PAGE
            s.pool[first + p % PAGE:first + PAGE] = 0x7FC0
            clean[first + p % PAGE:first + PAGE] = 0
    s.upload().run()
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    out = bits(s.out)
    s.pool = clean
    for t, row, p in s.tokens():
        if row == 2 and p >= 106:
            assert np.isnan(bf16.to_f64(out[t])).all() if bad == 0x7FC0 else not np.isfinite(bf16.to_f64(out[t])).all()
            continue
        want, spread, size = latent.attention_at(s.q[t], row, p, s.table, clean, s.c, s.scale)
        check(out[t], want, spread, size, p + 1, s.c + s.r, f"token {t}")


@pytest.mark.parametrize("heads", [16, 128], ids=["one-sm", "pairs"])
def test_a_long_row_with_a_key_that_is_not_finite_in_a_cut_share(heads):
    """The keys that a piece's first tokens do not see lie in a part whose sums are joined later."""
    s = Step(8, heads, 512, 64, pieces=[(4, 9000)])
    clean = s.pool.copy()
    s.pool[s.table[0, 9002 // PAGE] * PAGE + 9002 % PAGE, :5] = 0x7FC0
    s.upload().run()
    torch.cuda.synchronize()
    out = bits(s.out)
    _numbers_where(out, [0, 1], [2, 3])
    for t in (0, 1):
        want, spread, size = latent.attention_at(s.q[t], 0, 9000 + t, s.table, clean, s.c, s.scale)
        check(out[t], want, spread, size, 9001, s.c + s.r, f"token {t}")


@pytest.mark.parametrize("heads", [16, 128], ids=["one-sm", "pairs"])
def test_keys_that_are_not_finite_cost_no_wait(heads):
    """Behind a long context, and in the context of all of a piece's tokens: no wait of the kernel runs out."""
    s = Step(12, heads, 256, 32, pieces=[(6, 60000), (40, 8000)], dec=[9000])
    clean = s.pool.copy()
    s.pool[s.table[1, 60004 // PAGE] * PAGE + 60004 % PAGE] = 0x7FC0
    s.pool[s.table[2, 0] * PAGE + 5, :7] = 0x7F80
    s.pool[s.table[0, 0] * PAGE + 5, :7] = 0x7FC0
    s.upload().run()
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    out = bits(s.out)
    f = bf16.to_f64(out)
    assert np.isnan(f[4:6]).all()
    assert np.isnan(f[s.P]).all()  # (NaN among a key's numbers: its score, and all of the row)
    assert not np.isfinite(f[6:46, :, :7]).any()
    for t in (0, 3):
        want, spread, size = latent.attention_at(s.q[t][:2], 1, 60000 + t, s.table, clean, s.c, s.scale)
        check(out[t][:2], want, spread, size, 60001 + t, s.c + s.r, f"token {t}")


def test_graph_replays_on_another_stream_and_two_workspaces():
    """A captured step replayed on new inputs, with another step's calls beside it on another stream."""
    a = Step(9, 40, 512, 64, pieces=[(7, 200)], dec=[900, 300]).upload()
    b = Step(10, 100, 256, 32, dec=[1500, 20, 64]).upload()
    a.run().verify()
    b.run().verify()
    want_a, want_b = bits(a.out).copy(), bits(b.out).copy()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
        a.run()
    other = torch.cuda.Stream()
    for _ in range(5):
        a.out.fill_(0x7FC1)
        b.out.fill_(0x7FC1)
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(other):
            b.run()
            b.run()
        torch.cuda.synchronize()
        assert (bits(a.out) == want_a).all() and (bits(b.out) == want_b).all()


def test_append_then_decode_then_the_pager():
    """A row of a model's layer as it is served: reserve, append token by token, attend, fork, copy on write."""
    import paged_kv_gqa_row_gb300 as lnk
    rng = np.random.default_rng(11)
    heads, c, r, rows = 20, 256, 64, 3
    pager = lnk.Pager(12, rows, 4)
    pager.reserve(0, 70)
    table = pager.table()
    pool = np.zeros((12 * PAGE, c + r), np.uint16)
    inv = rope.inv_freq(1e4, r)
    w = normal(rng, c)
    desc = lnk.latent_desc(heads, c, r, 12, rows, 4, scale=0.1)
    size = lnk.lnk_latent_workspace_size(desc)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    dpool, status = d16(pool), torch.zeros(1, dtype=torch.int32, device="cuda")
    dw = d16(w)

    def step(q, kv, positions, rws):
        nonlocal pool
        t = len(positions)
        dq = d16(q)
        lnk.lnk_latent_append(desc, lnk.rope_desc(1e4), dq[:, :, c:], c + r, d16(kv), d32(positions), d32(rws), None,
                              d32(table), dw, 1e-6, dpool, dq[:, :, c:], c + r, None, t, status)
        out = torch.empty((t, heads, c), dtype=torch.int16, device="cuda")
        lnk.lnk_latent_step_attn(desc, dq, d32(rws), d32(positions), None, d32(table), dpool, out, t, 0, ws, size, status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        want_q, _, pool = latent.append(q[:, :, c:], kv, positions, rws, table, pool, inv, c, None, w, float(np.float32(1e-6)))
        _ulp1(bits(dpool), pool, "pool")
        pool = bits(dpool).copy()
        full = np.concatenate([q[:, :, :c], bits(dq)[:, :, c:]], axis=2)
        for i in range(t):
            want, spread, sz = latent.attention_at(full[i], rws[i], positions[i], table, pool, c, float(np.float32(0.1)))
            check(bits(out)[i], want, spread, sz, positions[i] + 1, c + r, f"token {i}")

    step(normal(rng, 70, heads, c + r), normal(rng, 70, c + r), list(range(70)), [0] * 70)
    pager.fork(0, 2, 70)
    copies = pager.prepare_append([0, 2], [70, 70])
    assert len(copies) == 1
    table = pager.table()
    lnk.lnk_latent_copy_pages(desc, [dpool], d32([copies[0][0]]), d32([copies[0][1]]), 1, status)
    for s, d in copies:
        pool[d * PAGE:(d + 1) * PAGE] = pool[s * PAGE:(s + 1) * PAGE]
    step(normal(rng, 2, heads, c + r), normal(rng, 2, c + r), [70, 70], [0, 2])

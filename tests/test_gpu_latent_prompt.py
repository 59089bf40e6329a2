"""Expanded attention of packed prompts (lnk_latent_prompt_attn) against the oracle in 64 bits, and
against the absorbed form on the same weights (tolerances: latent_harness)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from latent_harness import PAGE, bits, check, d16, d32, normal  # noqa: E402
from oracle import bf16, latent, rope  # noqa: E402

pytestmark = pytest.mark.gpu


class Prompts:
    """pieces: (queries, keys before them); `gap` tokens that no prompt holds behind them all."""

    def __init__(self, seed, heads, d, r, pieces, gap=0, scale=None, rope_stride=None, q_scale=1.0):
        rng = np.random.default_rng(seed)
        self.heads, self.d, self.r, self.pieces = heads, d, r, pieces
        self.scale = (d + r) ** -0.5 if scale is None else scale
        self.qs = np.cumsum([0] + [n for n, _ in pieces]).astype(np.int32)
        self.ks = np.cumsum([0] + [max(0, n + b) for n, b in pieces]).astype(np.int32)
        self.tq, self.tk = int(self.qs[-1]) + gap, int(self.ks[-1]) + gap
        self.stride = rope_stride or r
        self.q = normal(rng, self.tq, heads, d + r, scale=q_scale)
        self.kv, self.kr = normal(rng, self.tk, heads, 2 * d), normal(rng, self.tk, self.stride)

    def upload(self):
        import paged_kv_gqa_row_gb300 as lnk
        self.lnk = lnk
        self.dev = dict(q=d16(self.q), kv=d16(self.kv), kr=d16(self.kr), qs=d32(self.qs), ks=d32(self.ks))
        self.out = torch.full((self.tq, self.heads, self.d), 0x7FC1, dtype=torch.int16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self

    def run(self, stream=None):
        e = self.dev
        self.lnk.lnk_latent_prompt_attn(self.heads, self.d, self.r, self.scale, e["q"], e["kv"],
                                        e["kr"][:, self.stride - self.r:], self.stride, e["qs"], e["ks"], self.out, self.tq,
                                        self.tk, len(self.pieces), self.status, stream)
        return self

    def verify(self, clean=None, skip=lambda prompt, i: False):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        out, kv = bits(self.out), self.kv if clean is None else clean
        for n, (count, before) in enumerate(self.pieces):
            k = slice(self.ks[n], self.ks[n + 1])
            for i in range(count):
                got = out[self.qs[n] + i]
                if before + i < 0:
                    assert not got.any()
                    continue
                if skip(n, i):
                    continue
                want, spread, size = latent.expanded_at(self.q[self.qs[n] + i], kv[k], self.kr[k][:, self.stride - self.r:],
                                                        self.d, before + i, self.scale)
                check(got, want, spread, size, before + i + 1, self.d + self.r, f"prompt {n}, query {i}")
        assert (out[self.qs[-1]:] == 0x7FC1).all(), "queries that no prompt holds are left as they were"
        return out


CASES = [
    ("one-token", 1, 128, 64, [(1, 0)]),
    ("small", 3, 128, 64, [(17, 0), (150, 0), (83, 0)]),
    ("tile-edges", 2, 128, 64, [(255, 0), (256, 0), (257, 0), (1, 0)]),
    ("d64-r32", 3, 64, 32, [(100, 0), (300, 0)]),
    ("d64-r64", 2, 64, 64, [(129, 0), (0, 0), (5, 0)]),
    ("d128-r32", 2, 128, 32, [(127, 0), (128, 0)]),
    ("prefixes", 2, 128, 64, [(5, 700), (130, 63), (1, 127), (2, 126)]),
    ("empty-ones", 2, 128, 64, [(0, 0), (3, 0), (0, 10), (0, 0), (40, 1)]),
    ("fewer-keys", 2, 128, 64, [(20, -5), (6, -6), (4, -9), (300, -260)]),
    ("many", 1, 64, 32, [(1 + (7 * i) % 40, i % 3) for i in range(90)]),
]


@pytest.mark.parametrize("name,heads,d,r,pieces", CASES, ids=[c[0] for c in CASES])
def test_prompts(name, heads, d, r, pieces):
    Prompts(len(name), heads, d, r, pieces, gap=3).upload().run().verify()


def test_more_tiles_than_are_ordered_by_cost():
    Prompts(8, 1, 64, 32, [(1 + i % 5, i % 7 - 2) for i in range(700)]).upload().run().verify()


def test_tiles_without_keys_between_others():
    """A tile's outputs leave through the place of the values: the next tile's may come only then, whatever
    lies between the two."""
    pieces = [(3, -3) if i % 2 else (200 + i % 57, i % 5) for i in range(600)]
    s = Prompts(10, 4, 128, 64, pieces).upload().run()
    s.verify(skip=lambda n, i: (n + i) % 61 != 0)
    want = bits(s.out).copy()
    for _ in range(30):
        s.out.fill_(0x7FC1)
        s.run()
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0 and (bits(s.out) == want).all()


@pytest.mark.parametrize("d,r", [(128, 64), (64, 32)])
def test_many_tiles_a_worker(d, r):
    s = Prompts(9, 48, d, r, [(900, 0), (513, 130), (257, 3), (1300, 0)]).upload().run()
    s.verify(skip=lambda n, i: i % 97 and i not in (127, 128, 255, 256, 511, 512))
    want = bits(s.out).copy()
    for _ in range(20):  # (whatever the two workers of a cluster meet: the same numbers)
        s.out.fill_(0x7FC1)
        s.run()
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0 and (bits(s.out) == want).all()


def test_rotated_keys_inside_wider_rows():
    Prompts(1, 3, 128, 64, [(70, 0), (40, 30)], rope_stride=576).upload().run().verify()


def test_growing_scores():
    s = Prompts(2, 2, 128, 64, [(400, 0), (100, 300)], scale=0.3)
    s.kv[:, :, :128] = bf16.from_f64(bf16.to_f64(s.kv[:, :, :128]) * np.linspace(0.05, 4, s.tk)[:, None, None])
    s.upload().run().verify()


@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80, 0xFF80], ids=["nan", "inf", "-inf"])
def test_values_that_are_not_finite_reach_only_those_who_see_them(bad):
    s = Prompts(3, 2, 128, 64, [(300, 0), (40, 20)])
    clean = s.kv.copy()
    s.kv[200, 1, 128 + 5] = bad    # a value of prompt 0, head 1
    s.kv[330, 0, :256] = bad       # a whole key and value of prompt 1, head 0: its key 30
    out = s.upload().run().verify(clean=clean, skip=lambda n, i: (n == 0 and i >= 200) or (n == 1 and 20 + i >= 30))
    f = bf16.to_f64(out)
    for i in range(200, 300):
        assert np.isfinite(f[i, 0]).all() and np.isfinite(np.delete(f[i, 1], 5)).all() and not np.isfinite(f[i, 1, 5])
    for i in range(310, 340):
        assert not np.isfinite(f[i, 0]).any() and np.isfinite(f[i, 1]).all()


def test_values_that_are_not_finite_cost_no_wait():
    """At the start and near the end of a long prompt: those that see them, and no wait of the kernel runs out."""
    s = Prompts(7, 2, 128, 64, [(600, 30000)])
    clean = s.kv.copy()
    s.kv[5, 0, 128 + 70] = 0x7FC0
    s.kv[30550, 1, 128 + 9] = 0x7FC0
    s.upload().run()
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    out = bits(s.out)
    f = bf16.to_f64(out)
    own = np.delete(np.arange(128), 70)  # (number 70 of head 0 is NaN for all: the 6th key's is)
    for i in range(49, 550, 100):
        want, spread, size = latent.expanded_at(s.q[i], clean, s.kr, 128, 30000 + i, s.scale)
        check(out[i, 0, own], want[0, own], spread[0, own], size[0], 30001 + i, 192, f"query {i}, head 0")
        check(out[i, 1], want[1], spread[1], size[1], 30001 + i, 192, f"query {i}, head 1")
    assert np.isnan(f[:, 0, 70]).all() and np.isfinite(np.delete(f[:, 0], 70, axis=1)).all()
    assert np.isnan(f[550:, 1, 9]).all() and np.isfinite(f[:550, 1]).all() and np.isfinite(np.delete(f[:, 1], 9, axis=1)).all()


def test_starts_that_do_not_ascend_or_lie_outside():
    s = Prompts(4, 2, 64, 64, [(30, 0), (40, 0), (50, 0)]).upload()
    want = bits(s.run().out).copy()
    torch.cuda.synchronize()
    for qs, ks, good in (([0, 30, 70, 121], [0, 30, 70, 120], (0, 1)), ([0, 30, 70, 120], [0, 30, 70, 121], (0, 1)),
                         ([0, 30, 70, 120], [0, 30, 20, 120], (0,)), ([0, 30, 70, 120], [0, -1, 70, 120], ())):
        s.out.fill_(0x7FC1)
        s.status.zero_()
        s.dev["qs"], s.dev["ks"] = d32(qs), d32(ks)
        s.run()
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0x10
        got = bits(s.out)
        for n in good:
            assert (got[s.qs[n]:s.qs[n + 1]] == want[s.qs[n]:s.qs[n + 1]]).all()
    # no keys at all
    s.status.zero_()
    s.lnk.lnk_latent_prompt_attn(2, 64, 64, 0.1, s.dev["q"], None, None, 64, d32([0, 30, 70, 120]), d32([0, 0, 0, 0]), s.out,
                                 120, 0, 3, s.status)
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0 and not bits(s.out).any()


def test_captured_and_beside_another_stream():
    a = Prompts(5, 2, 128, 64, [(300, 10)]).upload()
    b = Prompts(6, 3, 64, 32, [(70, 0), (500, 0)]).upload()
    a.run().verify()
    b.run().verify()
    want_a, want_b = bits(a.out).copy(), bits(b.out).copy()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
    other = torch.cuda.Stream()
    for _ in range(5):
        a.out.fill_(0)
        b.out.fill_(0)
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(other):
            b.run()
        torch.cuda.synchronize()
        assert (bits(a.out) == want_a).all() and (bits(b.out) == want_b).all()


def test_both_forms_of_one_layer():
    """A prompt appended and attended in the expanded form, then its last tokens again in the absorbed form,
    as a user runs them: both against exact attention, from their own (rounded) keys or queries."""
    import paged_kv_gqa_row_gb300 as lnk
    rng = np.random.default_rng(12)
    heads, c, r, d, n = 6, 256, 64, 128, 150
    scale = float(np.float32((d + r) ** -0.5))
    q, kv = normal(rng, n, heads, d + r), normal(rng, n, c + r)
    up, vp = normal(rng, heads, d, c, scale=c ** -0.5), normal(rng, heads, d, c, scale=c ** -0.5)
    w = normal(rng, c)
    pages = -(-n // PAGE)
    desc = lnk.latent_desc(heads, c, r, pages, 1, pages, scale=scale)
    table, positions = np.arange(pages, dtype=np.int32)[None], np.arange(n, dtype=np.int32)
    dq, dpool, status = d16(q), torch.zeros((pages * PAGE, c + r), dtype=torch.int16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    rows_out = torch.empty((n, c + r), dtype=torch.int16, device="cuda")
    lnk.lnk_latent_append(desc, lnk.rope_desc(1e4), dq[:, :, d:], d + r, d16(kv), d32(positions), d32(np.zeros(n)), None,
                          d32(table), d16(w), 1e-6, dpool, dq[:, :, d:], d + r, rows_out, n, status)
    lat = rows_out.view(torch.bfloat16)[:, :c].float()
    u, v = d16(up).view(torch.bfloat16).float(), d16(vp).view(torch.bfloat16).float()
    ex = torch.cat([torch.einsum("tc,hdc->thd", lat, u), torch.einsum("tc,hdc->thd", lat, v)], dim=2).bfloat16().contiguous()
    out = torch.empty((n, heads, d), dtype=torch.int16, device="cuda")
    starts = d32([0, n])
    lnk.lnk_latent_prompt_attn(heads, d, r, scale, dq, ex, rows_out[:, c:], c + r, starts, starts, out, n, n, 1, status)
    # the last 20 tokens in the absorbed form, from the pool
    m = 20
    full = dq.view(torch.bfloat16).float()[n - m:]
    qa = torch.cat([torch.einsum("thd,hdc->thc", full[:, :, :d], u), full[:, :, d:]], dim=2).bfloat16().contiguous()
    oa = torch.empty((m, heads, c), dtype=torch.int16, device="cuda")
    size = lnk.lnk_latent_workspace_size(desc)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    lnk.lnk_latent_step_attn(desc, qa, d32(np.zeros(m)), d32(positions[n - m:]), None, d32(table), dpool, oa, m, 0, ws, size,
                             status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got, exb, qb, qab, oab, pool = bits(out), bits(ex.view(torch.int16)), bits(dq), bits(qa.view(torch.int16)), bits(oa), bits(dpool)
    krb = bits(rows_out)[:, c:]
    for i in range(n):
        want, spread, sz = latent.expanded_at(qb[i], exb, krb, d, i, scale)
        check(got[i], want, spread, sz, i + 1, d + r, f"expanded {i}")
    for i in range(m):
        want, spread, sz = latent.attention_at(qab[i], 0, n - m + i, table, pool, c, scale)
        check(oab[i], want, spread, sz, n, c + r, f"absorbed {i}")
    # and the two forms are one attention: they differ by the roundings of keys, values and queries to bf16, 2^-8 each of
    # what the products add up to in magnitude (z of the scores, A of the values), with the exact products between them
    f64 = lambda b: bf16.to_f64(b)
    lat64, u64, v64 = f64(bits(rows_out))[:, :c], f64(up), f64(vp)
    for i in (0, 7, m - 1):
        for h in range(heads):
            keys = np.concatenate([lat64 @ u64[h].T, f64(krb)], axis=1)[:n - m + i + 1]
            vals = (lat64 @ v64[h].T)[:n - m + i + 1]
            qh = f64(qb[n - m + i, h])
            want, spread, sz = latent.attend(qh[None], keys, vals, scale)
            a = f64(got[n - m + i, h])
            b = f64(oab[i, h]) @ v64[h].T
            mass = np.abs(f64(oab[i, h])) @ np.abs(v64[h]).T
            big = max(float((np.abs(qh) @ np.abs(keys).T).max()), float((np.abs(f64(qab[i, h])) @ np.abs(f64(pool[:n])).T).max()))
            bound = 2.0 ** -8 * np.abs(want[0]) + (2.0 ** -7 + 2.0 ** -11 + 4 * 2.0 ** -8 * scale * big) * spread[0] + 2.0 ** -8 * mass
            wide = (2.0 ** -7 + 2.0 ** -11 + 4 * 2.0 ** -8 * scale * big) * mass + bound
            assert (np.abs(a - want[0]) <= bound).all() and (np.abs(b - want[0]) <= wide).all()

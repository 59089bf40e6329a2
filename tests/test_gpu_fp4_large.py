"""4-bit (E2M1) pools at sizes where one cluster works through many tiles, where
offsets pass 32 bits, at the most decode rows, and with calls side by side.

The references are float64 on the GPU, written from the format and the formulas:
the stored value of a code is e2m1(code) e4m3(scale) pool scale, and attention is
softmax(q k / sqrt(D)) v over the visible keys.  The tolerance per element is that
of test_gpu_fp4_attention.py: 2^-8 |out| for the result's rounding, 2^-10 of
A = sum p |v| / sum p for P's rounding (2^-11) and the float32 work (half of it
allowed), and 2^-25 of max |v| per key for P below f16's normal range.
"""
import numpy as np
import pytest

from oracle import fp4 as ofp4
from oracle import fp8 as ofp8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

K_SCALE, V_SCALE = 0.25, 0.5


def values_of(pool, ps, hkv, pages, d):
    """[hkv][pages * 64][d] float64 of a pool of bytes (on its device)."""
    page = pool.view(hkv, pages, 36 * d)
    codes = page[:, :, : 32 * d].reshape(hkv, pages, 64, d // 2)
    lut = torch.from_numpy(ofp4.decode(np.arange(16))).to(pool.device)
    e4m3 = torch.from_numpy(ofp8.decode(np.arange(256, dtype=np.uint8)).astype(np.float64)).to(pool.device)
    v = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), -1).reshape(hkv, pages, 64, d // 16, 16)
    s = e4m3[page[:, :, 32 * d:].long()].reshape(hkv, pages, 4, d // 16, 16)  # [j % 4][block][j / 4]
    s = s.permute(0, 1, 4, 2, 3).reshape(hkv, pages, 64, d // 16, 1)
    return (v * s * ps).reshape(hkv, pages * 64, d)


def random_pool(hkv, pages, d, gen):
    """Random codes with scales of 2^-3 .. 2^3 (finite, both signs of codes)."""
    pool = torch.randint(0, 256, (hkv, pages, 36 * d), generator=gen, device="cuda", dtype=torch.int32).to(torch.uint8)
    scales = torch.randint(4 << 3, 10 << 3, (hkv, pages, 4 * d), generator=gen, device="cuda", dtype=torch.int32)
    pool[:, :, 32 * d:] = scales.to(torch.uint8)
    return pool.reshape(-1)


class Case:
    """A table of random pages, queries and outputs for `rows` and `positions`."""

    def __init__(self, hq, hkv, d, pages_per_row, num_rows, positions, rows=None, window=0, seed=1, scale=0.0):
        import paged_kv_gqa_row_gb300 as lnk
        self.lnk, self.hq, self.hkv, self.d, self.window = lnk, hq, hkv, d, window
        self.scale = scale or d ** -0.5
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.pages = pages_per_row * num_rows + 3
        self.table = torch.randperm(self.pages, generator=gen, device="cuda")[: num_rows * pages_per_row]
        self.table = self.table.to(torch.int32).reshape(num_rows, pages_per_row).contiguous()
        self.k_pool, self.v_pool = (random_pool(hkv, self.pages, d, gen) for _ in range(2))
        self.positions = torch.tensor(positions, dtype=torch.int32, device="cuda")
        self.rows = torch.tensor(list(range(len(positions))) if rows is None else rows, dtype=torch.int32, device="cuda")
        self.T = len(positions)
        self.q = torch.randn((self.T, hq, d), generator=gen, device="cuda").to(torch.bfloat16)
        self.out = torch.full_like(self.q, float("nan"))
        self.desc = lnk.attn_desc(hq, hkv, d, self.pages, num_rows, pages_per_row, window=window, kv_dtype=lnk.KV_E2M1,
                                  scale=scale, k_scale=K_SCALE, v_scale=V_SCALE)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws_bytes = max(256, lnk.lnk_paged_workspace_size(self.desc, min(self.T, 4096)))
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device="cuda")

    def chunks(self, stream=None, out=None):
        self.lnk.lnk_paged_step_attn(self.desc, self.q, self.rows, self.positions, None, None, self.table, self.k_pool,
                                     self.v_pool, self.out if out is None else out, None, None, self.T, 0, 0, None, 0,
                                     self.status, stream)

    def decode(self, stream=None, out=None, ws=None):
        self.lnk.lnk_paged_decode_attn(self.desc, self.q, self.positions, self.table, self.k_pool, self.v_pool,
                                       self.out if out is None else out, self.T, self.ws if ws is None else ws,
                                       self.ws_bytes, self.status, stream)

    def check(self, skip=()):
        torch.cuda.synchronize()
        k = values_of(self.k_pool, K_SCALE, self.hkv, self.pages, self.d)
        v = values_of(self.v_pool, V_SCALE, self.hkv, self.pages, self.d)
        g = self.hq // self.hkv
        got = self.out.double()
        positions, rows = self.positions.long(), self.rows.long()
        ok = torch.ones(self.T, dtype=torch.bool, device="cuda")
        ok[list(skip)] = False
        idle = (positions < 0) & ok
        assert not self.out[idle].view(torch.int16).any(), "an inactive token's output is zero"
        for r in torch.unique(rows[ok & ~idle]).tolist():
            ts = torch.nonzero(ok & ~idle & (rows == r)).flatten()
            n = int(positions[ts].max()) + 1
            slots = (self.table[r].long().repeat_interleave(64) * 64 + torch.arange(64, device="cuda").repeat(self.table.shape[1]))[:n]
            kr, vr = k[:, slots], v[:, slots]
            q = self.q[ts].double().view(len(ts), self.hkv, g, self.d)
            s = torch.einsum("thgd,hnd->thgn", q, kr) * self.scale
            j = torch.arange(n, device="cuda")
            pos = positions[ts].view(-1, 1)
            seen = j <= pos
            if self.window:
                seen &= j > pos - self.window
            p = torch.softmax(s.masked_fill(~seen[:, None, None], float("-inf")), -1)
            want = torch.einsum("thgn,hnd->thgd", p, vr).reshape(len(ts), self.hq, self.d)
            spread = torch.einsum("thgn,hnd->thgd", p, vr.abs()).reshape(len(ts), self.hq, self.d)
            bound = 2.0 ** -8 * want.abs() + 2.0 ** -10 * spread + n * 2.0 ** -25 * float(vr.abs().max())
            off = (got[ts] - want).abs()
            assert bool((off <= bound).all()), f"row {r}: worst {float((off - bound).max()):.3g} beyond its bound"


def prompts(rng, total, num_rows, longest, pages_per_row):
    """Prompts in rows of their own (some with keys before them), a stretch of tokens
    of no row that covers whole tiles, single inactive tokens, and tokens whose row
    changes from one to the next."""
    rows, positions = [], []
    r = 0
    while len(rows) < total and r < num_rows:
        n = int(rng.integers(1, longest + 1))
        first = int(rng.integers(0, pages_per_row * 64 - n + 1))
        rows += [r] * n
        positions += list(range(first, first + n))
        r += 1
        if r == num_rows // 2:
            rows += [0] * 600
            positions += [-1] * 600
    mixed = 90
    rows += [int(x) for x in rng.integers(0, num_rows, mixed)]
    positions += [int(x) for x in rng.integers(0, pages_per_row * 64, mixed)]
    for t in rng.integers(0, len(rows), 40):
        positions[int(t)] = -1
    return rows, positions


@pytest.mark.parametrize("hq,hkv,d,window", [(32, 4, 128, 0), (16, 4, 96, 130), (32, 16, 64, 0), (7, 7, 128, 64)])
def test_many_tiles_in_each_cluster(hq, hkv, d, window):
    rng = np.random.default_rng(hq + d)
    rows, positions = prompts(rng, 256 * 8 * hkv // hq * 12, 60, 400, 12)
    c = Case(hq, hkv, d, 12, 60, positions, rows, window, seed=hq)
    c.chunks()
    c.check()
    assert int(c.status.item()) == 0
    first = c.out.clone()
    c.out.fill_(float("nan"))
    c.chunks()
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), c.out.view(torch.int16))


def test_running_maxima_that_jump_in_many_tiles():
    """Scores of several hundred: the accumulated output is rescaled at many steps.
    (Their float32 sums are good to 2^-24 of a few hundred times eight, a factor of
    1 + 2^-12 on a probability: within what the tolerance allows.)"""
    rng = np.random.default_rng(9)
    rows, positions = prompts(rng, 1500, 30, 300, 14)
    c = Case(16, 8, 128, 14, 30, positions, rows, scale=1.0)
    c.chunks()
    c.check()


def test_more_tiles_than_are_ordered_by_cost():
    rng = np.random.default_rng(5)
    n = 520 * 32 + 7  # tiles of 32 tokens
    rows = [int(x) for x in np.repeat(rng.integers(0, 30, n // 50 + 1), 50)[:n]]
    positions = [int(x) for x in rng.integers(0, 192, n)]
    c = Case(8, 1, 64, 3, 30, positions, rows)
    c.chunks()
    c.check()


def test_bad_rows_and_positions_among_many_tiles():
    rng = np.random.default_rng(6)
    rows, positions = prompts(rng, 3000, 40, 200, 6)
    c = Case(16, 8, 128, 6, 40, positions, rows)
    bad = [5, 700, 701, 2000]
    c.rows[5], c.rows[700] = 40, -1
    c.positions[701], c.positions[2000] = 6 * 64, 2 ** 30
    c.chunks()
    torch.cuda.synchronize()
    assert int(c.status.item()) == c.lnk.binding.DEV_BAD_ROW | c.lnk.binding.DEV_BAD_POSITION
    assert not c.out[bad].view(torch.int16).any()
    c.check(skip=bad)


@pytest.mark.parametrize("rows,hq,hkv,d,window", [(4096, 8, 1, 64, 0), (4096, 4, 4, 128, 0), (1500, 8, 2, 96, 40)])
def test_the_most_decode_rows(rows, hq, hkv, d, window):
    rng = np.random.default_rng(rows + d)
    positions = [int(x) for x in rng.integers(-1, 128, rows)]
    c = Case(hq, hkv, d, 2, rows, positions, window=window)
    c.decode()
    c.check()
    assert int(c.status.item()) == 0


def test_bad_positions_of_decode_rows_are_skipped_and_reported():
    c = Case(8, 2, 128, 4, 12, [3, 255, 256, 17, 2 ** 30, -1, 64, 63, 100, 200, 0, 1])
    c.decode()
    torch.cuda.synchronize()
    assert int(c.status.item()) == c.lnk.binding.DEV_BAD_POSITION
    assert not c.out[[2, 4, 5]].view(torch.int16).any()
    c.check(skip=[2, 4])


def test_calls_on_two_streams_and_graphs_that_share_a_workspace():
    rng = np.random.default_rng(8)
    dec = Case(32, 8, 128, 40, 24, [int(x) for x in rng.integers(500, 2560, 24)])
    rows, positions = prompts(rng, 1500, 20, 300, 8)
    chk = Case(32, 8, 128, 8, 20, positions, rows)
    dec.decode()
    chk.chunks()
    torch.cuda.synchronize()
    want_d, want_c = dec.out.clone(), chk.out.clone()
    # side by side, with a workspace each
    streams = [torch.cuda.Stream() for _ in range(3)]
    ws2 = torch.zeros_like(dec.ws)
    out2 = torch.full_like(dec.out, float("nan"))
    dec.out.fill_(float("nan"))
    chk.out.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(5):
        dec.decode(stream=streams[0])
        dec.decode(stream=streams[1], out=out2, ws=ws2)
        chk.chunks(stream=streams[2])
    torch.cuda.synchronize()
    for got, want in ((dec.out, want_d), (out2, want_d), (chk.out, want_c)):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    # two graphs with one workspace, replayed one after the other
    outs, graphs = [torch.full_like(dec.out, float("nan")) for _ in range(2)], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dec.decode(out=o)
            chk.chunks()
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want_d.view(torch.int16))
    assert torch.equal(chk.out.view(torch.int16), want_c.view(torch.int16))


def test_pools_past_32_bit_offsets():
    """Pages at the end of pools of more than 2^32 bytes: append, read back, decode,
    chunk and copy give what the same pages give in a small pool, bit for bit."""
    import paged_kv_gqa_row_gb300 as lnk
    hq, hkv, d, ppr = 16, 8, 128, 6
    gen = torch.Generator(device="cuda").manual_seed(3)
    lengths = [300, 64, 129, 1]
    T = sum(lengths)
    rows = torch.tensor(np.repeat(np.arange(4), lengths), dtype=torch.int32, device="cuda")
    positions = torch.tensor(np.concatenate([np.arange(n) for n in lengths]), dtype=torch.int32, device="cuda")
    last = torch.tensor([n - 1 for n in lengths], dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn((T, h, d), generator=gen, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    perm = torch.randperm(4 * ppr, generator=gen, device="cuda").to(torch.int32).reshape(4, ppr)
    results = []
    for pages in (4 * ppr + 2, 125000):
        k_pool, v_pool = (torch.zeros(hkv * pages * 36 * d, dtype=torch.uint8, device="cuda") for _ in range(2))
        table = (perm + (pages - 4 * ppr)).contiguous()
        desc = lnk.attn_desc(hq, hkv, d, pages, 4, ppr, kv_dtype=lnk.KV_E2M1, k_scale=K_SCALE, v_scale=V_SCALE)
        assert lnk.lnk_paged_page_bytes(desc) == 36 * d
        rope = lnk.rope_desc(10000.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out = torch.zeros_like(q)
        k_back, v_back = torch.zeros_like(k), torch.zeros_like(v)
        lnk.lnk_paged_append_rope(desc, rope, q, k, v, positions, rows, None, table, None, None, 1e-6, k_pool, v_pool,
                                  q_out, T, status)
        lnk.lnk_paged_read_tokens(desc, k_pool, v_pool, positions, rows, None, table, k_back, v_back, T, status)
        out = torch.zeros_like(q)
        lnk.lnk_paged_step_attn(desc, q_out, rows, positions, None, None, table, k_pool, v_pool, out, None, None, T, 0, 0,
                                None, 0, status)
        size = lnk.lnk_paged_workspace_size(desc, 4)
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        dec = torch.zeros((4, hq, d), dtype=torch.bfloat16, device="cuda")
        lnk.lnk_paged_decode_attn(desc, q_out[:4].contiguous(), last, table, k_pool, v_pool, dec, 4, ws, size, status)
        # the last page onto the first one
        src = torch.tensor([pages - 1], dtype=torch.int32, device="cuda")
        dst = torch.tensor([0], dtype=torch.int32, device="cuda")
        lnk.lnk_paged_copy_pages_layers(desc, [k_pool], [v_pool], src, dst, 1, status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        ends = [p.view(hkv, pages, 36 * d) for p in (k_pool, v_pool)]
        for e in ends:
            assert torch.equal(e[:, 0], e[:, pages - 1])
        results.append([q_out, k_back, v_back, out, dec] + [e[:, pages - 4 * ppr:].clone() for e in ends])
        del k_pool, v_pool, ends
    for small, large in zip(*results):
        assert torch.equal(small.view(torch.uint8) if small.dtype == torch.uint8 else small.view(torch.int16),
                           large.view(torch.uint8) if large.dtype == torch.uint8 else large.view(torch.int16))


FIRST_CALL = """
import sys
sys.path[:0] = ["tests", "."]
import torch
from test_gpu_fp4_large import Case
rng = __import__("numpy").random.default_rng(1)
rows, positions = [0] * 100 + [1] * 30, list(range(100)) + list(range(30))
chk = Case(8, 2, 128, 4, 2, positions, rows)
dec = Case(8, 2, 128, 4, 6, [5, 100, 255, 0, 64, -1])
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    chk.chunks()
    dec.decode()
    chk.lnk.lnk_paged_read_tokens(chk.desc, chk.k_pool, chk.v_pool, chk.positions, chk.rows, None, chk.table,
                                  torch.empty((130, 2, 128), dtype=torch.bfloat16, device="cuda"), None, 130, chk.status)
graph.replay()
chk.check()
dec.check()
print("captured")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    """What a kernel's launch sets up once per device is allowed inside a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]

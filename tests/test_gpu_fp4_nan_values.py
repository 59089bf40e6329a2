"""Keys and values of 4-bit pools whose block scale is NaN (as the append stores a
block that holds one): they reach exactly the outputs that see them.  A masked key
adds nothing, whichever prompts and tokens share its tile, and a NaN value block
makes NaN of its own 16 dimensions alone.

Finite outputs are held to the bound of test_gpu_fp4_attention."""
import numpy as np
import pytest

import synth
from harness import to_bits
from oracle import bf16 as obf16
from oracle import fp4 as ofp4
from oracle import paged as opaged
from test_gpu_fp4 import K_SCALE, V_SCALE, F4Step, d8, u8
from test_gpu_fp4_attention import decode, step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def poison(pool, slot, head, blocks, code=0x7F):
    """NaN scales for `blocks` of one slot and kv head of a pool on the host."""
    page = pool[head, slot // 64]
    d = page.shape[-1] // 36
    for b in blocks:
        page[ofp4.scale_offset(slot % 64, b, d)] = code


def check(w, dev, k_host, v_host, tokens=None):
    torch.cuda.synchronize()
    assert int(dev.status.item()) == 0
    with np.errstate(all="ignore"):
        kv, vv = ofp4.pool_values(k_host, K_SCALE), ofp4.pool_values(v_host, V_SCALE)
    out, q = obf16.to_f64(to_bits(dev.out)), to_bits(dev.q_out)
    rows, positions = w.token_rows(), w.token_positions()
    clean = 0
    for t in range(w.T) if tokens is None else tokens:
        r, p = int(rows[t]), int(positions[t])
        what = f"token {t} of row {r} at {p}"
        with np.errstate(all="ignore"):
            want = ofp4.attention_at(q[t], r, p, w.table, kv, vv, w.window)
            spread = ofp4.attention_at(q[t], r, p, w.table, kv, np.abs(vv), w.window)
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(out[t]), nan), \
            f"{what}: {int((np.isnan(out[t]) & ~nan).sum())} NaN too many, {int((~np.isnan(out[t]) & nan).sum())} missing"
        lo, hi = opaged.visible_range(p, w.window)
        top = np.abs(np.nan_to_num(vv[:, opaged.row_slots(w.table, r, lo, hi)])).max()
        bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * spread + (hi - lo + 1) * 2.0 ** -25 * top
        assert (np.abs(out[t] - want) <= bound + 1e-30)[~nan].all(), f"{what}: outside the bound"
        clean += not nan.any()
    return clean


CASES = [
    # hq, hkv, d, decode lengths, chunks (start, tokens), window, poisoned (chunk, position)
    ("two-prompts-one-tile", 8, 2, 128, [], [(0, 30), (0, 20)], 0, [(0, 10)]),
    ("three-prompts-96", 4, 2, 96, [200, 3], [(0, 40), (70, 9), (500, 40)], 0, [(0, 7), (2, 515)]),
    ("mha64-steps", 3, 3, 64, [], [(0, 257), (1000, 3)], 0, [(0, 0), (0, 130), (1, 999)]),
    ("window-96", 4, 2, 96, [300], [(90, 150), (0, 99), (640, 70)], 100, [(0, 95), (1, 50), (2, 600), (2, 700)]),
    ("gqa8", 16, 2, 128, [40], [(17, 33), (0, 31), (300, 40)], 0, [(1, 30), (2, 127), (2, 128)]),
    ("many-steps", 2, 1, 128, [], [(900, 260)], 0, [(0, 1000), (0, 1100)]),
]


@pytest.mark.parametrize("which", ["values", "keys", "both"])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_nan_blocks_reach_only_the_tokens_that_see_them(case, which):
    name, hq, hkv, d, lengths, chunks, window, where = case
    w = synth.custom(seed=300 + len(name), hq=hq, hkv=hkv, head_dim=d, dec_lengths=lengths, chunks=chunks, window=window)
    dev = F4Step(w)
    dev.append()
    torch.cuda.synchronize()
    pools = [u8(dev.k_pool), u8(dev.v_pool)]
    starts = np.concatenate([[0], np.cumsum([n for _, n in chunks])])
    for i, (c, p) in enumerate(where):
        row = int(w.ch_rows[starts[c]])
        slot = int(w.table[row, p // 64]) * 64 + p % 64
        # first, last and all blocks of some heads in turn
        blocks = [[0], [d // 16 - 1], list(range(d // 16)), [1, d // 16 - 2]][i % 4]
        for pool, use in zip(pools, (which != "values", which != "keys")):
            if use:
                poison(pool, slot, i % hkv, blocks, 0x7F if i % 2 == 0 else 0xFF)
    dev.k_pool.copy_(d8(pools[0]))
    dev.v_pool.copy_(d8(pools[1]))
    step(dev)
    check(w, dev, *pools)


@pytest.mark.parametrize("poisoned", [(0,), (0, 5, 6, 12), (3, 4, 9)])
def test_pages_of_nan_values_among_many_tiles(poisoned):
    """More items than clusters, so that tiles follow one another in a cluster: all
    values of some prompts' first pages are NaN, the others' rows stay as they were."""
    w = synth.custom(seed=52, hq=8, hkv=4, head_dim=64, dec_lengths=[], chunks=[(0, 64)] + [(100, 500)] * 12)
    dev = F4Step(w)
    dev.append()
    step(dev)
    torch.cuda.synchronize()
    clean = dev.out.clone()
    pools = [u8(dev.k_pool), u8(dev.v_pool)]
    ends = np.cumsum([64] + [500] * 12)
    bad = np.zeros(w.T, dtype=bool)
    for c in poisoned:
        first = ends[c - 1] if c else 0
        bad[first:ends[c]] = True
        pools[1][:, int(w.table[int(w.ch_rows[first]), 0]), 32 * 64:] = 0x7F
    dev.v_pool.copy_(d8(pools[1]))
    dev.out.fill_(0)
    step(dev)
    check(w, dev, *pools, tokens=[0, 63, 64, 100, 700, 2600, 6000])
    bad = torch.from_numpy(bad).cuda()
    assert torch.equal(dev.out[~bad], clean[~bad])
    assert torch.isnan(dev.out[bad].view(torch.bfloat16)).all()


def test_decode_keeps_nan_to_its_row_and_dimensions():
    w = synth.custom(seed=53, hq=8, hkv=2, head_dim=128, dec_lengths=[5, 64, 130, 300, 1000], window=200)
    dev = F4Step(w)
    dev.append()
    torch.cuda.synchronize()
    pools = [u8(dev.k_pool), u8(dev.v_pool)]
    for row, p, blocks in ((0, 2, [3]), (3, 250, [0, 7]), (4, 100, range(8))):  # (the last one before its window)
        poison(pools[1], int(w.table[row, p // 64]) * 64 + p % 64, 1, blocks)
    poison(pools[0], int(w.table[2, 1]) * 64 + 5, 0, [2])
    for dst, src in zip((dev.k_pool, dev.v_pool), pools):
        dst.copy_(d8(src))
    decode(dev)
    assert check(w, dev, *pools) == 2

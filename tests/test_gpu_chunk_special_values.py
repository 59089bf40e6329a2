"""Prompt chunks over bf16 pools whose cached values hold NaN or infinities, or whose
keys hold NaN: they reach exactly the outputs that see them.  (A product multiplies
every value row of a step into all rows of a tile, those whose weight for it is
zero among them.)

Expectation: exact attention in float64 over the pool's values, with IEEE's rules."""
import numpy as np
import pytest

import synth
from harness import ATT_MAX_ABS, DeviceStep, to_bits
from oracle import bf16 as obf16
from oracle import paged as opaged
from test_gpu_fp4 import d16

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NAN, INF, NEG = 0x7FC0, 0x7F80, 0xFF80

CASES = [
    # hq, hkv, d, decode lengths, chunks (start, tokens), window, poisoned (chunk, position, dimensions, bits)
    ("two-prompts-one-tile", 8, 2, 128, [], [(0, 30), (0, 20)], 0, [(0, 10, [0, 77], NAN)]),
    ("three-prompts-96", 4, 2, 96, [200, 3], [(0, 40), (70, 9), (500, 40)], 0,
     [(0, 7, [95], INF), (2, 515, range(96), NAN)]),
    ("mha64-steps", 3, 3, 64, [], [(0, 257), (1000, 3)], 0, [(0, 0, [3], NEG), (0, 130, [3, 40], INF), (1, 999, [63], NAN)]),
    ("window-96", 4, 2, 96, [300], [(90, 150), (0, 99), (640, 70)], 100,
     [(0, 95, [1], NAN), (1, 50, [48], INF), (2, 600, [0], NAN), (2, 700, [47, 48], NEG)]),
    ("gqa8", 16, 2, 128, [40], [(17, 33), (0, 31), (300, 40)], 0,
     [(1, 30, [64], NAN), (2, 127, [63], INF), (2, 128, [127], NAN)]),
    ("many-steps", 2, 1, 128, [], [(900, 260)], 0, [(0, 1000, [5], NAN), (0, 1100, [6], INF)]),
]


@pytest.mark.parametrize("which", ["values", "keys"])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_special_values_reach_only_the_tokens_that_see_them(case, which):
    name, hq, hkv, d, lengths, chunks, window, where = case
    w = synth.custom(seed=400 + len(name), hq=hq, hkv=hkv, head_dim=d, dec_lengths=lengths, chunks=chunks, window=window)
    dev = DeviceStep(w, fill="host")
    dev.step()
    torch.cuda.synchronize()
    k, v = to_bits(dev.k_pool).copy(), to_bits(dev.v_pool).copy()
    starts = np.concatenate([[0], np.cumsum([n for _, n in chunks])])
    for i, (c, p, dims, bits) in enumerate(where):
        row = int(w.ch_rows[starts[c]])
        slot = int(w.table[row, p // 64]) * 64 + p % 64
        if which == "values":
            v[i % hkv, slot, list(dims)] = bits
        else:
            k[i % hkv, slot, list(dims)] = NAN
    dev.k_pool.copy_(d16(k))
    dev.v_pool.copy_(d16(v))
    dev.out.fill_(0x1234)
    dev.attend()
    torch.cuda.synchronize()
    assert int(dev.status.item()) == 0
    got, q = obf16.to_f64(to_bits(dev.out)), to_bits(dev.q_out)
    rows, positions = w.token_rows(), w.token_positions()
    for t in range(w.T):
        with np.errstate(all="ignore"):
            want = opaged.attention_at(q[t], int(rows[t]), int(positions[t]), w.table, k, v, w.window)
        what = f"token {t} of row {rows[t]} at {positions[t]}"
        finite = np.isfinite(want)
        assert np.array_equal(np.isnan(got[t]), np.isnan(want)), \
            f"{what}: {int(np.isnan(got[t]).sum())} NaN for {int(np.isnan(want).sum())}"
        assert np.array_equal(got[t][~finite & ~np.isnan(want)], want[~finite & ~np.isnan(want)]), f"{what}: infinities"
        assert np.abs(got[t] - want)[finite].max(initial=0) <= ATT_MAX_ABS, what


def test_a_prompt_of_nan_values_among_others():
    w = synth.custom(seed=9, hq=8, hkv=4, head_dim=64, dec_lengths=[], chunks=[(0, 64)] + [(100, 300)] * 6)
    dev = DeviceStep(w, fill="host")
    dev.step()
    torch.cuda.synchronize()
    clean = dev.out.clone()
    page = int(w.table[int(w.ch_rows[0]), 0])
    dev.v_pool[:, page * 64:page * 64 + 64] = NAN
    dev.out.fill_(0)
    dev.attend()
    torch.cuda.synchronize()
    assert torch.isnan(dev.out[:64].view(torch.bfloat16)).all()
    err = (dev.out[64:].view(torch.bfloat16).float() - clean[64:].view(torch.bfloat16).float()).abs().max()
    assert float(err) <= 2 * ATT_MAX_ABS  # (both within the bound of exact attention; NaN fails it too)

"""Absorbed latent attention where the rows of one tile see different keys: what some of them
do not see adds nothing to them, whatever it is (tolerances: latent_harness)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from latent_harness import PAGE, Step, bits, check, d32  # noqa: E402
from oracle import bf16, latent  # noqa: E402

pytestmark = pytest.mark.gpu

NAN, INF, MINUS_INF = 0x7FC0, 0x7F80, 0xFF80

# A tile holds so many tokens: 64 query rows on one SM, or 128 on a pair of them in launches of
# at least 16 piece rows an SM.
KINDS = {"one-sm": (16, 4, 8), "pairs": (40, 3, 90)}  # heads, tokens a tile, tokens of the piece


def slot(s, row, position):
    return s.table[row, position // PAGE] * PAGE + position % PAGE


def piece(kind, before, seed, **kw):
    heads, per_tile, count = KINDS[kind]
    s = Step(seed, heads, 256, 64, pieces=[(count, before)], dec=[500], **kw)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert (count * heads >= 16 * sms) == (kind == "pairs")
    return s, per_tile


def compare(s, out, t, row, p, clean):
    want, spread, size = latent.attention_at(s.q[t], row, p, s.table, clean, s.c, s.scale, s.window)
    check(out[t], want, spread, size, p + 1, s.c + s.r, f"token {t}, row {row} at {p}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("before", [100, 4000], ids=["whole", "cut"])
def test_tokens_without_keys_among_others(kind, before):
    """Inactive tokens and tokens behind the table's end are zero, with a key that is not finite
    in what all the other tokens of their tile see."""
    s, per_tile = piece(kind, before, 31)
    s.pool[slot(s, 1, 70), :5] = NAN
    past = s.table.shape[1] * PAGE
    empty = {0: -1, per_tile + 1: past, per_tile + 2: -1, 2 * per_tile - 1: past, s.P - 1: -1}
    for t, p in empty.items():
        s.positions[t] = p
    s.upload().run()
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0x02
    out = bits(s.out)
    for t in range(s.P):
        if t in empty:
            assert not out[t].any(), f"token {t}"
        else:
            assert np.isnan(bf16.to_f64(out[t])).all(), f"token {t}"
    compare(s, out, s.P, 0, 499, s.pool)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("before", [100, 4000], ids=["whole", "cut"])
@pytest.mark.parametrize("bad", [NAN, INF, MINUS_INF], ids=["nan", "inf", "-inf"])
def test_keys_that_only_a_tiles_last_tokens_see(kind, before, bad):
    s, per_tile = piece(kind, before, 32)
    first = per_tile + 2  # the first token that sees the key: neither first nor alone in its tile
    assert first % per_tile != 0
    clean = s.pool.copy()
    s.pool[slot(s, 1, before + first)] = bad
    s.upload().run()
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    out = bits(s.out)
    for t, row, p in s.tokens():
        if row == 1 and t >= first:
            f = bf16.to_f64(out[t])
            assert np.isnan(f).all() if bad == NAN else not np.isfinite(f).all()
        elif row == 0 or t >= first - per_tile:
            compare(s, out, t, row, p, clean)
        else:
            assert np.isfinite(bf16.to_f64(out[t])).all(), f"token {t}"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("before,window", [(300, 65), (4000, 2000)], ids=["whole", "cut"])
def test_keys_that_leave_the_window_inside_a_tile(kind, before, window):
    s, per_tile = piece(kind, before, 33, window=window)
    last = per_tile + 1  # the last token that sees the key: one behind it in its tile does not
    assert last % per_tile != per_tile - 1
    clean = s.pool.copy()
    s.pool[slot(s, 1, before + last - window + 1), 3:7] = NAN
    s.upload().run()
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    out = bits(s.out)
    for t, row, p in s.tokens():
        if row == 1 and t <= last:
            assert np.isnan(bf16.to_f64(out[t])).all(), f"token {t}"
        elif row == 0 or t <= last + 2 * per_tile:
            compare(s, out, t, row, p, clean)


@pytest.mark.parametrize("kind", KINDS)
def test_pages_between_two_windows_need_not_be_there(kind):
    """Two tokens of one tile far apart in their row: the pages that neither's window reaches."""
    s, per_tile = piece(kind, 500, 34, window=65)
    s.positions[:] = -1
    s.positions[:2] = 70, 500
    s.table[1, 2:6] = (-1, s.pages, -1, -1)
    s.upload().run().verify()


@pytest.mark.parametrize("heads,pieces,dec", [(16, [(5, 100)], [700]), (16, [], [5000, 64]), (40, [(90, 100)], [700]),
                                              (128, [(2, 70)], [3000])], ids=["one-sm", "cut", "pairs", "cut-pairs"])
def test_large_latents_behind_a_first_key_of_low_score(heads, pieces, dec):
    """Sums stay in float32's range where the softmax of the same numbers does: weights relative to the
    first key's score, 2^26 to 2^30 for the others here, and latents of 2^100."""
    s = Step(35, heads, 256, 64, pieces=pieces, dec=dec, scale=1.0)
    rng = np.random.default_rng(36)
    s.q[:, :, :s.c] = 0
    s.q[:, :, s.c:] = bf16.from_f64(np.ones((1,)))[0]
    s.pool[:, :s.c] = bf16.from_f64(bf16.to_f64(s.pool[:, :s.c]) * 2.0 ** 100)
    s.pool[:, s.c:] = bf16.from_f64(rng.choice([-1, 1], (len(s.pool), s.r)) * rng.uniform(0.02, 0.06, (len(s.pool), s.r)))
    for row in range(s.table.shape[0]):
        s.pool[slot(s, row, 0), s.c:] = bf16.from_f64(np.full(s.r, -0.3))
    s.upload().run().verify()

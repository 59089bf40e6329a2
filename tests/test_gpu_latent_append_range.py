"""lnk_latent_append where numbers are small, large or not finite, and far positions: what lnk.h says of
lnk_paged_append_rope holds for it, with the norm over the latent's C numbers."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from latent_harness import bits, d16, d32, normal  # noqa: E402
from oracle import bf16, latent, rope  # noqa: E402

pytestmark = pytest.mark.gpu

PAGE = 64
NAN, INF, MINUS_INF = 0x7FC0, 0x7F80, 0xFF80


def append(q, kv, positions, c, w=None, eps=0.0, theta=1e4):
    """Token t into slot t; q's and the pool's bits after the call."""
    import paged_kv_gqa_row_gb300 as lnk
    t, heads, r = q.shape
    pages = -(-t // PAGE)
    desc = lnk.latent_desc(heads, c, r, pages, 1, 1, scale=1.0)
    pool = torch.full((pages * PAGE, c + r), 0x1234, dtype=torch.int16, device="cuda")
    q_out, kv_out = torch.empty((t, heads, r), dtype=torch.int16, device="cuda"), torch.empty((t, c + r), dtype=torch.int16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lnk.lnk_latent_append(desc, lnk.rope_desc(theta), d16(q), r, d16(kv), d32(positions), None, d32(np.arange(t)), None,
                          None if w is None else d16(w), eps, pool, q_out, r, kv_out, t, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = bits(pool)
    assert (got[:t] == bits(kv_out)).all() and (got[t:] == 0x1234).all()
    return bits(q_out), got[:t]


def close(got, want, what):
    d = bf16.ulp_distance(got, want)
    assert d.max(initial=0) <= 1 and (d != 0).sum() <= 1 + d.size // 1000000, f"{what}: {int((d != 0).sum())} differ"


def rows_of_magnitudes(rng, t, n, low, high):
    x = rng.standard_normal((t, n))
    x = np.where(np.abs(x) < 2.0 ** -10, 2.0 ** -10, x)
    return bf16.from_f64(x * np.exp2(rng.integers(low, high + 1, (t, 1))))


@pytest.mark.parametrize("t", [7, 900], ids=["few", "many"])
@pytest.mark.parametrize("c,r", [(512, 64), (128, 32), (384, 64)])
def test_rows_in_the_stated_range_match_the_oracle(t, c, r):
    """Mean squares of 2^-96 to 2^118 without an epsilon (their sum over 512 numbers stays in float32's range)."""
    rng = np.random.default_rng(t + c)
    kv = np.concatenate([rows_of_magnitudes(rng, t, c, -45, 57), normal(rng, t, r)], axis=1)
    q, w, positions = normal(rng, t, 6, r), bf16.from_f64(1 + 0.1 * rng.standard_normal(c)), np.arange(t) * 7
    got_q, got = append(q, kv, positions, c, w)
    want_q, want, _ = latent.append(q, kv, positions, None, None, np.zeros_like(kv), rope.inv_freq(1e4, r), c, np.arange(t), w, 0.0)
    close(got_q, want_q, "queries")
    close(got, want, "rows")


@pytest.mark.parametrize("t", [7, 900], ids=["few", "many"])
def test_rows_that_are_not_finite_or_whose_squares_are_not(t):
    rng = np.random.default_rng(t)
    c, r = 256, 64
    kv, q, w, positions = normal(rng, t, c + r), normal(rng, t, 5, r), normal(rng, c), np.arange(t) * 3
    want_q, want, _ = latent.append(q, kv, positions, None, None, np.zeros_like(kv), rope.inv_freq(1e4, r), c, np.arange(t), w, 0.0)
    bad = {0: (17, INF), 2: (255, NAN), 3: (0, MINUS_INF), 5: (100, bf16.from_f64(np.array([2.0 ** 64]))[0])}
    for row, (at, x) in bad.items():
        kv[row, at] = x
    kv[1, :c] = bf16.from_f64(np.full(c, 2.0 ** 61))  # each square is in range, their sum is not
    kv[4, :c] = 0                                     # no mean and no epsilon: 0 / 0
    nan = np.array([0, 1, 2, 3, 4, 5])
    got_q, got = append(q, kv, positions, c, w)
    assert np.isnan(bf16.to_f64(got[nan, :c])).all()
    others = np.setdiff1d(np.arange(t), nan)
    close(got[others], want[others], "rows")
    close(got[nan, c:], want[nan, c:], "rotated parts of the rows that are not")
    close(got_q, want_q, "queries")
    # without a norm the latent is copied bit for bit, and an epsilon makes zeros of a row of zeros
    assert (append(q, kv, positions, c)[1][:, :c] == kv[:, :c]).all()
    assert not append(q, kv, positions, c, w, 1e-6)[1][4, :c].any()


@pytest.mark.parametrize("t", [9, 900], ids=["few", "many"])
def test_rotations_of_numbers_that_are_not_finite(t):
    """Each result by the float32 expression where an element is not finite or the result is beyond float32's
    range; the pairs beside it as ever."""
    rng = np.random.default_rng(50 + t)
    c, r, heads = 128, 64, 3
    h = r // 2
    kv, q, positions = normal(rng, t, c + r), normal(rng, t, heads, r), np.arange(t) * 5
    big = bf16.from_f64(np.array([3.3e38]))[0]
    inv = rope.inv_freq(1e4, r)
    spots = [(0, 0, (INF, None)), (1, 3, (None, NAN)), (2, 5, (MINUS_INF, INF)), (3, 31, (NAN, INF)), (4, 1, (None, MINUS_INF)),
             (5, 0, (big, big)), (6, 2, (big, big | 0x8000)), (8, 7, (INF, INF))]
    want_q, want, _ = latent.append(q, kv, positions, None, None, np.zeros_like(kv), inv, c, np.arange(t))
    want_q, want_k = bf16.to_f64(want_q), bf16.to_f64(want[:, c:])
    for token, e, (x1, x2) in spots:
        ang = rope.angles(int(positions[token]), inv)
        for src, to in ((q[token, 1], want_q[token, 1]), (kv[token, c:], want_k[token])):
            if x1 is not None:
                src[e] = x1
            if x2 is not None:
                src[e + h] = x2
            a, b = np.float32(bf16.to_f64(src[e])), np.float32(bf16.to_f64(src[e + h]))
            cs, sn = np.float32(np.cos(np.float64(ang[e]))), np.float32(np.sin(np.float64(ang[e])))
            with np.errstate(all="ignore"):
                to[e], to[e + h] = a * cs - b * sn, b * cs + a * sn
    got_q, got = append(q, kv, positions, c)
    for got64, want64, what in ((bf16.to_f64(got_q), want_q, "queries"), (bf16.to_f64(got[:, c:]), want_k, "keys")):
        top = 3.3961775292304961e38  # from here on float32 rounds to infinity in bf16
        want64 = np.where(np.abs(want64) >= top, np.copysign(np.inf, want64), want64)
        same = (got64 == want64) | (np.isnan(got64) & np.isnan(want64)) | (np.abs(got64 - want64) <= 2.0 ** -8 * np.abs(want64))
        assert same.all(), f"{what}: {got64[~same]} for {want64[~same]}"


@pytest.mark.parametrize("t", [8, 800], ids=["few", "many"])
@pytest.mark.parametrize("theta", [1e4, 1e6])
def test_far_positions(t, theta):
    rng = np.random.default_rng(60 + t)
    c, r = 128, 64
    some = np.array([2 ** 20 - 1, 2 ** 20, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 27 - 5, 2 ** 31 - 1, 12345678, 2 ** 30])
    positions = np.resize(some, t)
    kv, q, w = normal(rng, t, c + r), normal(rng, t, 9, r), normal(rng, c)
    got_q, got = append(q, kv, positions, c, w, 1e-6, theta)
    want_q, want, _ = latent.append(q, kv, positions, None, None, np.zeros_like(kv), rope.inv_freq(theta, r), c, np.arange(t), w,
                                    float(np.float32(1e-6)))
    close(got_q, want_q, "queries")
    close(got, want, "rows")

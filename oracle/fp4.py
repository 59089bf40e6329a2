"""4-bit (E2M1) page pools for the oracle (test infrastructure only).

The pages define the pool as bf16; a 4-bit pool is a variant this library adds.
The readings taken, each stated once here and in the design notes:

  * Codes: OCP E2M1: 1 sign bit, 2 exponent bits with bias 1, 1 mantissa bit;
    exponent field 0 holds 0 and 0.5; no infinities, no NaN; largest 6.
  * Blocks: 16 consecutive dimensions of one head's row share one E4M3 scale
    code (oracle/fp8.py); each pool has one float32 scale ps besides.
  * Quantizer, on the bf16 values x a bf16 pool would hold, every operation one
    IEEE float32 operation:
        s = E4M3(max|x| / (6 ps)),  d = e4m3(s) * ps,  code = E2M1(x / d)
    both formats rounding to nearest even and saturating; d = 0 stores s = 0
    and zero codes; a NaN in the block stores the NaN scale and zero codes.
  * Page of one head, 36 D bytes: 64 rows of D / 2 code bytes (even dimension in
    the low four bits), then 4 D scale codes, position j's scale of block b at
    ((j % 4) * (D / 16) + b) * 16 + j / 4.
  * Attention over a 4-bit pool is the exact attention of the dequantized keys
    and values.
"""
import numpy as np

from . import bf16
from . import fp8
from . import paged

BLOCK = 16
PAGE = paged.PAGE_SIZE
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
NAN_SCALE = 0x7F


def decode(codes) -> np.ndarray:
    """Value of each E2M1 code (0..15), float64."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, m = (c >> 1) & 3, (c & 1).astype(np.float64)
    mag = np.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * np.exp2(e.astype(np.float64) - 1.0))
    return np.where(c & 8, -mag, mag)


def encode(x) -> np.ndarray:
    """Nearest E2M1 code, ties to the even code, magnitudes above 6 saturating."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 6.0)
    hi = np.searchsorted(MAGNITUDES, a, side="left")
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - MAGNITUDES[lo], MAGNITUDES[hi] - a
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    return code.astype(np.uint8) | (np.signbit(x).astype(np.uint8) << 3)


def quantize(bits, ps: float):
    """(codes [..., D], scale codes [..., D / 16]) of bf16 rows ``bits`` [..., D]."""
    bits = np.asarray(bits, dtype=np.uint16)
    x = bf16.to_f64(bits).astype(np.float32).reshape(*bits.shape[:-1], -1, BLOCK)
    ps32 = np.float32(ps)
    nan = np.isnan(x).any(-1)
    with np.errstate(all="ignore"):
        a = np.abs(np.where(nan[..., None], np.float32(0), x)).max(-1)
        t = a / (np.float32(6.0) * ps32)
        s = fp8.encode(t.astype(np.float64))
        d = fp8.decode(s).astype(np.float32) * ps32
        dead = ~(d > 0)
        s = np.where(nan, NAN_SCALE, np.where(dead, 0, s)).astype(np.uint8)
        u = x / np.where(dead, np.float32(1), d)[..., None]
    codes = np.where((nan | dead)[..., None], 0, encode(np.where(nan[..., None], 0.0, u.astype(np.float64))))
    return codes.astype(np.uint8).reshape(bits.shape), s


def row_values(codes, scales, ps: float) -> np.ndarray:
    """float64 values of codes [..., D] with scale codes [..., D / 16]."""
    return decode(codes) * np.repeat(fp8.decode(scales), BLOCK, axis=-1) * float(np.float32(ps))


def scale_offset(j: int, b: int, d: int) -> int:
    return 32 * d + ((j % 4) * (d // BLOCK) + b) * 16 + j // 4


def write_row(page: np.ndarray, j: int, codes, scales) -> None:
    """Writes one position's row into a page of one head (36 D bytes, in place)."""
    d = page.shape[-1] // 36
    page[j * (d // 2):(j + 1) * (d // 2)] = codes[0::2] | (codes[1::2] << 4)
    for b in range(d // BLOCK):
        page[scale_offset(j, b, d)] = scales[b]


def read_row(page: np.ndarray, j: int):
    """(codes [D], scale codes [D / 16]) of one position."""
    d = page.shape[-1] // 36
    raw = page[j * (d // 2):(j + 1) * (d // 2)]
    codes = np.stack([raw & 15, raw >> 4], axis=-1).reshape(d)
    return codes, np.array([page[scale_offset(j, b, d)] for b in range(d // BLOCK)], dtype=np.uint8)


def pack_pool(codes, scales) -> np.ndarray:
    """Pool bytes [Hkv, pages, 36 D] of codes [Hkv, slots, D], scales [Hkv, slots, D / 16]."""
    h, n, d = codes.shape
    pool = np.empty((h, n // PAGE, 36 * d), dtype=np.uint8)
    c = codes.reshape(h, n // PAGE, PAGE, d)
    pool[..., :32 * d] = (c[..., 0::2] | (c[..., 1::2] << 4)).reshape(h, n // PAGE, 32 * d)
    s = scales.reshape(h, n // PAGE, PAGE, d // BLOCK)
    for j in range(PAGE):
        for b in range(d // BLOCK):
            pool[..., scale_offset(j, b, d)] = s[:, :, j, b]
    return pool


def pool_values(pool: np.ndarray, ps: float) -> np.ndarray:
    """float64 values [Hkv, slots, D] of a whole pool."""
    h, n, size = pool.shape
    d = size // 36
    raw = pool[..., :32 * d].reshape(h, n, PAGE, d // 2)
    codes = np.stack([raw & 15, raw >> 4], axis=-1).reshape(h, n, PAGE, d)
    scales = np.empty((h, n, PAGE, d // BLOCK), dtype=np.uint8)
    for j in range(PAGE):
        for b in range(d // BLOCK):
            scales[:, :, j, b] = pool[..., scale_offset(j, b, d)]
    return row_values(codes, scales, ps).reshape(h, n * PAGE, d)


def append_rope(q, k, v, positions, rows, table, k_pool, v_pool, inv, k_scale, v_scale,
                slots=None, gamma_q=None, gamma_k=None, eps=1e-6):
    """The bf16 append (oracle.paged.append_rope), then the quantizer on the
    rows it writes.  Pools: bytes [Hkv, pages, 36 D] (not modified).  Returns
    (q_out, k_pool', v_pool')."""
    hkv, n = k_pool.shape[:2]
    scratch = np.zeros((hkv, n * PAGE, q.shape[-1]), dtype=np.uint16)
    q_out, kb, vb = paged.append_rope(q, k, v, positions, rows, table, scratch, scratch, inv,
                                      slots=slots, gamma_q=gamma_q, gamma_k=gamma_k, eps=eps)
    k_pool, v_pool = k_pool.copy(), v_pool.copy()
    for t in range(q.shape[0]):
        p = int(positions[t])
        if p < 0:
            continue
        s = int(slots[t]) if slots is not None else paged.slot_of(table, int(rows[t]), p)
        for pool, bits, ps in ((k_pool, kb, k_scale), (v_pool, vb, v_scale)):
            codes, scales = quantize(bits[:, s, :], ps)
            for h in range(hkv):
                write_row(pool[h, s // PAGE], s % PAGE, codes[h], scales[h])
    return q_out, k_pool, v_pool


def attention_at(q_bits, row, position, table, k_values, v_values, window, scale=None):
    """Output of one token over its row's visible keys; ``k_values`` and
    ``v_values`` are a pool's values (pool_values).  Returns float64 [Hq, D]."""
    hq, d = q_bits.shape
    hkv = k_values.shape[0]
    group = hq // hkv
    if scale is None:
        scale = paged.default_scale(d)
    out = np.zeros((hq, d), dtype=np.float64)
    if position < 0:
        return out
    lo, hi = paged.visible_range(position, window)
    slots = paged.row_slots(table, row, lo, hi)
    qf = bf16.to_f64(q_bits)
    for kvh in range(hkv):
        heads = [h for h in range(hq) if paged.kv_head_of(h, group, hkv) == kvh]
        out[heads] = paged.attend(qf[heads], k_values[kvh, slots, :], v_values[kvh, slots, :], scale)
    return out


def step_attention(q_out, rows, positions, step_positions, table, k_values, v_values, window, scale=None):
    """P chunk tokens followed by B decode rows (row b = table row b)."""
    every = list(zip(rows, positions)) + list(enumerate(step_positions))
    out = np.zeros(q_out.shape, dtype=np.float64)
    for t, (r, p) in enumerate(every):
        out[t] = attention_at(q_out[t], int(r), int(p), table, k_values, v_values, window, scale)
    return out

"""The latent cache for the oracle (test infrastructure only).

A pool row is [c, k]: a latent vector of C numbers, the value of every head and the
first part of its key, and R rotated numbers.  float64 throughout; tensors are bf16
bit patterns.  Rows of pages and rotations are those of ``paged`` and ``rope``.
"""
import numpy as np

from . import bf16, paged, rope


def append(q, kv, positions, rows, table, pool, inv, latent_dim, slots=None, norm_w=None, eps=1e-6):
    """q: bf16 [T, H, R]; kv: bf16 [T, C + R]; pool: bf16 [S, C + R] (not modified).

    Returns (q_out, kv_out, pool') as bf16 arrays; inactive tokens give zeros.
    """
    c = latent_dim
    q_out, kv_out = np.zeros_like(q, dtype=np.uint16), np.zeros_like(kv, dtype=np.uint16)
    pool = np.array(pool, dtype=np.uint16, copy=True)
    for t in range(q.shape[0]):
        p = int(positions[t])
        if p < 0:
            continue
        ang = rope.angles(p, inv)
        q_out[t] = bf16.from_f64(rope.rotate(bf16.to_f64(q[t]), ang))
        kv_out[t, :c] = kv[t, :c]
        if norm_w is not None:
            kv_out[t, :c] = bf16.from_f64(rope.qk_norm(bf16.to_f64(kv[t, :c]), bf16.to_f64(norm_w), eps))
        kv_out[t, c:] = bf16.from_f64(rope.rotate(bf16.to_f64(kv[t, c:]), ang))
        s = int(slots[t]) if slots is not None else paged.slot_of(table, int(rows[t]), p)
        pool[s] = kv_out[t]
    return q_out, kv_out, pool


def attend(q, keys, values, scale):
    """softmax(q keys^T scale) values and the same of |values|, with what the products of
    the scores add up to in magnitude (the largest of a row).  q: [H, W]."""
    s = (q @ keys.T) * scale
    w = np.exp(s - np.max(s, axis=1, keepdims=True))
    w /= np.sum(w, axis=1, keepdims=True)
    size = np.max((np.abs(q) @ np.abs(keys).T) * scale, axis=1, keepdims=True)
    return w @ values, w @ np.abs(values), size


def attention_at(q_bits, row, position, table, pool, latent_dim, scale, window=0):
    """One token's absorbed attention, [H, C] (and the two magnitudes of attend)."""
    lo, hi = paged.visible_range(position, window)
    keys = bf16.to_f64(pool[paged.row_slots(table, row, lo, hi)])
    return attend(bf16.to_f64(q_bits), keys, keys[:, :latent_dim], scale)


def expanded_at(q_bits, kv_bits, k_rope_bits, head_dim, index, scale):
    """One token's expanded attention over its prompt's first index + 1 keys, [H, D].

    q_bits: [H, D + R]; kv_bits: [n, H, 2 D] (keys, then values); k_rope_bits: [n, R].
    """
    d = head_dim
    kv, kr = bf16.to_f64(kv_bits[:index + 1]), bf16.to_f64(k_rope_bits[:index + 1])
    q = bf16.to_f64(q_bits)
    out, spread, size = [], [], []
    for h in range(q.shape[0]):
        keys = np.concatenate([kv[:, h, :d], kr], axis=1)
        o, a, z = attend(q[h:h + 1], keys, kv[:, h, d:], scale)
        out.append(o[0])
        spread.append(a[0])
        size.append(z[0])
    return np.array(out), np.array(spread), np.array(size)

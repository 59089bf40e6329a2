"""Shared by the latent-cache tests: seeded inputs, device copies, tolerances.

Tolerance of an attention output, per element, against exact arithmetic on the same
bf16 inputs (A = sum p |v| / sum p):
  * the result is rounded to bf16: 2^-8 |out|;
  * the probabilities are rounded to bf16 on their way into the product: 2^-8 A (the
    sum that divides is of the unrounded ones);
  * a score is a float32 sum of W products of 8 significant bits (exact in float32),
    off by at most W 2^-23 of what the products add up to in magnitude (z, in units of
    the exponent): a probability and the sum it is divided by are off by that, relative;
  * the value product is a float32 sum of n terms: n 2^-23 A;
  * exponential, reference, factors of raises and of joined parts: 2^-12 A.
"""
import numpy as np
import torch

from oracle import bf16

PAGE = 64


def check(got_bits, want, spread, size, n, width, what):
    got = bf16.to_f64(got_bits)
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -12 + n * 2.0 ** -23 + 2 * width * 2.0 ** -23 * size) * spread
    bad = ~(np.abs(got - want) <= bound + 1e-30)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, worst "
                           f"{np.nanmax(np.abs(got - want)):.3g} of {bound.max():.3g}")


def normal(rng, *shape, scale=1.0):
    """bf16 bits of normal numbers, away from the subnormal ones."""
    x = rng.standard_normal(shape) * scale
    x = np.where(np.abs(x) < 2.0 ** -60, 2.0 ** -60, x)
    return bf16.from_f64(x)


def d16(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda()


def d32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def bits(t):
    return t.detach().cpu().numpy().view(np.uint16)


def tables(rng, lengths, extra=2):
    """Rows of distinct pages in random order, -1 past each row's last page; (table, pages)."""
    need = [-(-n // PAGE) for n in lengths]
    pages = sum(need) + extra
    perm = rng.permutation(pages)
    table = np.full((len(lengths), max(max(need), 1)), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, pages


class Step:
    """Pieces of prompts [(tokens, positions before them)] and decode rows over one pool."""

    def __init__(self, seed, heads, c, r, pieces=(), dec=(), window=0, scale=None, q_scale=1.0, idle=()):
        import paged_kv_gqa_row_gb300 as lnk
        rng = np.random.default_rng(seed)
        self.lnk, self.heads, self.c, self.r, self.window = lnk, heads, c, r, window
        self.scale = (3 * r) ** -0.5 if scale is None else scale
        self.B = len(dec)
        self.table, self.pages = tables(rng, list(dec) + [n + before for n, before in pieces])
        self.rows = np.concatenate([[self.B + i] * n for i, (n, _) in enumerate(pieces)] or [[]]).astype(np.int32)
        self.positions = np.concatenate([np.arange(b, b + n) for n, b in pieces] or [[]]).astype(np.int32)
        self.step_positions = np.array([-1 if b in idle else n - 1 for b, n in enumerate(dec)], dtype=np.int32)
        self.P = len(self.rows)
        self.q = normal(rng, self.P + self.B, heads, c + r, scale=q_scale)
        self.pool = normal(rng, self.pages * PAGE, c + r)
        self.desc = lnk.latent_desc(heads, c, r, self.pages, self.table.shape[0], self.table.shape[1], scale=self.scale,
                                    window=window)

    def upload(self):
        self.d = dict(q=d16(self.q), pool=d16(self.pool), table=d32(self.table), rows=d32(self.rows),
                      positions=d32(self.positions), step=d32(self.step_positions))
        self.out = torch.full((self.P + self.B, self.heads, self.c), 0x7FC1, dtype=torch.int16, device="cuda")
        self.ws_bytes = self.lnk.lnk_latent_workspace_size(self.desc)
        # whatever the workspace holds must not matter
        self.ws = torch.full((self.ws_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self

    def run(self, stream=None):
        d = self.d
        if self.P == 0:
            self.lnk.lnk_latent_decode_attn(self.desc, d["q"], d["step"], d["table"], d["pool"], self.out, self.B, self.ws,
                                            self.ws_bytes, self.status, stream)
        else:
            self.lnk.lnk_latent_step_attn(self.desc, d["q"], d["rows"], d["positions"], d["step"] if self.B else None,
                                          d["table"], d["pool"], self.out, self.P, self.B, self.ws, self.ws_bytes,
                                          self.status, stream)
        return self

    def tokens(self):
        for t in range(self.P + self.B):
            if t < self.P:
                yield t, int(self.rows[t]), int(self.positions[t])
            else:
                yield t, t - self.P, int(self.step_positions[t - self.P])

    def verify(self, some=None, status=0):
        from oracle import latent
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        out = bits(self.out)
        for t, row, p in self.tokens():
            if some is not None and t not in some:
                continue
            if p < 0:
                assert not out[t].any(), f"token {t}: an inactive token's output is zero"
                continue
            want, spread, size = latent.attention_at(self.q[t], row, p, self.table, self.pool, self.c, self.scale,
                                                     self.window)
            check(out[t], want, spread, size, p + 1, self.c + self.r, f"token {t}, row {row} at {p}")
        return out

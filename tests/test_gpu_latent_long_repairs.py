"""Rows that are computed again behind very long contexts: longer than a pipeline's wait may take (two
seconds), while other tiles of the same blocks wait for them.  No wait runs out, and every tile gets its
outputs (tolerances: latent_harness)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from latent_harness import PAGE, bits, check, d16, d32, normal  # noqa: E402
from oracle import bf16, latent  # noqa: E402

pytestmark = pytest.mark.gpu

NAN = 0x7FC0
# Computing the rows again takes 2.6 to 2.8 s behind so many keys (184, 144 and 168 ms behind 30 000)
KEYS = {"one-sm": 440000, "pairs": 560000, "expanded": 480000}


def absorbed(heads, tokens, others, keys, rows):
    """One piece of `tokens` behind `keys` keys, the last of which its own last token alone sees and is not finite;
    `others` short tokens beside it; and `rows` decode rows over the same pages, so that a share of the pages is
    longer than the piece's tile."""
    import paged_kv_gqa_row_gb300 as lnk
    rng = np.random.default_rng(heads)
    c, r = 128, 32
    per_row = -(-(keys + tokens) // PAGE)
    pages = per_row + 2
    g = torch.Generator(device="cuda").manual_seed(heads)
    dpool = torch.empty((pages * PAGE, c + r), dtype=torch.bfloat16, device="cuda").normal_(generator=g).view(torch.int16)
    clean = bits(dpool).copy()
    table = np.tile(np.arange(per_row, dtype=np.int32), (rows + 2, 1))
    table[rows, -1] = per_row          # the piece's last page is its own
    table[rows + 1, 0] = per_row + 1   # the short ones'
    last = keys + tokens - 1
    assert (keys // PAGE, last // PAGE) == (per_row - 1, per_row - 1)
    at = per_row * PAGE + last % PAGE
    dpool[at] = NAN
    q = normal(rng, tokens + others + rows, heads, c + r)
    trow = np.array([rows] * tokens + [rows + 1] * others, dtype=np.int32)
    pos = np.concatenate([np.arange(keys, keys + tokens), np.arange(others) % PAGE]).astype(np.int32)
    dec = np.full(rows, keys - 1, dtype=np.int32)
    scale = float(np.float32(0.1))
    desc = lnk.latent_desc(heads, c, r, pages, rows + 2, per_row, scale=scale)
    size = lnk.lnk_latent_workspace_size(desc)
    d = [d16(q), d32(trow), d32(pos), d32(dec), d32(table), dpool]
    out = torch.full((tokens + others + rows, heads, c), 0x7FC1, dtype=torch.int16, device="cuda")
    ws, status = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    lnk.lnk_latent_step_attn(desc, *d, out, tokens + others, rows, ws, size, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = bits(out)
    assert np.isnan(bf16.to_f64(got[tokens - 1])).all()
    for t, row, p in ((tokens - 2, rows, keys + tokens - 2), *([(tokens + others - 1, rows + 1, int(pos[-1]))] if others else []),
                      (tokens + others, 0, keys - 1)):
        some = [0, heads - 1]
        want, spread, z = latent.attention_at(q[t][some], row, p, table, clean, c, scale)
        check(got[t][some], want, spread, z, p + 1, c + r, f"token {t}")
    # every other decode row has the same keys, and its own query
    f = bf16.to_f64(got[tokens - 1 + others + 1:])
    assert np.isfinite(f).all() and (np.abs(f).max(axis=(1, 2)) > 0).all()


@pytest.mark.parametrize("kind", ["one-sm", "pairs"])
def test_absorbed(kind):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if kind == "one-sm":
        absorbed(16, 4, 0, KEYS[kind], sms + sms // 4)
    else:
        absorbed(40, 3, 16 * sms // 40 + 3, KEYS[kind], sms // 2 + sms // 8)


def test_expanded():
    import paged_kv_gqa_row_gb300 as lnk
    keys, many = KEYS["expanded"], 400  # so many short prompts that every worker has more than one tile
    rng = np.random.default_rng(5)
    d, r, n = 128, 64, 256
    qs, ks = np.concatenate([[0], n + np.arange(many + 1)]), np.concatenate([[0], keys + np.arange(many + 1)])
    q = normal(rng, n + many, 1, d + r)
    g = torch.Generator(device="cuda").manual_seed(3)
    kv = torch.empty((keys + many, 1, 2 * d), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    kr = torch.empty((keys + many, r), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    clean = bits(kv.view(torch.int16)).copy()
    kv[keys - 1, 0, d + 9] = float("nan")
    out = torch.full((n + many, 1, d), 0x7FC1, dtype=torch.int16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = float(np.float32((d + r) ** -0.5))
    args = [d16(q), kv, kr]
    starts = [d32(qs), d32(ks)]
    lnk.lnk_latent_prompt_attn(1, d, r, scale, *args, r, *starts, out, n + many, keys + many, many + 1, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got, krb = bits(out), bits(kr.view(torch.int16))
    f = bf16.to_f64(got)
    assert np.isnan(f[n - 1, 0, 9]) and np.isfinite(np.delete(f[n - 1, 0], 9)).all() and np.isfinite(np.delete(f, n - 1, axis=0)).all()
    for i in (0, n - 2):
        seen = keys - n + i + 1
        want, spread, z = latent.expanded_at(q[i], clean[:seen], krb[:seen], d, seen - 1, scale)
        check(got[i], want, spread, z, seen, d + r, f"query {i}")
    # a prompt of one token: its own value
    assert (got[n:, 0] == clean[keys:, 0, d:]).all()

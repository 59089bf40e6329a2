"""The 4-bit cache operators and the page copies of every layer, as measured cases.

Where ``own`` is false the operators run in their plain form (elementary torch
operations in 32 or 64 bits); where it is true they run through this package's
public calls.  The 4-bit pool, as both forms read and write it:

  * a block is 16 consecutive dimensions of one head's row; with a = max |x| over
    the block and ps the pool's scale, its scale code is s = E4M3(a / (6 ps)) and
    an element's code is E2M1(x / (s ps)), both rounded to nearest even and
    saturating, every division one float32 division;
  * a page of one head is 64 rows of D / 2 code bytes (the low four bits hold the
    even dimension), then 64 * D / 16 scale bytes, the scale of block b of
    position j at ((j % 4) * (D / 16) + b) * 16 + j / 4.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
K_SCALE, V_SCALE = 0.5, 0.25


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one decode step's tokens of 64 rows written and read back (8 kv heads)
        dict(name="append 64 decode tokens", op="append", tokens=64, hq=32, hkv=8, d=128, theta=1e6, norm=False, start=4000),
        # a prompt of 2048 tokens with QK-norm, behind a shared prefix
        dict(name="append 2048 prompt tokens", op="append", tokens=2048, hq=32, hkv=8, d=128, theta=1e6, norm=True, start=512),
        # an odd prompt, a kv head for every query head
        dict(name="append 333 tokens d96 mha", op="append", tokens=333, hq=32, hkv=32, d=96, theta=1e4, norm=False, start=1),
        # the smallest decode step: 4 rows of up to 300 positions, where latency counts
        dict(name="decode 4 short rows", op="decode", rows=4, hq=32, hkv=32, d=96, shortest=1, longest=300, window=0, idle=0),
        # a serving batch of 64 rows of 512 to 8192 positions
        dict(name="decode 64 rows", op="decode", rows=64, hq=32, hkv=8, d=128, shortest=512, longest=8192, window=0, idle=0),
        # a sliding window of 2047 positions; one row in eight waits for work
        dict(name="decode 32 rows window", op="decode", rows=32, hq=32, hkv=32, d=96, shortest=1000, longest=4096, window=2047, idle=8),
        # two very long rows: the work of a row spread over the whole device
        dict(name="decode 2 long rows", op="decode", rows=2, hq=32, hkv=8, d=128, shortest=100001, longest=131072, window=0, idle=0),
        # three short prompts of odd lengths behind almost nothing
        dict(name="prompts 3 short", op="step", chunks=3, short=17, long=150, near=0, far=70, rows=0, shortest=0, longest=0, hq=16, hkv=2, d=64, window=0),
        # a step of four prompt pieces behind long contexts, and 32 decode rows beside them
        dict(name="step 4 prompts and 32 rows", op="step", chunks=4, short=512, long=512, near=1024, far=7168, rows=32, shortest=1024, longest=8192, hq=32, hkv=8, d=128, window=0),
        # four whole prompts of 1024 and more, no decode rows
        dict(name="prompts 4 long", op="step", chunks=4, short=1024, long=2047, near=0, far=0, rows=0, shortest=0, longest=0, hq=32, hkv=8, d=128, window=0),
        # copy on write after a fork: three pages, in 32 layers
        dict(name="copy 3 pages 32 layers", op="copy", layers=32, pages=64, moved=3, hkv=8, d=128),
        # compaction: a quarter of the pool moves below a lower limit, in 32 layers
        dict(name="compact 160 of 640 pages", op="copy", layers=32, pages=640, moved=160, hkv=8, d=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice((64, 96, 128))
    hkv = rng.choice((1, 2, 3, 4, 8))
    hq = hkv * rng.choice((1, 2, 4, 8))
    op = rng.choice(("append", "decode", "step", "copy"))
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 1900), hq=min(hq, 32), hkv=hkv if hq <= 32 else hq // 8, d=d,
                    theta=rng.choice((1e4, 5e5, 1e6)), norm=rng.random() < 0.5, start=_log(rng, 1, 20000))
    if op == "decode":
        rows = _log(rng, 1, 160)
        longest = _log(rng, 1, max(1, min(120000, 400000 // rows)))
        return dict(op=op, rows=rows, hq=hq, hkv=hkv, d=d, shortest=_log(rng, 1, longest), longest=longest,
                    window=rng.choice((0, 0, _log(rng, 1, 4000))), idle=rng.choice((0, 0, 3)))
    if op == "step":
        rows = rng.choice((0, _log(rng, 1, 40)))
        long = _log(rng, 1, 700)
        far = _log(rng, 1, 5000)
        longest = _log(rng, 1, 6000)
        chunks = rng.randint(1, 4)
        while chunks * long * (far + long) * hq * d > 3e10:  # no more than the largest listed step
            far, long = 1 + far // 2, 1 + long * 3 // 4
        return dict(op=op, chunks=chunks, short=_log(rng, 1, long), long=long, near=_log(rng, 1, far), far=far,
                    rows=rows, shortest=_log(rng, 1, longest), longest=longest, hq=hq, hkv=hkv, d=d,
                    window=rng.choice((0, 0, _log(rng, 1, 4000))))
    layers = _log(rng, 1, 32)
    pages = _log(rng, 8, 500)
    return dict(op=op, layers=layers, pages=pages, moved=max(1, min(pages // 2, _log(rng, 1, 150))), hkv=hkv, d=d)


def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


# ----------------------------------------------------------------- inputs ----

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)


def _permutation(gen, n):
    return torch.randperm(n, generator=gen, device=DEV).to(torch.int32)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _table(gen, lengths, per_row):
    """Rows of distinct pages in random order; -1 past each row's last page."""
    need = [-(-n // PAGE) for n in lengths]
    pages = sum(need) + 3
    perm = _permutation(gen, pages)
    table = torch.full((len(lengths), per_row), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, pages


def _filled_pool(gen, hkv, pages, d, ps):
    """A pool whose rows are N(0, 1) tokens in 4 bits, as an append leaves them."""
    pool = torch.empty((hkv, pages, 36 * d), dtype=torch.uint8, device=DEV)
    for h in range(hkv):
        codes, scales = _quantize(_normal(gen, pages, PAGE, d).float(), ps)
        pool[h] = _pack(codes, scales)
    return pool


def _pack(codes, scales):
    """Page bytes [n, 36 d] of codes [n, 64, d] and scale codes [n, 64, d / 16]."""
    n, _, d = codes.shape
    rows = codes[..., 0::2] | (codes[..., 1::2] << 4)
    tail = scales.reshape(n, PAGE // 4, 4, d // 16).permute(0, 2, 3, 1)
    return torch.cat([rows.reshape(n, -1), tail.reshape(n, -1)], dim=1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    host = np.random.RandomState(int(seed) % (1 << 32))
    if case["op"] == "append":
        return _prepare_append(case, gen)
    if case["op"] == "decode":
        return _prepare_decode(case, gen, host)
    if case["op"] == "step":
        return _prepare_step(case, gen, host)
    return _prepare_copy(case, gen)


def _prepare_append(case, gen):
    t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    if t <= 256:  # one token of each row, at its own position
        positions = [case["start"] + (37 * i) % 61 for i in range(t)]
        rows = list(range(t))
    else:  # one row's prompt
        positions = list(range(case["start"], case["start"] + t))
        rows = [0] * t
    lengths = [0] * (max(rows) + 1)
    for p, r in zip(positions, rows):
        lengths[r] = max(lengths[r], p + 1)
    # only the written pages of each row are mapped: the others are not read
    per_row = -(-max(lengths) // PAGE)
    wanted = sorted({(r, p // PAGE) for p, r in zip(positions, rows)})
    pages = len(wanted) + 3
    perm = _permutation(gen, pages).tolist()
    table = np.full((len(lengths), per_row), -1, dtype=np.int32)
    for (r, lp), pg in zip(wanted, perm):
        table[r, lp] = pg
    i = np.arange(d // 2, dtype=np.float32)
    exponent = -(i * np.float32(2) / np.float32(d)) * np.float32(np.log(np.float64(np.float32(case["theta"]))))
    inv = np.exp(exponent.astype(np.float64)).astype(np.float32)
    s = dict(case=case, q=_normal(gen, t, hq, d), k=_normal(gen, t, hkv, d), v=_normal(gen, t, hkv, d),
             positions=_i32(positions), rows=_i32(rows), table=torch.from_numpy(table).to(DEV), pages=pages,
             inv=torch.from_numpy(inv).to(DEV), gq=None, gk=None,
             k_pool=torch.zeros((hkv, pages, 36 * d), dtype=torch.uint8, device=DEV),
             v_pool=torch.zeros((hkv, pages, 36 * d), dtype=torch.uint8, device=DEV),
             q_out=torch.empty((t, hq, d), dtype=torch.bfloat16, device=DEV),
             k_out=torch.empty((t, hkv, d), dtype=torch.bfloat16, device=DEV),
             v_out=torch.empty((t, hkv, d), dtype=torch.bfloat16, device=DEV))
    if case["norm"]:
        s["gq"] = (1 + 0.1 * torch.randn(d, generator=gen, device=DEV)).to(torch.bfloat16)
        s["gk"] = (1 + 0.1 * torch.randn(d, generator=gen, device=DEV)).to(torch.bfloat16)
    return s


def _decode_positions(case, host):
    lengths = _spread(case["shortest"], case["longest"], case["rows"])
    lengths = [lengths[i] for i in host.permutation(len(lengths))]
    idle = case.get("idle", 0)
    return lengths, [-1 if idle and b % idle == idle - 1 else n - 1 for b, n in enumerate(lengths)]


def _pools(case, gen, pages):
    return dict(k_pool=_filled_pool(gen, case["hkv"], pages, case["d"], K_SCALE),
                v_pool=_filled_pool(gen, case["hkv"], pages, case["d"], V_SCALE), pages=pages)


def _prepare_decode(case, gen, host):
    lengths, positions = _decode_positions(case, host)
    table, pages = _table(gen, lengths, -(-max(lengths) // PAGE))
    return dict(case=case, q=_normal(gen, case["rows"], case["hq"], case["d"]), positions=_i32(positions), table=table,
                out=torch.empty((case["rows"], case["hq"], case["d"]), dtype=torch.bfloat16, device=DEV),
                **_pools(case, gen, pages))


def _chunks(case):
    """(tokens, positions before them) of each prompt piece."""
    n = case["chunks"]
    return list(zip(_spread(case["short"], case["long"], n), reversed(_spread(case["near"], case["far"], n))))


def _prepare_step(case, gen, host):
    chunks = _chunks(case)
    lengths, dec = _decode_positions(case, host) if case["rows"] else ([], [])
    ends = [before + n for n, before in chunks]
    table, pages = _table(gen, lengths + ends, -(-max(lengths + ends) // PAGE))
    rows, positions, segments = [], [], []
    for c, (n, before) in enumerate(chunks):
        rows += [len(lengths) + c] * n
        positions += list(range(before, before + n))
        segments += [c] * n
    t = len(rows) + len(dec)
    most = max(n for n, _ in chunks)
    # where each prompt piece's tokens lie in the pack (-1: none), for the plain form
    first = np.cumsum([0] + [n for n, _ in chunks])
    place = np.full((len(chunks), most), -1, dtype=np.int64)
    for c, (n, _) in enumerate(chunks):
        place[c, :n] = np.arange(first[c], first[c] + n)
    return dict(case=case, q=_normal(gen, t, case["hq"], case["d"]), rows=_i32(rows), positions=_i32(positions),
                segments=_i32(segments), step_positions=_i32(dec) if dec else None, table=table,
                place=torch.from_numpy(place).to(DEV),
                out=torch.empty((t, case["hq"], case["d"]), dtype=torch.bfloat16, device=DEV), **_pools(case, gen, pages))


def _prepare_copy(case, gen):
    n, layers, hkv, d = case["pages"], case["layers"], case["hkv"], case["d"]
    # moved pages leave the upper part for free places in the lower one
    low = n - case["moved"]
    src = low + torch.randperm(n - low, generator=gen, device=DEV)[:case["moved"]]
    dst = torch.randperm(low, generator=gen, device=DEV)[:case["moved"]]
    pools = {}
    for which in ("k_pools", "v_pools"):
        pools[which] = torch.empty((layers, hkv, n * PAGE, d), dtype=torch.bfloat16, device=DEV)
        for layer in range(layers):
            pools[which][layer] = _normal(gen, hkv, n * PAGE, d)
    return dict(case=case, src=src.to(torch.int32), dst=dst.to(torch.int32), **pools,
                k_list=list(pools["k_pools"]), v_list=list(pools["v_pools"]))


# -------------------------------------------------------------- plain form ----

def _quantize(x, ps):
    """4-bit codes (0..15) and scale codes of float32 values whose last axis is D."""
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    t = blocks.abs().amax(-1) / torch.tensor(6.0 * ps, dtype=torch.float32, device=x.device)
    scale = t.clamp(max=448.0).to(torch.float8_e4m3fn)
    step = scale.float() * ps
    u = torch.where(step[..., None] > 0, blocks / step[..., None], torch.zeros_like(blocks))
    a = u.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code.to(torch.uint8) | (torch.signbit(u).to(torch.uint8) << 3)
    return code.reshape(x.shape), scale.view(torch.uint8)


def _values(pages, d, ps):
    """float32 values [..., 64, d] of page bytes [..., 36 d]."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float32, device=pages.device)
    rows = pages[..., :32 * d].reshape(*pages.shape[:-1], PAGE, d // 2)
    codes = torch.stack([rows & 15, rows >> 4], dim=-1).reshape(*rows.shape[:-1], d)
    tail = pages[..., 32 * d:].reshape(*pages.shape[:-1], 4, d // 16, 16)
    scale = tail.movedim(-1, -3).reshape(*pages.shape[:-1], PAGE, d // 16).contiguous().view(torch.float8_e4m3fn).float()
    return lut[codes.int()] * scale.repeat_interleave(16, dim=-1) * ps


def _to_bf16(x):
    """float64 to bfloat16 in one rounding, to nearest even."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256.0), e - 8).to(torch.bfloat16)


def _rotated(x, positions, inv, gamma, eps=1e-6):
    """QK-norm (with gamma) and rotation of heads [t, h, d], in 64 bits."""
    y = x.double()
    if gamma is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * gamma.double()
    angle = (positions.float()[:, None] * inv[None, :]).double()[:, None, :]
    half = y.shape[-1] // 2
    lo, hi = y[..., :half], y[..., half:]
    return torch.cat([lo * angle.cos() - hi * angle.sin(), hi * angle.cos() + lo * angle.sin()], dim=-1)


def _plain_append(s):
    case = s["case"]
    d, blocks = case["d"], case["d"] // 16
    eps = float(np.float32(1e-6))
    q_out = _to_bf16(_rotated(s["q"], s["positions"], s["inv"], s["gq"], eps))
    k_new = _to_bf16(_rotated(s["k"], s["positions"], s["inv"], s["gk"], eps))
    page = s["table"][s["rows"].long(), (s["positions"] // PAGE).long()].long()
    j = (s["positions"] % PAGE).long()
    at_codes = (j * (d // 2))[:, None] + torch.arange(d // 2, device=DEV)
    at_scales = 32 * d + ((j % 4)[:, None] * blocks + torch.arange(blocks, device=DEV)) * 16 + (j // 4)[:, None]
    back = []
    for pool, new, ps in ((s["k_pool"], k_new, K_SCALE), (s["v_pool"], s["v"], V_SCALE)):
        codes, scales = _quantize(new.float(), ps)
        pool[:, page[:, None], at_codes] = (codes[..., 0::2] | (codes[..., 1::2] << 4)).transpose(0, 1)
        pool[:, page[:, None], at_scales] = scales.transpose(0, 1)
        lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float32, device=DEV)
        rows = pool[:, page[:, None], at_codes].transpose(0, 1)
        held = torch.stack([rows & 15, rows >> 4], dim=-1).reshape(new.shape)
        scale = pool[:, page[:, None], at_scales].transpose(0, 1).contiguous().view(torch.float8_e4m3fn).float()
        back.append((lut[held.int()] * scale.repeat_interleave(16, dim=-1) * ps).to(torch.bfloat16))
    return {"q": q_out, "k": back[0], "v": back[1]}


def _attend(q, first, last, keys, values):
    """Softmax attention of queries [c, t, hkv, g, d] over keys [hkv, c, l, d]; a query
    sees keys first..last ([c, t]); one that sees none answers zero."""
    scores = torch.einsum("cthgd,hcld->cthgl", q.float(), keys) / math.sqrt(q.shape[-1])
    at = torch.arange(keys.shape[2], device=DEV)
    seen = ((at >= first[..., None]) & (at <= last[..., None]))[:, :, None, None, :]
    scores = scores.masked_fill(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("cthgl,hcld->cthgd", p, values)
    return out / torch.where(total > 0, total, torch.ones_like(total))


def _row_values(s, pool, rows, ps):
    """float32 values [hkv, rows, l, d] of the table rows' pages."""
    entries = s["table"][rows].long().clamp(min=0)
    got = _values(s[pool][:, entries], s["case"]["d"], ps)
    return got.reshape(got.shape[0], got.shape[1], -1, got.shape[-1])


def _visible(positions, window):
    first = (positions - window + 1).clamp(min=0) if window else torch.zeros_like(positions)
    return first, positions


def _plain_decode(s, q, positions):
    case = s["case"]
    b, hkv, d = positions.shape[0], case["hkv"], case["d"]
    rows = slice(0, b)
    first, last = _visible(positions, case["window"])
    out = _attend(q.reshape(b, 1, hkv, -1, d), first[:, None], last[:, None], _row_values(s, "k_pool", rows, K_SCALE),
                  _row_values(s, "v_pool", rows, V_SCALE))
    return out.reshape(b, case["hq"], d).to(torch.bfloat16)


def _plain_step(s):
    case = s["case"]
    place, hkv, d = s["place"], case["hkv"], case["d"]
    b = case["rows"]
    rows = slice(b, b + place.shape[0])
    packed = place.clamp(min=0)
    positions = torch.where(place >= 0, s["positions"][packed].long(), torch.full_like(place, -1))
    first, last = _visible(positions, case["window"])
    got = _attend(s["q"][packed].reshape(*place.shape, hkv, -1, d), first, last, _row_values(s, "k_pool", rows, K_SCALE),
                  _row_values(s, "v_pool", rows, V_SCALE))
    out = torch.empty_like(s["q"])
    out[place[place >= 0]] = got.reshape(*place.shape, case["hq"], d)[place >= 0].to(torch.bfloat16)
    if b:
        out[-b:] = _plain_decode(s, s["q"][-b:], s["step_positions"])
    return out


def _plain_copy(s):
    for which in ("k_pools", "v_pools"):
        pools = s[which].unflatten(2, (-1, PAGE))
        pools[:, :, s["dst"].long()] = pools[:, :, s["src"].long()]
    return {"k": s["k_pools"], "v": s["v_pools"]}


# ----------------------------------------------------- the package's calls ----

def _handle(s):
    """The descriptor and the workspace that a program makes once and keeps."""
    import paged_kv_gqa_row_gb300 as lnk
    case = s["case"]
    if case["op"] == "copy":
        desc = lnk.attn_desc(case["hkv"], case["hkv"], case["d"], case["pages"], 1, 1)
    else:
        desc = lnk.attn_desc(case["hq"], case["hkv"], case["d"], s["pages"], s["table"].shape[0], s["table"].shape[1],
                             window=case.get("window", 0), kv_dtype=lnk.KV_E2M1, k_scale=K_SCALE, v_scale=V_SCALE)
    rope = lnk.rope_desc(case["theta"]) if case["op"] == "append" else None
    size = lnk.lnk_paged_workspace_size(desc, case["rows"]) if case.get("rows") else 0
    return lnk, desc, rope, torch.zeros(size, dtype=torch.uint8, device=DEV) if size else None, size


def _own_append(s, lnk, desc, rope, t):
    lnk.lnk_paged_append_rope(desc, rope, s["q"], s["k"], s["v"], s["positions"], s["rows"], None, s["table"], s["gq"],
                              s["gk"], 1e-6, s["k_pool"], s["v_pool"], s["q_out"], t)
    lnk.lnk_paged_read_tokens(desc, s["k_pool"], s["v_pool"], s["positions"], s["rows"], None, s["table"], s["k_out"],
                              s["v_out"], t)
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _own(s):
    if "handle" not in s:
        s["handle"] = _handle(s)
    lnk, desc, rope, ws, size = s["handle"]
    case = s["case"]
    if case["op"] == "append":
        return _own_append(s, lnk, desc, rope, case["tokens"])
    if case["op"] == "copy":
        lnk.lnk_paged_copy_pages_layers(desc, s["k_list"], s["v_list"], s["src"], s["dst"], case["moved"])
        return {"k": s["k_pools"], "v": s["v_pools"]}
    if case["op"] == "decode":
        lnk.lnk_paged_decode_attn(desc, s["q"], s["positions"], s["table"], s["k_pool"], s["v_pool"], s["out"], case["rows"],
                                  ws, size)
    else:
        lnk.lnk_paged_step_attn(desc, s["q"], s["rows"], s["positions"], s["segments"], s["step_positions"], s["table"],
                                s["k_pool"], s["v_pool"], s["out"], None, None, s["rows"].shape[0], case["rows"], 0, ws, size)
    return s["out"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "append":
        return _plain_append(state)
    if op == "copy":
        return _plain_copy(state)
    if op == "decode":
        return _plain_decode(state, state["q"], state["positions"])
    return _plain_step(state)


# ------------------------------------------------------------ work, exact ----

def _seen(position, window):
    return min(position + 1, window) if window else position + 1


def work(case):
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "copy":
        return {"bytes": 2 * 2 * case["layers"] * hkv * case["moved"] * PAGE * d * 2, "flops": 0}
    hq, row4 = case["hq"], d // 2 + d // 16
    if case["op"] == "append":
        t = case["tokens"]
        read = t * (hq + 2 * hkv) * d * 2 + 8 * t
        written = t * hq * d * 2 + t * hkv * 2 * row4 + t * hkv * 2 * d * 2
        return {"bytes": read + written, "flops": t * (hq + 3 * hkv) * d * 6}
    window, total, flops = case["window"], 0, 0
    if case["rows"]:
        lengths = _spread(case["shortest"], case["longest"], case["rows"])
        idle = case.get("idle", 0)
        live = case["rows"] - (case["rows"] // idle if idle else 0)
        seen = sum(_seen(n - 1, window) for n in lengths) * live // case["rows"]
        total += seen * hkv * 2 * row4 + case["rows"] * hq * d * 4 + 4 * (seen // PAGE + case["rows"])
        flops += 4 * hq * d * seen
    if case["op"] == "step":
        for n, before in _chunks(case):
            flops += 4 * hq * d * sum(_seen(p, window) for p in range(before, before + n))
            first = max(0, before - window + 1) if window else 0
            total += (before + n - first) * hkv * 2 * row4 + n * hq * d * 4 + 12 * n
    return {"bytes": total, "flops": flops}


def _exact_values(page_bytes, d, ps):
    """Values [64, d] of one head's page, byte by byte as the layout says."""
    b = page_bytes.cpu().numpy()
    value = np.empty((PAGE, d))
    for j in range(PAGE):
        code = b[j * (d // 2) + np.arange(d) // 2].astype(np.int64) >> (4 * (np.arange(d) % 2))
        sign = np.where(code & 8, -1.0, 1.0)
        e, m = (code >> 1) & 3, code & 1
        mag = np.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e - 1))
        sc = b[32 * d + ((j % 4) * (d // 16) + np.arange(d) // 16) * 16 + j // 4].astype(np.int64)
        se, sm = (sc >> 3) & 15, sc & 7
        value[j] = sign * mag * np.where(se == 0, sm * 2.0 ** -9, (1 + sm / 8.0) * 2.0 ** (se - 7.0)) * ps
    return torch.from_numpy(value).to(DEV)


def _exact_rows(s, q, rows, positions):
    """Attention of queries [t, hq, d], query i at positions[i] of table row rows[i], in 64 bits."""
    case = s["case"]
    hkv, d, window = case["hkv"], case["d"], case["window"]
    group = case["hq"] // hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    for r in sorted(set(rows)):
        mine = [i for i, x in enumerate(rows) if x == r and positions[i] >= 0]
        if not mine:
            continue
        length = max(positions[i] for i in mine) + 1
        pages = s["table"][r, :-(-length // PAGE)].tolist()
        at = torch.tensor([positions[i] for i in mine], device=DEV)[:, None]
        j = torch.arange(length, device=DEV)[None, :]
        seen = (j <= at) & (j > at - window) if window else j <= at
        for h in range(hkv):
            k = _cached(s, "k_pool", h, pages, K_SCALE)[:length]
            v = _cached(s, "v_pool", h, pages, V_SCALE)[:length]
            for g in range(h * group, (h + 1) * group):
                z = (q[mine, g].double() @ k.T) * d ** -0.5
                z = torch.where(seen, z, torch.full_like(z, -math.inf))
                out[mine, g] = torch.softmax(z, dim=-1) @ v
    return out


def _cached(s, pool, h, pages, ps):
    d = s["case"]["d"]
    key = (pool, h)
    got = s.setdefault("exact", {}).get(key)
    if got is None:
        raw = s[pool][h].cpu().numpy()
        n = raw.shape[0]
        code = raw[:, :32 * d].reshape(n, PAGE, d // 2)
        code = np.repeat(code, 2, axis=-1) >> np.tile(np.array([0, 4], dtype=np.uint8), d // 2)
        mag = np.array(E2M1)[code & 7] * np.where(code & 8, -1.0, 1.0)
        j, b = np.arange(PAGE)[:, None], np.arange(d)[None, :] // 16
        sc = raw[:, (32 * d + ((j % 4) * (d // 16) + b) * 16 + j // 4)].astype(np.int64)
        se, sm = (sc >> 3) & 15, sc & 7
        got = torch.from_numpy(mag * np.where(se == 0, sm * 2.0 ** -9, (1 + sm / 8.0) * 2.0 ** (se - 7.0)) * ps).to(DEV)
        # one page against the layout written out byte by byte
        assert torch.equal(got[0], _exact_values(s[pool][h, 0], d, ps))
        s["exact"][key] = got
    return got[torch.tensor(pages, device=DEV)].reshape(-1, d)


def _exact_append(s):
    case = s["case"]
    d = case["d"]
    pos = s["positions"].cpu().numpy()
    angle = (pos.astype(np.float32)[:, None] * s["inv"].cpu().numpy()[None, :]).astype(np.float32).astype(np.float64)
    turn = (np.cos(angle) + 1j * np.sin(angle))[:, None, :]
    answers = {}
    for name, gamma in (("q", s["gq"]), ("k", s["gk"])):
        x = s[name].float().cpu().numpy().astype(np.float64)
        if gamma is not None:
            x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + float(np.float32(1e-6))) * gamma.float().cpu().numpy().astype(np.float64)
        z = (x[..., :d // 2] + 1j * x[..., d // 2:]) * turn
        answers[name] = np.concatenate([z.real, z.imag], axis=-1)
    m, e = np.frexp(answers["k"])
    stored = {"k": np.ldexp(np.rint(m * 256), e - 8), "v": s["v"].float().cpu().numpy().astype(np.float64)}
    e4m3 = np.array([(1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) if c >> 3 else (c & 7) * 2.0 ** -9 for c in range(127)])
    for name, ps in (("k", K_SCALE), ("v", V_SCALE)):
        x = stored[name].reshape(*stored[name].shape[:-1], d // 16, 16)
        t = (np.abs(x).max(-1).astype(np.float32) / np.float32(6 * ps)).astype(np.float64)
        sc = e4m3[_nearest(e4m3, t)]
        u = np.divide(x.astype(np.float32), (sc * ps).astype(np.float32)[..., None], out=np.zeros(x.shape, np.float32),
                      where=sc[..., None] > 0).astype(np.float64)
        mag = np.array(E2M1)[_nearest(np.array(E2M1), np.abs(u))]
        answers[name] = (np.sign(u) * mag * sc[..., None] * ps).reshape(stored[name].shape)
    return {n: torch.from_numpy(x) for n, x in answers.items()}


def _nearest(values, x):
    """Index of the value nearest to x, the even one of two equally near."""
    hi = np.searchsorted(values, x).clip(1, len(values) - 1)
    below, above = x - values[hi - 1], values[hi] - x
    return np.where((below < above) | ((below == above) & ((hi - 1) % 2 == 0)), hi - 1, hi)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "copy":
        for which in ("k_pools", "v_pools"):
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                s[which][:, :, b * PAGE:(b + 1) * PAGE] = s[which][:, :, a * PAGE:(a + 1) * PAGE]
        return {"k": s["k_pools"], "v": s["v_pools"]}
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "decode":
        return _exact_rows(s, s["q"], list(range(case["rows"])), s["positions"].tolist())
    rows = s["rows"].tolist() + list(range(case["rows"]))
    positions = s["positions"].tolist() + (s["step_positions"].tolist() if case["rows"] else [])
    return _exact_rows(s, s["q"], rows, positions)

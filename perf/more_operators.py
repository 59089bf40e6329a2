"""The latent-cache operators, as measured cases.

A latent pool holds one row of C + R bf16 numbers a token, which every query head
shares: a latent vector of C numbers (normalised, it is the value and the first C
numbers of the key) and R rotated numbers (the key's last R).  A page is 64 rows;
position j of table row r lies in page table[r, j / 64], row j % 64.

  append   c = latent * w / sqrt(mean(latent^2) + eps), the key's R numbers and each
           head's R query numbers turned by the token's position, and [c, k] written
           into the token's place;
  decode   absorbed attention, one token a row: scores q . [c, k] * scale over the
           row's keys up to the token's position, softmax, output sum p c (C numbers);
  step     the same for pieces of prompts, with decode rows behind them;
  prompt   the expanded form: every head has keys [k_nope, k_rope] and values of its
           own, computed from the latents by the caller; packed prompts, causal, a
           prompt's queries being the last of its keys;
  copy     whole pages moved in the pools of all layers.

Where ``own`` is false the operators run in their plain form (elementary torch
operations in 32 or 64 bits); where it is true they run through this package's
public calls.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one decode step's tokens of 64 rows
        dict(name="append 64 decode tokens", op="append", tokens=64, heads=64, c=512, r=64, theta=1e4, start=4000),
        # a prompt of 2000 tokens behind a shared prefix
        dict(name="append 2000 prompt tokens", op="append", tokens=2000, heads=40, c=512, r=64, theta=5e5, start=512),
        # the smallest decode step: 4 rows of up to 300 positions, where latency counts
        dict(name="decode 4 short rows", op="decode", rows=4, heads=32, c=256, r=32, shortest=1, longest=300, window=0, idle=0),
        # a serving batch of 64 rows of 512 to 8192 positions
        dict(name="decode 64 rows", op="decode", rows=64, heads=32, c=512, r=64, shortest=512, longest=8192, window=0, idle=0),
        # many heads share each latent; one row in eight waits for work
        dict(name="decode 32 rows 128 heads", op="decode", rows=32, heads=128, c=512, r=64, shortest=1000, longest=8000, window=0, idle=8),
        # two very long rows: the work of a row spread over the whole device
        dict(name="decode 2 long rows", op="decode", rows=2, heads=40, c=512, r=64, shortest=100001, longest=131072, window=0, idle=0),
        # three short pieces of odd lengths behind almost nothing
        dict(name="pieces 3 short", op="step", chunks=3, short=17, long=150, near=0, far=70, rows=0, shortest=0, longest=0, heads=24, c=256, r=64, window=0),
        # proposed tokens of four rows checked behind long contexts, beside 32 decode rows
        dict(name="step 4 pieces and 32 rows", op="step", chunks=4, short=8, long=128, near=1024, far=7168, rows=32, shortest=1024, longest=8192, heads=64, c=512, r=64, window=0),
        # three whole prompts of odd lengths
        dict(name="prompts 3 short", op="prompt", chunks=3, short=17, long=150, near=0, far=0, heads=16, d=128, r=64),
        # four whole prompts of 1024 and more
        dict(name="prompts 4 long", op="prompt", chunks=4, short=1024, long=2047, near=0, far=0, heads=32, d=128, r=64),
        # copy on write after a fork: three pages, in 32 layers
        dict(name="copy 3 pages 32 layers", op="copy", layers=32, pages=64, moved=3, c=512, r=64),
        # compaction: a quarter of the pool moves below a lower limit, in 32 layers
        dict(name="compact 160 of 640 pages", op="copy", layers=32, pages=640, moved=160, c=512, r=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c, r = rng.choice((128, 256, 384, 512)), rng.choice((32, 64))
    heads = rng.choice((1, 3, 8, 20, 24, 32, 40, 64, 96, 128, 160))
    op = rng.choice(("append", "decode", "step", "prompt", "copy"))
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 1900), heads=min(heads, 40), c=c, r=r, theta=rng.choice((1e4, 5e5, 1e6)),
                    start=_log(rng, 1, 20000))
    if op == "decode":
        rows = _log(rng, 1, 160)
        longest = _log(rng, 1, max(1, min(120000, 18000000 // (rows * max(heads, 32)))))
        return dict(op=op, rows=rows, heads=heads, c=c, r=r, shortest=_log(rng, 1, longest), longest=longest,
                    window=rng.choice((0, 0, _log(rng, 1, 4000))), idle=rng.choice((0, 0, 3)))
    if op == "step":
        rows = rng.choice((0, _log(rng, 1, 30)))
        long, far, longest = _log(rng, 1, 300), _log(rng, 1, 5000), _log(rng, 1, 5000)
        chunks = rng.randint(1, 4)
        while chunks * long * (far + long) * heads > 1.2e8:  # no more than the largest listed step
            far, long = 1 + far // 2, 1 + long * 3 // 4
        return dict(op=op, chunks=chunks, short=_log(rng, 1, long), long=long, near=_log(rng, 1, far), far=far, rows=rows,
                    shortest=_log(rng, 1, longest), longest=longest, heads=min(heads, 128), c=c, r=r,
                    window=rng.choice((0, 0, _log(rng, 1, 4000))))
    if op == "prompt":
        long = _log(rng, 1, 1500)
        far = rng.choice((0, _log(rng, 1, 500)))
        return dict(op=op, chunks=rng.randint(1, 4), short=_log(rng, 1, long), long=long, near=far // 3, far=far,
                    heads=min(heads, 32), d=rng.choice((64, 128)), r=r)
    pages = _log(rng, 8, 500)
    return dict(op=op, layers=_log(rng, 1, 32), pages=pages, moved=max(1, min(pages // 2, _log(rng, 1, 150))), c=c, r=r)


def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _chunks(case):
    """(tokens, positions before them) of each piece of a prompt."""
    n = case["chunks"]
    return list(zip(_spread(case["short"], case["long"], n), reversed(_spread(case["near"], case["far"], n))))


def _scale(case):
    """The softmax scale: that of expanded heads of 128 + 64, or in proportion."""
    return (3 * case["r"]) ** -0.5 if case["op"] != "prompt" else (case["d"] + case["r"]) ** -0.5


# ----------------------------------------------------------------- inputs ----

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _table(gen, lengths):
    """Rows of distinct pages in random order; -1 past each row's last page."""
    need = [-(-n // PAGE) for n in lengths]
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lengths), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for row, n in enumerate(need):
        table[row, :n] = perm[at:at + n]
        at += n
    return table, pages


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    host = np.random.RandomState(int(seed) % (1 << 32))
    make = dict(append=_prepare_append, decode=_prepare_step, step=_prepare_step, prompt=_prepare_prompt, copy=_prepare_copy)
    s = make[case["op"]](case, gen, host)
    s["case"] = case
    return s


def _prepare_append(case, gen, host):
    t, heads, c, r = case["tokens"], case["heads"], case["c"], case["r"]
    if t <= 256:  # one token of each row, at its own position
        positions, rows = [case["start"] + (37 * i) % 61 for i in range(t)], list(range(t))
    else:  # one row's prompt
        positions, rows = list(range(case["start"], case["start"] + t)), [0] * t
    # only the written pages of each row are mapped: the others are not read
    wanted = sorted({(row, p // PAGE) for p, row in zip(positions, rows)})
    pages = len(wanted) + 3
    perm = torch.randperm(pages, generator=gen, device=DEV).tolist()
    table = np.full((max(rows) + 1, max(positions) // PAGE + 1), -1, dtype=np.int32)
    for (row, lp), pg in zip(wanted, perm):
        table[row, lp] = pg
    i = np.arange(r // 2, dtype=np.float32)
    exponent = -(i * np.float32(2) / np.float32(r)) * np.float32(np.log(np.float64(np.float32(case["theta"]))))
    inv = np.exp(exponent.astype(np.float64)).astype(np.float32)
    # projected queries: each head's 128 (or 64) other numbers lie before the rotated ones
    return dict(q=_normal(gen, t, heads, 2 * r + r), kv=_normal(gen, t, c + r), positions=_i32(positions), rows=_i32(rows),
                table=torch.from_numpy(table).to(DEV), pages=pages, inv=torch.from_numpy(inv).to(DEV),
                w=(1 + 0.1 * torch.randn(c, generator=gen, device=DEV)).to(torch.bfloat16),
                pool=torch.zeros((pages * PAGE, c + r), dtype=torch.bfloat16, device=DEV),
                q_out=torch.zeros((t, heads, c + r), dtype=torch.bfloat16, device=DEV),
                kv_out=torch.empty((t, c + r), dtype=torch.bfloat16, device=DEV))


def _prepare_step(case, gen, host):
    chunks = _chunks(case) if case["op"] == "step" else []
    lengths = _spread(case["shortest"], case["longest"], case["rows"]) if case["rows"] else []
    lengths = [lengths[i] for i in host.permutation(len(lengths))]
    idle = case.get("idle", 0)
    dec = [-1 if idle and b % idle == idle - 1 else n - 1 for b, n in enumerate(lengths)]
    table, pages = _table(gen, lengths + [before + n for n, before in chunks])
    rows, positions = [], []
    for i, (n, before) in enumerate(chunks):
        rows += [len(lengths) + i] * n
        positions += list(range(before, before + n))
    t, w = len(rows) + len(dec), case["c"] + case["r"]
    return dict(q=_normal(gen, t, case["heads"], w), pool=_normal(gen, pages * PAGE, w), table=table, pages=pages,
                rows=_i32(rows) if rows else None, positions=_i32(positions) if rows else None,
                step_positions=_i32(dec) if dec else None, pieces=chunks,
                out=torch.empty((t, case["heads"], case["c"]), dtype=torch.bfloat16, device=DEV))


def _prepare_prompt(case, gen, host):
    chunks = _chunks(case)
    heads, d, r = case["heads"], case["d"], case["r"]
    q_starts = np.cumsum([0] + [n for n, _ in chunks]).tolist()
    k_starts = np.cumsum([0] + [n + before for n, before in chunks]).tolist()
    tq, tk = q_starts[-1], k_starts[-1]
    return dict(q=_normal(gen, tq, heads, d + r), kv=_normal(gen, tk, heads, 2 * d), k_rope=_normal(gen, tk, r),
                q_starts=_i32(q_starts), k_starts=_i32(k_starts), pieces=chunks,
                out=torch.empty((tq, heads, d), dtype=torch.bfloat16, device=DEV))


def _prepare_copy(case, gen, host):
    n, low = case["pages"], case["pages"] - case["moved"]
    # moved pages leave the upper part for free places in the lower one
    src = low + torch.randperm(n - low, generator=gen, device=DEV)
    dst = torch.randperm(low, generator=gen, device=DEV)[:case["moved"]]
    pools = torch.empty((case["layers"], n * PAGE, case["c"] + case["r"]), dtype=torch.bfloat16, device=DEV)
    for layer in range(case["layers"]):
        pools[layer] = _normal(gen, n * PAGE, case["c"] + case["r"])
    return dict(src=src.to(torch.int32), dst=dst.to(torch.int32), pools=pools, list=list(pools))


# -------------------------------------------------------------- plain form ----

def _to_bf16(x):
    """float64 to bfloat16 in one rounding, to nearest even."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256.0), e - 8).to(torch.bfloat16)


def _rotated(x, positions, inv):
    """The last axis of x [t, h, r] turned by the tokens' positions, in 64 bits."""
    y = x.double()
    angle = (positions.float()[:, None] * inv[None, :]).double()[:, None, :]
    half = y.shape[-1] // 2
    lo, hi = y[..., :half], y[..., half:]
    return torch.cat([lo * angle.cos() - hi * angle.sin(), hi * angle.cos() + lo * angle.sin()], dim=-1)


def _plain_append(s):
    c, r = s["case"]["c"], s["case"]["r"]
    latent = s["kv"][:, :c].double()
    latent = latent * torch.rsqrt(latent.square().mean(-1, keepdim=True) + EPS) * s["w"].double()
    s["kv_out"][:, :c] = _to_bf16(latent)
    s["kv_out"][:, c:] = _to_bf16(_rotated(s["kv"][:, None, c:], s["positions"], s["inv"]))[:, 0]
    s["q_out"][:, :, c:] = _to_bf16(_rotated(s["q"][:, :, -r:], s["positions"], s["inv"]))
    page = s["table"][s["rows"].long(), (s["positions"] // PAGE).long()].long()
    s["pool"][page * PAGE + (s["positions"] % PAGE).long()] = s["kv_out"]
    return {"q": s["q_out"], "kv": s["kv_out"], "pool": s["pool"]}


def _attend(q, first, last, keys, values, scale):
    """Softmax attention of q [n, t, h, w] over keys [n, l, w] with values [n, l, c]; token t
    sees keys first..last ([n, t]); one that sees none answers zero."""
    n, t, h, w = q.shape
    scores = torch.bmm(q.reshape(n, t * h, w).float(), keys.transpose(1, 2)).reshape(n, t, h, -1) * scale
    at = torch.arange(keys.shape[1], device=DEV)
    seen = ((at >= first[..., None]) & (at <= last[..., None]))[:, :, None, :]
    scores = scores.masked_fill(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p.reshape(n, t * h, -1), values).reshape(n, t, h, -1)
    return out / torch.where(total > 0, total, torch.ones_like(total))


def _visible(positions, window):
    first = (positions - window + 1).clamp(min=0) if window else torch.zeros_like(positions)
    return first, positions


def _plain_rows(s, q, table, positions):
    """Tokens [n, t] of n table rows: one row's tokens share its keys."""
    case = s["case"]
    pool = s["pool"].reshape(-1, PAGE, case["c"] + case["r"])
    keys = pool[table.long().clamp(min=0)].reshape(table.shape[0], -1, pool.shape[-1]).float()
    first, last = _visible(positions, case["window"])
    return _attend(q, first, last, keys, keys[..., :case["c"]], _scale(case)).to(torch.bfloat16)


def _plain_step(s):
    b, at = s["case"]["rows"], 0
    for i, (n, before) in enumerate(s["pieces"]):
        pages = -(-(before + n) // PAGE)
        s["out"][at:at + n] = _plain_rows(s, s["q"][None, at:at + n], s["table"][b + i:b + i + 1, :pages],
                                          s["positions"][None, at:at + n])[0]
        at += n
    if b:
        s["out"][at:] = _plain_rows(s, s["q"][at:, None], s["table"][:b], s["step_positions"][:, None])[:, 0]
    return s["out"]


def _plain_prompt(s):
    case = s["case"]
    d, at, kat = case["d"], 0, 0
    for n, before in s["pieces"]:
        kv = s["kv"][kat:kat + before + n].transpose(0, 1).float()
        rope = s["k_rope"][kat:kat + before + n].float()
        keys = torch.cat([kv[..., :d], rope[None].expand(kv.shape[0], -1, -1)], dim=-1)
        q = s["q"][at:at + n].transpose(0, 1)[:, :, None]
        last = torch.arange(before, before + n, device=DEV)[None].expand(kv.shape[0], -1)
        got = _attend(q, torch.zeros_like(last), last, keys, kv[..., d:], _scale(case))
        s["out"][at:at + n] = got[:, :, 0].transpose(0, 1).to(torch.bfloat16)
        at, kat = at + n, kat + before + n
    return s["out"]


def _plain_copy(s):
    pools = s["pools"].unflatten(1, (-1, PAGE))
    pools[:, s["dst"].long()] = pools[:, s["src"].long()]
    return s["pools"]


# ----------------------------------------------------- the package's calls ----

def _handle(s):
    """The descriptor and the workspace that a program makes once and keeps."""
    import paged_kv_gqa_row_gb300 as lnk
    case = s["case"]
    heads = case.get("heads", 1)
    if case["op"] == "prompt":
        return lnk, None, None, None, 0
    if case["op"] == "copy":
        return lnk, lnk.latent_desc(heads, case["c"], case["r"], case["pages"], 1, 1, scale=1.0), None, None, 0
    desc = lnk.latent_desc(heads, case["c"], case["r"], s["pages"], s["table"].shape[0], s["table"].shape[1],
                           scale=_scale(case), window=case.get("window", 0))
    if case["op"] == "append":
        return lnk, desc, lnk.rope_desc(case["theta"]), None, 0
    size = lnk.lnk_latent_workspace_size(desc)
    return lnk, desc, None, torch.zeros(size, dtype=torch.uint8, device=DEV), size


def _own(s):
    if "handle" not in s:
        s["handle"] = _handle(s)
    lnk, desc, rope, ws, size = s["handle"]
    case = s["case"]
    if case["op"] == "append":
        c, r = case["c"], case["r"]
        lnk.lnk_latent_append(desc, rope, s["q"][:, :, -r:], s["q"].stride(1), s["kv"], s["positions"], s["rows"], None,
                              s["table"], s["w"], EPS, s["pool"], s["q_out"][:, :, c:], c + r, s["kv_out"], case["tokens"])
        return {"q": s["q_out"], "kv": s["kv_out"], "pool": s["pool"]}
    if case["op"] == "copy":
        lnk.lnk_latent_copy_pages(desc, s["list"], s["src"], s["dst"], case["moved"])
        return s["pools"]
    if case["op"] == "prompt":
        lnk.lnk_latent_prompt_attn(case["heads"], case["d"], case["r"], _scale(case), s["q"], s["kv"], s["k_rope"],
                                   case["r"], s["q_starts"], s["k_starts"], s["out"], s["q"].shape[0], s["kv"].shape[0],
                                   case["chunks"])
    elif case["op"] == "decode":
        lnk.lnk_latent_decode_attn(desc, s["q"], s["step_positions"], s["table"], s["pool"], s["out"], case["rows"], ws, size)
    else:
        lnk.lnk_latent_step_attn(desc, s["q"], s["rows"], s["positions"], s["step_positions"], s["table"], s["pool"],
                                 s["out"], s["rows"].shape[0], case["rows"], ws, size)
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return dict(append=_plain_append, decode=_plain_step, step=_plain_step, prompt=_plain_prompt,
                copy=_plain_copy)[state["case"]["op"]](state)


# ------------------------------------------------------------ work, exact ----

def _seen(position, window):
    return min(position + 1, window) if window else position + 1


def work(case):
    if case["op"] == "copy":
        return {"bytes": 2 * case["layers"] * case["moved"] * PAGE * (case["c"] + case["r"]) * 2, "flops": 0}
    heads, r = case["heads"], case["r"]
    if case["op"] == "prompt":
        d, pairs, total = case["d"], 0, 0
        for n, before in _chunks(case):
            pairs += n * before + n * (n + 1) // 2
            total += n * heads * (2 * d + r) * 2 + (n + before) * (heads * 2 * d + r) * 2
        return {"bytes": total, "flops": 2 * heads * (2 * d + r) * pairs}
    c = case["c"]
    w = c + r
    if case["op"] == "append":
        t = case["tokens"]
        return {"bytes": t * (2 * heads * r * 2 + 3 * w * 2 + 8), "flops": t * (heads * r * 3 + r * 3 + c * 4)}
    window, total, flops = case["window"], 0, 0
    if case["rows"]:
        lengths = _spread(case["shortest"], case["longest"], case["rows"])
        idle = case.get("idle", 0)
        live = case["rows"] - (case["rows"] // idle if idle else 0)
        seen = sum(_seen(n - 1, window) for n in lengths) * live // case["rows"]
        total += seen * w * 2 + case["rows"] * heads * (w + c) * 2 + 4 * (seen // PAGE + case["rows"])
        flops += 2 * heads * (w + c) * seen
    if case["op"] == "step":
        for n, before in _chunks(case):
            flops += 2 * heads * (w + c) * sum(_seen(p, window) for p in range(before, before + n))
            first = max(0, before - window + 1) if window else 0
            total += (before + n - first) * w * 2 + n * heads * (w + c) * 2 + 8 * n
    return {"bytes": total, "flops": flops}


def _exact_append(s):
    case = s["case"]
    c, r = case["c"], case["r"]
    pos = s["positions"].cpu().numpy()
    angle = (pos.astype(np.float32)[:, None] * s["inv"].cpu().numpy()[None, :]).astype(np.float32).astype(np.float64)
    turn = (np.cos(angle) + 1j * np.sin(angle))[:, None, :]

    def turned(x):
        x = x.float().cpu().numpy().astype(np.float64)
        z = (x[..., :r // 2] + 1j * x[..., r // 2:]) * turn
        return np.concatenate([z.real, z.imag], axis=-1)

    x = s["kv"].float().cpu().numpy().astype(np.float64)
    latent = x[:, :c] / np.sqrt(np.mean(x[:, :c] ** 2, axis=-1, keepdims=True) + EPS) * s["w"].float().cpu().numpy()
    kv = np.concatenate([latent, turned(s["kv"][:, None, c:])[:, 0]], axis=-1)
    q = np.zeros(tuple(s["q_out"].shape))
    q[:, :, c:] = turned(s["q"][:, :, -r:])
    pool = np.zeros(tuple(s["pool"].shape))
    table, rows = s["table"].cpu().numpy(), s["rows"].cpu().numpy()
    for i, (p, row) in enumerate(zip(pos, rows)):
        pool[table[row, p // PAGE] * PAGE + p % PAGE] = kv[i]
    return {"q": torch.from_numpy(q), "kv": torch.from_numpy(kv), "pool": torch.from_numpy(pool)}


def _exact_step(s):
    """Token by token, in 64 bits."""
    case = s["case"]
    c, window, b = case["c"], case["window"], case["rows"]
    rows = (s["rows"].tolist() if s["rows"] is not None else []) + list(range(b))
    positions = (s["positions"].tolist() if s["rows"] is not None else []) + (s["step_positions"].tolist() if b else [])
    table = s["table"].cpu()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    held = (None, None)
    for t, (row, p) in enumerate(zip(rows, positions)):
        if p < 0:
            continue
        if held[0] != row:
            slots = (table[row].long()[:, None] * PAGE + torch.arange(PAGE)).reshape(-1)
            held = (row, s["pool"][slots.clamp(min=0).to(DEV)].double())
        keys = held[1][max(0, p - window + 1) if window else 0:p + 1]
        z = (s["q"][t].double() @ keys.T) * _scale(case)
        out[t] = torch.softmax(z, dim=-1) @ keys[:, :c]
    return out


def _exact_prompt(s):
    case = s["case"]
    d = case["d"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    qs, ks = s["q_starts"].tolist(), s["k_starts"].tolist()
    for i in range(case["chunks"]):
        n, m = qs[i + 1] - qs[i], ks[i + 1] - ks[i]
        hidden = torch.ones((n, m), dtype=torch.bool, device=DEV).triu(m - n + 1)
        for h in range(case["heads"]):
            q = s["q"][qs[i]:qs[i + 1], h].double()
            kv = s["kv"][ks[i]:ks[i + 1], h].double()
            z = (q[:, :d] @ kv[:, :d].T + q[:, d:] @ s["k_rope"][ks[i]:ks[i + 1]].double().T) * _scale(case)
            out[qs[i]:qs[i + 1], h] = torch.softmax(z.masked_fill(hidden, -math.inf), dim=-1) @ kv[:, d:]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "copy":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            s["pools"][:, b * PAGE:(b + 1) * PAGE] = s["pools"][:, a * PAGE:(a + 1) * PAGE]
        return s["pools"]
    return dict(append=_exact_append, decode=_exact_step, step=_exact_step, prompt=_exact_prompt)[case["op"]](s)

"""The latent cache where offsets pass 32 bits, with the most heads, and on streams of its own
(tolerances: latent_harness)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from latent_harness import PAGE, Step, bits, check, d16, d32, normal  # noqa: E402
from oracle import bf16, latent, rope  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,c,r,dec,pieces", [
    (1024, 128, 32, [70, 5], []),
    (1000, 512, 64, [200], [(2, 130)]),
    (300, 256, 64, [9000, 64], []),
    (129, 384, 32, [4000], [(1, 4000)]),
], ids=["1024", "1000-step", "300-cut", "129-cut"])
def test_many_heads(heads, c, r, dec, pieces):
    Step(heads, heads, c, r, pieces=pieces, dec=dec).upload().run().verify()


@pytest.mark.parametrize("heads", [16, 128], ids=["one-sm", "pairs"])
def test_a_stream_of_its_own(heads):
    """Inputs made, a call and its outputs read on one side stream."""
    s = Step(20 + heads, heads, 512, 64, pieces=[(3, 700)], dec=[2000, 65])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.upload()
        s.run()
        s.run(side)
        s.run(side.cuda_stream)
    side.synchronize()
    s.verify()


def test_a_pool_of_more_than_32_bits():
    """Appended to, copied and read behind 2^32 bytes and 2^31 numbers of a pool."""
    import paged_kv_gqa_row_gb300 as lnk
    heads, c, r, pages = 20, 512, 64, 60000  # 2.2e9 numbers
    rng = np.random.default_rng(1)
    t = 150
    pool = torch.zeros((pages * PAGE, c + r), dtype=torch.int16, device="cuda")
    table = np.array([[pages - 1, pages - 7, 3], [pages - 2, 5, pages - 3]], dtype=np.int32)
    desc = lnk.latent_desc(heads, c, r, pages, 2, 3, scale=0.05)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, kv = normal(rng, t, heads, c + r), normal(rng, t, c + r)
    dq = d16(q)
    positions, rows = np.arange(t, dtype=np.int32), np.zeros(t, np.int32)
    lnk.lnk_latent_append(desc, lnk.rope_desc(1e4), dq[:, :, c:], c + r, d16(kv), d32(positions), d32(rows), None, d32(table),
                          None, 0.0, pool, dq[:, :, c:], c + r, None, t, status)
    lnk.lnk_latent_copy_pages(desc, [pool], d32(table[0]), d32(table[1]), 3, status)
    size = lnk.lnk_latent_workspace_size(desc)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = torch.empty((t + 2, heads, c), dtype=torch.int16, device="cuda")
    qq = torch.cat([dq, dq[:2]])
    lnk.lnk_latent_step_attn(desc, qq, d32(rows), d32(positions), d32([149, 149]), d32(table), pool, out, t, 2, ws, size, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    _, want, _ = latent.append(q[:, :, c:], kv, positions, rows, table, np.zeros((t, c + r), np.uint16), rope.inv_freq(1e4, r),
                               c, slots=np.arange(t))
    for row in (0, 1):
        got = np.concatenate([bits(pool[p * PAGE:(p + 1) * PAGE]) for p in table[row]])
        assert bf16.ulp_distance(got[:t], want).max() <= 1 and not got[t:].any()
    keys, full = bf16.to_f64(got[:t]), bits(qq)
    for i, p in ((0, 0), (63, 63), (64, 64), (130, 130), (149, 149), (150, 149), (151, 149)):
        o, spread, z = latent.attend(bf16.to_f64(full[i]), keys[:p + 1], keys[:p + 1, :c], float(np.float32(0.05)))
        check(bits(out[i]), o, spread, z, p + 1, c + r, f"token {i}")


def test_prompts_whose_keys_pass_32_bits():
    import paged_kv_gqa_row_gb300 as lnk
    heads, d, r, n, m = 128, 128, 64, 70000, 5  # 2.3e9 numbers of keys and values
    g = torch.Generator(device="cuda").manual_seed(2)
    kv = torch.empty((n, heads, 2 * d), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    kr = torch.empty((n, r), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q = torch.empty((m, heads, d + r), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    out = torch.empty((m, heads, d), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = float(np.float32((d + r) ** -0.5))
    lnk.lnk_latent_prompt_attn(heads, d, r, scale, q, kv, kr, r, d32([0, 1, m]), d32([0, 69000, n]), out, m, n, 2, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    for h in (0, 127):
        for i, lo, hi in ((0, 0, 69000), (1, 69000, n - 3), (4, 69000, n)):
            keys = np.concatenate([f(kv[lo:hi, h, :d]), f(kr[lo:hi])], axis=1)
            want, spread, z = latent.attend(f(q[i, h])[None], keys, f(kv[lo:hi, h, d:]), scale)
            check(bits(out[i, h].view(torch.int16))[None], want, spread, z, hi - lo, d + r, f"head {h}, query {i}")

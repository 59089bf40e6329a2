"""Page copies in every layer's pools, and a run of the cache operators together:
prompts, forks, copy on write, compaction and decoding over 4-bit pools of
several layers."""
import numpy as np
import pytest

import synth
from harness import to_bits
from oracle import fp4 as ofp4
from oracle import pager as opager
from test_gpu_fp4 import d16, d32, u8
from test_gpu_fp4_attention import check_token

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "e2m1"]


def _dtype(lnk, kind):
    return {"bf16": lnk.KV_BF16, "e4m3": lnk.KV_E4M3, "e2m1": lnk.KV_E2M1}[kind]


def _pools(lnk, desc, layers, seed):
    """Random bytes, [layers][Hkv][pages][page bytes], in one allocation that the layers share."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    size = lnk.lnk_paged_page_bytes(desc)
    return torch.randint(0, 256, (layers, desc.num_kv_heads, desc.num_pages, size), dtype=torch.uint8, device="cuda",
                         generator=g)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hkv,d,pages,layers", [(1, 64, 5, 1), (3, 96, 11, 7), (2, 128, 40, 130)])
def test_copies_every_layer_and_nothing_else(kind, hkv, d, pages, layers):
    import paged_kv_gqa_row_gb300 as lnk
    desc = lnk.attn_desc(hkv, hkv, d, pages, 1, 1, kv_dtype=_dtype(lnk, kind))
    k, v = _pools(lnk, desc, layers, 1), _pools(lnk, desc, layers, 2)
    order = np.random.RandomState(pages).permutation(pages)
    n = pages // 2
    src, dst = order[:n], order[n:2 * n]
    want_k, want_v = k.clone(), v.clone()
    for a, b in zip(src.tolist(), dst.tolist()):
        want_k[:, :, b] = k[:, :, a]
        want_v[:, :, b] = v[:, :, a]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # bad pairs and a page onto itself among the good ones
    src = list(src) + [pages, 0, -1, int(order[-1])]
    dst = list(dst) + [0, pages, 1, int(order[-1])]
    lnk.lnk_paged_copy_pages_layers(desc, list(k), list(v), d32(src), d32(dst), len(src), status)
    torch.cuda.synchronize()
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    assert int(status.item()) == lnk.binding.DEV_BAD_PAGE


def test_one_layer_of_4_bit_pools_through_copy_pages():
    import paged_kv_gqa_row_gb300 as lnk
    desc = lnk.attn_desc(4, 2, 96, 6, 1, 6, kv_dtype=lnk.KV_E2M1)
    k, v = _pools(lnk, desc, 1, 3)[0], _pools(lnk, desc, 1, 4)[0]
    wk, wv = k.clone(), v.clone()
    for a, b in ((4, 0), (1, 5)):
        wk[:, b], wv[:, b] = k[:, a], v[:, a]
    lnk.lnk_paged_copy_pages(desc, k, v, d32([4, 1]), d32([0, 5]), 2)
    torch.cuda.synchronize()
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_a_captured_copy_keeps_its_pools_and_reads_new_pairs():
    import paged_kv_gqa_row_gb300 as lnk
    desc = lnk.attn_desc(2, 2, 128, 12, 1, 1)
    k, v = _pools(lnk, desc, 3, 5), _pools(lnk, desc, 3, 6)
    src, dst = d32([1, 2]), d32([3, 4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lnk.lnk_paged_copy_pages_layers(desc, list(k), list(v), src, dst, 2)
    for a, b in (([1, 2], [3, 4]), ([11, 3], [0, 5])):
        src.copy_(d32(a))
        dst.copy_(d32(b))
        wk, wv = k.clone(), v.clone()
        wk[:, :, b], wv[:, :, b] = k[:, :, a], v[:, :, a]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(k, wk) and torch.equal(v, wv)


def test_a_serving_run_over_4_bit_pools_with_forks_and_compaction():
    """Two layers share one table.  Row 0 takes a prompt of 150 tokens, rows 1 and 2
    fork it, all decode; row 0 leaves, the pools are compacted below page 7, and
    the rows go on.  Every appended token reads back as the quantizer's values,
    outputs match exact attention over what each row's history stores, and a
    decode before the moves equals the same decode after them bit for bit."""
    import paged_kv_gqa_row_gb300 as lnk
    hq, hkv, d, pages, n_rows, per_row, layers = 8, 2, 128, 16, 3, 5, 2
    ks, vs = 0.25, 0.5
    desc = lnk.attn_desc(hq, hkv, d, pages, n_rows, per_row, kv_dtype=lnk.KV_E2M1, k_scale=ks, v_scale=vs)
    rope = lnk.rope_desc(1e4)
    k_pools, v_pools = _pools(lnk, desc, layers, 7), _pools(lnk, desc, layers, 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws_bytes = lnk.lnk_paged_workspace_size(desc, n_rows)
    ws = torch.zeros(ws_bytes, dtype=torch.uint8, device="cuda")
    pg, model = lnk.Pager(pages, n_rows, per_row), opager.Pager(pages, n_rows, per_row)

    def copy(moves):
        if moves:
            lnk.lnk_paged_copy_pages_layers(desc, list(k_pools), list(v_pools), d32([a for a, _ in moves]),
                                            d32([b for _, b in moves]), len(moves), status)

    def write(seed, rows, positions):
        """The tokens in both layers; their rotated queries, one tensor per layer."""
        moves = pg.prepare_append(rows, positions)
        assert moves == model.prepare_append(rows, positions)
        copy(moves)
        table = d32(pg.table())
        t, queries = len(rows), []
        for layer in range(layers):
            q = d16(synth.tensor_bf16(seed, 10 * layer, (t, hq, d)))
            k = d16(synth.tensor_bf16(seed, 10 * layer + 1, (t, hkv, d)))
            v_host = synth.tensor_bf16(seed, 10 * layer + 2, (t, hkv, d))
            q_out = torch.empty_like(q)
            back = [torch.empty_like(k) for _ in range(2)]
            lnk.lnk_paged_append_rope(desc, rope, q, k, d16(v_host), d32(positions), d32(rows), None, table, None, None,
                                      1e-6, k_pools[layer], v_pools[layer], q_out, t, status)
            lnk.lnk_paged_read_tokens(desc, k_pools[layer], v_pools[layer], d32(positions), d32(rows), None, table,
                                      back[0], back[1], t, status)
            stored = ofp4.row_values(*ofp4.quantize(v_host, vs), vs)
            stored[np.array(positions) < 0] = 0  # an inactive token reads as zeros
            # (5 significant bits times a power of two: exact in bf16)
            same = np.array_equal(back[1].view(torch.bfloat16).double().cpu().numpy(), stored)
            assert same
            queries.append(q_out)
        return table, queries

    def decode(table, queries, positions):
        outs = []
        for layer in range(layers):
            out = torch.full_like(queries[layer], 0x7FC0)
            lnk.lnk_paged_decode_attn(desc, queries[layer], d32(positions), table, k_pools[layer], v_pools[layer], out,
                                      n_rows, ws, ws_bytes, status)
            outs.append(out)
        return outs

    def check(table, queries, positions, outs):
        torch.cuda.synchronize()
        host = table.cpu().numpy()
        for layer in range(layers):
            kv, vv = ofp4.pool_values(u8(k_pools[layer]), ks), ofp4.pool_values(u8(v_pools[layer]), vs)
            for b, p in enumerate(positions):
                check_token(to_bits(outs[layer])[b], to_bits(queries[layer])[b], b, p, host, kv, vv, 0,
                            f"layer {layer} row {b}")

    write(1, [0] * 150, list(range(150)))
    for dst in (1, 2):
        pg.fork(0, dst, 150)
        model.fork(0, dst, 150)
    for step in range(3):
        positions = [150 + step] * 3
        table, queries = write(20 + step, [0, 1, 2], positions)
        outs = decode(table, queries, positions)
        check(table, queries, positions, outs)
    pg.reserve(0, 300)  # scatter: row 0 takes more pages, and leaves
    model.reserve(0, 300)
    pg.reserve(1, 300)
    model.reserve(1, 300)
    pg.release(0)
    model.release(0)
    positions = [-1, 152, 152]
    before = decode(d32(pg.table()), queries, positions)
    moves = pg.compact(7)
    assert moves == model.compact(7) and len(moves) >= 2
    copy(moves)
    for pools in (k_pools, v_pools):
        pools[:, :, 7:] = 0x7F  # the upper part is given back
    after = decode(d32(pg.table()), queries, positions)
    torch.cuda.synchronize()
    for a, b in zip(before, after):
        assert torch.equal(a, b)
    # 40 more tokens of each row, into a page mapped before the moves or after them
    table, written = write(60, [1] * 40 + [2] * 40, list(range(153, 193)) * 2)
    queries = [torch.stack([torch.zeros_like(q[0]), q[39], q[79]]) for q in written]
    positions = [-1, 192, 192]
    check(table, queries, positions, decode(table, queries, positions))
    assert int(status.item()) == 0

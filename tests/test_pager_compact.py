"""Compaction of the host page allocator: a worked example, the library against
the oracle's model on seeded random sequences, and refusals (no GPU)."""
import ctypes

import numpy as np
import pytest

from oracle import pager as opager
from test_pager import _apply, _invariants, _lib_err, _lib_pager, _oracle_err, _random_ops

UNMAPPED = -1


def _worked_example(make, err):
    pg = make(8, 4, 4)
    pg.reserve(0, 256)                 # row 0: pages 0 1 2 3
    pg.reserve(1, 128)                 # row 1: pages 4 5
    pg.fork(1, 2, 100)                 # row 2 shares 4 and 5
    pg.reserve(3, 64)                  # row 3: page 6
    pg.release(0)                      # 0 1 2 3 are free
    assert err(lambda: pg.compact(-1)) == "EINVAL" and err(lambda: pg.compact(9)) == "EINVAL"
    before = [list(r) for r in pg.table()]
    assert err(lambda: pg.compact(2)) == "ENOSPACE"  # three pages, two places
    assert [list(r) for r in pg.table()] == before
    assert pg.compact(8) == [] and pg.compact(7) == []
    assert pg.compact(5) == [(5, 0), (6, 1)]
    assert [list(r)[:2] for r in pg.table()] == [[UNMAPPED] * 2, [4, 0], [4, 0], [1, UNMAPPED]]
    assert [pg.refcount(p) for p in range(8)] == [2, 1, 0, 0, 2, 0, 0, 0] and pg.free_pages() == 5
    assert pg.compact(3) == [(4, 2)]
    assert [pg.refcount(p) for p in range(8)] == [2, 1, 2, 0, 0, 0, 0, 0]
    # the next write into a shared page copies it, as before the moves
    assert pg.prepare_append([2], [70]) == [(0, 3)]


def test_oracle_compact_worked_example():
    _worked_example(opager.Pager, _oracle_err)


def test_library_compact_worked_example():
    _worked_example(_lib_pager().Pager, _lib_err)


def _call(pg, limit, err):
    got = {}

    def go():
        got["moves"] = pg.compact(limit)
    e = err(go)
    return e if e else got["moves"]


@pytest.mark.parametrize("seed", [21, 22, 23, 24])
def test_library_compact_matches_the_model_between_other_calls(seed):
    lnk = _lib_pager()
    rng = np.random.default_rng(seed)
    num_pages, num_rows, ppr = [(24, 6, 5), (9, 4, 3), (64, 8, 9)][seed % 3]
    want, got = opager.Pager(num_pages, num_rows, ppr), lnk.Pager(num_pages, num_rows, ppr)
    moved = 0
    for i, op in enumerate(_random_ops(rng, num_rows, ppr, 500)):
        assert _apply(want, op, _oracle_err) == _apply(got, op, _lib_err)
        if i % 3 == 0:
            limit = int(rng.integers(-1, num_pages + 2))
            a, b = _call(want, limit, _oracle_err), _call(got, limit, _lib_err)
            assert a == b, (i, limit, a, b)
            if isinstance(a, list):
                moved += len(a)
                assert not {x for x, _ in a} & {y for _, y in a}
                assert all(want.refcount(p) == 0 for p in range(max(0, limit), num_pages))
        _invariants(want)
        assert np.array_equal(np.asarray(want.table(), dtype=np.int32), got.table())
        assert [want.refcount(p) for p in range(num_pages)] == [got.refcount(p) for p in range(num_pages)]
        assert want.free_pages() == got.free_pages()
    assert moved > 0


def test_compact_refuses_bad_buffers_and_changes_nothing():
    lnk = _lib_pager()
    pg = lnk.Pager(6, 2, 3)
    pg.reserve(0, 192)
    pg.reserve(1, 192)
    pg.release(0)
    i32p = ctypes.POINTER(ctypes.c_int32)
    buf = (ctypes.c_int32 * 8)()
    n = ctypes.c_int32(7)
    einval, erange = 1, 2
    table = pg.table()

    def status(h, limit, src, dst, cap, out):
        return lnk.binding.raw_status("lnk_pager_compact", h, limit, src, dst, cap, out)

    p = ctypes.cast(buf, i32p)
    assert status(None, 3, p, p, 8, ctypes.byref(n)) == einval
    assert status(pg._h, 3, p, p, 8, None) == einval
    assert status(pg._h, 3, None, p, 8, ctypes.byref(n)) == einval and n.value == 0
    assert status(pg._h, 3, p, None, 8, ctypes.byref(n)) == einval
    assert status(pg._h, 3, p, p, -1, ctypes.byref(n)) == einval
    assert status(pg._h, 3, p, p, 2, ctypes.byref(n)) == erange
    assert status(pg._h, 6, None, None, 0, ctypes.byref(n)) == 0  # nothing to move, nothing to write
    assert np.array_equal(pg.table(), table) and pg.free_pages() == 3
    assert pg.compact(3) == [(3, 0), (4, 1), (5, 2)]


class _KeepsTheSharers(opager.Pager):
    def compact(self, limit):
        table = [list(r) for r in self.rows]
        moves = super().compact(limit)
        for old, new in moves:  # only the first entry follows
            hit = [(r, i) for r, row in enumerate(table) for i, e in enumerate(row) if e == old]
            for r, i in hit[1:]:
                self.rows[r][i] = old
        return moves


class _LosesTheCount(opager.Pager):
    def compact(self, limit):
        moves = super().compact(limit)
        for _, new in moves:
            self.count[new] = 1
        return moves


@pytest.mark.parametrize("cls", [_KeepsTheSharers, _LosesTheCount])
def test_worked_example_catches_planted_mistakes(cls):
    with pytest.raises(AssertionError):
        _worked_example(cls, _oracle_err)


def test_copy_pages_layers_refuses_bad_arguments_without_a_launch():
    lnk = _lib_pager()
    good = dict(head_dim=96, num_kv_heads=2, num_pages=4, page_size=64, kv_dtype=lnk.KV_E2M1)

    def status(k=(16, 32), v=(48, 64), src=16, dst=16, n=1, **kw):
        d = dict(good, **kw)
        desc = lnk.attn_desc(d["num_kv_heads"], d["num_kv_heads"], d["head_dim"], d["num_pages"], 1, 1,
                             page_size=d["page_size"], kv_dtype=d["kv_dtype"])
        try:
            lnk.lnk_paged_copy_pages_layers(desc, list(k), list(v), src, dst, n, stream=0)
        except lnk.LnkError as e:
            return e.status
        return 0

    einval, erange, eunsupported = 1, 2, 4
    assert status(n=0) == 0 and status(k=(), v=()) == 0  # nothing to do, nothing enqueued
    assert status(k=(16, None)) == einval and status(v=(48, 72)) == einval and status(k=(20, 32)) == einval
    assert status(src=None) == einval and status(dst=None) == einval and status(n=-1) == einval
    assert status(num_kv_heads=0) == einval and status(num_pages=0) == einval
    assert status(kv_dtype=3) == eunsupported and status(head_dim=80) == eunsupported and status(page_size=32) == eunsupported
    assert status(n=65535 * 1024 + 1) == erange
    with pytest.raises(ValueError):
        status(v=(48,))

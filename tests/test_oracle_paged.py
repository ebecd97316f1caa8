"""Pins of the paged cache's plain definitions: against the dense oracle, by invariants of the
page operations, and by small worked cases."""

import numpy as np
import pytest

import oracle
from oracle import PageTable, paged_attention


def _paged_copy(x, ps, rng, spare=2):
    """Pages in scattered order holding the tokens of x (B, H_kv, N, d); unused slots are NaN."""
    B, h, n, d = x.shape
    per = -(-n // ps)
    order = rng.permutation(B * per + spare)
    pages = np.full((B * per + spare, h, ps, d), np.nan)
    table = np.full((B, per), -1)
    for b in range(B):
        for e in range(per):
            table[b, e] = order[b * per + e]
            part = x[b, :, e * ps:(e + 1) * ps]
            pages[table[b, e], :, :part.shape[1]] = part
    return pages, table


@pytest.mark.parametrize("n,ps,causal", [(7, 8, True), (37, 8, True), (40, 16, False), (1, 8, True)])
def test_all_tokens_as_queries_is_the_dense_attention(n, ps, causal):
    rng = np.random.default_rng(n)
    B, H, hkv, d = 2, 4, 2, 8
    q = rng.standard_normal((B, H, n, d))
    k, v = rng.standard_normal((2, B, hkv, n, d))
    kp, table = _paged_copy(k, ps, np.random.default_rng(5))
    vp, _ = _paged_copy(v, ps, np.random.default_rng(5))
    o, lse, *_ = paged_attention(q, kp, vp, table, [n] * B, [], 0, 0.3, causal)
    O, L = oracle.attention_forward_gqa(q, k, v, 0.3, causal)
    np.testing.assert_allclose(o, O, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse, L, rtol=1e-12, atol=1e-12)


def test_a_shared_prefix_is_the_same_as_its_tokens_in_front_of_every_sequence():
    rng = np.random.default_rng(3)
    B, hkv, d, ps, P, n, T = 3, 2, 8, 8, 21, 13, 2
    pre = rng.standard_normal((2, 1, hkv, P, d))
    own = rng.standard_normal((2, B, hkv, n, d))
    q = rng.standard_normal((B, 4, T, d))
    whole = np.concatenate([np.repeat(pre, B, axis=1), own], axis=3)
    pools, tables = [], None
    for x in whole:
        p, tables = _paged_copy(x, ps, np.random.default_rng(1))
        pools.append(p)
    want = paged_attention(q, *pools, tables, [P + n] * B, [], 0, 0.5, True)
    pools, prefix_table, own_table = [], None, None
    for i in range(2):
        a, prefix_table = _paged_copy(pre[i], ps, np.random.default_rng(2))
        b, own_table = _paged_copy(own[i], ps, np.random.default_rng(2))
        pools.append(np.concatenate([a, b]))
    got = paged_attention(q, *pools, own_table + a.shape[0], [n] * B, prefix_table[0], P, 0.5, True)
    np.testing.assert_allclose(got[0], want[0], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(got[1], want[1], rtol=1e-12, atol=1e-12)


def test_queries_without_keys_and_rows_without_a_sequence():
    q = np.ones((3, 1, 2, 4))
    pages = np.ones((1, 1, 8, 4))
    o, lse, *_ = paged_attention(q, pages, pages, [[0]] * 3, [1, 0, -1], [], 0, 1.0, True)
    assert (o[0, 0, 0] == 0).all() and lse[0, 0, 0] == -np.inf  # position 1 - 2 + 0 < 0
    assert (o[0, 0, 1] == 1).all() and lse[0, 0, 1] == 4.0
    assert (o[1] == 0).all() and np.isnan(o[2]).all()


def _consistent(t):
    """Counts are the numbers of entries that name a page, tails are not shared."""
    refs = [0] * len(t.refs)
    tails = []
    for b in range(len(t.lens)):
        for e in range(t.owned(b)):
            refs[t.table[b][e]] += 1
        if t.lens[b] > 0 and t.lens[b] % t.ps:
            tails.append(t.table[b][t.owned(b) - 1])
    assert refs == t.refs
    assert all(t.refs[p] == 1 for p in tails)


def test_page_operations_keep_the_table_consistent():
    rng = np.random.default_rng(11)
    rows, width, pages = 9, 6, 30
    t = PageTable(8, np.full((rows, width), -1), [-1] * rows, [0] * pages)
    for step in range(300):
        what = rng.integers(0, 4)
        if what == 0:
            t.reserve([int(x) if rng.random() < 0.4 else -1 for x in rng.integers(0, 8 * width + 1, rows)])
        elif what == 1:
            live = [b for b in range(rows) if t.lens[b] >= 0]
            empty = [b for b in range(rows) if t.lens[b] < 0]
            if live and empty:
                kids = list(rng.permutation(empty))[:3]
                t.fork([int(rng.choice(live)) for _ in kids], kids)
        elif what == 2:
            t.free([int(b) for b in rng.permutation(rows)[:2]])
        else:
            before = [[t.content[p] for p in row[:t.owned(b)]] for b, row in enumerate(t.table)]
            n = sum(r > 0 for r in t.refs)
            t.compact()
            assert all(r > 0 for r in t.refs[:n]) and not any(t.refs[n:])
            assert before == [[t.content[p] for p in row[:t.owned(b)]] for b, row in enumerate(t.table)]
        _consistent(t)


def test_pages_go_to_rows_in_order_and_lowest_first():
    t = PageTable(8, [[4, -1, -1], [-1, -1, -1], [-1, -1, -1]], [8, -1, 0], [1, 0, 0, 1, 1, 0])
    refused = t.reserve([9, 24, 8])
    assert refused == [1, 2]  # 1 + 3 > 3 free pages, and so is everything after it
    assert t.table == [[4, 1, -1], [-1, -1, -1], [-1, -1, -1]] and t.lens == [9, -1, 0]
    assert t.refs == [1, 1, 0, 1, 1, 0]


def test_compaction_moves_the_last_pages_into_the_first_holes():
    t = PageTable(8, [[5, 2], [5, 0]], [16, 12], [1, 0, 1, 0, 0, 2])
    assert t.compact() == [0, -1, 2, -1, -1, 1]
    assert t.table == [[1, 2], [1, 0]] and t.refs == [1, 2, 1, 0, 0, 0] and t.content[1] == 5

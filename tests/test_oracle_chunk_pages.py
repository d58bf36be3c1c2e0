"""Pins of the chunk-attention and page oracles: closed forms, the tree
oracle on a chain, library softmax, and the pool's invariants."""

import random

import numpy as np
import pytest

import oracle
from oracle.attention import bf16_to_f64


def _paged(rng, lens, Hkv, D, page=16, spare=3):
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), max(max(need), 1)), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, rng.standard_normal((pages, Hkv, page, D)), rng.standard_normal((pages, Hkv, page, D))


def test_one_token_is_library_softmax():
    rng = np.random.default_rng(0)
    table, k, v = _paged(rng, [38], 2, 8)
    q = rng.standard_normal((1, 4, 8))
    out, lse = oracle.chunk_attention(q, k, v, table, [37], [0, 1])
    pos = np.arange(38)
    for h in range(4):
        K, V = k[table[0, pos // 16], h // 2, pos % 16], v[table[0, pos // 16], h // 2, pos % 16]
        s = K @ q[0, h] / np.sqrt(8)
        w = np.exp(s) / np.exp(s).sum()
        np.testing.assert_allclose(out[0, h], w @ V, rtol=1e-12)
        np.testing.assert_allclose(lse[0, h], np.log(np.exp(s).sum()), rtol=1e-12)


def test_a_chunk_is_a_chain_tree():
    """A chunk's tokens are a chain: the tree oracle with parents i - 1 and the
    chunk's K/V beside the cache must agree with the appended cache."""
    rng = np.random.default_rng(1)
    lens, new = [21, 0], [7, 18]
    table, _, _ = _paged(rng, [a + b for a, b in zip(lens, new)], 2, 8)
    pages = int(table.max()) + 4

    def bits(*shape):
        return (rng.standard_normal(shape).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)

    k, v = bits(pages, 2, 16, 8), bits(pages, 2, 16, 8)
    tk, tv, q = bits(25, 2, 8), bits(25, 2, 8), bits(25, 4, 8)
    cu = np.array([0, 7, 25])
    parents = np.concatenate([np.arange(-1, 6), np.arange(-1, 17)])
    want = oracle.tree_verify_attention(q, tk, tv, k, v, table, lens, cu, parents)
    k2, v2, after = oracle.kv_append(tk[None], tv[None], k[None], v[None], table, lens, cu)
    assert after.tolist() == [28, 18]
    got = oracle.chunk_attention(bf16_to_f64(q), bf16_to_f64(k2[0]), bf16_to_f64(v2[0]), table, lens, cu)
    np.testing.assert_allclose(got[0], want[0], rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(got[1], want[1], rtol=1e-10)


def test_visible_closed_form():
    m = oracle.chunk_visible(10, 4, window=3, sink=2)
    for i in range(4):
        assert np.flatnonzero(m[i]).tolist() == [0, 1] + list(range(10 + i - 2, 10 + i + 1))
    assert oracle.chunk_visible(5, 3).sum() == 6 + 7 + 8
    assert np.array_equal(oracle.chunk_visible(5, 3, window=8), oracle.chunk_visible(5, 3))
    assert oracle.chunk_visible(0, 1, window=1).tolist() == [[True]]


def test_equal_keys_give_the_mean_of_the_visible_values():
    table = np.array([[2, 0]], dtype=np.int32)
    k, v = np.ones((3, 1, 16, 4)), np.arange(3 * 16 * 4, dtype=float).reshape(3, 1, 16, 4)
    out, lse = oracle.chunk_attention(np.ones((2, 1, 4)), k, v, table, [17], [0, 2], window=4, sink=1)
    flat = v[[2, 0], 0].reshape(32, 4)
    for i in range(2):
        seen = [0] + list(range(17 + i - 3, 17 + i + 1))
        np.testing.assert_allclose(out[i, 0], flat[seen].mean(0))
        np.testing.assert_allclose(lse[i, 0], 2.0 + np.log(5))


def _pool(rng, rows, width, pages):
    pool = oracle.Pool([[-1] * width for _ in range(rows)], [0] * rows, [0] * rows, [0] * pages)
    return pool


@pytest.mark.parametrize("seed", range(8))
def test_pool_keeps_its_invariant(seed):
    """Random forks, growth, rollbacks and compactions: references equal
    entries, written ranges are private, shared prefixes read the same."""
    rng = random.Random(seed)
    rows, width, pages = 6, 12, 60
    pool = _pool(rng, rows, width, pages)
    tokens = np.full((1, pages, 16), -1)  # what each slot holds, tagged by (owner, position)
    texts = [[] for _ in range(rows)]
    for step in range(60):
        what = rng.choice(["grow", "fork", "release", "compact"])
        if what == "grow":
            new = [c + rng.choice([0, 1, 5, 20]) for c in pool.ctx]
            new = [min(n, width * 16) for n in new]
            try:
                copies = pool.reserve(new)
            except MemoryError:
                pool.check()
                continue
            assert len({z for _, z in copies}) == len(copies) and not {a for a, _ in copies} & {z for _, z in copies}
            tokens = oracle.copy_pages(tokens, copies)
            for b in range(rows):
                for slot in range(pool.ctx[b], new[b]):
                    page = pool.table[b][slot // 16]
                    assert pool.refs[page] == 1
                    tokens[0, page, slot % 16] = step * 1000 + b
                    texts[b].append(step * 1000 + b)
                pool.ctx[b] = max(pool.ctx[b], new[b])
        elif what == "fork":
            parent, child = rng.randrange(rows), rng.randrange(rows)
            if parent != child and pool.held[child] == 0:
                pool.fork([parent], [child])
                texts[child] = list(texts[parent])
        elif what == "release":
            keep = [rng.choice([c, c, c // 2, 0]) for c in pool.ctx]
            pool.release(keep)
            for b in range(rows):
                pool.ctx[b] = keep[b]
                texts[b] = texts[b][:keep[b]]
        else:
            moves, live = pool.compact()
            tokens = oracle.copy_pages(tokens, moves)
            assert all(r > 0 for r in pool.refs[:live]) and not any(pool.refs[live:])
        pool.check()
        for b in range(rows):
            got = [tokens[0, pool.table[b][s // 16], s % 16] for s in range(pool.ctx[b])]
            assert got == texts[b]


def test_the_lowest_row_keeps_a_shared_page_only_when_every_sharer_grows():
    pool = _pool(None, 3, 4, 8)
    pool.reserve([20, 0, 0])
    pool.ctx[0] = 20
    pool.fork([0, 0], [1, 2])
    assert pool.reserve([21, 21, 21]) == [(1, 2), (1, 3)] and pool.table[0][:2] == [0, 1]
    pool.release([20, 0, 0])
    pool.ctx[1] = pool.ctx[2] = 0
    pool.fork([0], [1])
    assert pool.reserve([20, 21, 0]) == [(1, 2)]  # row 0 does not write: row 1 takes its own
    with pytest.raises(MemoryError):
        pool.reserve([20 + 16 * 7, 21, 0])
    pool.check()

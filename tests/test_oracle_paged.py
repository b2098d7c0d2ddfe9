"""Pins of the fp64 oracle of the paged attention path: facts that its formulas have to give,
none of them a copy of its code."""
import numpy as np
import pytest
import torch

from oracle import paged


def _pool(n):
    return np.arange(n, dtype=np.int32)[::-1].copy()


def test_plan_by_hand():
    # pages of 4; sequence 0 holds pages 7, 8 for 6 tokens of which 1 is accepted, sequence 1 ends
    table = np.full((2, 4), -1, np.int32)
    table[0, :2], table[1, :1] = (7, 8), 9
    free = np.array([0, 1, 2, -1, -1, -1, -1, -1, -1, -1], np.int32)
    r = paged.kv_plan(np.array([2, 1], np.int32), np.array([2, 1], np.int32), table, free, 3, 4, 4,
                      commit=np.array([1, 0], np.int32), add=np.array([4, -1], np.int32))
    assert r["seq_len"].tolist() == [3, 0] and r["n_pages"].tolist() == [2, 0]
    assert r["kv_len"].tolist() == [7, 0] and r["q_len"].tolist() == [4, 0]
    assert r["slots"].tolist() == [[31, 32, 33, 34], [-1] * 4]
    assert r["free_count"] == 4 and r["free"][:4].tolist() == [0, 1, 2, 9] and r["status"] == 0
    # the page pushed last is the first popped
    r = paged.kv_plan(r["seq_len"], r["n_pages"], r["table"], r["free"], r["free_count"], 4, 4,
                      commit=np.array([4, 0], np.int32), add=np.array([2, 3], np.int32))
    assert r["table"][0, :3].tolist() == [7, 8, 9] and r["table"][1, 0] == 2
    assert r["slots"].tolist() == [[35, 36, -1, -1], [8, 9, 10, -1]]


def test_plan_keeps_every_page_once():
    rng = np.random.default_rng(5)
    B, T, page, n = 7, 6, 3, 40
    table, seq, held = np.full((B, 12), -1, np.int32), np.zeros(B, np.int32), np.zeros(B, np.int32)
    free, count, commit = _pool(n), n, None
    for _ in range(60):
        add = rng.integers(-1, T + 1, B).astype(np.int32)
        r = paged.kv_plan(seq, held, table, free, count, T, page, commit, add)
        seq, held, table, free, count = r["seq_len"], r["n_pages"], r["table"], r["free"], r["free_count"]
        mine = [table[b, i] for b in range(B) for i in range(held[b])]
        assert sorted(mine + free[:count].tolist()) == list(range(n))
        used = r["slots"][r["slots"] >= 0]
        assert len(set(used.tolist())) == len(used)
        commit = np.minimum(rng.integers(0, T + 1, B), r["q_len"]).astype(np.int32)


def test_rotation_is_relative_and_keeps_lengths():
    rng = np.random.default_rng(1)
    f = 100.0 ** (-np.arange(8) / 8)
    x, y = rng.standard_normal((1, 24)), rng.standard_normal((1, 24))
    for pairs in (False, True):
        r = lambda z, p: paged.rotate(z, None, [p], f, [8], False, pairs, 0.0)[0]  # noqa: E731
        assert np.allclose(r(x, 0), x[0])
        assert np.isclose((r(x, 77) ** 2).sum(), (x ** 2).sum())
        assert np.isclose(r(x, 40) @ r(y, 33), r(x, 17) @ r(y, 10))
        assert np.array_equal(r(x, 5)[16:], x[0, 16:])


def test_axis_layouts():
    assert [paged.pair_axis(i, [2, 1, 1], False) for i in range(4)] == [0, 0, 1, 2]
    assert [paged.pair_axis(i, [4, 2, 2], True) for i in range(8)] == [0, 1, 2, 0, 1, 2, 0, 0]
    # with one position on all axes the layout does not matter
    f = 10.0 ** (-np.arange(8) / 8)
    x = np.random.default_rng(2).standard_normal((3, 16))
    a = paged.rotate(x, None, [9] * 3, f, [4, 2, 2], True, False, 0.0)
    assert np.allclose(a, paged.rotate(x, None, [9], f, [8], False, False, 0.0))


def test_norm_of_a_head():
    x = np.zeros((1, 16))
    x[0, :2] = 3.0, 4.0                                  # mean square 25 / 16
    r = paged.rotate(x, np.full(16, 2.0), [0], np.ones(8), [8], False, False, 0.0)
    assert np.allclose(r[0, :2], [3 / 1.25 * 2, 4 / 1.25 * 2])


@pytest.mark.parametrize("window", [0, 5])
def test_attention_agrees_with_a_dense_softmax(window):
    rng = np.random.default_rng(3)
    B, T, Hq, Hk, d, page, n = 2, 3, 4, 2, 8, 4, 11
    q = rng.standard_normal((B, T, Hq, d))
    kc, vc = rng.standard_normal((2, 8, page, Hk, d))
    table = np.array([[5, 2, 7], [0, 3, 1]])
    o, lse, written = paged.paged_attention(q, kc, vc, table, [n, n], window=window)
    assert written.all()
    k = torch.tensor(np.stack([kc[t].reshape(-1, Hk, d)[:n] for t in table])).repeat_interleave(Hq // Hk, 2)
    v = torch.tensor(np.stack([vc[t].reshape(-1, Hk, d)[:n] for t in table])).repeat_interleave(Hq // Hk, 2)
    pos = torch.arange(n - T, n)[:, None]
    mask = torch.arange(n) <= pos
    if window:
        mask &= torch.arange(n) > pos - window
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.tensor(q).transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), attn_mask=mask).transpose(1, 2)
    assert np.allclose(o, ref.numpy(), atol=1e-12)
    s = torch.einsum("bthd,bnhd->bthn", torch.tensor(q), k) / d ** 0.5
    s = s.masked_fill(~mask[None, :, None, :], -torch.inf)
    assert np.allclose(lse, torch.logsumexp(s, -1).numpy(), atol=1e-12)


def test_attention_rows_that_see_nothing():
    rng = np.random.default_rng(4)
    q = rng.standard_normal((1, 4, 2, 8))
    kc, vc = rng.standard_normal((2, 2, 4, 1, 8))
    o, lse, written = paged.paged_attention(q, kc, vc, np.array([[1]]), [1], q_len=[3])
    assert written.tolist() == [[True, True, True, False]]
    assert (o[0, :2] == 0).all() and np.isneginf(lse[0, :2]).all()
    assert np.allclose(o[0, 2], vc[1, 0, 0]) and np.isfinite(lse[0, 2]).all()

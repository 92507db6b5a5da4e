"""The oracle of drafted trees and bounded caches, pinned: hand-worked masks, paths
and evictions, masked attention against the causal oracle in C, weights against
attention to indicator values, selections against a brute-force search."""
import itertools

import numpy as np
import pytest
import torch

from oracle import oracle as orc
from paged_kv_attention_16_gb300 import inputs
from tests import spans


def test_hand_worked_masks():
    # request 0: 0 -> (1, 2), 2 -> 3; request 1: two roots, 0 and 1, and 1 -> 2
    mask, pos, st = orc.tree_masks([-1, 0, 0, 2, -1, -1, 1], [0, 4, 7], 8, 1, [10, 3])
    assert st == 0
    assert mask[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1101, 0b1, 0b10, 0b110, 0]
    assert pos.tolist() == [6, 7, 7, 8, 0, 0, 1, 0]


def test_chain_masks_are_causal_and_words_run_on():
    mask, pos, st = orc.tree_masks(np.arange(-1, 129), [0, 130], 130, 3, [140])
    seen = orc.mask_rows(mask, 0, 130)
    assert st == 0 and np.array_equal(seen, np.tril(np.ones((130, 130), bool)))
    assert np.array_equal(pos, 10 + np.arange(130)) and not (mask[:, 2] >> np.uint64(2)).any()


def test_bad_parents_hide_their_subtree_alone():
    mask, pos, st = orc.tree_masks([-1, 1, 1, 0], [0, 4], 4, 1, [4])
    assert st == orc.DEV_BAD_TREE
    assert mask[:, 0].tolist() == [1, 0, 0, 0b1001] and pos.tolist() == [0, 0, 0, 1]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_causal_attention_is_that_of_the_c_oracle(dtype):
    b = spans.batch([5, 1, 20], [30, 9, 20], 4, 2, 64, 16, dtype, seed=3)
    want = orc.paged_attention(
        inputs.storage_array(b.q), inputs.storage_array(b.k_cache), inputs.storage_array(b.v_cache),
        b.block_table.numpy(), b.seq_lens.numpy(), b.query_start_loc.numpy(), 4, 2, 64, 16, b.scale,
        sinks=np.array([0.5, -1.0, 2.0, 0.0])).reshape(-1, 4, 64)
    sinks = [0.5, -1.0, 2.0, 0.0]
    chain = orc.tree_masks(spans.random_trees(None, [5, 1, 20], chain=True), b.query_start_loc.numpy(), 26, 1)[0]
    for mask in (None, chain):
        got = np.concatenate([r["out"] for r in spans.oracle(b, mask, sinks)])
        assert np.abs(got - want).max() < 1e-12


def test_a_tree_row_is_the_causal_row_of_its_own_path():
    """Attention of a node equals the last row of a sequence made of its ancestors."""
    n, cached = 9, 21
    b = spans.batch([n], [n + cached], 2, 1, 64, 16, "f32", seed=4)
    parents = spans.random_trees(np.random.default_rng(4), [n])
    mask = orc.tree_masks(parents, [0, n], n, 1)[0]
    got = spans.oracle(b, mask)[0]["out"]
    page, slot = spans.slots_of(b, 0)
    for i in range(n):
        path = [j for j in range(n) if int(mask[i, 0]) >> j & 1]
        at = list(range(cached)) + [cached + j for j in path]
        k, v = (c[page[at], slot[at], 0].double().numpy() for c in (b.k_cache, b.v_cache))
        for h in range(2):
            x = b.scale * (k @ b.q[i, h].double().numpy())
            w = np.exp(x - x.max())
            assert np.abs(got[i, h] - (w / w.sum()) @ v).max() < 1e-12


def test_rows_that_see_nothing_are_zero():
    b = spans.batch([3], [3], 2, 1, 64, 16, "f32", seed=5)
    r = spans.oracle(b, np.array([[0], [1], [0]], np.uint64))[0]
    assert not r["out"][0].any() and not r["out"][2].any() and r["out"][1].any()


def test_weights_are_attention_to_indicator_values():
    """W_j is the sum over rows of attention with value 1 at position j, 0 elsewhere."""
    b = spans.batch([3], [70], 4, 2, 64, 16, "f32", seed=6)
    want = spans.oracle(b)[0]["weights"]
    page, slot = spans.slots_of(b, 0)
    for j in (0, 1, 40, 66, 67, 69):
        b.v_cache[page, slot] = 0.0
        b.v_cache[page[j], slot[j]] = 1.0
        out = spans.oracle(b)[0]["out"]
        for h in range(2):
            assert abs(out[:, 2 * h:2 * h + 2, 0].sum() - want[h, j]) < 1e-12
    assert np.abs(want.sum(1) - 3 * 2).max() < 1e-12  # each row's weights sum to one


def test_weights_with_a_sink_sum_to_less():
    b = spans.batch([2], [50], 2, 1, 64, 16, "f32", seed=7)
    r = spans.oracle(b, sinks=[1.0, -40.0])[0]
    plain = spans.oracle(b)[0]
    share = np.exp(plain["lse"] - r["lse"])  # of the denominator that the keys hold
    assert abs(r["weights"].sum() - share.sum()) < 1e-12 and share[:, 0].max() < 1 - 1e-3


def test_hand_worked_acceptance():
    # block size 4, one request of 3 cached and 6 drafted positions on pages 2, 0, 1
    k = np.arange(3 * 4, dtype=np.float32).reshape(3, 4, 1, 1)
    table = [[2, 0, 1]]
    kn, vn, after, freed, st = orc.cache_accept(k, k + 100, table, [9], [0, 6], [[1, 3, 5, -1]], [3], 4, 3, 9)
    flat = [int(kn[table[0][p // 4], p % 4, 0, 0]) for p in range(9)]
    was = [table[0][p // 4] * 4 + p % 4 for p in range(9)]
    assert st == 0 and after == [6] and freed == [1]
    assert flat == was[:3] + [was[4], was[6], was[8]] + was[6:]
    assert np.array_equal(vn, kn + 100)


@pytest.mark.parametrize("path,n,st", [([0, 2, 1], 3, 0x100), ([0, 0, 1], 3, 0x100), ([4, 5, 6], 3, 0x100),
                                       ([-1, 0, 1], 3, 0x100), ([0, 1, 2], 4, 0x100), ([0, 1, 2], -1, 0x100),
                                       ([0, 5, 9], 2, 0)])
def test_bad_paths_move_nothing(path, n, st):
    k = np.arange(12, dtype=np.float32).reshape(3, 4, 1, 1)
    got = orc.cache_accept(k, k, [[0, 1, 2]], [9], [0, 6], [path], [n], 4, 3, 9)
    assert got[4] == st
    if st:
        assert np.array_equal(got[0], k) and got[2] == [9] and got[3] == []


def test_kept_positions_by_brute_force():
    """Of all choices that hold the first and the recent ones the kept set weighs most."""
    rng = np.random.default_rng(8)
    for _ in range(30):
        n = int(rng.integers(1, 9))
        w = rng.integers(0, 4, n).astype(float)
        keep, first, recent = (int(x) for x in rng.integers(0, n + 2, 3))
        got = orc.kept_positions(w, keep, first, recent)
        assert got == sorted(set(got)) and len(got) == min(n, keep)
        if n <= keep:
            continue
        f = min(first, keep)
        r = min(recent, keep - f)
        must = set(range(f)) | set(range(n - r, n))
        best = max(sum(w[list(c)]) for c in itertools.combinations(range(n), keep) if must <= set(c))
        assert must <= set(got) and sum(w[got]) == best


def test_ties_nan_and_zeros():
    nan = float("nan")
    assert orc.kept_positions([1, 2, 2, 2, 0], 2, 0, 0) == [1, 2]
    assert orc.kept_positions([nan, -np.inf, 0.0, -0.0, nan], 3, 0, 0) == [1, 2, 3]
    assert orc.kept_positions([0.0, -0.0, 0.0], 2, 0, 0) == [0, 1]
    assert orc.kept_positions([nan, nan, nan], 2, 0, 0) == [0, 1]
    assert orc.kept_positions([9, 1, 5, 1, 1], 3, 1, 1) == [0, 2, 4]
    assert orc.kept_positions([9, 1, 5], 1, 0, 5) == [2] and orc.kept_positions([9, 1], 0, 3, 3) == []


def test_hand_worked_eviction():
    # block size 2, two KV heads that keep other positions; pages 3, 1, 0
    k = np.arange(4 * 2 * 2, dtype=np.float32).reshape(4, 2, 2, 1)
    w = np.zeros((4, 2, 2), np.float32)
    at = [(3, 0), (3, 1), (1, 0), (1, 1), (0, 0)]
    for pos, (p, s) in enumerate(at):
        w[p, 0, s], w[p, 1, s] = [0, 3, 1, 5, 2][pos], [4, 0, 0, 0, 1][pos]
    kn, vn, wn, after, freed, st = orc.cache_evict(k, -k, w, w, [[3, 1, 0]], [5], [3], 2, 4, 8, 5)
    assert st == 0 and after == [3] and freed == [0]
    for h, kept in ((0, [1, 3, 4]), (1, [0, 1, 4])):
        for i, j in enumerate(kept):
            assert kn[at[i][0], at[i][1], h] == k[at[j][0], at[j][1], h] == -vn[at[i][0], at[i][1], h]
            assert wn[at[i][0], h, at[i][1]] == w[at[j][0], h, at[j][1]]


def plant(find, put):
    import inspect
    import types
    src = inspect.getsource(orc)
    assert src.count(find) == 1, src.count(find)
    m = types.ModuleType("planted")
    m.__dict__.update(__name__="oracle.planted", __package__="oracle", __file__=orc.__file__)
    exec(compile(src.replace(find, put), "planted", "exec"), m.__dict__)
    return m


@pytest.mark.parametrize("find,put,test", [
    ("positions[qsl[s] + i] = length - n + len(chain) - 1", "positions[qsl[s] + i] = length - n + len(chain)",
     test_hand_worked_masks),
    ("mask[qsl[s] + i, j // 64] |= np.uint64(1 << (j % 64))", "mask[qsl[s] + i, 0] |= np.uint64(1 << (j % 64))",
     test_chain_masks_are_causal_and_words_run_on),
    ("r[\"weights\"][h, see] += e / den", "r[\"weights\"][h, see] += e / e.sum()",
     test_weights_with_a_sink_sum_to_less),
    ("return (1, 0.0, j) if w != w else (0, -w, j)", "return (1, 0.0, j) if w != w else (0, -w, -j)",
     test_ties_nan_and_zeros),
    ("            a, b = prefix + node, prefix + i", "            a, b = prefix + node, prefix + i + 1",
     test_hand_worked_acceptance),
])
def test_pins_catch_mistakes(find, put, test, monkeypatch):
    bad = plant(find, put)
    for name in ("tree_masks", "mask_rows", "span_attention", "cache_accept", "kept_positions", "cache_evict"):
        monkeypatch.setattr(orc, name, getattr(bad, name))
    with pytest.raises(AssertionError):
        test()

"""Drafted trees on the GPU against the oracle: pa_tree_masks (exact),
pa_forward_tree (elementwise bounds derived from the arithmetic), pa_cache_accept
(bit for bit)."""
import numpy as np
import pytest
import torch

from oracle import oracle as orc
from paged_kv_attention_16_gb300 import inputs, pa
from tests import spans

pytestmark = pytest.mark.gpu
i32 = spans.i32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_attention_16_gb300 import build
    build.build()
    pa.lib()
    pa.pa_get_device_status()  # clear


# ---------------------------------------------------------------------------
# pa_tree_masks
# ---------------------------------------------------------------------------

def masks(parents, qsl, T, words, lens=None):
    mask = torch.full((T, words), 0x1234567, dtype=torch.int64, device="cuda")
    pos = torch.full((T,), 99, dtype=torch.int32, device="cuda") if lens is not None else None
    par = np.full(T, 0x7ffffff)
    par[:len(parents)] = parents
    pa.pa_tree_masks(i32(par), i32(qsl), mask, seq_lens=None if lens is None else i32(lens),
                     positions=pos)
    return mask.cpu().numpy().view(np.uint64), None if pos is None else pos.cpu().numpy()


@pytest.mark.parametrize("q_lens,words,pad,chain", [
    ([1], 1, 0, False), ([8], 1, 3, False), ([64], 1, 0, True), ([65], 2, 0, True), ([64, 63], 3, 1, False),
    ([0, 5, 0, 129, 1], 3, 17, False), ([250, 250], 4, 5, True), ([16] * 64, 1, 0, False),
    ([700], 11, 0, False), ([3] * 1030, 2, 9, False), ([256, 192, 128], 4, 0, False),
])
def test_masks_equal_the_oracle(q_lens, words, pad, chain):
    rng = np.random.default_rng(sum(q_lens) + words)
    parents = spans.random_trees(rng, q_lens, chain)
    qsl = np.concatenate([[0], np.cumsum(q_lens)])
    T = int(qsl[-1]) + pad
    lens = np.asarray(q_lens) + rng.integers(0, 5000, len(q_lens))
    want, pos, status = orc.tree_masks(parents, qsl, T, words, lens)
    got, gpos = masks(parents, qsl, T, words, lens)
    assert pa.pa_get_device_status() == status == 0
    assert np.array_equal(got, want) and np.array_equal(gpos, pos)
    assert np.array_equal(masks(parents, qsl, T, words)[0], want)  # without positions


@pytest.mark.parametrize("what", ["parent_self", "parent_low", "parent_later", "decreasing", "first",
                                  "last", "q_len", "words", "negative"])
def test_masks_bad_metadata(what):
    rng = np.random.default_rng(3)
    q_lens = [9, 70, 20]
    parents = spans.random_trees(rng, q_lens)
    qsl, lens, words = np.array([0, 9, 79, 99]), np.array([30, 90, 20]), 2
    if what == "parent_self":
        parents[9 + 40] = 40
    elif what == "parent_low":
        parents[9 + 5] = -2
    elif what == "parent_later":
        parents[3] = 8
    elif what == "decreasing":
        qsl[1] = 80
    elif what == "first":
        qsl[0] = 1
    elif what == "last":
        qsl[3] = 120
    elif what == "q_len":
        lens[1] = 69
    elif what == "words":
        words = 1
    else:
        lens[0] = -1
    want, pos, status = orc.tree_masks(parents, qsl, 105, words, lens)
    got, gpos = masks(parents, qsl, 105, words, lens)
    assert pa.pa_get_device_status() == status != 0
    assert np.array_equal(got, want) and np.array_equal(gpos, pos)


def test_masks_without_requests():
    got, pos = masks([], [0], 5, 2, [])
    assert not got.any() and not pos.any() and pa.pa_get_device_status() == 0


# ---------------------------------------------------------------------------
# pa_forward_tree
# ---------------------------------------------------------------------------

SHAPES = [(32, 8, 128, 16), (64, 4, 128, 64), (8, 1, 128, 64), (16, 4, 64, 32), (8, 8, 128, 128),
          (2, 1, 64, 48), (16, 1, 64, 16)]


def check_tree(q_lens, cached, shape, dtype="bf16", layout="nhd", seed=0, sinks=None, mask=None,
               max_query_len=0, scale=None):
    H, Hk, D, bs = shape
    b = spans.batch(q_lens, [n + c for n, c in zip(q_lens, cached)], H, Hk, D, bs, dtype, layout, seed,
                    scale)
    if mask is None:
        words = -(-max(q_lens) // 64)
        parents = spans.random_trees(np.random.default_rng(seed), q_lens)
        mask = orc.tree_masks(parents, b.query_start_loc.numpy(), b.num_tokens, max(words, 1))[0]
    got = spans.run_tree(b, mask, sinks=sinks, max_query_len=max_query_len)
    spans.check_out(b, got, spans.oracle(b, mask, sinks), dtype)
    return b, mask, got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("shape", SHAPES)
def test_equals_the_oracle(shape, layout, dtype):
    check_tree([1, 7, 16, 3], [300, 64, 1000, 0], shape, dtype, layout, seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 129])
def test_tree_sizes(n, dtype):
    check_tree([n], [130], (8, 2, 64, 16), dtype, seed=n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ctx", [0, 1, 15, 63, 64, 112, 119, 120, 121, 127, 128, 129, 247, 248, 255, 256, 500])
def test_contexts_around_the_tiles(ctx, dtype):
    check_tree([9, 2], [ctx, ctx + 3], (8, 2, 128, 16), dtype, seed=ctx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_wide_trees_over_row_blocks(dtype):
    check_tree([200, 65], [333, 90], (16, 1, 64, 16), dtype, "hnd", seed=5)
    check_tree([129, 130], [100, 700], (4, 4, 128, 64), dtype, seed=6)


def test_long_contexts_are_split():
    check_tree([5], [9000], (8, 1, 128, 64), seed=7)
    check_tree([12, 1, 3], [20000, 3, 700], (4, 1, 64, 32), seed=8)


def test_many_requests():
    rng = np.random.default_rng(9)
    q = rng.integers(0, 5, 300).tolist()
    check_tree(q, rng.integers(0, 90, 300).tolist(), (4, 2, 64, 16), seed=9)


@pytest.mark.parametrize("S", [20, 21, 27, 28, 29, 32, 33])
def test_batches_around_the_planned_sizes(S):
    """Some requests are planned in the kernel itself, more by a kernel before it."""
    rng = np.random.default_rng(S)
    q = rng.integers(0, 20, S).tolist()
    q[-1] = 0 if S % 2 else 3
    check_tree(q, rng.integers(0, 400, S).tolist(), (8, 2, 64, 16), seed=S)


@pytest.mark.parametrize("S", [28, 40])
def test_bad_requests_among_many(S):
    q_lens = [6] * S
    b = spans.batch(q_lens, [90] * S, 8, 2, 64, 16, seed=S)
    mask = np.full((6 * S, 1), 0x3f, np.uint64)
    want = spans.oracle(b, mask)
    b.seq_lens[S - 1] = 5
    b.seq_lens[3] = b.max_seq_len + 1
    b.block_table[9, 2] = b.num_blocks
    got = spans.run_tree(b, mask, expect=7)
    b.seq_lens[S - 1] = b.seq_lens[3] = 90
    zero_rows(b, got, want, {3, 9, S - 1}, "bf16")
    spans.check_out(b, got, want, "bf16")
    b.query_start_loc[S // 2] = 1
    assert not spans.run_tree(b, mask, expect=pa.PA_DEV_BAD_QSL).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_any_mask(dtype):
    """Masks that are no trees: later tokens seen, own ones hidden, rows without any."""
    q_lens, cached = [40, 70, 1, 2], [0, 65, 0, 200]
    rng = np.random.default_rng(10)
    mask = spans.random_mask(rng, q_lens, 2)
    mask[3] = 0    # sees nothing at all: zeros
    mask[110] = 0  # a single new token without a context that hides itself
    _, _, got = check_tree(q_lens, cached, (8, 2, 64, 16), dtype, seed=10, mask=mask)
    assert not got[3].any() and not got[110].any()


def test_causal_mask_agrees_with_pa_forward():
    q_lens, ctx = [20, 64, 1], [500, 64, 300]
    b = spans.batch(q_lens, ctx, 32, 8, 128, 16, seed=11)
    parents = spans.random_trees(None, q_lens, chain=True)
    mask = orc.tree_masks(parents, b.query_start_loc.numpy(), b.num_tokens, 1)[0]
    got = spans.run_tree(b, mask)
    spans.check_out(b, got, spans.oracle(b), "bf16")
    ref = pa.forward(pa.to_device(b)).float().cpu().numpy()
    assert np.abs(got - ref).max() < 2e-2 and pa.pa_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sinks(dtype):
    sinks = np.linspace(-60.0, 60.0, 8).astype(np.float32)
    check_tree([7, 33], [50, 400], (8, 2, 128, 16), dtype, seed=12, sinks=sinks)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
def test_scales(scale):
    check_tree([7, 12], [50, 400], (8, 2, 64, 16), seed=13, scale=scale)


@pytest.mark.parametrize("max_query_len", [16, 17, 64])
def test_a_bound_on_the_new_tokens(max_query_len):
    check_tree([16, 2, 9], [700, 5, 128], (32, 8, 128, 16), seed=14, max_query_len=max_query_len)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("garbage", [float("nan"), float("inf"), -float("inf"), 3.0e38])
def test_hidden_tokens_may_hold_anything(garbage, dtype):
    """K and V of new tokens that no row of a request sees, and of one that some see."""
    q_lens, cached = [40, 130], [100, 7]
    b = spans.batch(q_lens, [n + c for n, c in zip(q_lens, cached)], 8, 2, 64, 16, dtype, seed=15)
    rng = np.random.default_rng(15)
    mask = orc.tree_masks(spans.random_trees(rng, q_lens), b.query_start_loc.numpy(), 170, 3)[0]
    hidden = {0: [5, 39], 1: [0, 64, 129]}
    qsl = b.query_start_loc.numpy()
    for s, nodes in hidden.items():
        for n in nodes:
            mask[qsl[s]:qsl[s + 1], n // 64] &= ~np.uint64(1 << (n % 64))
    want = spans.oracle(b, mask)
    for s, nodes in hidden.items():
        page, slot = spans.slots_of(b, s)
        for n in nodes:
            b.k_cache[page[cached[s] + n], slot[cached[s] + n]] = garbage
            b.v_cache[page[cached[s] + n], slot[cached[s] + n]] = garbage
    spans.check_out(b, spans.run_tree(b, mask), want, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_value_reaches_those_that_see_it(value, dtype):
    """One new token's V is not finite: rows that see it show that, the others are
    as without it."""
    q_lens, cached = [40, 130], [100, 7]
    b = spans.batch(q_lens, [n + c for n, c in zip(q_lens, cached)], 8, 2, 64, 16, dtype, seed=16)
    rng = np.random.default_rng(16)
    mask = orc.tree_masks(spans.random_trees(rng, q_lens), b.query_start_loc.numpy(), 170, 3)[0]
    want = spans.oracle(b, mask)
    qsl = b.query_start_loc.numpy()
    at = {0: 3, 1: 66}
    for s, n in at.items():
        page, slot = spans.slots_of(b, s)
        b.v_cache[page[cached[s] + n], slot[cached[s] + n], 0, 7] = value
    got = spans.run_tree(b, mask)
    for s, n in at.items():
        seen = orc.mask_rows(mask, qsl[s], q_lens[s])[:, n]
        g = got[qsl[s]:qsl[s + 1]]
        hit = g[seen][:, :4, 7]
        assert (np.isnan(hit) if value != value else hit == value).all()
        g[np.ix_(seen, np.arange(4), [7])] = want[s]["out"][np.ix_(seen, np.arange(4), [7])]
    spans.check_out(b, got, want, dtype)


@pytest.mark.parametrize("max_query_len", [0, 8])
@pytest.mark.parametrize("shape,S", [((32, 8, 128, 16), 60), ((64, 4, 128, 64), 80), ((16, 8, 64, 32), 70),
                                     ((8, 8, 128, 128), 50)])
def test_units_that_one_block_finishes(shape, S, max_query_len):
    """More units than blocks, several tiles each: hidden tokens that hold anything, values
    that are not finite where some see them, a bad page and sinks among them."""
    H, Hk, D, bs = shape
    G = H // Hk
    rng = np.random.default_rng(S)
    q_lens = rng.integers(1, 9, S).tolist()
    q_lens[3:8] = [8, 1, 8, 6, 7]
    cached = rng.integers(60, 700, S).tolist()
    b = spans.batch(q_lens, [n + c for n, c in zip(q_lens, cached)], H, Hk, D, bs, seed=S)
    qsl = b.query_start_loc.numpy()
    mask = orc.tree_masks(spans.random_trees(rng, q_lens), qsl, b.num_tokens, 1)[0]
    mask[qsl[3]:qsl[4]] &= ~np.uint64(1)
    sinks = rng.standard_normal(H)
    want = spans.oracle(b, mask, sinks)
    page, slot = spans.slots_of(b, 3)
    b.k_cache[page[cached[3]], slot[cached[3]]] = float("nan")
    b.v_cache[page[cached[3]], slot[cached[3]]] = float("inf")
    page, slot = spans.slots_of(b, 5)
    b.v_cache[page[-1], slot[-1], 0, 7] = float("inf")  # (the last token's: itself alone sees it)
    b.block_table[7, 0] = -1
    got = spans.run_tree(b, mask, sinks=sinks, expect=1, max_query_len=max_query_len)
    row = qsl[6] - 1
    assert (got[row, :G, 7] == np.inf).all()
    got[row, :G, 7] = want[5]["out"][-1, :G, 7]
    zero_rows(b, got, want, {7}, "bf16")
    spans.check_out(b, got, want, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_in_a_cached_key_stays_visible(dtype):
    b = spans.batch([3, 4], [300, 200], 4, 2, 64, 16, dtype, seed=17)
    page, slot = spans.slots_of(b, 0)
    b.k_cache[page[140], slot[140], 1, 3] = float("nan")
    mask = np.full((7, 1), 0xffff, np.uint64)
    got = spans.run_tree(b, mask)
    assert np.isnan(got[:3, 2:]).all() and np.isfinite(got[:3, :2]).all() and np.isfinite(got[3:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 200, 255, 256, 700, 903])
def test_one_key_takes_the_weight(at, dtype):
    """A key far above all others, wherever it lies: references move."""
    b = spans.batch([6], [904], 4, 1, 64, 16, dtype, seed=18)
    b.q[:] = 1.0
    page, slot = spans.slots_of(b, 0)
    b.k_cache[page[at], slot[at]] = 40.0
    mask = np.full((6, 1), 0x3f, np.uint64)
    spans.check_out(b, spans.run_tree(b, mask), spans.oracle(b, mask), dtype)


@pytest.mark.parametrize("pad", [1, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_last_request_are_left_as_they_were(pad, dtype):
    q_lens = [5, 9]
    b = spans.batch(q_lens, [40, 300], 8, 2, 64, 16, dtype, seed=19)
    mask = orc.tree_masks(spans.random_trees(np.random.default_rng(19), q_lens),
                          b.query_start_loc.numpy(), 14, 1)[0]
    want = spans.oracle(b, mask)
    q = torch.cat([b.q, torch.full((pad, 8, 64), float("nan")).to(b.q.dtype)])
    b.q = q
    out = torch.full((14 + pad, 8, 64), 7.0).to(q.dtype).cuda()
    got = spans.run_tree(b, np.concatenate([mask, np.full((pad, 1), ~np.uint64(0))]), out=out)
    assert (got[14:] == 7.0).all()
    spans.check_out(b, got[:14], want, dtype)


def zero_rows(b, got, want, bad, dtype):
    qsl = b.query_start_loc.numpy()
    for s in range(b.num_seqs):
        if s in bad:
            assert not got[qsl[s]:qsl[s + 1]].any(), s
            want[s] = dict(want[s], out=want[s]["out"] * 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what,bit", [("page", 1), ("negative_page", 1), ("q_len", 2), ("bound", 2),
                                      ("words", 2), ("long", 4), ("negative", 6)])
def test_bad_metadata_zeroes_its_rows(what, bit, dtype):
    q_lens, cached = [6, 70, 9], [200, 50, 400]
    b = spans.batch(q_lens, [n + c for n, c in zip(q_lens, cached)], 8, 2, 64, 16, dtype, seed=20)
    mask = orc.tree_masks(spans.random_trees(np.random.default_rng(20), q_lens),
                          b.query_start_loc.numpy(), 85, 2)[0]
    want, bad, kw = spans.oracle(b, mask), {1}, {}
    if what == "page":
        b.block_table[1, 3] = b.num_blocks
    elif what == "negative_page":
        b.block_table[1, 0] = -1
    elif what == "q_len":
        b.seq_lens[1] = 69
    elif what == "bound":
        kw["max_query_len"] = 69
    elif what == "words":
        mask = np.ascontiguousarray(mask[:, :1])
        want = want[:1] + [want[1]] + want[2:]
    elif what == "long":
        b.seq_lens[1] = b.max_seq_len + 1
    else:
        b.seq_lens[1] = -4
    got = spans.run_tree(b, mask, expect=bit, **kw)
    b.seq_lens[1] = 120
    zero_rows(b, got, want, bad, dtype)
    want = [w for w in want]
    spans.check_out(b, got, want, dtype)


@pytest.mark.parametrize("at,value", [(0, 1), (1, 30), (2, 99)])
def test_bad_starts_zero_every_row(at, value):
    b = spans.batch([6, 8], [200, 50], 8, 2, 64, 16, seed=21)
    b.query_start_loc[at] = value
    got = spans.run_tree(b, np.full((14, 1), 1, np.uint64), expect=pa.PA_DEV_BAD_QSL)
    assert not got.any()


def test_lengths_beyond_the_bound_do_not_leave_the_workspace():
    b = spans.batch([2] * 8, [900] * 8, 8, 2, 64, 16, seed=22)
    b.max_seq_len = 300
    got = spans.run_tree(b, np.full((16, 1), 3, np.uint64), expect=pa.PA_DEV_BAD_SEQLEN)
    assert not got.any()


def test_two_calls_give_the_same_bits():
    b = spans.batch([16] * 20, [1500] * 20, 32, 8, 128, 16, seed=23)
    mask = orc.tree_masks(spans.random_trees(np.random.default_rng(23), [16] * 20),
                          b.query_start_loc.numpy(), 320, 1)[0]
    assert np.array_equal(spans.run_tree(b, mask), spans.run_tree(b, mask))


def tree_call(d, mask, out, stream=None, workspace=None, max_query_len=0):
    pa.pa_forward_tree(d.q, d.k_cache, d.v_cache, d.block_table, d.seq_lens, d.query_start_loc, mask,
                       d.num_heads, d.num_kv_heads, d.head_dim, d.block_size, d.scale, out, stream,
                       max_seq_len=d.max_seq_len, kv_layout=d.kv_layout, workspace=workspace,
                       max_query_len=max_query_len)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_captured_graphs_replayed_at_once(dtype):
    cases = []
    for seed in (24, 25):
        q_lens = [5 + seed % 2, 16, 3]
        b = spans.batch(q_lens, [400, 900, 60], 8, 2, 128, 16, dtype, seed=seed)
        mask = orc.tree_masks(spans.random_trees(np.random.default_rng(seed), q_lens),
                              b.query_start_loc.numpy(), b.num_tokens, 1)[0]
        d, words = pa.to_device(b), spans.to_words(mask)
        out = torch.zeros_like(d.q)
        tree_call(d, words, out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tree_call(d, words, out)
        cases.append((b, mask, d, words, out, g, torch.cuda.Stream()))
    for _ in range(5):
        for c in cases:
            c[4].zero_()
        torch.cuda.synchronize()
        for c in cases:
            with torch.cuda.stream(c[6]):
                c[5].replay()
        torch.cuda.synchronize()
        for b, mask, _, _, out, _, _ in cases:
            spans.check_out(b, out.float().cpu().numpy().astype(np.float64), spans.oracle(b, mask), dtype)
    assert pa.pa_get_device_status() == 0


def test_calls_on_two_streams_at_once_and_a_workspace_of_the_caller():
    b = spans.batch([16] * 6, [2000] * 6, 8, 2, 128, 16, seed=26)
    mask = np.full((96, 1), 0xffff, np.uint64)
    want = spans.oracle(b, mask)
    d, words = pa.to_device(b), spans.to_words(mask)
    outs = [torch.zeros_like(d.q) for _ in range(3)]
    need = pa.pa_forward_tree_workspace_bytes(pa.PA_BF16, 6, 96, 8, 2, 128, b.max_seq_len)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        tree_call(d, words, outs[0], streams[0], ws)
        tree_call(d, words, outs[1], streams[1])
        tree_call(d, words, outs[2], streams[1], max_query_len=16)
    torch.cuda.synchronize()
    for out in outs:
        spans.check_out(b, out.float().cpu().numpy().astype(np.float64), want, "bf16")
    with pytest.raises(pa.PaError):
        tree_call(d, words, outs[0], None, ws[:need - 256])


def test_cache_offsets_past_32_bits():
    """Pages whose element offsets pass 2^31."""
    Hk, D, bs = 8, 128, 64
    pages = (1 << 31) // (bs * Hk * D) + 40
    k = torch.zeros((pages, bs, Hk, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    b = spans.batch([6], [150], 8, Hk, D, bs, seed=27)
    far = torch.tensor([pages - 1, pages - 7, pages - 3])
    old = b.block_table[0, :3].long()
    k[far.cuda()], v[far.cuda()] = b.k_cache[old].cuda(), b.v_cache[old].cuda()
    mask = np.full((6, 1), 0x3f, np.uint64)
    want = spans.oracle(b, mask)
    d = pa.to_device(b)
    d.k_cache, d.v_cache = k, v
    d.block_table = far.to(torch.int32).view(1, 3).cuda()
    out = torch.zeros_like(d.q)
    tree_call(d, spans.to_words(mask), out)
    spans.check_out(b, out.float().cpu().numpy().astype(np.float64), want, "bf16")
    assert pa.pa_get_device_status() == 0


# ---------------------------------------------------------------------------
# pa_cache_accept
# ---------------------------------------------------------------------------

def accept_case(seed, q_lens, cached, Hk, D, bs, dtype, layout, max_path):
    rng = np.random.default_rng(seed)
    b = spans.batch(q_lens, [n + c for n, c in zip(q_lens, cached)], Hk, Hk, D, bs, dtype, layout, seed)
    path = np.full((len(q_lens), max_path), -77)
    lens = np.zeros(len(q_lens), np.int64)
    for s, n in enumerate(q_lens):
        lens[s] = rng.integers(0, min(n, max_path) + 1)
        path[s, :lens[s]] = np.sort(rng.permutation(n)[:lens[s]])
    return b, path, lens


def check_accept(b, path, path_lens, capacity=None, expect=None):
    cap = b.block_table.numel() if capacity is None else capacity
    ks, vs = inputs.storage_array(b.k_cache), inputs.storage_array(b.v_cache)
    want = orc.cache_accept(ks, vs, b.block_table.numpy(), b.seq_lens.numpy(), b.query_start_loc.numpy(),
                            path, path_lens, b.block_size, b.num_blocks, cap, b.kv_layout)
    d = pa.to_device(b)
    after = i32([-5] * b.num_seqs)
    freed, count = i32([-9] * cap), i32([-9])
    pa.pa_cache_accept(d.k_cache, d.v_cache, d.block_table, d.seq_lens, d.query_start_loc, i32(path),
                       i32(path_lens), after, b.block_size, freed_pages=freed, num_freed=count,
                       kv_layout=b.kv_layout)
    assert pa.pa_get_device_status() == want[4]
    if expect is not None:
        assert want[4] == expect
    assert after.tolist() == want[2]
    assert int(count) == len(want[3]) and freed.tolist()[:len(want[3])] == want[3]
    assert (freed[len(want[3]):] == -9).all()
    assert np.array_equal(inputs.storage_array(d.k_cache.cpu()).view(np.uint8), want[0].view(np.uint8))
    assert np.array_equal(inputs.storage_array(d.v_cache.cpu()).view(np.uint8), want[1].view(np.uint8))
    return want


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("q_lens,cached,Hk,D,bs,max_path", [
    ([1], [0], 1, 64, 16, 1), ([8, 1, 0, 16], [100, 15, 7, 0], 8, 128, 16, 8),
    ([250, 40, 99], [3, 64, 17], 2, 64, 64, 250), ([64] * 9, list(range(9)), 4, 128, 32, 30),
    ([5] * 600, [11] * 600, 1, 64, 16, 5),
])
def test_accept_equals_the_oracle(q_lens, cached, Hk, D, bs, max_path, layout, dtype):
    b, path, lens = accept_case(len(q_lens) + D, q_lens, cached, Hk, D, bs, dtype, layout, max_path)
    check_accept(b, path, lens, expect=0)


@pytest.mark.parametrize("D,bs", [(8, 16), (80, 7), (576, 64), (2048, 1)])
def test_accept_other_rows_and_blocks(D, bs):
    b, path, lens = accept_case(D, [30, 50], [9, 0], 3, D, bs, "bf16", "nhd", 50)
    check_accept(b, path, lens, expect=0)


@pytest.mark.parametrize("what,bit", [
    ("falls", 0x100), ("repeats", 0x100), ("beyond", 0x100), ("below", 0x100), ("path_len", 0x100),
    ("path_len_negative", 0x100), ("long", 4), ("q_len", 2), ("page", 1), ("starts", 8)])
def test_accept_bad_metadata(what, bit):
    b, path, lens = accept_case(31, [12, 40, 9], [20, 33, 5], 2, 64, 16, "bf16", "nhd", 20)
    lens[1], path[1] = 20, np.arange(0, 40, 2)
    if what == "falls":
        path[1, 10] = path[1, 8]
    elif what == "repeats":
        path[1, 19] = path[1, 18]
    elif what == "beyond":
        path[1, 19] = 40
    elif what == "below":
        path[1, 0] = -1
    elif what == "path_len":
        lens[1] = 21
    elif what == "path_len_negative":
        lens[1] = -1
    elif what == "long":
        b.seq_lens[1] = b.block_table.shape[1] * 16 + 1
    elif what == "q_len":
        b.seq_lens[1] = 39
    elif what == "page":
        b.block_table[1, 3] = b.num_blocks
    else:
        b.query_start_loc[1], b.query_start_loc[2] = 30, 20
    if what in ("starts", "q_len"):  # (path lengths of the other requests still fit)
        lens[0] = lens[2] = 0
    want = check_accept(b, path, lens)
    assert want[4] & bit


def test_accept_list_overflow_and_no_list():
    b, path, lens = accept_case(32, [100, 100], [5, 9], 1, 64, 16, "bf16", "nhd", 4)
    check_accept(b, path, lens, capacity=3, expect=0x10)
    d, after = pa.to_device(b), i32([0, 0])
    pa.pa_cache_accept(d.k_cache, d.v_cache, d.block_table, d.seq_lens, d.query_start_loc, i32(path),
                       i32(lens), after, 16)
    assert after.tolist() == [5 + lens[0], 9 + lens[1]] and pa.pa_get_device_status() == 0


@pytest.mark.parametrize("S,n", [(1, 1), (256, 8), (257, 8), (64, 32), (65, 32)])
def test_accept_lists_in_one_launch_or_two(S, n):
    b, path, lens = accept_case(S + n, [n] * S, [11] * S, 1, 64, 16, "bf16", "nhd", n)
    check_accept(b, path, lens, expect=0)


def test_accept_bad_paths_leave_their_pages():
    b, path, lens = accept_case(33, [40] * 30, [16] * 30, 2, 64, 16, "bf16", "hnd", 8)
    lens[:] = 3
    path[:, :3] = [0, 7, 39]
    path[4, 1] = 0
    path[9, 2] = 40
    lens[11] = 9
    b.block_table[20, 3] = b.num_blocks
    want = check_accept(b, path, lens, expect=0x101)
    assert want[2][4] == want[2][9] == want[2][11] == 56 and want[2][5] == 19


def test_accepts_captured_and_on_two_streams():
    cases = []
    for seed in (34, 35):
        b, path, lens = accept_case(seed, [30] * 20, [50] * 20, 2, 128, 16, "bf16", "nhd", 12)
        want = orc.cache_accept(inputs.storage_array(b.k_cache), inputs.storage_array(b.v_cache),
                                b.block_table.numpy(), b.seq_lens.numpy(), b.query_start_loc.numpy(), path,
                                lens, 16, b.num_blocks, 200, "nhd")
        d, after, freed, count = pa.to_device(b), i32([0] * 20), i32([-9] * 200), i32([-9])
        d_path, d_lens, st = i32(path), i32(lens), torch.cuda.Stream()
        saved = d.k_cache.clone(), d.v_cache.clone()

        def call(d=d, p=d_path, n=d_lens, after=after, freed=freed, count=count):
            pa.pa_cache_accept(d.k_cache, d.v_cache, d.block_table, d.seq_lens, d.query_start_loc, p, n, after,
                               16, freed_pages=freed, num_freed=count)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        cases.append((want, d, saved, after, freed, count, st, g, d_path, d_lens))
    for _ in range(3):
        for _, d, saved, after, freed, count, *_ in cases:
            d.k_cache.copy_(saved[0])
            d.v_cache.copy_(saved[1])
            for t in (after, freed, count):
                t.fill_(-9)
        torch.cuda.synchronize()
        for c in cases:
            with torch.cuda.stream(c[6]):
                c[7].replay()
        torch.cuda.synchronize()
        for want, d, _, after, freed, count, *_ in cases:
            assert after.tolist() == want[2] and int(count) == len(want[3])
            assert freed.tolist()[:len(want[3])] == want[3]
            assert np.array_equal(inputs.storage_array(d.k_cache.cpu()).view(np.uint8), want[0].view(np.uint8))
            assert np.array_equal(inputs.storage_array(d.v_cache.cpu()).view(np.uint8), want[1].view(np.uint8))
    assert pa.pa_get_device_status() == 0


def test_accept_offsets_past_32_bits():
    """Pages whose element offsets pass 2^31."""
    Hk, D, bs = 8, 128, 64
    pages = (1 << 31) // (bs * Hk * D) + 40
    b, path, lens = accept_case(36, [100], [60], Hk, D, bs, "bf16", "nhd", 50)
    want = orc.cache_accept(inputs.storage_array(b.k_cache), inputs.storage_array(b.v_cache),
                            b.block_table.numpy(), b.seq_lens.numpy(), b.query_start_loc.numpy(), path, lens,
                            bs, b.num_blocks, 8, "nhd")
    far, old = torch.tensor([pages - 1, pages - 7, pages - 3]), b.block_table[0, :3].long()
    k = torch.zeros((pages, bs, Hk, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[far.cuda()], v[far.cuda()] = b.k_cache[old].cuda(), b.v_cache[old].cuda()
    after = i32([0])
    pa.pa_cache_accept(k, v, far.to(torch.int32).view(1, 3).cuda(), b.seq_lens.cuda(), b.query_start_loc.cuda(),
                       i32(path), i32(lens), after, bs)
    assert pa.pa_get_device_status() == 0 and after.tolist() == want[2]
    for got, ref in ((k, want[0]), (v, want[1])):
        assert np.array_equal(inputs.storage_array(got[far.cuda()].cpu()), ref[old.numpy()])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout,block_size", [("nhd", 16), ("hnd", 64)])
def test_speculative_steps_together(layout, block_size):
    """Three steps in one captured graph each size-independent: tables and slots, masks
    and positions, the cache write, tree attention, acceptance; every step's attention
    against the oracle on a cache kept by the host."""
    H, Hk, D, bs, S, n, mp = 8, 2, 64, block_size, 3, 12, 5
    rng = np.random.default_rng(40)
    nb, width = 60, 12
    shape = (nb, bs, Hk, D) if layout == "nhd" else (nb, Hk, bs, D)
    cached = np.array([3, 40, 0])
    perm = rng.permutation(nb)
    table = np.full((S, width), -1)
    used = 0
    for s in range(S):
        k = -(-cached[s] // bs)
        table[s, :k] = perm[used:used + k]
        used += k
    k_cache = torch.randn(shape, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    v_cache = torch.randn(shape, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    d_table, free = i32(table), list(perm[used:])
    T = S * n
    lens, qsl = i32(cached + n), i32(np.arange(S + 1) * n)
    parents, mask = i32(np.zeros(T)), torch.zeros((T, 1), dtype=torch.int64, device="cuda")
    pos, slots = i32(np.zeros(T)), torch.zeros(T, dtype=torch.int64, device="cuda")
    q, kn, vn = (torch.zeros((T, h, D), dtype=torch.bfloat16, device="cuda") for h in (H, Hk, Hk))
    out = torch.zeros_like(q)
    path, path_lens, after = i32(np.zeros((S, mp))), i32(np.zeros(S)), i32(np.zeros(S))
    d_free, start, end = i32(np.zeros(nb)), i32([0]), i32([0])
    freed, count = i32(np.zeros(nb)), i32([0])

    def step():
        pa.pa_block_tables(lens, qsl, d_table, slots, bs, num_blocks=nb, free_pages=d_free,
                           free_start=start, free_end=end)
        pa.pa_tree_masks(parents, qsl, mask, seq_lens=lens, positions=pos)
        pa.pa_cache_write_slots(kn, vn, k_cache, v_cache, slots, bs, kv_layout=layout)
        pa.pa_forward_tree(q, k_cache, v_cache, d_table, lens, qsl, mask, H, Hk, D, bs, 0.125, out,
                           max_seq_len=width * bs, kv_layout=layout, max_query_len=n)
        pa.pa_cache_accept(k_cache, v_cache, d_table, lens, qsl, path, path_lens, after, bs,
                           freed_pages=freed, num_freed=count, kv_layout=layout)

    graph = None
    for turn in range(3):
        par = spans.random_trees(rng, [n] * S)
        parents.copy_(i32(par))
        for t in (q, kn, vn):
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32)).bfloat16())
        pl = rng.integers(1, mp + 1, S)
        chosen = np.full((S, mp), -1)
        for s in range(S):
            chosen[s, :pl[s]] = np.sort(rng.permutation(n)[:pl[s]])
        path.copy_(i32(chosen))
        path_lens.copy_(i32(pl))
        lens.copy_(i32(cached + n))
        d_free.fill_(-1)
        d_free[:len(free)] = i32(free)
        if graph is None:
            saved = [x.clone() for x in (k_cache, v_cache, d_table)]
            step()  # (first calls are made outside capture)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for x, y in zip((k_cache, v_cache, d_table), saved):
                x.copy_(y)
        before = [x.cpu() for x in (k_cache, v_cache, d_table)]
        graph.replay()
        torch.cuda.synchronize()
        assert pa.pa_get_device_status() == 0
        # the same step on the host
        tbl, want_slots, _, taken, _ = orc.block_tables(cached + n, np.arange(S + 1) * n, before[2].numpy(),
                                                        bs, nb, T, np.array(free), 0)
        assert np.array_equal(slots.cpu().numpy(), want_slots)
        ks, vs, _ = orc.cache_write_slots(inputs.storage_array(kn.cpu()), inputs.storage_array(vn.cpu()),
                                          inputs.storage_array(before[0]), inputs.storage_array(before[1]),
                                          want_slots, bs, layout)
        m, want_pos, _ = orc.tree_masks(par, np.arange(S + 1) * n, T, 1, cached + n)
        assert np.array_equal(mask.cpu().numpy().view(np.uint64), m)
        assert np.array_equal(pos.cpu().numpy(), want_pos)
        want = orc.span_attention(inputs.storage_array(q.cpu()), ks, vs, tbl, cached + n,
                                  np.arange(S + 1) * n, H, Hk, D, bs, 0.125, mask=m, kv_layout=layout)
        b = inputs.PagedBatch(q.cpu(), None, None, None, torch.tensor(cached + n), qsl.cpu(), H, Hk, D, bs,
                              0.125, "bf16", width * bs)
        spans.check_out(b, out.float().cpu().numpy().astype(np.float64), want, "bf16")
        ks, vs, new, gone, _ = orc.cache_accept(ks, vs, tbl, cached + n, np.arange(S + 1) * n, chosen, pl, bs,
                                                nb, nb, layout)
        assert after.tolist() == new and freed.tolist()[:int(count)] == gone
        assert np.array_equal(inputs.storage_array(k_cache.cpu()), ks)
        assert np.array_equal(inputs.storage_array(v_cache.cpu()), vs)
        free = list(free[taken:]) + gone
        cached = np.array(new)

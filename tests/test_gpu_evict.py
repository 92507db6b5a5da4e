"""Bounded caches on the GPU against the oracle: pa_forward_weights (elementwise
bounds derived from the arithmetic) and pa_cache_evict (bit for bit)."""
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
# pa_forward_weights
# ---------------------------------------------------------------------------

def check_votes(q_lens, ctx, shape, dtype="bf16", layout="nhd", seed=0, sinks=None, output=True,
                accumulate=True, max_query_len=0, scale=None):
    H, Hk, D, bs = shape
    b = spans.batch(q_lens, ctx, H, Hk, D, bs, dtype, layout, seed, scale)
    before = np.random.default_rng(seed).random((b.num_blocks, Hk, bs)).astype(np.float32)
    before[np.random.default_rng(seed + 1).random(before.shape) < 0.02] = np.nan
    for s in range(b.num_seqs):  # what is added to is finite
        page, slot = spans.slots_of(b, s)
        n = q_lens[s]
        old = len(page) - n if accumulate else 0
        before[page[:old], :, slot[:old]] = np.nan_to_num(before[page[:old], :, slot[:old]])
        before[page[old:], :, slot[old:]] = np.nan  # what is set may be anything
        if n == 0:
            before[page, :, slot] = 0.5
    want = spans.oracle(b, sinks=sinks, values=output)
    out, got = spans.run_weights(b, before, accumulate, output, sinks, max_query_len)
    if output:
        spans.check_out(b, out, want, dtype)
    spans.check_weights(b, got, before, want, accumulate)
    return b, before, want, out, got


SHAPES = [(32, 8, 128, 16), (64, 4, 128, 64), (8, 1, 128, 64), (16, 4, 64, 32), (8, 8, 128, 128),
          (2, 1, 64, 48), (16, 1, 64, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("output", [True, False])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("shape", SHAPES)
def test_equals_the_oracle(shape, layout, output, dtype):
    check_votes([1, 1, 5, 0, 17], [300, 1, 130, 9, 17], shape, dtype, layout, 1, output=output)


@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_steps(dtype, accumulate):
    check_votes([1] * 9, [1, 2, 63, 64, 127, 128, 129, 1000, 255], (8, 2, 128, 16), dtype, seed=2,
                accumulate=accumulate, max_query_len=1)


@pytest.mark.parametrize("output", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [7, 8, 9, 16, 31, 32, 33, 64, 65, 128, 129, 200])
def test_windows_of_rows(n, dtype, output):
    """Around the rows whose scores are kept (32 of a KV head), and whole blocks."""
    check_votes([n, n], [n, n + 300], (8, 2, 64, 16), dtype, seed=n, output=output, accumulate=False)


@pytest.mark.parametrize("output", [True, False])
@pytest.mark.parametrize("shape", [(16, 1, 64, 16), (8, 2, 128, 32), (4, 2, 64, 64)])
def test_windows_of_all_sizes_in_one_call(shape, output):
    """Kept scores, rows whose sums stay in shared memory and rows whose sums pass."""
    check_votes([1, 150, 40, 300, 9, 0, 33, 200], [700, 150, 41, 900, 500, 8, 260, 1000], shape, "bf16", "nhd", 44,
                output=output)


@pytest.mark.parametrize("S", [20, 21, 28, 29])
def test_batches_around_the_planned_sizes(S):
    rng = np.random.default_rng(S)
    q = rng.integers(0, 12, S)
    check_votes(q.tolist(), (q + rng.integers(0, 500, S)).tolist(), (8, 2, 64, 16), seed=S)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_whole_prompt(dtype):
    check_votes([300], [300], (4, 2, 64, 16), dtype, seed=4)


def test_long_contexts_are_split():
    check_votes([1], [30000], (8, 1, 128, 64), seed=5)
    check_votes([20, 1], [9000, 700], (4, 1, 64, 32), seed=6, output=False)


def test_many_requests():
    rng = np.random.default_rng(7)
    q = rng.integers(0, 3, 400)
    check_votes(q.tolist(), (q + rng.integers(0, 60, 400)).tolist(), (4, 2, 64, 16), seed=7)


@pytest.mark.parametrize("output", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sinks(dtype, output):
    sinks = np.linspace(-60.0, 30.0, 8).astype(np.float32)
    check_votes([1, 33, 4], [50, 400, 700], (8, 2, 128, 16), dtype, seed=8, sinks=sinks, output=output)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
def test_scales(scale):
    check_votes([1, 40], [300, 400], (8, 2, 64, 16), seed=9, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 200, 255, 256, 700, 903])
@pytest.mark.parametrize("n", [1, 40])
def test_one_key_takes_the_weight(at, n, dtype):
    b = spans.batch([n], [904 + n], 4, 1, 64, 16, dtype, seed=10)
    b.q[:] = 1.0
    page, slot = spans.slots_of(b, 0)
    b.k_cache[page[at], slot[at]] = 20.0
    before = np.zeros((b.num_blocks, 1, 16), np.float32)
    want = spans.oracle(b)
    out, got = spans.run_weights(b, before, True)
    spans.check_out(b, out, want, dtype)
    spans.check_weights(b, got, before, want, True)
    assert abs(got[page[at], 0, slot[at]] - 4 * n) < 1e-3 * n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("garbage", [float("nan"), float("inf")])
def test_later_tokens_may_hold_anything(garbage, dtype):
    """The last new token's K and V: rows before it are as if they were not there."""
    n = 40
    b = spans.batch([n, 1], [130 + n, 60], 8, 2, 64, 16, dtype, seed=11)
    want = spans.oracle(b)
    page, slot = spans.slots_of(b, 0)
    b.k_cache[page[-1], slot[-1]] = garbage
    b.v_cache[page[-1], slot[-1]] = garbage
    out, _ = spans.run_weights(b, np.zeros((b.num_blocks, 2, 16), np.float32), True)
    assert np.isnan(out[n - 1]).all()
    out[n - 1] = want[0]["out"][-1]
    spans.check_out(b, out, want, dtype)


def test_rows_behind_the_last_request_are_left_as_they_were():
    b = spans.batch([1, 3], [40, 300], 8, 2, 64, 16, seed=12)
    want = spans.oracle(b)
    b.q = torch.cat([b.q, torch.full((5, 8, 64), float("nan")).bfloat16()])
    d = pa.to_device(b)
    out = torch.full_like(d.q, 7.0)
    w = torch.zeros((b.num_blocks, 2, 16), device="cuda")
    pa.pa_forward_weights(d.q, d.k_cache, d.v_cache, d.block_table, d.seq_lens, d.query_start_loc, 8, 2,
                          64, 16, b.scale, out, w, accumulate=True, max_seq_len=300)
    assert (out[4:] == 7.0).all() and pa.pa_get_device_status() == 0
    spans.check_out(b, out[:4].float().cpu().numpy().astype(np.float64), want, "bf16")
    spans.check_weights(b, w.cpu().numpy(), np.zeros((b.num_blocks, 2, 16), np.float32), want, True)


@pytest.mark.parametrize("n", [6, 70])
@pytest.mark.parametrize("what,bit", [("page", 1), ("q_len", 2), ("bound", 2), ("long", 4), ("negative", 6)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_metadata_leaves_the_weights(what, bit, n, dtype):
    q_lens, cached = [1, n, 9], [200, 50, 400]
    b = spans.batch(q_lens, [x + c for x, c in zip(q_lens, cached)], 8, 2, 64, 16, dtype, seed=13)
    before = np.full((b.num_blocks, 2, 16), 0.25, np.float32)
    want, kw = spans.oracle(b), {}
    if what == "page":
        b.block_table[1, 2] = b.num_blocks
    elif what == "q_len":
        b.seq_lens[1] = n - 1
    elif what == "bound":
        kw["max_query_len"] = n - 1 if n > 9 else 9
        if n <= 9:
            kw["max_query_len"] = 5
    elif what == "long":
        b.seq_lens[1] = b.max_seq_len + 1
    else:
        b.seq_lens[1] = -4
    skip = {1, 2} if what == "bound" and n <= 9 else {1}
    out, got = spans.run_weights(b, before, True, expect=bit, **kw)
    b.seq_lens[1] = n + 50
    qsl = b.query_start_loc.numpy()
    for s in skip:
        assert not out[qsl[s]:qsl[s + 1]].any()
        want[s] = dict(want[s], out=want[s]["out"][:0], mass=want[s]["mass"][:0])
        out[qsl[s]:qsl[s + 1]] = 0
    spans.check_weights(b, got, before, want, True)


def test_two_calls_give_the_same_bits():
    b = spans.batch([1] * 30 + [70], [1500] * 31, 32, 8, 128, 16, seed=14)
    before = np.zeros((b.num_blocks, 8, 16), np.float32)
    a, c = spans.run_weights(b, before, True), spans.run_weights(b, before, True)
    assert np.array_equal(a[0], c[0]) and np.array_equal(a[1], c[1])


@pytest.mark.parametrize("n", [1, 40])
def test_two_captured_graphs_replayed_at_once(n):
    cases = []
    for seed in (15, 16):
        b = spans.batch([n, n, n], [400, 900, 60], 8, 2, 128, 16, seed=seed)
        d = pa.to_device(b)
        out, w = torch.zeros_like(d.q), torch.zeros((b.num_blocks, 2, 16), device="cuda")

        def call(d=d, out=out, w=w, b=b):
            pa.pa_forward_weights(d.q, d.k_cache, d.v_cache, d.block_table, d.seq_lens, d.query_start_loc,
                                  8, 2, 128, 16, b.scale, out, w, accumulate=True, max_seq_len=900)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        cases.append((b, out, w, g, torch.cuda.Stream(), d))  # (a graph does not hold its inputs)
    for _ in range(4):
        for c in cases:
            c[2].zero_()
        torch.cuda.synchronize()
        for c in cases:
            with torch.cuda.stream(c[4]):
                c[3].replay()
        torch.cuda.synchronize()
        for b, out, w, _, _, _ in cases:
            want = spans.oracle(b)
            spans.check_out(b, out.float().cpu().numpy().astype(np.float64), want, "bf16")
            spans.check_weights(b, w.cpu().numpy(), np.zeros((b.num_blocks, 2, 16), np.float32), want, True)
    assert pa.pa_get_device_status() == 0


# ---------------------------------------------------------------------------
# pa_cache_evict
# ---------------------------------------------------------------------------

def evict_case(seed, lens, Hk, D, bs, dtype="bf16", layout="nhd", kind="spread"):
    b = spans.batch([0] * len(lens), lens, Hk, Hk, D, bs, dtype, layout, seed)
    rng = np.random.default_rng(seed)
    shape = (b.num_blocks, Hk, bs)
    w = np.exp(1.5 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 3, shape).astype(np.float32)
    elif kind == "equal":
        w = np.zeros(shape, np.float32)
        w[rng.random(shape) < 0.5] = -0.0
    elif kind == "odd":  # NaN, infinities, negative ones, the smallest and the largest
        pick = rng.integers(0, 9, shape)
        for i, x in enumerate([np.nan, np.inf, -np.inf, -1.0, 1e-45, 3.4e38, -3.4e38]):
            w[pick == i] = x
    return b, w


def check_evict(b, w, keep, first=0, recent=0, in_place=False, capacity=None, max_seq_len=None):
    cap = max(b.block_table.numel(), 1) if capacity is None else capacity
    msl = b.max_seq_len if max_seq_len is None else max_seq_len
    blank = w if in_place else np.full_like(w, -3.0)
    want = orc.cache_evict(inputs.storage_array(b.k_cache), inputs.storage_array(b.v_cache), w, blank,
                           b.block_table.numpy(), b.seq_lens.numpy(), keep, b.block_size, b.num_blocks, cap,
                           msl, first, recent, b.kv_layout)
    d = pa.to_device(b)
    d_w = torch.from_numpy(w.copy()).cuda()
    w_out = d_w if in_place else torch.from_numpy(blank.copy()).cuda()
    after, freed, count = i32([-5] * b.num_seqs), i32([-9] * cap), i32([-9])
    pa.pa_cache_evict(d.k_cache, d.v_cache, d_w, d.block_table, d.seq_lens, i32(keep), after, b.block_size,
                      max_seq_len=msl, weights_out=None if in_place else w_out, num_first=first,
                      num_recent=recent, freed_pages=freed, num_freed=count, kv_layout=b.kv_layout)
    assert pa.pa_get_device_status() == want[5]
    assert after.tolist() == want[3]
    assert int(count) == len(want[4]) and freed.tolist()[:len(want[4])] == want[4]
    assert (freed[len(want[4]):] == -9).all()
    for got, ref in ((d.k_cache, want[0]), (d.v_cache, want[1])):
        assert np.array_equal(inputs.storage_array(got.cpu()).view(np.uint8), ref.view(np.uint8))
    assert np.array_equal(w_out.cpu().numpy().view(np.uint32), want[2].view(np.uint32))
    if not in_place:
        assert np.array_equal(d_w.cpu().numpy().view(np.uint32), w.view(np.uint32))
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("D,bs", [(128, 16), (64, 64)])
def test_evict_equals_the_oracle(D, bs, layout, dtype, in_place):
    lens, keep = [1000, 64, 0, 333, 2000, 1], [200, 64, 5, 332, 129, 0]
    b, w = evict_case(D, lens, 3, D, bs, dtype, layout)
    check_evict(b, w, keep, 4, 32, in_place)


@pytest.mark.parametrize("kind", ["ties", "equal", "odd"])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_orders_weights(kind, in_place):
    b, w = evict_case(3, [700, 500, 90, 2049], 2, 64, 16, kind=kind)
    if kind == "odd":  # (copied NaN patterns are compared bit for bit)
        assert np.isnan(w).any()
    check_evict(b, w, [100, 250, 89, 1024], 3, 10, in_place)


@pytest.mark.parametrize("first,recent", [(0, 0), (0, 100), (100, 0), (64, 36), (99, 99), (5000, 5000), (1, 1)])
def test_evict_first_and_recent(first, recent):
    b, w = evict_case(4, [700, 101, 100, 99], 2, 64, 16)
    check_evict(b, w, [100] * 4, first, recent)


@pytest.mark.parametrize("keep", [0, 1, 2, 63, 64, 65, 127, 128, 511, 512, 513, 2046, 2047])
def test_evict_budgets(keep):
    b, w = evict_case(5, [2047, 600], 1, 128, 32)
    check_evict(b, w, [keep] * 2, 1, 1, in_place=True)


def test_evict_long_requests():
    """More positions than a step of the selection, more chunks than blocks wait for."""
    b, w = evict_case(6, [30000, 9000], 2, 64, 64)
    check_evict(b, w, [20000, 10], 4, 64, in_place=True)


@pytest.mark.parametrize("D,bs", [(8, 16), (80, 7), (2048, 1), (4096, 3)])
def test_evict_other_rows_and_blocks(D, bs):
    b, w = evict_case(7, [150, 90], 3, D, bs)
    check_evict(b, w, [40, 70], 2, 9)


def test_evict_many_requests():
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 60, 700).tolist()
    b, w = evict_case(8, lens, 1, 64, 16)
    check_evict(b, w, rng.integers(0, 50, 700).tolist(), 1, 3)


def test_everything_moves_and_nothing_moves():
    b, w = evict_case(9, [3000], 1, 128, 16)
    page, slot = spans.slots_of(b, 0)
    w[page, 0, slot] = np.arange(3000)           # the tail stays: every row moves
    check_evict(b, w, [1500], in_place=True)
    w[page, 0, slot] = -np.arange(3000.0)        # the front stays: no row moves
    check_evict(b, w, [1500], in_place=True)
    w[page, 0, slot] = np.arange(3000) % 2       # every other row
    check_evict(b, w, [1500], in_place=True)


@pytest.mark.parametrize("what", ["negative", "long", "bound", "keep", "page", "capacity"])
def test_evict_bad_metadata(what):
    b, w = evict_case(10, [300, 500, 90], 2, 64, 16)
    keep, kw = [100, 100, 20], {}
    if what == "negative":
        b.seq_lens[1] = -1
    elif what == "long":
        b.seq_lens[1] = b.block_table.shape[1] * 16 + 1
        kw["max_seq_len"] = 5000
    elif what == "bound":
        kw["max_seq_len"] = 499
    elif what == "keep":
        keep[1] = -1
    elif what == "page":
        b.block_table[1, 2] = -1
        b.block_table[1, 20] = b.num_blocks
    else:
        kw["capacity"] = 7
    want = check_evict(b, w, keep, 4, 8, **kw)
    assert want[5] != 0


def test_evict_without_a_list_on_another_stream():
    b, w = evict_case(11, [900, 800], 2, 64, 16)
    want = orc.cache_evict(inputs.storage_array(b.k_cache), inputs.storage_array(b.v_cache), w, w,
                           b.block_table.numpy(), b.seq_lens.numpy(), [100, 300], 16, b.num_blocks, 10 ** 6,
                           900)
    d, d_w, after = pa.to_device(b), torch.from_numpy(w).cuda(), i32([0, 0])
    keep = i32([100, 300])
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    pa.pa_cache_evict(d.k_cache, d.v_cache, d_w, d.block_table, d.seq_lens, keep, after, 16, st,
                      max_seq_len=900)
    torch.cuda.synchronize()
    assert after.tolist() == [100, 300] and pa.pa_get_device_status(st) == 0
    assert np.array_equal(inputs.storage_array(d.k_cache.cpu()), want[0])


def test_evict_offsets_past_32_bits():
    """Pages whose element offsets pass 2^31."""
    Hk, D, bs = 8, 128, 64
    pages = (1 << 31) // (bs * Hk * D) + 40
    b, w = evict_case(17, [180], Hk, D, bs)
    want = orc.cache_evict(inputs.storage_array(b.k_cache), inputs.storage_array(b.v_cache), w, w,
                           b.block_table.numpy(), b.seq_lens.numpy(), [70], bs, b.num_blocks, 10, 180, 2, 9)
    far, old = torch.tensor([pages - 1, pages - 7, pages - 3]), b.block_table[0, :3].long()
    k = torch.zeros((pages, bs, Hk, D), dtype=torch.bfloat16, device="cuda")
    v, d_w = torch.zeros_like(k), torch.zeros((pages, Hk, bs), device="cuda")
    at = far.cuda()
    k[at], v[at], d_w[at] = b.k_cache[old].cuda(), b.v_cache[old].cuda(), torch.from_numpy(w)[old].cuda()
    after = i32([0])
    pa.pa_cache_evict(k, v, d_w, far.to(torch.int32).view(1, 3).cuda(), b.seq_lens.cuda(), i32([70]), after, bs,
                      max_seq_len=180, num_first=2, num_recent=9)
    assert pa.pa_get_device_status() == 0 and after.tolist() == [70]
    for got, ref in ((k, want[0]), (v, want[1]), (d_w, want[2])):
        assert np.array_equal(inputs.storage_array(got[at].cpu()), ref[old.numpy()])


def test_evictions_captured_and_replayed_at_once():
    cases = []
    for seed in (12, 13):
        b, w = evict_case(seed, [3000, 2000], 4, 128, 16)
        d, d_w, w_out = pa.to_device(b), torch.from_numpy(w).cuda(), torch.zeros(w.shape, device="cuda")
        keep, after = i32([700, 1500]), i32([0, 0])
        saved = d.k_cache.clone(), d.v_cache.clone()

        def call(d=d, d_w=d_w, w_out=w_out, keep=keep, after=after):
            pa.pa_cache_evict(d.k_cache, d.v_cache, d_w, d.block_table, d.seq_lens, keep, after, 16,
                              max_seq_len=3000, weights_out=w_out, num_first=4, num_recent=50)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        want = orc.cache_evict(inputs.storage_array(b.k_cache), inputs.storage_array(b.v_cache), w,
                               np.zeros_like(w), b.block_table.numpy(), b.seq_lens.numpy(), [700, 1500], 16,
                               b.num_blocks, 10 ** 6, 3000, 4, 50)
        cases.append((d, saved, g, torch.cuda.Stream(), want, w_out, (keep, after, d_w)))
    for _ in range(3):
        for d, saved, *_ in cases:
            d.k_cache.copy_(saved[0])
            d.v_cache.copy_(saved[1])
        torch.cuda.synchronize()
        for c in cases:
            with torch.cuda.stream(c[3]):
                c[2].replay()
        torch.cuda.synchronize()
        for d, _, _, _, want, w_out, _ in cases:
            assert np.array_equal(inputs.storage_array(d.k_cache.cpu()).view(np.uint8), want[0].view(np.uint8))
            assert np.array_equal(inputs.storage_array(d.v_cache.cpu()).view(np.uint8), want[1].view(np.uint8))
            assert np.array_equal(w_out.cpu().numpy(), want[2])
    assert pa.pa_get_device_status() == 0


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout,bs", [("nhd", 16), ("hnd", 32)])
def test_a_bounded_cache_together(layout, bs):
    """A prompt's last rows vote, the cache is cut down, decode steps attend to what is
    left and add to its weights, and it is cut down again, the pages going round."""
    H, Hk, D, n, window, budget = 8, 2, 64, 400, 32, 96
    b = spans.batch([window], [n], H, Hk, D, bs, "f32", layout, seed=20)
    width = b.block_table.shape[1]
    d = pa.to_device(b)
    rng = np.random.default_rng(20)
    w = torch.full((b.num_blocks, Hk, bs), float("nan"), device="cuda")  # stale
    pa.pa_forward_weights(d.q, d.k_cache, None, d.block_table, d.seq_lens, d.query_start_loc, H, Hk, D, bs,
                          b.scale, None, w, accumulate=False, max_seq_len=n, kv_layout=layout)
    want = spans.oracle(b, values=False)
    host_w = np.full(w.shape, np.nan, np.float32)
    spans.check_weights(b, w.cpu().numpy(), host_w, want, False)
    lens, freed, count = d.seq_lens, i32(np.zeros(width)), i32([0])
    free = i32([])
    for _ in range(2):
        before = [x.cpu() for x in (d.k_cache, d.v_cache, w, lens, d.block_table)]
        after = i32([0])
        pa.pa_cache_evict(d.k_cache, d.v_cache, w, d.block_table, lens, i32([budget]), after, bs,
                          max_seq_len=width * bs, num_first=2, num_recent=16, freed_pages=freed,
                          num_freed=count, kv_layout=layout)
        ref = orc.cache_evict(inputs.storage_array(before[0]), inputs.storage_array(before[1]),
                              before[2].numpy(), before[2].numpy(), before[4].numpy(), before[3].numpy(),
                              [budget], bs, b.num_blocks, width, width * bs, 2, 16, layout)
        assert np.array_equal(d.k_cache.cpu().numpy(), ref[0], equal_nan=True)
        assert np.array_equal(w.cpu().numpy(), ref[2], equal_nan=True)
        assert after.tolist() == [budget] and freed.tolist()[:int(count)] == ref[4]
        free = torch.cat([free, freed[:int(count)]])
        lens = after
        at = 0
        for _ in range(bs + 3):  # decode
            lens = lens + 1
            slots = torch.zeros(1, dtype=torch.int64, device="cuda")
            start, end = i32([at]), i32([0])
            qsl = i32([0, 1])
            pa.pa_block_tables(lens, qsl, d.block_table, slots, bs, num_blocks=b.num_blocks,
                               free_pages=free, free_start=start, free_end=end)
            at = int(end)
            k, v = (torch.from_numpy(rng.standard_normal((1, Hk, D)).astype(np.float32)).cuda() for _ in "kv")
            pa.pa_cache_write_slots(k, v, d.k_cache, d.v_cache, slots, bs, kv_layout=layout)
            q = torch.from_numpy(rng.standard_normal((1, H, D)).astype(np.float32)).cuda()
            step = inputs.PagedBatch(q.cpu(), d.k_cache.cpu(), d.v_cache.cpu(), d.block_table.cpu(), lens.cpu(),
                                     qsl.cpu(), H, Hk, D, bs, b.scale, "f32", width * bs, kv_layout=layout)
            host_w, out = w.cpu().numpy(), torch.zeros_like(q)
            pa.pa_forward_weights(q, d.k_cache, d.v_cache, d.block_table, lens, qsl, H, Hk, D, bs, b.scale,
                                  out, w, accumulate=True, max_seq_len=width * bs, kv_layout=layout,
                                  max_query_len=1)
            want = spans.oracle(step)
            spans.check_out(step, out.cpu().numpy().astype(np.float64), want, "f32")
            spans.check_weights(step, w.cpu().numpy(), host_w, want, True)
        free = free[at:]
    assert pa.pa_get_device_status() == 0

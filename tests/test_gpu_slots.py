"""pa_block_tables and pa_cache_write_slots on the GPU against the oracle:
whole numbers and copied bits, so every result must be equal."""
import numpy as np
import pytest
import torch

from oracle import oracle as orc
from paged_kv_attention_16_gb300 import inputs, pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_attention_16_gb300 import build
    build.build()
    pa.lib()
    pa.pa_get_device_status()  # clear


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def step(lens, qsl, table, bs, nb, T, free=None, start=None, stream=None):
    """The device's (table, slots, positions, free_end) for one step; outputs
    start as garbage."""
    d_table = i32(table)
    slots = torch.full((T,), 12345, dtype=torch.int64, device="cuda")
    pos = torch.full((T,), 777, dtype=torch.int32, device="cuda")
    kw, end = {}, None
    if start is not None:
        end = i32([-9])
        kw = dict(free_pages=i32(free), free_start=i32([start]), free_end=end)
    pa.pa_block_tables(i32(lens), i32(qsl), d_table, slots, bs, stream, num_blocks=nb, positions=pos,
                       **kw)
    torch.cuda.synchronize()
    return (d_table.cpu().numpy(), slots.cpu().numpy(), pos.cpu().numpy(),
            None if end is None else int(end))


def check(lens, qsl, table, bs, nb, T, free=None, start=None):
    want = orc.block_tables(lens, qsl, table, bs, nb, T, free, start)
    got = step(lens, qsl, table, bs, nb, T, free, start)
    assert pa.pa_get_device_status() == want[4]
    for g, w, name in zip(got[:3], want[:3], ("table", "slots", "positions")):
        assert np.array_equal(g, w), name
    assert got[3] == want[3]
    return want


def batch(seed, S, new, cached, bs, slack=0):
    """Lengths, starts, a table holding the pages before the step, a pool and its free pages."""
    rng = np.random.default_rng(seed)
    q = np.ones(S, int) if new == 1 else rng.integers(0, new + 1, S)
    lens = q + rng.integers(0, cached + 1, S)
    held, need = -(-(lens - q) // bs), -(-lens // bs)
    nb = int(need.sum()) + 5
    perm = rng.permutation(nb)
    table = np.full((S, max(int(need.max(initial=1)), 1) + slack), -1)
    at = 0
    for s in range(S):
        table[s, :held[s]] = perm[at:at + held[s]]
        at += held[s]
    return lens, np.concatenate([[0], np.cumsum(q)]), table, nb, perm[at:]


@pytest.mark.parametrize("S,new,cached,bs,pad", [
    (1, 1, 0, 16, 0), (1, 1, 15, 16, 0), (1, 1, 16, 16, 3), (64, 1, 500, 16, 0), (3, 700, 40, 16, 65),
    (37, 90, 333, 64, 1), (513, 1, 90, 16, 0), (700, 9, 50, 7, 100), (1025, 3, 20, 1, 0),
    (2, 9000, 10, 256, 0), (16384, 2, 33, 16, 9),
])
def test_tables_equal_the_oracle(S, new, cached, bs, pad):
    lens, qsl, table, nb, free = batch(S + new, S, new, cached, bs, slack=2)
    T = int(qsl[-1]) + pad
    check(lens, qsl, table, bs, nb, T, np.concatenate([[nb + 7], free]), 1)
    # the slot map alone, over the completed table
    done = orc.block_tables(lens, qsl, table, bs, nb, T, np.concatenate([[nb], free]), 1)[0]
    check(lens, qsl, done, bs, nb, T)


@pytest.mark.parametrize("share", [0.0, 0.3, 0.9])
def test_free_pages_run_out(share):
    lens, qsl, table, nb, free = batch(5, 40, 60, 100, 16)
    need = int((-(-lens // 16)).sum() - (table >= 0).sum())
    want = check(lens, qsl, table, 16, nb, int(qsl[-1]), free[:int(need * share)], 0)
    assert want[4] == orc.DEV_NO_PAGES


@pytest.mark.parametrize("start", [-3, 10, 99])
def test_start_outside_the_list_takes_nothing(start):
    lens, qsl, table, nb, free = batch(6, 12, 30, 100, 16)
    want = check(lens, qsl, table, 16, nb, int(qsl[-1]) + 2, free[:10], start)
    assert want[3] == start


@pytest.mark.parametrize("what", ["decreasing", "first", "last", "q_len", "negative", "long", "page",
                                  "free_page"])
def test_bad_metadata(what):
    lens, qsl, table, nb, free = batch(7, 9, 40, 100, 16)
    T = int(qsl[-1])
    lens, qsl, free = lens.copy(), qsl.copy(), free.copy()
    if what == "decreasing":
        qsl[3], qsl[4] = qsl[4] + 1, qsl[3]
    elif what == "first":
        qsl[0] = 1
    elif what == "last":
        qsl[-1] = T + 1
    elif what == "q_len":
        lens[2] = (qsl[3] - qsl[2]) - 1
    elif what == "negative":
        lens[2] = -5
    elif what == "long":
        lens[4] = 16 * table.shape[1] + 1
    elif what == "page":
        table[:, :] = np.where(table >= 0, nb, table)
    else:
        free[1], free[3] = -2, nb
    want = check(lens, qsl, table, 16, nb, T, free, 0)
    assert want[4] != 0


def test_starts_whose_difference_wraps():
    """Decreasing starts that a 32-bit difference would call a length."""
    lens, qsl, table, nb, free = batch(7, 3, 40, 100, 16)
    top = 2 ** 31 - 1
    want = check(np.array([top, top, 40]), np.array([0, top, -5, 3]), table, 16, nb, 3, free, 0)
    assert want[4] == pa.PA_DEV_BAD_QSL


def test_no_requests_and_no_tokens():
    e = np.zeros(0, int)
    got = step(e, [0], np.zeros((0, 4), int), 16, 8, 5, [3, 4], 1)
    assert (got[1] == -1).all() and (got[2] == 0).all() and got[3] == 1
    got = step([5, 0], [0, 0, 0], np.full((2, 4), -1), 16, 8, 0, [3, 4], 1)
    assert got[3] == 1 and pa.pa_get_device_status() == 0


def test_a_chain_of_captured_steps():
    """One captured step replayed as its inputs move on: lengths grow in place,
    the two counters alternate (two steps to a graph)."""
    S, bs, nb = 5, 16, 64
    rng = np.random.default_rng(2)
    pages = rng.permutation(nb)
    lens, qsl, table = i32([3, 15, 31, 16, 1]), i32(np.arange(S + 1)), i32(np.full((S, 8), -1))
    free, a, b = i32(pages), i32([0]), i32([0])
    slots = torch.empty((2, S), dtype=torch.int64, device="cuda")
    kw = dict(num_blocks=nb, free_pages=free)
    all_new = i32([0, 3, 18, 49, 65, 66])
    first = torch.empty(66, dtype=torch.int64, device="cuda")
    pa.pa_block_tables(lens, all_new, table, first, bs, free_start=a, free_end=b, **kw)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        lens.add_(1)
        pa.pa_block_tables(lens, qsl, table, slots[0], bs, free_start=b, free_end=a, **kw)
        lens.add_(1)
        pa.pa_block_tables(lens, qsl, table, slots[1], bs, free_start=a, free_end=b, **kw)
    w_table, _, _, end, _ = orc.block_tables([3, 15, 31, 16, 1], [0, 3, 18, 49, 65, 66],
                                             np.full((S, 8), -1), bs, nb, 66, pages, 0)
    now = np.array([3, 15, 31, 16, 1])
    for _ in range(6):
        g.replay()
        torch.cuda.synchronize()
        for step_ in range(2):
            now = now + 1
            w_table, w_slots, _, end, st = orc.block_tables(now, np.arange(S + 1), w_table, bs, nb, S,
                                                            pages, end)
            assert st == 0 and np.array_equal(slots[step_].cpu().numpy(), w_slots)
        assert np.array_equal(table.cpu().numpy(), w_table) and int(b) == end
    assert pa.pa_get_device_status() == 0


# ---------------------------------------------------------------------------
# pa_cache_write_slots
# ---------------------------------------------------------------------------

def rows_of(T, Hk, D, dtype, seed, fused=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, fused + 2 * Hk, D), generator=g).to(inputs.DTYPES[dtype])
    if fused:
        x = x.cuda()
        return x[:, fused:fused + Hk], x[:, fused + Hk:]
    return x[:, :Hk].contiguous().cuda(), x[:, Hk:].contiguous().cuda()


def write_both(k, v, bs, nb, layout, slots, seed, status=0, stream=None):
    Hk, D = k.shape[1:]
    g = torch.Generator().manual_seed(seed)
    shape = (nb, bs, Hk, D) if layout == "nhd" else (nb, Hk, bs, D)
    kc, vc = (torch.randn(shape, generator=g).to(k.dtype) for _ in range(2))
    want = orc.cache_write_slots(*(inputs.storage_array(x) for x in (k, v, kc, vc)), slots, bs, layout)
    d_k, d_v = kc.cuda(), vc.cuda()
    d_slots = torch.tensor(slots, dtype=torch.int64).cuda()
    torch.cuda.synchronize()
    pa.pa_cache_write_slots(k, v, d_k, d_v, d_slots, bs, stream, kv_layout=layout)
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == want[2] == status
    for got, w in ((d_k, want[0]), (d_v, want[1])):
        assert np.array_equal(inputs.storage_array(got.cpu()).view(np.uint8), w.view(np.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("T,Hk,D,bs,fused", [
    (1, 1, 8, 1, 0), (1, 2, 64, 16, 8), (7, 3, 40, 5, 1), (64, 8, 128, 16, 32), (333, 4, 64, 64, 0),
    (50, 5, 72, 48, 3), (3000, 1, 128, 16, 7),
])
def test_write_equals_the_oracle(T, Hk, D, bs, fused, layout, dtype):
    k, v = rows_of(T, Hk, D, dtype, T + D, fused)
    nb = -(-T // bs) + 3
    slots = np.random.default_rng(T).permutation(nb * bs)[:T]
    slots[::5] = np.where(np.arange(len(slots[::5])) % 2 == 0, -1, -(1 << 40))
    write_both(k, v, bs, nb, layout, slots, T)


def test_slots_past_the_pool_are_skipped():
    k, v = rows_of(6, 2, 64, "bf16", 1)
    write_both(k, v, 16, 3, "nhd", [0, 48, 5, 1 << 40, 47, -1], 2, status=orc.DEV_BAD_BLOCK)


def test_a_repeated_row_and_odd_strides():
    """A token stride of 0 repeats one row; K and V may have different strides."""
    k, _ = rows_of(1, 2, 64, "bf16", 3)
    wide = torch.randn((9, 5, 64), device="cuda").to(torch.bfloat16)
    write_both(k.expand(9, 2, 64), wide[:, 1:3], 16, 2, "hnd", list(range(20, 29)), 4)


def test_rows_with_gaps_between_heads_are_refused():
    x = torch.zeros((4, 6, 64), dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros((2, 16, 3, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        pa.pa_cache_write_slots(x[:, ::2], x[:, 1::2], cache, cache, torch.zeros(4, dtype=torch.int64, device="cuda"), 16)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: its last slots are reached."""
    Hk, D, bs = 8, 128, 16
    nb = (1 << 32) // (bs * Hk * D * 2) + 3
    kc = torch.zeros((nb, bs, Hk, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    k, v = rows_of(3, Hk, D, "bf16", 9)
    slots = torch.tensor([nb * bs - 1, nb * bs - 17, 0], device="cuda")
    pa.pa_cache_write_slots(k, v, kc, vc, slots, bs)
    assert pa.pa_get_device_status() == 0
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // bs, s % bs], k[t]) and torch.equal(vc[s // bs, s % bs], v[t])
    # in the head-major layout the same bytes
    kh, vh = kc.view(nb, Hk, bs, D).zero_(), vc.view(nb, Hk, bs, D).zero_()
    pa.pa_cache_write_slots(k, v, kh, vh, slots, bs, kv_layout="hnd")
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(kh[s // bs, :, s % bs], k[t]) and torch.equal(vh[s // bs, :, s % bs], v[t])


def test_on_a_side_stream():
    side = torch.cuda.Stream()
    k, v = rows_of(40, 2, 64, "f32", 8)
    write_both(k, v, 16, 4, "nhd", np.random.default_rng(1).permutation(64)[:40], 9, stream=side)
    lens, qsl, table, nb, free = batch(9, 20, 30, 60, 16)
    want = orc.block_tables(lens, qsl, table, 16, nb, int(qsl[-1]), free, 0)
    got = step(lens, qsl, table, 16, nb, int(qsl[-1]), free, 0, stream=side)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[3] == want[3]

"""pa_forward_shared_prefix against the fp64 oracle on the same contexts
written out in full (every request's block-table row naming its prefix's pages).

Tolerances, per output element, with A = sum_j p_j |v_j| of the exact row (the
oracle run on |V|), out the exact output:
  bf16: every weight is rounded to bf16 once (half a step, 2^-8 relative) before
        the value product while the sum of weights is kept in fp32, and the
        output is rounded once: 2^-8 (A + |out|).
  both: a score is a sum of D products in fp32, off by at most (D + 2) 2^-24
        s_max with s_max = scale max|q| max|k| (2-norms bound sum |q_d k_d|); a
        weight is then off by that, times 2 for weight and denominator; sums
        over N keys of weights and of weighted values are each off by N 2^-24,
        and 64 more roundings cover exponentials, rescaling and the merge:
        2^-24 (2 (D + 2) s_max + 2 N + 64) A.
"""
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


def oracle(b, rows=None, sinks=None, absolute=False):
    v = b.v_cache.abs() if absolute else b.v_cache
    return orc.paged_attention(
        inputs.storage_array(b.q), inputs.storage_array(b.k_cache), inputs.storage_array(v),
        b.full_table.numpy(), b.seq_lens.numpy(), b.query_start_loc.numpy(), b.num_heads,
        b.num_kv_heads, b.head_dim, b.block_size, b.scale, rows=rows, kv_layout=b.kv_layout,
        sinks=None if sinks is None else np.asarray(sinks, np.float64))


def tolerance(b, want, absolute):
    q, k = b.q.float(), torch.nan_to_num(b.k_cache.float())
    s_max = abs(b.scale) * float(q.norm(dim=-1).max()) * float(k.norm(dim=-1).max())
    N = int(b.seq_lens.max())
    tol = 2.0 ** -24 * (2 * (b.head_dim + 2) * s_max + 2 * N + 64) * absolute
    if b.dtype == "bf16":
        tol = tol + 2.0 ** -8 * (absolute + np.abs(want))
    return tol


def check(b, got, rows=None, sinks=None, what=""):
    want, absolute = oracle(b, rows, sinks), oracle(b, rows, sinks, absolute=True)
    g = got.float().cpu().numpy().astype(np.float64).reshape(-1, b.head_dim)
    w, a = want.reshape(g.shape), absolute.reshape(g.shape)
    if rows is not None:
        g, w, a = g[rows], w[rows], a[rows]
    assert np.isfinite(g).all(), what
    over = np.abs(g - w) - tolerance(b, w, a)
    assert over.max(initial=-1.0) <= 0, f"{what}: {int((over > 0).sum())} elements off, worst {over.max()}"


def run(b, status=0, sinks=None, **kw):
    d = pa.to_device(b)
    out = torch.full_like(d.q, float("nan"))
    s = None if sinks is None else torch.as_tensor(np.asarray(sinks), dtype=torch.float32).cuda()
    pa.forward_shared_prefix(d, out=out, sinks=s, **kw)
    got = pa.pa_get_device_status()
    assert got == status, f"device status {got:#x}"
    return out


def make(groups, H, Hk, D, bs, dtype="bf16", layout="nhd", seed=0, **kw):
    b = inputs.shared_prefix_batch(groups, H, Hk, D, bs, dtype=dtype, seed=seed, **kw)
    return inputs.as_hnd(b) if layout == "hnd" else b


def decodes(n, lo, hi, seed):
    rng = np.random.default_rng(seed)
    return [(1, int(x)) for x in rng.integers(lo, hi + 1, n)]


BATCHES = {
    # one group of decodes; own parts from a single position on
    "decode": lambda bs: [(20 * bs, [(1, 1), (1, 2), (1, bs), (1, bs + 1), (1, 70)])],
    # groups with and without a prefix, of one request, empty, with idle requests
    "groups": lambda bs: [(0, [(1, 5), (3, 9)]), (bs, [(1, 1)]), (3 * bs, []),
                          (7 * bs, [(0, 0), (1, 33), (0, 8), (1, 4)]), (11 * bs, [(0, 3)])],
    # extends: own part all new, one token, many tokens, mixed with decodes
    "extend": lambda bs: [(5 * bs, [(40, 40), (1, 17), (2, 300), (130, 150)]), (bs, [(9, 9), (1, 1)])],
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,D,bs,layout", [
    (8, 2, 128, 16, "nhd"), (4, 4, 64, 16, "hnd"), (16, 1, 64, 64, "nhd"), (8, 4, 128, 128, "hnd"),
    (16, 2, 128, 48, "nhd"), (2, 1, 64, 256, "nhd"),
])
@pytest.mark.parametrize("kind", sorted(BATCHES))
def test_equals_the_oracle(kind, H, Hk, D, bs, layout, dtype):
    b = make(BATCHES[kind](bs), H, Hk, D, bs, dtype, layout, seed=H + D + bs)
    check(b, run(b), what=kind)


@pytest.mark.parametrize("n,H,Hk,D,bs", [
    (3, 8, 8, 128, 16), (31, 8, 2, 64, 16), (33, 8, 2, 128, 16), (64, 16, 4, 64, 64),
    (65, 16, 4, 128, 16), (130, 16, 1, 128, 64), (257, 2, 2, 64, 16),
])
def test_row_block_edges(n, H, Hk, D, bs):
    """Row counts around the 128-row tiles and the 256-row items."""
    b = make([(9 * bs, decodes(n, 1, 40, n))], H, Hk, D, bs, seed=n)
    check(b, run(b, max_query_len=1))


@pytest.mark.parametrize("pages", [1, 7, 8, 9, 15, 16, 17, 63, 64, 65, 200])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_lengths_around_the_tiles(pages, dtype):
    b = make([(16 * pages, decodes(4, 1, 30, pages))], 8, 1, 128, 16, dtype, seed=pages)
    check(b, run(b))


@pytest.mark.parametrize("D,bs,layout", [(128, 16, "nhd"), (64, 64, "hnd"), (128, 128, "nhd")])
def test_long_prefix_is_split_over_the_grid(D, bs, layout):
    b = make([(24576, decodes(20, 1, 600, 4))], 8, 1, D, bs, layout=layout, seed=4)
    rows = np.random.default_rng(0).choice(160, 24, replace=False)
    check(b, run(b, max_query_len=1), rows=np.sort(rows).astype(np.int64))


@pytest.mark.parametrize("D,G,layout", [(128, 4, "nhd"), (64, 8, "hnd"), (128, 1, "hnd"), (64, 16, "nhd")])
def test_more_items_than_sms(D, G, layout):
    """A block goes through several items, of one and of two row tiles, with
    tiles that wrap the rings of both."""
    rng = np.random.default_rng(D + G)
    groups = [(16 * int(rng.integers(1, 90)), decodes(int(rng.integers(1, 600 // G)), 1, 40, i))
              for i in range(30)]
    b = make(groups, 8 * G, 8, D, 16, layout=layout, seed=D + G)
    check(b, run(b), rows=np.sort(rng.choice(b.num_tokens * 8 * G, 500, replace=False)).astype(np.int64))


def test_many_groups():
    """More groups than the split model looks at, more requests than the merge caches."""
    rng = np.random.default_rng(8)
    groups = [(16 * int(rng.integers(0, 30)), decodes(int(rng.integers(1, 11)), 1, 30, i))
              for i in range(220)]
    b = make(groups, 4, 2, 64, 16, seed=8)
    assert b.num_seqs > 1024
    check(b, run(b), rows=np.sort(rng.choice(b.num_tokens * 4, 600, replace=False)).astype(np.int64))


@pytest.mark.parametrize("H,Hk,D,bs,layout", [(64, 4, 128, 16, "nhd"), (4, 2, 64, 64, "hnd"),
                                              (8, 8, 128, 128, "nhd"), (16, 1, 64, 48, "nhd")])
def test_few_long_rows_are_cut_over_their_own_positions(H, Hk, D, bs, layout):
    """Requests of more than one token whose own parts are many positions: several
    splits a row, the last tokens' rows seeing more of them than the first's."""
    b = make([(4 * bs, [(15, 1368), (3, 700), (1, 50), (130, 131)]), (0, [(40, 901), (2, 2)])],
             H, Hk, D, bs, layout=layout, seed=12)
    sinks = np.linspace(-3, 3, H).astype(np.float32)
    check(b, run(b, sinks=sinks), sinks=sinks)
    assert torch.equal(run(b).view(torch.int16), run(b).view(torch.int16))


def test_more_groups_than_the_planner_keeps():
    rng = np.random.default_rng(9)
    b = make([(16 * int(rng.integers(0, 12)), [(1, int(rng.integers(1, 20)))]) for _ in range(1100)],
             2, 1, 64, 16, seed=9)
    check(b, run(b, max_query_len=1), rows=np.sort(rng.choice(2200, 500, replace=False)).astype(np.int64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_group_shares_anything(dtype):
    b = make([(0, [(1, 40), (7, 90)]), (0, [(3, 3)])], 8, 2, 128, 16, dtype, seed=10)
    assert b.max_prefix_len == 0
    check(b, run(b))
    b = make([(0, [(0, 17), (1, 1)])], 4, 4, 64, 16, dtype, seed=11)
    check(b, run(b, max_query_len=1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sinks(dtype):
    b = make(BATCHES["extend"](16), 8, 2, 128, 16, dtype, seed=3)
    sinks = np.linspace(-60, 60, 8).astype(np.float32)
    check(b, run(b, sinks=sinks), sinks=sinks)


@pytest.mark.parametrize("scale", [0.0, -0.09, 2.0])
def test_scales(scale):
    b = make(BATCHES["extend"](16), 8, 2, 128, 16, seed=6, scale=scale)
    check(b, run(b))


def test_agrees_with_pa_forward_on_the_full_table():
    b = make([(640, decodes(9, 1, 200, 1)), (48, [(20, 60), (1, 5)])], 16, 4, 128, 16, seed=9)
    got = run(b).float()
    d = pa.to_device(b)
    d.block_table = d.full_table
    want = pa.forward(d).float()
    # both within the stated distance of the exact rows, so within twice that of each other
    w, a = oracle(b), oracle(b, absolute=True)
    assert (np.abs((got - want).cpu().numpy()) <= 2 * tolerance(b, w, a)).all()


def test_largest_values_and_masked_garbage():
    """Scores spread over hundreds of units; NaN and infinities everywhere the
    call must not look."""
    b = make([(512, decodes(6, 1, 40, 2)), (16, [(30, 31)])], 8, 2, 128, 16, seed=12, scale=3.0)
    k = b.k_cache
    k[torch.isnan(k)] = float("inf")
    check(b, run(b))


def _scores(prefix, own, profile, D=128, G=4, dtype="bf16"):
    """A batch whose scores are `profile`(position) exactly, for every row: q is
    the first unit vector, keys carry the score in that column (profile values
    are whole numbers that bf16 holds), scale is 1."""
    b = make([(prefix, [(1, own), (1, own)])], G, 1, D, 16, dtype, seed=70, scale=1.0)
    b.q.zero_()
    b.q[..., 0] = 1.0
    n = prefix + own
    for s in range(2):
        for p in range(n):
            page, at = int(b.full_table[s, p // 16]), p % 16
            b.k_cache[page, at] = 0.0
            b.k_cache[page, at, 0, 0] = float(profile(p))
    return b


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", ["rising", "falling", "steps", "sawtooth"])
def test_scores_that_leave_the_reference_behind(shape, dtype):
    """The running reference has to follow scores that grow by hundreds within a
    tile of positions and from tile to tile, and to hold when they fall."""
    profile = {"rising": lambda p: p // 4, "falling": lambda p: 200 - p // 4,
               "steps": lambda p: 100 * (p // 96), "sawtooth": lambda p: 64 * ((p // 32) % 3)}[shape]
    b = _scores(640, 9, lambda p: min(max(profile(p), 0), 255), dtype=dtype)
    check(b, run(b), what=shape)


@pytest.mark.parametrize("at", [0, 1, 63, 64, 65, 127, 128, 191, 192, 255, 256, 383, 500, 639, 645])
def test_one_key_takes_the_weight(at):
    """One score 200 above the others, in either half of the first, a middle or
    the last tile, or behind the prefix: the row is that key's value."""
    b = _scores(640, 9, lambda p: 200 if p == at else 0)
    out = run(b).float().cpu()
    for s in range(2):
        want = b.v_cache[int(b.full_table[s, at // 16]), at % 16, 0].float()
        assert torch.equal(out[s], want.expand(4, -1))


# Scores of one query row by position, the first of them that holds; a score of None is -inf.
# A row's reference is its maximum over positions 0 .. 127, the first tile of its item.
PROFILES = [
    lambda p: 0,
    lambda p: 30 if p == 130 else 0,                        # grows in the first half of a tile
    lambda p: 200 if p == 200 else 0,                       # in the second half of the same tile
    lambda p: None if p < 128 else 90 if p == 200 else 0,   # nothing to see in the first tile
    lambda p: None if p < 192 else 0,
    lambda p: 100 if p == 140 else 250 if p == 220 else 0,  # in both halves
    lambda p: 250 if p == 140 else 100 if p == 220 else 0,
    lambda p: 255 - p // 4,
    lambda p: p // 4,
    lambda p: 150 if p == 330 else 0,                       # the next tile's second half
    lambda p: 40 if p == 260 else 0,                        # and its first
    lambda p: 13 if 192 <= p < 256 else 0,                  # just below what moves a reference,
    lambda p: 16 if 192 <= p < 256 else 0,                  # and just above
    lambda p: 64 * (p // 32 % 4),
    lambda p: 120 if p in (191, 447) else 255 if p == 639 else 0,
    lambda p: None if p < 640 else 0,
    lambda p: None,
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,layout", [(128, "nhd"), (64, "hnd")])
def test_rows_of_one_warp_with_other_scores_each(D, layout, dtype):
    """32 rows side by side (8 requests x 4 heads) whose scores leave their
    references behind at different places, if at all: what one row needs, the
    rows beside it neither get in its place nor miss.  Twenty groups of 8 KV
    heads on the same pages: more row blocks than SMs, so that no prefix is
    split and an item goes through all five tiles."""
    n, NG, Hk, own, none = len(PROFILES), 20, 8, 9, 32
    N = 640 + own
    b = make([(640, [(1, own)] * 8)] * NG, 4 * Hk, Hk, D, 16, dtype, seed=73, scale=1.0)
    for t in (b.block_table, b.full_table):
        for g in range(1, NG):
            t[8 * g:8 * g + 8] = t[:8]
    x = np.array([[-np.inf if f(p) is None else f(p) for p in range(N)] for f in PROFILES])
    keys = torch.zeros((N, D))
    keys[:, :n] = torch.from_numpy(np.where(np.isinf(x), 0.0, x)).T
    keys[:, none:none + n] = torch.from_numpy(np.where(np.isinf(x), -2e38, 0.0)).T
    pages = b.full_table[0, :40].long()
    b.k_cache[pages] = keys[:640].view(40, 16, 1, D).to(b.k_cache.dtype)
    tails = b.full_table[:8, 40].long()
    b.k_cache[tails, :own] = keys[640:].view(1, own, 1, D).to(b.k_cache.dtype)
    rng = np.random.default_rng(74)
    of = torch.from_numpy(rng.integers(0, n, (8 * NG, 4 * Hk)))
    of[:8, :4] = 1  # and warps whose rows have but two profiles
    of[3, 2] = 2
    of[8:16, 4:8] = 5
    of[9, 7] = 4
    b.q.zero_()
    b.q.scatter_(2, of[..., None], 1.0)
    b.q.scatter_(2, none + of[..., None], 2e38)  # times -2e38: an fp32 product of -inf
    top = x.max(axis=1, keepdims=True)
    w = np.where(np.isinf(x), 0.0, np.exp(x - np.where(np.isinf(top), 0.0, top)))
    w = torch.from_numpy(w / np.maximum(w.sum(axis=1, keepdims=True), 1.0))  # (all -inf: no weight)
    vp = b.v_cache[pages].double().reshape(640, Hk, D)
    vo = b.v_cache[tails, :own].double()  # [8, own, Hk, D]

    def rows(v_pre, v_own):
        all_ = (torch.einsum("fp,pkd->fkd", w[:, :640], v_pre)[:, None]
                + torch.einsum("fp,spkd->fskd", w[:, 640:], v_own))  # [profile, request, head, D]
        s = torch.arange(8 * NG)[:, None] % 8
        return all_[of, s, torch.arange(4 * Hk)[None, :] // 4]

    want, absolute = rows(vp, vo), rows(vp.abs(), vo.abs())
    # The scores are exact (one product of whole numbers).  A weight's exponent takes roundings
    # of log2 e, the product, the reference, its moves (two at most: a difference of near
    # references is exact, and what a far one leaves behind has no weight) and the log-sum-exp,
    # each of 2^-24 x 255 log2 e, and counts twice (weight and denominator); then as in
    # tolerance().
    tol = 2.0 ** -24 * (2 * 6 * 255 + 2 * N + 64) * absolute
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (absolute + want.abs())
    b = inputs.as_hnd(b) if layout == "hnd" else b
    got = run(b, max_query_len=1).double().cpu()
    bad = ~torch.isfinite(got).all(-1)
    assert not bad.any(), f"profiles of rows that are not finite: {sorted(set(of[bad].tolist()))}"
    over = ((got - want).abs() > tol).any(-1)
    assert not over.any(), f"profiles of rows that are off: {sorted(set(of[over].tolist()))}"


@pytest.mark.parametrize("hidden", [16, 64, 128, 129, 192, 300, 640])
def test_leading_scores_of_minus_infinity(hidden):
    """The first keys have a score of -inf (an overflowed product): no weight,
    and the reference is set by the first finite score."""
    b = _scores(640, 9, lambda p: 0)
    b.q[..., 1] = 2e38
    for s in range(2):
        for p in range(hidden):
            b.k_cache[int(b.full_table[s, p // 16]), p % 16, 0, 1] = -2e38
    out = run(b).float().cpu().double()
    for s in range(2):
        v = torch.stack([b.v_cache[int(b.full_table[s, p // 16]), p % 16, 0].double()
                         for p in range(hidden, 649)])
        # equal weights: their mean, one rounding of each weight and of the output
        tol = 2.0 ** -8 * (v.abs().mean(0) + v.mean(0).abs()) + 1e-6
        assert ((out[s] - v.mean(0)).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["q", "prefix_k", "prefix_v", "own_v"])
def test_nan_stays_visible(where, dtype):
    """A NaN in a visible input reaches the rows that see it, and no others."""
    b = make([(160, [(1, 9), (1, 20)]), (32, [(1, 5)])], 4, 2, 64, 16, dtype, seed=71)
    rows = [0, 1]
    if where == "q":
        b.q[1] = float("nan")
        rows = [1]
    elif where == "own_v":
        b.v_cache[int(b.full_table[1, 10]), 3] = float("nan")
        rows = [1]
    else:
        cache = b.k_cache if where == "prefix_k" else b.v_cache
        cache[int(b.full_table[0, 4]), 7] = float("nan")
    out = run(b).float().cpu()
    for t in range(3):
        assert torch.isnan(out[t]).all() if t in rows else torch.isfinite(out[t]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_and_a_bad_page_behind_the_first_tile_of_an_item(dtype):
    """More row blocks than SMs, so that an item goes through all five tiles of
    its prefix: what one group's later tiles hold reaches that group alone."""
    groups = [(640, [(1, 5 + s) for s in range(4)])] * 20
    b, good = (make(groups, 32, 8, 64, 16, dtype, seed=75) for _ in range(2))
    b.q[2, 7] = float("nan")
    b.k_cache[int(b.full_table[12, 17]), 3] = float("nan")  # group 3, position 275
    b.v_cache[int(b.full_table[20, 39]), 15] = float("nan")  # group 5, position 639
    b.block_table[28, 20] = b.num_blocks  # group 7, position 320
    out = run(b, status=pa.PA_DEV_BAD_BLOCK, max_query_len=1)
    nan, zero = torch.isnan(out.float()).all(-1).cpu(), (out == 0).all(-1).cpu()
    want = torch.zeros((80, 32), dtype=torch.bool)
    want[2, 7] = want[12:16] = want[20:24] = True
    assert torch.equal(nan, want)
    dead = torch.zeros((80, 32), dtype=torch.bool)
    dead[28:32] = True
    assert torch.equal(zero, dead)
    rows = (~(want | dead)).flatten().nonzero().flatten()[::7].numpy()
    check(good, out, rows=rows)


def test_cache_offsets_past_32_bits():
    """Pages beyond 2^32 bytes into the caches."""
    b = make([(1024, decodes(5, 1, 60, 1))], 8, 8, 128, 16, seed=72, poison=False)
    pages = (1 << 32) // (16 * 8 * 128 * 2) + b.num_blocks
    big = [torch.empty((pages, 16, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for dst, src in zip(big, (b.k_cache, b.v_cache)):
        dst[-b.num_blocks:] = src.cuda()
    d = pa.to_device(b)
    want = pa.forward_shared_prefix(d).clone()
    d.k_cache, d.v_cache = big
    d.block_table = torch.where(d.block_table >= 0, d.block_table + (pages - b.num_blocks), d.block_table)
    assert torch.equal(pa.forward_shared_prefix(d), want)
    check(b, want)
    assert pa.pa_get_device_status() == 0


def test_rows_with_no_finite_score_are_zero():
    """Every key -inf away from every query: no weight is left."""
    b = make([(64, [(1, 3), (4, 9)])], 4, 2, 64, 16, seed=13, poison=False)
    b.q[:], b.k_cache[:] = 0.0, 0.0
    b.q[..., 0], b.k_cache[..., 0] = 3e38, -3e38
    assert (run(b).float() == 0).all()


# ---------------------------------------------------------------------------
# bad metadata: a status bit, and zeros in the rows it concerns
# ---------------------------------------------------------------------------

def _zero_and_right(b, out, dead, what):
    """Rows of the requests in `dead` are zero, the others the oracle's."""
    H, qsl = b.num_heads, b.query_start_loc.tolist()
    zero = [t for s in dead for t in range(qsl[s], qsl[s + 1])]
    assert (out[zero].float() == 0).all(), what
    live = [t * H + h for s in range(b.num_seqs) if s not in dead
            for t in range(qsl[s], qsl[s + 1]) for h in range(H)]
    check(b, out, rows=np.asarray(live, np.int64), what=what)


def _bad(dtype):
    return make([(96, [(1, 5), (6, 20)]), (160, [(1, 40), (1, 1), (12, 12)]), (0, [(1, 9)])],
                8, 2, 64, 16, dtype, seed=21)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["prefix_page", "own_page", "not_whole_pages", "negative", "above_bound",
                                  "tokens_inside", "q_len", "q_bound", "length"])
def test_bad_group_or_request(what, dtype):
    b, kw, good = _bad(dtype), {}, _bad(dtype)
    if what == "prefix_page":
        b.block_table[2, 4] = b.num_blocks + 3
        dead, bit = [2, 3, 4], pa.PA_DEV_BAD_BLOCK
    elif what == "own_page":
        b.block_table[4, 10] = -1
        dead, bit = [4], pa.PA_DEV_BAD_BLOCK
    elif what in ("not_whole_pages", "negative", "above_bound"):
        b.prefix_lens[1] = {"not_whole_pages": 152, "negative": -16, "above_bound": 176}[what]
        dead, bit = [2, 3, 4], pa.PA_DEV_BAD_SEQLEN
    elif what == "tokens_inside":
        b.seq_lens[1] = 96 + 5  # six new tokens
        dead, bit = [1], pa.PA_DEV_BAD_SEQLEN
    elif what == "q_len":
        b.seq_lens[4] = 11
        dead, bit = [4], pa.PA_DEV_BAD_QLEN | pa.PA_DEV_BAD_SEQLEN
    elif what == "q_bound":
        kw, dead, bit = dict(max_query_len=6), [4], pa.PA_DEV_BAD_QLEN
    else:
        b.seq_lens[0] = b.max_seq_len + 1
        dead, bit = [0], pa.PA_DEV_BAD_SEQLEN
    _zero_and_right(good, run(b, status=bit, **kw), dead, what)


@pytest.mark.parametrize("field,at,value", [
    ("query_start_loc", 0, 1), ("query_start_loc", 6, 99), ("query_start_loc", 2, 30),
    ("group_start_loc", 0, 1), ("group_start_loc", 3, 5), ("group_start_loc", 1, 6),
])
def test_bad_starts_zero_every_row(field, at, value):
    b = _bad("bf16")
    getattr(b, field)[at] = value
    assert (run(b, status=pa.PA_DEV_BAD_QSL).float() == 0).all()


def test_lengths_beyond_the_bound_do_not_leave_the_workspace():
    """max_seq_len sizes the workspace; longer requests are refused one by one."""
    b = _bad("bf16")
    b.max_seq_len = 100  # the last request alone is shorter
    _zero_and_right(_bad("bf16"), run(b, status=pa.PA_DEV_BAD_SEQLEN), [0, 1, 2, 3, 4], "bound")


def test_a_prefix_beyond_the_bound_of_the_lengths():
    """max_prefix_len may be set above max_seq_len; no request can have such a prefix."""
    def batch():
        return make([(96, [(1, 5)]), (4096, [(1, 5), (9, 9)]), (48, [(3, 40)])], 8, 2, 64, 16, seed=22)
    b = batch()
    b.max_seq_len = 200
    assert b.max_prefix_len == 4096
    _zero_and_right(batch(), run(b, status=pa.PA_DEV_BAD_SEQLEN), [1, 2], "prefix")


# ---------------------------------------------------------------------------
# rows behind the last request: a batch padded to a captured size
# ---------------------------------------------------------------------------

def _padded(b, pad):
    """b with `pad` token rows behind its requests, holding NaN."""
    b.q = torch.cat([b.q, torch.full((pad, *b.q.shape[1:]), float("nan"), dtype=b.q.dtype)])
    return b


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,max_query_len,groups", [
    # few rows and many (another merge), decodes declared and not, more rows than real ones
    (3, 0, [(96, [(1, 5), (6, 20)]), (0, [(1, 9)])]),
    (1, 1, [(320, [(1, 5)] * 7), (64, [(1, 30)])]),
    (200, 1, [(320, [(1, 5), (1, 17)])]),
    (77, 0, [(640, [(1, 40)] * 500), (16, [(40, 77)])]),
    # as many tokens as requests, two of which have none; and no token at all
    (2, 1, [(160, [(1, 5), (0, 9), (1, 3), (0, 0)])]),
    (4, 0, [(160, [(0, 9), (0, 3)])]),
])
def test_rows_behind_the_last_request_are_left_as_they_were(pad, max_query_len, groups, dtype):
    H, D = 8, 64
    b = make(groups, H, 2, D, 16, dtype, seed=23)
    T = b.num_tokens
    d = pa.to_device(_padded(make(groups, H, 2, D, 16, dtype, seed=23), pad))
    out = torch.full_like(d.q, 7.0)
    pa.forward_shared_prefix(d, out=out, max_query_len=max_query_len)
    assert pa.pa_get_device_status() == 0
    assert (out[T:] == 7.0).all()
    if T:
        check(b, out[:T], rows=np.arange(0, T * H, max(1, T // 40)))


def test_starts_beyond_the_tokens_are_refused():
    b = make([(96, [(1, 5), (6, 20)]), (0, [(1, 9)])], 8, 2, 64, 16, seed=24)
    b.q = b.q[:-1].contiguous()
    assert (run(b, status=pa.PA_DEV_BAD_QSL).float() == 0).all()


@pytest.mark.parametrize("layout,block_size", [("nhd", 16), ("hnd", 64)])
def test_a_captured_step_of_changing_size(layout, block_size):
    """One graph of tables, cache write and attention for up to 24 tokens of up
    to 6 requests, replayed for steps of fewer: each against the oracle."""
    H, Hk, D, bs, S, T = 8, 2, 64, block_size, 6, 24
    prefix, nb, width = [4 * bs, 2 * bs], 64, 12
    g = torch.Generator().manual_seed(78)
    shape = (nb, bs, Hk, D) if layout == "nhd" else (nb, Hk, bs, D)
    kc, vc = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    free = torch.randperm(nb, generator=g).to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32)
    at = 0
    for s, p in ((0, prefix[0]), (3, prefix[1])):  # the shared pages, filled beforehand
        for j in range(p // bs):
            table[s, j] = free[at]
            at += 1
    pages = free[:at].long().cuda()
    for c in (kc, vc):
        c[pages] = torch.randn((at, *shape[1:]), generator=g).to(torch.bfloat16).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    seq, qsl, table, free = i32([0] * S), i32([0] * (S + 1)), table.cuda(), free.cuda()
    words = [i32([at]), i32([0])]
    rows = torch.zeros((T, H + 2 * Hk, D), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(T, dtype=torch.int64, device="cuda")
    out = torch.empty_like(q)
    starts, plens = i32([0, 3, S]), i32(prefix)

    def step():
        pa.pa_block_tables(seq, qsl, table, slots, bs, num_blocks=nb, free_pages=free,
                           free_start=words[0], free_end=words[1])
        pa.pa_cache_write_slots(rows[:, H:H + Hk], rows[:, H + Hk:], kc, vc, slots, bs, kv_layout=layout)
        pa.pa_forward_shared_prefix(q, kc, vc, table, seq, qsl, starts, plens, H, Hk, D, bs, 0.125,
                                    out, max_seq_len=width * bs, max_prefix_len=max(prefix),
                                    kv_layout=layout)
        words[0].copy_(words[1])
    step()  # (no tokens yet; the first call on a device cannot be captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens = [prefix[0]] * 3 + [prefix[1]] * 3
    for q_lens in ([9, 1, 0, 5, 7, 2], [1] * 6, [0, 3, 0, 0, 1, 0], [0] * 6, [1, 0, 20, 0, 0, 3]):
        n = sum(q_lens)
        lens = [a + b for a, b in zip(lens, q_lens)]
        seq.copy_(i32(lens))
        qsl.copy_(i32(np.cumsum([0] + q_lens).tolist()))
        rows.copy_(torch.randn((T, H + 2 * Hk, D), generator=g).to(torch.bfloat16))
        q.copy_(rows[:, :H])
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert pa.pa_get_device_status() == 0
        assert (slots[n:] == -1).all() and (slots[:n] >= 0).all() and (out[n:] == 7.0).all()
        if n == 0:
            continue
        full = table.cpu().clone()
        for s in range(S):
            p = prefix[s // 3] // bs
            full[s, :p] = full[s // 3 * 3, :p]
        b = inputs.SharedPrefixBatch(
            q=q[:n].cpu(), k_cache=kc.cpu(), v_cache=vc.cpu(), block_table=table.cpu(),
            seq_lens=seq.cpu(), query_start_loc=qsl.cpu(), num_heads=H, num_kv_heads=Hk, head_dim=D,
            block_size=bs, scale=0.125, dtype="bf16", max_seq_len=width * bs, full_table=full)
        b.kv_layout = layout
        check(b, out[:n], what=str(q_lens))


# ---------------------------------------------------------------------------
# streams, graphs, repeated calls
# ---------------------------------------------------------------------------

def test_two_calls_give_the_same_bits():
    b = make([(2048, decodes(40, 1, 500, 3)), (16, [(30, 80)])], 16, 4, 128, 16, seed=30)
    assert torch.equal(run(b).view(torch.int16), run(b).view(torch.int16))


@pytest.mark.parametrize("dtype,max_query_len", [("bf16", 0), ("bf16", 1), ("f32", 0)])
def test_a_run_of_calls_on_one_workspace_with_other_metadata_each(dtype, max_query_len):
    """Back to back calls whose metadata is written by the kernel before each of
    them: every kernel of a call goes by that call's plan, none by the last one's."""
    def batch(i):
        def reqs(n, lo, hi, j):
            one = decodes(n, lo, hi, 10 * i + j)
            return one if max_query_len == 1 else one[:-2] + [(9 + 3 * i, 40), (23 - 3 * i, 60 + i)]
        return make([(16 * (30 - 9 * i), reqs(9 + i, 1, 300, 1)), (16 * (5 + 20 * i), reqs(12 - i, 1, 200, 2))],
                    8, 2, 128, 16, dtype, seed=33)
    names = ("q", "block_table", "seq_lens", "query_start_loc", "group_start_loc", "prefix_lens")
    bs = [batch(i) for i in range(3)]
    T, NB, M = bs[0].num_tokens, max(b.num_blocks for b in bs), max(b.block_table.shape[1] for b in bs)
    for b in bs:
        assert b.num_tokens == T and b.num_seqs == bs[0].num_seqs
        b.block_table = torch.nn.functional.pad(b.block_table, (0, M - b.block_table.shape[1]), value=-1)
        b.max_seq_len = max(x.max_seq_len for x in bs)
        b.max_prefix_len = max(x.max_prefix_len for x in bs)
        for name in ("k_cache", "v_cache"):
            c = getattr(b, name)
            setattr(b, name, torch.cat([c, c.new_zeros((NB - c.shape[0], *c.shape[1:]))]))
    ds = [pa.to_device(b) for b in bs]
    want = [pa.forward_shared_prefix(d, max_query_len=max_query_len).clone() for d in ds]
    for b, w in zip(bs, want):
        check(b, w, rows=np.arange(0, T * 8, 7))
    live = [[getattr(d, n).clone() for n in names] for d in ds]
    kv = [torch.cat([getattr(d, n) for d in ds]) for n in ("k_cache", "v_cache")]
    for i, x in enumerate(live):  # one pool, the batches' pages one behind the other
        x[1] = torch.where(x[1] >= 0, x[1] + i * NB, x[1])
    d = pa.to_device(bs[0])
    d.k_cache, d.v_cache = kv
    outs = torch.full((60, *d.q.shape), 7.0, dtype=d.q.dtype, device="cuda")
    ws = torch.empty(pa.pa_forward_shared_prefix_workspace_bytes(
        pa.PA_BF16 if dtype == "bf16" else pa.PA_F32, d.num_seqs, 2, T, 8, 2, 128, d.max_seq_len),
        dtype=torch.uint8, device="cuda")

    def steps():
        for i in range(len(outs)):
            for name, x in zip(names, live[(i + i // 4) % 3]):
                getattr(d, name).copy_(x)
            pa.forward_shared_prefix(d, out=outs[i], max_query_len=max_query_len, workspace=ws)
    steps()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    eager = outs.clone()
    outs.fill_(7.0)
    with torch.cuda.graph(graph):
        steps()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for got in (eager, outs):
        for i in range(len(outs)):
            assert torch.equal(got[i], want[(i + i // 4) % 3]), i
    assert pa.pa_get_device_status() == 0


def test_calls_on_two_streams_at_once():
    made = [make([(4096, decodes(24, 1, 300, i))], 16, 4, 128, 16, seed=40 + i) for i in range(2)]
    d = [pa.to_device(b) for b in made]
    want = [pa.forward_shared_prefix(x).clone() for x in d]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in d]
    outs = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(pa.forward_shared_prefix(d[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])
    # an explicit stream that is not the current one
    out = torch.empty_like(d[0].q)
    streams[0].wait_stream(torch.cuda.current_stream())
    pa.forward_shared_prefix(d[0], out=out, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(out, want[0])
    assert pa.pa_get_device_status() == 0


def test_two_captured_graphs_replayed_at_once():
    made = [make([(4096, decodes(24, 1, 300, i))], 16, 4, 128, 16, seed=50 + i) for i in range(2)]
    d = [pa.to_device(b) for b in made]
    want = [pa.forward_shared_prefix(x).clone() for x in d]
    outs, graphs = [torch.empty_like(x.q) for x in d], []
    torch.cuda.synchronize()
    for x, o in zip(d, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.forward_shared_prefix(x, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in d]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    # the graph reads its metadata when it runs: shorter own parts
    b = made[0]
    b.seq_lens -= (b.seq_lens - b.max_prefix_len - 1) // 2
    d[0].seq_lens.copy_(b.seq_lens)
    graphs[0].replay()
    torch.cuda.synchronize()
    check(b, outs[0])
    assert pa.pa_get_device_status() == 0


def test_a_workspace_of_the_caller():
    b = make([(320, decodes(7, 1, 50, 5))], 8, 2, 128, 16, seed=60)
    need = pa.pa_forward_shared_prefix_workspace_bytes(pa.PA_BF16, b.num_seqs, 1, b.num_tokens, 8, 2,
                                                       128, b.max_seq_len)
    ws = torch.full((need + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    check(b, run(b, workspace=ws[:need]))
    assert (ws[need:] == 0xAB).all()
    with pytest.raises(pa.PaError, match="workspace"):
        run(b, workspace=ws[:need - 256])


# ---------------------------------------------------------------------------
# a serving loop: block tables, cache write and attention together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout,block_size,padded", [("nhd", 16, 0), ("hnd", 64, 3)])
def test_serving_steps_together(layout, block_size, padded):
    """Two prompts are written once (each by its group's first request), then
    every request of both groups extends and decodes a few steps: pages and
    slots from pa_block_tables, rows sliced from a fused projection and written
    by pa_cache_write_slots, attention by pa_forward_shared_prefix.  Every
    step's output is the oracle's on the whole history."""
    H, Hk, D, bs = 8, 2, 64, block_size
    sizes, prefix = [3, 4], [5 * bs, 2 * bs]
    S, nb = sum(sizes), 80
    g = torch.Generator().manual_seed(77)
    shape = (nb, bs, Hk, D) if layout == "nhd" else (nb, Hk, bs, D)
    kc = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    free = torch.randperm(nb, generator=g).to(torch.int32).cuda()
    counters = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
    table = torch.full((S, 12), -1, dtype=torch.int32, device="cuda")
    first = [0, sizes[0]]
    group_start = torch.tensor([0, sizes[0], S], dtype=torch.int32, device="cuda")
    prefix_lens = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    groups = [0] * sizes[0] + [1] * sizes[1]
    history = [[] for _ in range(S)]  # (k, v) rows of the request behind the prefix
    shared = [None, None]
    turn = 0

    def step(q_lens, lens, pad):
        nonlocal turn
        T = sum(q_lens) + pad
        qsl = torch.tensor(np.cumsum([0] + q_lens), dtype=torch.int32, device="cuda")
        seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
        slots = torch.empty(T, dtype=torch.int64, device="cuda")
        pa.pa_block_tables(seq, qsl, table, slots, bs, num_blocks=nb, free_pages=free,
                           free_start=counters[turn], free_end=counters[1 - turn])
        turn = 1 - turn
        rows = torch.randn((T, H + 2 * Hk, D), generator=g).to(torch.bfloat16).cuda()
        pa.pa_cache_write_slots(rows[:, H:H + Hk], rows[:, H + Hk:], kc, vc, slots, bs,
                                kv_layout=layout)
        return rows, qsl, seq

    # the prompts, by the groups' first requests
    q_lens = [prefix[groups[s]] if s in first else 0 for s in range(S)]
    rows, qsl, _ = step(q_lens, q_lens, 0)
    at = 0
    for gi in range(2):
        n = prefix[gi]
        shared[gi] = rows[at:at + n].float().cpu().numpy().astype(np.float64)
        at += n
    lens = [prefix[groups[s]] for s in range(S)]
    for q_lens in ([5, 1, 40, 2, 1, 17, 3], [1] * S, [1, 1, 0, 1, 1, 1, 1], [1] * S):
        lens = [a + b for a, b in zip(lens, q_lens)]
        rows, qsl, seq = step(q_lens, lens, padded)
        T = sum(q_lens)
        q = rows[:T, :H].contiguous()
        out = torch.empty_like(q)
        pa.pa_forward_shared_prefix(q, kc, vc, table, seq, qsl, group_start, prefix_lens, H, Hk, D,
                                    bs, 0.125, out, max_seq_len=max(lens),
                                    max_prefix_len=max(prefix), kv_layout=layout)
        r = rows.float().cpu().numpy().astype(np.float64)
        got = out.float().cpu().numpy().astype(np.float64)
        at = 0
        for s in range(S):
            history[s].append(r[at:at + q_lens[s], H:])
            ctx = np.concatenate([shared[groups[s]][:, H:]] + history[s])
            assert len(ctx) == lens[s]
            k, v = ctx[:, :Hk], ctx[:, Hk:]
            for i in range(q_lens[s]):
                seen = lens[s] - q_lens[s] + i + 1
                for h in range(H):
                    x = k[:seen, h // 4] @ r[at + i, h] * 0.125
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    want = w @ v[:seen, h // 4]
                    tol = 2.0 ** -8 * (w @ np.abs(v[:seen, h // 4]) + np.abs(want)) + 1e-4
                    assert (np.abs(got[at + i, h] - want) <= tol).all()
            at += q_lens[s]
    assert pa.pa_get_device_status() == 0

"""Values that are not finite in some of their columns: where a row sees such a token the
other columns are as exact as anywhere, rounded once."""
import numpy as np
import pytest
import torch

from paged_kv_attention_16_gb300 import pa
from tests import spans

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_attention_16_gb300 import build
    build.build()
    pa.lib()
    pa.pa_get_device_status()  # clear


@pytest.mark.parametrize("mode", ["tree", "weights"])
@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("at", [0, 1])  # the new token that holds the infinity
# units that a block finishes in one row tile, in two, and ones joined by the merge
@pytest.mark.parametrize("S,n,Hk", [(30, 5, 8), (4, 60, 2), (3, 5, 2)])
def test_other_columns_are_rounded_once(S, n, Hk, at, D, sink, mode):
    """Every row sees one cached position, of the larger score (its weight in the product
    is 1, which rounds to itself), and a new token, which holds an infinity in column 3
    and elsewhere values that cancel the cached one's: the sum is small beside them, so
    its own rounding alone is allowed, and fp32's of the parts.  (All rows of a causal
    call see the first new token: it stays in the product, where its weight w is rounded
    to bf16 like any other, by 2^-8 w |v| at most.)"""
    H = 4 * Hk
    b = spans.batch([n] * S, [n + 1] * S, H, Hk, D, 16, seed=n + D)
    gen = torch.Generator().manual_seed(n)
    b.q = (0.2 + torch.rand(b.q.shape, generator=gen)).bfloat16()
    for s in range(S):
        page, slot = spans.slots_of(b, s)
        b.k_cache[page[0], slot[0]] = 0.5
        b.k_cache[page[1:], slot[1:]] = 0.0
        b.k_cache[page[1 + at], slot[1 + at]] = 0.25
        v = 1.0 + torch.rand((Hk, D), generator=gen)
        b.v_cache[page[0], slot[0]] = v.bfloat16()
        b.v_cache[page[1:], slot[1:]] = 0.0
        b.v_cache[page[1 + at], slot[1 + at]] = (-v * (1.5 + torch.rand((Hk, D), generator=gen))).bfloat16()
        b.v_cache[page[1 + at], slot[1 + at], :, 3] = float("inf")
    sinks = np.linspace(-3.0, 3.0, H) if sink else None
    if mode == "tree":
        mask = np.full((b.num_tokens, 1), 1 << at, np.uint64)
        out = spans.run_tree(b, mask, sinks=sinks)
    else:  # causal: the rows from this token on see the two, and zeros
        mask = None
        out, _ = spans.run_weights(b, np.zeros((b.num_blocks, Hk, 16), np.float32), True, sinks=sinks)
    for s in range(S):
        page, slot = spans.slots_of(b, s)
        b.v_cache[page[1 + at], slot[1 + at], :, 3] = 0.0
    want = spans.oracle(b, mask, sinks)
    rows = range(n) if mode == "tree" else [0] if at == 0 else range(1, n)
    cols = [c for c in range(D) if c != 3]
    for s, r in enumerate(want):
        e = spans.weight_error(b, r, n + 1)
        page, slot = spans.slots_of(b, s)
        v = np.abs(b.v_cache[page[1 + at], slot[1 + at]].double().numpy()).repeat(4, 0)
        cached = np.abs(b.v_cache[page[0], slot[0]].double().numpy()).repeat(4, 0)
        for i in rows:
            got, ref, mass = out[s * n + i], r["out"][i], r["mass"][i]
            assert (got[:, 3] == np.inf).all()
            tol = 1.01 * e * mass + 2.0 ** -8 * 1.01 * (np.abs(ref) + e * mass) + 1e-30
            if mode == "weights" and at == 0:
                w = (ref + mass)[:, 0] / 2 / cached[:, 0]  # of the cached one, whose values are positive
                w = ((mass[:, 0] - w * cached[:, 0]) / v[:, 0])[:, None]
                tol += 1.01 ** 2 * 2.0 ** -8 * w * v
            bad = np.abs(got - ref)[:, cols] > tol[:, cols]
            assert not bad.any(), (s, i, bad.sum(), (np.abs(got - ref) / tol)[:, cols].max())

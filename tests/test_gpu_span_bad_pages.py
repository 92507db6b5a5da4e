"""A bad page and scores that are not numbers in one request: its rows are zero, its
weights are left as they were, whichever piece of the context holds which, and the
others are as they are without it."""
import numpy as np
import pytest
import torch

from paged_kv_attention_16_gb300 import pa
from tests import spans

pytestmark = pytest.mark.gpu

NAN = float("nan")
BAD = 1  # the request


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_attention_16_gb300 import build
    build.build()
    pa.lib()
    pa.pa_get_device_status()  # clear


def spoiled(n, dtype, where, page_at, S, D):
    """A batch whose request BAD has a bad page at page_at of its cached part, and NaN in
    its last query or in one cached key."""
    rng = np.random.default_rng(n + S)
    q_lens = [3, n, 9] + rng.integers(1, 6, S - 3).tolist()
    cached = [200, 2500, 400] + rng.integers(20, 900, S - 3).tolist()
    b = spans.batch(q_lens, [q + c for q, c in zip(q_lens, cached)], 8, 2, D, 16, dtype, seed=n)
    page, slot = spans.slots_of(b, BAD)
    if where == "last query":
        b.q[b.query_start_loc[BAD + 1] - 1] = NAN
    else:
        at = 40 if where == "key early" else 2400
        b.k_cache[page[at], slot[at], :, 5] = NAN
    b.block_table[BAD, page_at] = b.num_blocks if n % 2 else -1
    return b, page[page_at]


def clean(b):
    """The same batch with the request's own faults mended, for the oracle."""
    b.q[torch.isnan(b.q)] = 0.0
    b.k_cache[torch.isnan(b.k_cache)] = 0.0


@pytest.mark.parametrize("where", ["last query", "key early", "key late"])
@pytest.mark.parametrize("page_at", [0, 155])
@pytest.mark.parametrize("output", [True, False])
@pytest.mark.parametrize("n,S", [(1, 3), (8, 40), (9, 3), (70, 60)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights(dtype, n, S, output, page_at, where):
    b, real = spoiled(n, dtype, where, page_at, S, 64)
    before = np.random.default_rng(n).random((b.num_blocks, 2, 16)).astype(np.float32)
    out, got = spans.run_weights(b, before, True, output, expect=pa.PA_DEV_BAD_BLOCK)
    clean(b)
    b.block_table[BAD, page_at] = int(real)
    want = spans.oracle(b, values=output)
    qsl = b.query_start_loc.numpy()
    if output:
        assert not out[qsl[BAD]:qsl[BAD + 1]].any()
        want[BAD]["out"][:] = 0.0
        spans.check_out(b, out, want, dtype)
    want[BAD] = dict(want[BAD], out=want[BAD]["out"][:0])  # (its slots as they were)
    spans.check_weights(b, got, before, want, True)


@pytest.mark.parametrize("where", ["last query", "key early", "key late"])
@pytest.mark.parametrize("page_at", [0, 155])
@pytest.mark.parametrize("n,S,D", [(9, 3, 128), (9, 60, 128), (63, 40, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_trees(dtype, n, S, D, page_at, where):
    b, real = spoiled(n, dtype, where, page_at, S, D)
    mask = np.full((b.num_tokens, 1), ~np.uint64(0))
    out = spans.run_tree(b, mask, expect=pa.PA_DEV_BAD_BLOCK)
    clean(b)
    b.block_table[BAD, page_at] = int(real)
    want = spans.oracle(b, mask)
    qsl = b.query_start_loc.numpy()
    assert not out[qsl[BAD]:qsl[BAD + 1]].any()
    want[BAD]["out"][:] = 0.0
    spans.check_out(b, out, want, dtype)

"""pa_forward_weights with a query that is not a number: NaN at the positions that its
token sees, at the others, the later tokens' among them, what the other rows give; the same
whether a request's scores are kept or multiplied out again."""
import numpy as np
import pytest

from paged_kv_attention_16_gb300 import pa
from tests import spans

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_attention_16_gb300 import build
    build.build()
    pa.lib()
    pa.pa_get_device_status()  # clear


@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("at", [0, 0.5])
@pytest.mark.parametrize("n", [2, 5, 8, 9, 70, 150])  # (32 rows of a KV head are kept)
@pytest.mark.parametrize("S,output", [(2, True), (2, False), (40, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_are_not_numbers(dtype, S, output, n, at, accumulate):
    rng = np.random.default_rng(n + S)
    q_lens = [n, 3] + rng.integers(1, 6, S - 2).tolist()
    cached = [300, 40] + rng.integers(0, 900, S - 2).tolist()
    b = spans.batch(q_lens, [q + c for q, c in zip(q_lens, cached)], 8, 2, 64, 16, dtype, seed=n)
    row = int(at * n)
    b.q[row, 5] = float("nan")  # one head, of the second KV head
    before = rng.random((b.num_blocks, 2, 16)).astype(np.float32)
    want = spans.oracle(b, values=output)
    page, slot = spans.slots_of(b, 0)
    assert np.isnan(want[0]["weights"][1, :300 + row + 1]).all()
    assert np.isfinite(want[0]["weights"][1, 300 + row + 1:]).all() and np.isfinite(want[0]["weights"][0]).all()
    out, got = spans.run_weights(b, before, accumulate, output)
    spans.check_weights(b, got, before, want, accumulate)
    if output:
        assert np.isnan(out[row, 5]).all()
        out[row, 5] = want[0]["out"][row, 5] = want[0]["mass"][row, 5] = 0.0
        spans.check_out(b, out, want, dtype)

"""Calls of pa_forward_tree and pa_forward_weights that follow one another on one
workspace, each with a plan of its own: every call works from its own plan."""
import numpy as np
import pytest
import torch

from paged_kv_attention_16_gb300 import inputs, pa
from tests import spans

pytestmark = pytest.mark.gpu

H, HK, D, BS = 8, 2, 64, 16
MAX_LEN = 3000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_attention_16_gb300 import build
    build.build()
    pa.lib()
    pa.pa_get_device_status()  # clear


def batches(S, dtype):
    """Three batches of S requests whose units, tiles and pieces differ."""
    rng = np.random.default_rng(S)
    out = []
    for seed, q_most, c_most in ((1, 3, 40), (2, 12, MAX_LEN - 12), (3, 40 if S < 10 else 8, 700)):
        q = rng.integers(1, q_most + 1, S)
        ctx = q + rng.integers(0, c_most, S)
        out.append(spans.batch(q.tolist(), ctx.tolist(), H, HK, D, BS, dtype, seed=seed))
    return out


@pytest.mark.parametrize("mode", ["tree", "weights", "weights alone"])
@pytest.mark.parametrize("S", [1, 4, 30, 120])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_that_share_a_workspace(dtype, S, mode):
    cases, need = [], 0
    for b in batches(S, dtype):
        d = pa.to_device(b)
        T = b.num_tokens
        mask = spans.to_words(np.full((T, 1), (1 << 40) - 1, np.uint64))
        start = torch.rand((b.num_blocks, HK, BS), device="cuda")
        code = pa.PA_BF16 if dtype == "bf16" else pa.PA_F32
        size = (pa.pa_forward_tree_workspace_bytes if mode == "tree"
                else pa.pa_forward_weights_workspace_bytes)
        need = max(need, size(code, S, T, H, HK, D, MAX_LEN))
        cases.append((d, mask, start))

    def call(case, out, w, workspace):
        d, mask, _ = case
        if mode == "tree":
            pa.pa_forward_tree(d.q, d.k_cache, d.v_cache, d.block_table, d.seq_lens, d.query_start_loc,
                               mask, H, HK, D, BS, d.scale, out, max_seq_len=MAX_LEN, workspace=workspace)
        else:
            pa.pa_forward_weights(d.q, d.k_cache, d.v_cache, d.block_table, d.seq_lens, d.query_start_loc,
                                  H, HK, D, BS, d.scale, out if mode == "weights" else None, w,
                                  accumulate=True, max_seq_len=MAX_LEN, workspace=workspace)

    def results():
        return [(torch.zeros_like(c[0].q), c[2].clone()) for c in cases]

    want = results()
    for c, (out, w) in zip(cases, want):  # each on memory of its own, alone
        call(c, out, w, torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    got = [results() for _ in range(6)]
    for turn in got[:3]:  # called one by one
        for c, (out, w) in zip(cases, turn):
            call(c, out, w, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for turn in got[3:]:
            for c, (out, w) in zip(cases, turn):
                call(c, out, w, ws)
    for _ in range(3):
        for turn in got[3:]:
            for c, (out, w) in zip(cases, turn):
                out.zero_()
                w.copy_(c[2])
        graph.replay()
    torch.cuda.synchronize()
    assert pa.pa_get_device_status() == 0
    for turn in got:
        for (out, w), (ref_out, ref_w) in zip(turn, want):
            assert np.array_equal(inputs.storage_array(out.cpu()), inputs.storage_array(ref_out.cpu()))
            assert torch.equal(w, ref_w)

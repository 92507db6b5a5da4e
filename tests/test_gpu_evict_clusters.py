"""pa_cache_evict where a request's positions are shared out over a cluster of blocks:
every size of it, budgets that leave nothing to count (the first and the recent positions
fill them) and ones that do, launch after launch."""
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


# (clusters of 2, 4, 8 and 16 blocks on 152 SMs)
@pytest.mark.parametrize("longest", [2100, 5000, 9000, 17000])
@pytest.mark.parametrize("keep,first,recent", [
    (300, 4, 296),       # nothing to count: a window behind some first positions
    (300, 5000, 5000),   # more than fill it
    (0, 4, 64),          # nothing kept
    (301, 4, 296),       # one to find
    (700, 0, 0),
])
def test_clusters(longest, keep, first, recent):
    Hk, D, bs = 2, 8, 16
    rng = np.random.default_rng(longest + keep)
    lens = [longest, 40, longest - 900]
    b = spans.batch([0] * 3, lens, Hk, Hk, D, bs, seed=longest)
    w = np.exp(1.5 * rng.standard_normal((b.num_blocks, Hk, bs))).astype(np.float32)
    want = orc.cache_evict(inputs.storage_array(b.k_cache), inputs.storage_array(b.v_cache), w, w,
                           b.block_table.numpy(), b.seq_lens.numpy(), [keep] * 3, bs, b.num_blocks, 4000,
                           longest, first, recent)
    d, keeps = pa.to_device(b), i32([keep] * 3)
    need = pa.pa_cache_evict_workspace_bytes(pa.PA_BF16, 3, Hk, D, longest)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    turns = []
    for _ in range(20):
        turns.append((d.k_cache.clone(), d.v_cache.clone(), torch.from_numpy(w).cuda(), i32([-5] * 3),
                      i32([-9] * 4000), i32([-9])))
    for k, v, d_w, after, freed, count in turns:
        pa.pa_cache_evict(k, v, d_w, d.block_table, d.seq_lens, keeps, after, bs, max_seq_len=longest,
                          num_first=first, num_recent=recent, freed_pages=freed, num_freed=count,
                          workspace=ws)
    assert pa.pa_get_device_status() == want[5] == 0
    for k, v, d_w, after, freed, count in turns:
        assert np.array_equal(inputs.storage_array(k.cpu()), want[0])
        assert np.array_equal(inputs.storage_array(v.cpu()), want[1])
        assert np.array_equal(d_w.cpu().numpy(), want[2])
        assert after.tolist() == want[3] and int(count) == len(want[4])
        assert freed.tolist()[:len(want[4])] == want[4]

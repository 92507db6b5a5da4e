"""Arrays that a call writes and that overlap others of the same call are refused on the
host: blocks and launches of one call read what others of it write.  Counts that would
pass the kernels' 32-bit counters are refused too.  Nothing is launched, no GPU needed."""
import ctypes

import pytest

from paged_kv_attention_16_gb300 import build as pbuild
from paged_kv_attention_16_gb300 import pa
from tests.test_span_abi_cpu import ACCEPT, EVICT, MASKS, TREE, WEIGHTS, call

M = 1 << 24  # apart by more than any array of these calls


def at(i, offset=0):
    """Stands for a device address that is never followed."""
    return (i + 1) * M + offset


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.lib()


def apart(spec, pointers):
    order, defaults = spec
    a = dict(defaults)
    a.update({name: at(i) for i, name in enumerate(pointers.split())})
    return order, a


MASK_ARGS = apart(MASKS, "par qsl sl mask pos")       # 2 requests, 3 tokens, 1 word
ACCEPT_ARGS = apart(ACCEPT, "k v bt sl qsl path pl out freed count")  # 2 requests, 4 wide, list of 8
EVICT_ARGS = apart(EVICT, "k v w wo bt sl keep out freed count ws")
TREE_ARGS = apart(TREE, "q k v bt sl qsl mask out ws")   # 3 tokens of 8 heads of 128, bf16
WEIGHT_ARGS = apart(WEIGHTS, "q k v bt sl qsl out w ws")


@pytest.mark.parametrize("kw,want", [
    (dict(pos=at(0)), 1), (dict(pos=at(0, 8)), 1), (dict(pos=at(0, -8)), 1),  # over parents
    (dict(pos=at(1, 8)), 1), (dict(pos=at(2, 4)), 1), (dict(pos=at(3, 20)), 1),
    (dict(mask=at(0)), 1), (dict(mask=at(1, -16)), 1), (dict(mask=at(2)), 1),
    (dict(S=(1 << 30) + 1), 2),
])
def test_masks(lib, kw, want):
    assert call(lib.pa_tree_masks, *MASK_ARGS, kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(out=at(3)), 1), (dict(out=at(3, 4)), 1), (dict(out=at(3, -4)), 1),   # seq_lens
    (dict(out=at(4, 8)), 1), (dict(out=at(5, 28)), 1), (dict(out=at(6)), 1), (dict(out=at(2, 28)), 1),
    (dict(freed=at(2)), 1), (dict(freed=at(3, -28)), 1), (dict(freed=at(6)), 1),
    (dict(count=at(6, 4)), 1), (dict(count=at(7)), 1), (dict(count=at(8, 28)), 1), (dict(freed=at(7, -4)), 1),
    (dict(S=(1 << 30) + 1), 2),
])
def test_accept(lib, kw, want):
    assert call(lib.pa_cache_accept, *ACCEPT_ARGS, kw) == want


@pytest.mark.parametrize("kw", [
    dict(out=at(5)), dict(out=at(5, 4)), dict(out=at(6, -4)), dict(out=at(4, 28)), dict(freed=at(6)),
    dict(freed=at(4)), dict(count=at(5)), dict(count=at(7, 4)), dict(count=at(8)), dict(freed=at(7, -4)),
    dict(wo=at(2, 4)), dict(wo=at(2, -4)), dict(wo=at(2, 4 * 4 * 2 * 16 - 4)),
])
def test_evict(lib, kw):
    assert call(lib.pa_cache_evict, *EVICT_ARGS, kw) == 1


@pytest.mark.parametrize("kw", [dict(out=at(0)), dict(out=at(0, 16)), dict(out=at(0, 3 * 8 * 128 * 2 - 16)),
                                dict(out=at(0, 16 - 3 * 8 * 128 * 2))])
def test_outputs_over_queries(lib, kw):
    assert call(lib.pa_forward_tree, *TREE_ARGS, kw) == 1
    assert call(lib.pa_forward_weights, *WEIGHT_ARGS, kw) == 1


def test_options_change_nothing(lib):
    o = ctypes.byref(pa.ForwardOptions(None, 1, 0, None, 0, 1))
    assert call(lib.pa_forward_tree, *TREE_ARGS, dict(o=o, out=at(0))) == 1

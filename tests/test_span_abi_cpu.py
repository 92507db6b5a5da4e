"""Host-side argument checks of pa_tree_masks, pa_forward_tree, pa_cache_accept,
pa_forward_weights and pa_cache_evict, through the C ABI and through the binding:
refused calls launch nothing and need no GPU."""
import ctypes

import pytest
import torch

from paged_kv_attention_16_gb300 import build as pbuild
from paged_kv_attention_16_gb300 import pa

P = 1 << 20  # stands for an aligned device address that is never followed


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.lib()


def call(f, order, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return f(*[a[x] for x in order.split()])


MASKS = ("par qsl sl mask pos st S T W", dict(par=P, qsl=P, sl=P, mask=P, pos=P, st=None, S=2, T=3, W=1))


@pytest.mark.parametrize("kw,want", [
    (dict(W=0), 1), (dict(W=-1), 1), (dict(S=-1), 1), (dict(T=-1), 1), (dict(par=None), 1),
    (dict(mask=None), 1), (dict(qsl=None), 1), (dict(sl=None), 1), (dict(mask=P + 4), 1),
    (dict(par=P + 2), 1), (dict(qsl=P + 1), 1), (dict(sl=P + 2), 1), (dict(pos=P + 2), 1),
    (dict(T=0), 0), (dict(T=0, mask=None, par=None), 0), (dict(T=(1 << 30) + 1), 2),
])
def test_masks_argument_checks(lib, kw, want):
    assert call(lib.pa_tree_masks, *MASKS, kw) == want


TREE = ("q k v bt sl qsl mask H Hk D bs scale out st dt S T W mbps nb msl o ws wsb",
        dict(q=P, k=P, v=P, bt=P, sl=P, qsl=P, mask=P, H=8, Hk=2, D=128, bs=16, scale=0.1, out=P, st=None,
             dt=1, S=2, T=3, W=1, mbps=4, nb=4, msl=64, o=None, ws=P, wsb=1 << 40))
WEIGHTS = ("q k v bt sl qsl H Hk D bs scale out w acc st dt S T mbps nb msl o ws wsb",
           dict(q=P, k=P, v=P, bt=P, sl=P, qsl=P, H=8, Hk=2, D=128, bs=16, scale=0.1, out=P, w=P, acc=1,
                st=None, dt=1, S=2, T=3, mbps=4, nb=4, msl=64, o=None, ws=P, wsb=1 << 40))

BOTH = [
    (dict(H=0), 1), (dict(Hk=3), 1), (dict(S=-1), 1), (dict(T=-1), 1), (dict(dt=7), 1), (dict(D=96), 2),
    (dict(bs=8), 2), (dict(bs=512), 2), (dict(H=96, Hk=3), 2), (dict(T=0), 0), (dict(T=0, ws=None), 0),
    (dict(S=0), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(bt=None), 1),
    (dict(sl=None), 1), (dict(qsl=None), 1), (dict(nb=0), 1), (dict(mbps=0), 1), (dict(q=P + 8), 1),
    (dict(k=P + 8), 1), (dict(v=P + 8), 1), (dict(out=P + 8), 1), (dict(ws=None), 3), (dict(wsb=100), 3),
    (dict(ws=P + 128), 1), (dict(bt=P + 1), 1), (dict(sl=P + 2), 1), (dict(qsl=P + 3), 1),
    (dict(S=1 << 20, T=1 << 20, msl=1 << 30), 2), (dict(msl=-1), 1),
    (dict(S=1, T=1, H=1, Hk=1, msl=(1 << 30) + 1), 2), (dict(S=1, T=1, H=1, Hk=1, msl=1 << 30, ws=None), 3),
]


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(W=0), 1), (dict(W=-1), 1), (dict(mask=None), 1), (dict(mask=P + 4), 1), (dict(out=None), 1),
])
def test_tree_argument_checks(lib, kw, want):
    assert call(lib.pa_forward_tree, *TREE, kw) == want


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(w=None), 1), (dict(w=P + 8), 1), (dict(acc=2), 1), (dict(acc=-1), 1),
    (dict(out=None, v=None, ws=None), 3), (dict(out=None, v=P + 1, ws=None), 3),
])
def test_weights_argument_checks(lib, kw, want):
    assert call(lib.pa_forward_weights, *WEIGHTS, kw) == want


@pytest.mark.parametrize("f,spec", [("pa_forward_tree", TREE), ("pa_forward_weights", WEIGHTS)])
@pytest.mark.parametrize("opts,want", [
    ((None, 0, 0, None, 0, 0), 0), ((None, 1, 0, None, 0, 1), 0), ((P + 2, 0, 0, None, 0, 0), 1),
    ((None, 2, 0, None, 0, 0), 1), ((None, 0, -1, None, 0, 0), 1), ((None, 0, 16, None, 0, 0), 2),
    ((None, 0, 0, P, 0, 0), 2), ((None, 0, 0, None, 2, 0), 1), ((None, 0, 0, None, 0, -1), 1),
])
def test_option_checks(lib, f, spec, opts, want):
    o = ctypes.byref(pa.ForwardOptions(*opts))
    assert call(getattr(lib, f), *spec, dict(o=o, T=0)) == want


ACCEPT = ("k v bt sl qsl path pl out freed count Hk D bs st dt S mp mbps nb cap layout",
          dict(k=P, v=P, bt=P, sl=P, qsl=P, path=P, pl=P, out=P + 64, freed=P, count=P, Hk=2, D=128, bs=16,
               st=None, dt=1, S=2, mp=4, mbps=4, nb=4, cap=8, layout=0))


@pytest.mark.parametrize("kw,want", [
    (dict(S=-1), 1), (dict(mp=-1), 1), (dict(Hk=0), 1), (dict(D=0), 1), (dict(bs=0), 1), (dict(mbps=-1), 1),
    (dict(nb=-1), 1), (dict(cap=-1), 1), (dict(dt=3), 1), (dict(layout=2), 1), (dict(D=4), 2),
    (dict(D=16384), 2), (dict(count=None), 1), (dict(freed=None), 1), (dict(freed=None, count=None), 1),
    (dict(k=None), 1), (dict(v=None), 1), (dict(bt=None), 1), (dict(sl=None), 1), (dict(qsl=None), 1),
    (dict(path=None), 1), (dict(pl=None), 1), (dict(out=None), 1), (dict(mbps=0), 1), (dict(nb=0), 1),
    (dict(k=P + 8), 1), (dict(v=P + 8), 1), (dict(bt=P + 2), 1), (dict(out=P), 1), (dict(out=P + 2), 1),
    (dict(freed=P + 1), 1), (dict(count=P + 2), 1), (dict(path=P + 2), 1),
    (dict(S=0, freed=None, count=None, cap=0), 0), (dict(mp=1 << 27), 2),
])
def test_accept_argument_checks(lib, kw, want):
    assert call(lib.pa_cache_accept, *ACCEPT, kw) == want


EVICT = ("k v w wo bt sl keep out freed count first recent Hk D bs st dt S mbps nb cap msl layout ws wsb",
         dict(k=P, v=P, w=P, wo=P, bt=P, sl=P, keep=P + 32, out=P + 64, freed=P, count=P, first=4, recent=8,
              Hk=2, D=128, bs=16, st=None, dt=1, S=2, mbps=4, nb=4, cap=8, msl=64, layout=0, ws=P,
              wsb=1 << 40))


@pytest.mark.parametrize("kw,want", [
    (dict(S=-1), 1), (dict(first=-1), 1), (dict(recent=-1), 1), (dict(Hk=0), 1), (dict(D=0), 1),
    (dict(bs=0), 1), (dict(mbps=-1), 1), (dict(nb=-1), 1), (dict(cap=-1), 1), (dict(msl=-1), 1),
    (dict(dt=3), 1), (dict(layout=2), 1), (dict(D=4), 2), (dict(D=16384), 2), (dict(count=None), 1),
    (dict(freed=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(w=None), 1), (dict(wo=None), 1),
    (dict(bt=None), 1), (dict(sl=None), 1), (dict(keep=None), 1), (dict(out=None), 1), (dict(mbps=0), 1),
    (dict(nb=0), 1), (dict(k=P + 8), 1), (dict(w=P + 2), 1), (dict(wo=P + 1), 1), (dict(out=P), 1),
    (dict(out=P + 32), 1), (dict(keep=P + 2), 1), (dict(ws=None), 3), (dict(wsb=100), 3),
    (dict(ws=P + 16), 1), (dict(S=1 << 20, Hk=1 << 10, msl=1 << 20), 2),
    (dict(S=1, Hk=1, D=8, msl=(1 << 30) + 1), 2), (dict(S=1, Hk=1, D=8, msl=1 << 30, ws=None), 3),
    (dict(S=0, freed=None, count=None, cap=0), 0),
])
def test_evict_argument_checks(lib, kw, want):
    assert call(lib.pa_cache_evict, *EVICT, kw) == want


def test_workspace_bytes(lib):
    tree, votes = pa.pa_forward_tree_workspace_bytes, pa.pa_forward_weights_workspace_bytes
    base = tree(pa.PA_BF16, 64, 1024, 32, 8, 128, 8192, 16)
    # two partials (128 values and a log-sum-exp) of 64 rows for each KV head of a request
    assert 64 * 8 * 2 * 64 * 129 * 4 <= base < tree(pa.PA_BF16, 64, 1024, 32, 8, 128, 8192)
    assert tree(pa.PA_BF16, 64, 2048, 32, 8, 128, 8192, 32) > base
    # a decode step keeps its rows' scores: 4 of a KV head, each on 8192 positions
    assert votes(pa.PA_BF16, 64, 64, 32, 8, 128, 8192, 1) >= 64 * 8 * 4 * 8192 * 4
    # scores of at most 32 rows of a KV head are kept
    assert votes(pa.PA_BF16, 4, 4096, 32, 8, 128, 8192) < 4 * 8 * 32 * 8192 * 4 + (1 << 28)
    evict = pa.pa_cache_evict_workspace_bytes
    assert evict(pa.PA_BF16, 4, 8, 128, 8192) >= 4 * 8 * 8192 * 8
    top = 2 ** 31 - 1
    assert tree(pa.PA_BF16, top, top, top, top, 128, top) == 0
    assert votes(pa.PA_BF16, top, top, 32, 8, 128, top) == 0
    assert evict(pa.PA_BF16, top, top, 128, top) == 0 and evict(pa.PA_BF16, 1, 1, 16384, 64) == 0
    assert tree(pa.PA_BF16, -1, 1, 32, 8, 128, 64) == 0 and tree(1, 1, 1, 32, 5, 128, 64) == 0
    assert tree(1, 1, 1, 32, 8, 128, 64, -1) == 0 and evict(1, 1, 0, 128, 64) == 0


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


CACHES, Q, MASK = torch.zeros(4, 16, 2, 64), torch.zeros(3, 4, 64), torch.zeros(3, 1, dtype=torch.int64)
W = torch.zeros(4, 2, 16)


def test_binding_refuses_tensors_off_the_device():
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.pa_tree_masks(i32(3), i32(3), MASK)
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.pa_forward_tree(Q, CACHES, CACHES, i32(2, 4), i32(2), i32(3), MASK, 4, 2, 64, 16, 0.1,
                           torch.zeros(3, 4, 64), max_seq_len=64)
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.pa_forward_weights(Q, CACHES, None, i32(2, 4), i32(2), i32(3), 4, 2, 64, 16, 0.1, None, W,
                              accumulate=True, max_seq_len=64)
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.pa_cache_accept(CACHES, CACHES, i32(2, 4), i32(2), i32(3), i32(2, 5), i32(2), i32(2), 16)
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.pa_cache_evict(CACHES, CACHES, W, i32(2, 4), i32(2), i32(2), i32(2), 16, max_seq_len=64)


def refused(f, args, kw, changes):
    for at, bad, err in changes:
        a, k = list(args), dict(kw)
        if isinstance(at, str):
            k[at] = bad
        else:
            a[at] = bad
        with pytest.raises(err):
            f(*a, **k)


def test_binding_refuses_shapes_types_and_strides():
    refused(pa.pa_tree_masks, [i32(3), i32(3), MASK], {}, [
        (0, i32(2), ValueError), (0, i32(3).long(), TypeError), (2, MASK.int(), TypeError),
        (2, torch.zeros(3, 2, dtype=torch.int64)[:, :1], ValueError), ("positions", i32(3), ValueError),
        ("seq_lens", i32(3), ValueError)])
    args = [Q, CACHES, CACHES, i32(2, 4), i32(2), i32(3), MASK, 4, 2, 64, 16, 0.1, torch.zeros(3, 4, 64)]
    refused(pa.pa_forward_tree, args, dict(max_seq_len=64), [
        (0, torch.zeros(3, 64, 4).transpose(1, 2), ValueError), (0, Q.half(), TypeError),
        (1, torch.zeros(4, 16, 1, 64), ValueError), (2, torch.zeros(5, 16, 2, 64), ValueError),
        (3, i32(3, 4), ValueError), (4, i32(2).long(), TypeError), (5, i32(4), ValueError),
        (6, torch.zeros(2, 1, dtype=torch.int64), ValueError), (6, MASK.int(), TypeError),
        (10, 32, ValueError), (12, torch.zeros(3, 4, 32), ValueError), ("kv_layout", "hnd", ValueError),
        ("num_blocks", 5, ValueError), ("sinks", torch.zeros(3), TypeError)])
    args = [Q, CACHES, CACHES, i32(2, 4), i32(2), i32(3), 4, 2, 64, 16, 0.1, torch.zeros(3, 4, 64), W]
    refused(pa.pa_forward_weights, args, dict(accumulate=True, max_seq_len=64), [
        (2, None, ValueError), (2, CACHES.bfloat16(), TypeError), (12, torch.zeros(4, 16, 2), ValueError),
        (12, W.double(), TypeError), (12, torch.zeros(4, 16, 2).transpose(1, 2), ValueError),
        (5, i32(2), ValueError)])
    args = [CACHES, CACHES, i32(2, 4), i32(2), i32(3), i32(2, 5), i32(2), i32(2), 16]
    refused(pa.pa_cache_accept, args, {}, [
        (1, torch.zeros(4, 16, 2, 32), ValueError), (5, i32(3, 5), ValueError), (6, i32(3), ValueError),
        (7, i32(1), ValueError), (4, i32(2), ValueError), (8, 32, ValueError), (5, i32(5, 2).t(), ValueError),
        ("freed_pages", i32(4), ValueError), ("num_blocks", 9, ValueError), (0, CACHES.half(), TypeError)])
    args = [CACHES, CACHES, W, i32(2, 4), i32(2), i32(2), i32(2), 16]
    refused(pa.pa_cache_evict, args, dict(max_seq_len=64), [
        (2, torch.zeros(4, 16, 2), ValueError), ("weights_out", torch.zeros(3, 2, 16), ValueError),
        (5, i32(3), ValueError), (6, i32(1), ValueError), (7, 8, ValueError), ("num_freed", i32(1), ValueError),
        (4, i32(2).long(), TypeError)])

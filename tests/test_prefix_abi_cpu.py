"""Host-side argument checks of pa_forward_shared_prefix, pa_block_tables and
pa_cache_write_slots, through the C ABI and through the binding: refused calls
launch nothing and need no GPU."""
import ctypes

import pytest
import torch

from paged_kv_attention_16_gb300 import build as pbuild
from paged_kv_attention_16_gb300 import pa

P = 1 << 20  # stands for an aligned device address that is never followed
VP, CI, CL = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pa.lib()


def _prefix(lib, opts=None, **kw):
    a = dict(q=P, k=P, v=P, bt=P, sl=P, qsl=P, gsl=P, pl=P, H=8, Hk=2, D=128, bs=16, scale=0.1,
             out=P, stream=None, dtype=1, S=2, NG=1, T=2, mbps=4, nb=4, msl=64, mpl=32, ws=P,
             wsb=1 << 40)
    a.update(kw)
    o = None if opts is None else ctypes.byref(pa.ForwardOptions(*opts))
    return lib.pa_forward_shared_prefix(
        a["q"], a["k"], a["v"], a["bt"], a["sl"], a["qsl"], a["gsl"], a["pl"], a["H"], a["Hk"],
        a["D"], a["bs"], a["scale"], a["out"], a["stream"], a["dtype"], a["S"], a["NG"], a["T"],
        a["mbps"], a["nb"], a["msl"], a["mpl"], o, a["ws"], a["wsb"])


@pytest.mark.parametrize("kw,want", [
    (dict(H=0), 1), (dict(Hk=3), 1), (dict(S=-1), 1), (dict(NG=-1), 1), (dict(mpl=-1), 1),
    (dict(dtype=7), 1), (dict(D=96), 2), (dict(bs=8), 2), (dict(H=96, Hk=3), 2), (dict(T=0), 0),
    (dict(T=0, ws=None), 0), (dict(NG=0), 1), (dict(S=0), 1), (dict(gsl=None), 1),
    (dict(pl=None), 1), (dict(q=None), 1), (dict(out=P + 4), 1), (dict(ws=None), 3),
    (dict(wsb=1000), 3), (dict(ws=P + 16), 1), (dict(k=None), 1), (dict(nb=0), 1),
    (dict(bt=None), 1),
])
def test_prefix_argument_checks(lib, kw, want):
    assert _prefix(lib, **kw) == want


@pytest.mark.parametrize("name", ["bt", "sl", "qsl", "gsl", "pl"])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_prefix_metadata_alignment(lib, name, off):
    assert _prefix(lib, **{name: P + off}) == 1


@pytest.mark.parametrize("opts,want", [
    ((None, 0, 0, None, 0, 0), 0), ((None, 1, 0, None, 0, 1), 0), ((P + 2, 0, 0, None, 0, 0), 1),
    ((None, 2, 0, None, 0, 0), 1), ((None, 0, -1, None, 0, 0), 1), ((None, 0, 16, None, 0, 0), 2),
    ((None, 0, 0, P, 0, 0), 2), ((None, 0, 0, None, 2, 0), 1), ((None, 0, 0, None, 0, -1), 1),
])
def test_prefix_option_checks(lib, opts, want):
    assert _prefix(lib, opts, T=0) == want


def test_prefix_workspace_bytes(lib):
    f = pa.pa_forward_shared_prefix_workspace_bytes
    base = f(pa.PA_BF16, 64, 1, 64, 32, 8, 128, 8192)
    assert base > 0 and f(pa.PA_BF16, 64, 1, 4096, 32, 8, 128, 8192) > base
    # (fp32 has no tiles to cut, whose partials are 304 x 128 rows at most)
    assert f(pa.PA_F32, 64, 1, 64, 32, 8, 128, 8192) + 304 * 128 * 129 * 4 >= base
    # 256 rows of partials (head_dim values and a log-sum-exp) for every item of the prefix
    # part: at least one per KV head and group, and 152 where the prefix has tiles for them
    assert base >= 152 * 256 * (128 + 1) * 4
    assert f(pa.PA_BF16, 1, 1, 1, 32, 8, 128, 100) < base / 10
    # one tile of positions cannot be split: an item for each KV head and group, their partials alone
    one = f(pa.PA_BF16, 64, 64, 64, 32, 8, 128, 128)
    assert 8 * 64 * 256 * 129 * 4 < one < 8 * 66 * 256 * 129 * 4 * 2
    # sizes whose products pass what a call takes
    top = 2 ** 31 - 1
    assert f(pa.PA_BF16, top, top, top, top, top, 128, top) == 0
    assert f(pa.PA_BF16, 1, top, 1, 64, 64, 64, top) == 0
    assert f(pa.PA_BF16, -1, 1, 1, 32, 8, 128, 64) == 0 and f(1, 1, 1, 1, 32, 5, 128, 64) == 0


def _tables(lib, **kw):
    a = dict(sl=P, qsl=P, free=P, fs=P, fe=P + 4, bt=P, slots=P, pos=P, bs=16, stream=None, S=2,
             T=2, mbps=4, nb=4, nf=8)
    a.update(kw)
    return lib.pa_block_tables(a["sl"], a["qsl"], a["free"], a["fs"], a["fe"], a["bt"], a["slots"],
                               a["pos"], a["bs"], a["stream"], a["S"], a["T"], a["mbps"], a["nb"],
                               a["nf"])


NO_FREE = dict(fs=None, fe=None, free=None, nf=0)


@pytest.mark.parametrize("kw,want", [
    (dict(bs=0), 1), (dict(S=-1), 1), (dict(T=-1), 1), (dict(mbps=-1), 1), (dict(nb=-1), 1),
    (dict(nf=-1), 1), (dict(fe=P), 1), (dict(fe=None), 1), (dict(free=None), 1),
    (dict(fs=None), 1), (dict(sl=None), 1), (dict(qsl=None), 1), (dict(bt=None), 1),
    (dict(slots=None), 1), (dict(slots=P + 4), 1), (dict(pos=P + 2), 1), (dict(fs=P + 2), 1),
    (dict(mbps=0), 1), (dict(S=16385), 2), (dict(T=0, **NO_FREE), 0), (dict(sl=P + 1), 1),
])
def test_tables_argument_checks(lib, kw, want):
    assert _tables(lib, **kw) == want


def _write(lib, **kw):
    a = dict(kn=P, vn=P, kc=P, vc=P, slots=P, Hk=2, D=128, bs=16, stream=None, dtype=1, T=1,
             ks=256, vs=256, nb=4, layout=0)
    a.update(kw)
    return lib.pa_cache_write_slots(a["kn"], a["vn"], a["kc"], a["vc"], a["slots"], a["Hk"], a["D"],
                                    a["bs"], a["stream"], a["dtype"], a["T"], a["ks"], a["vs"],
                                    a["nb"], a["layout"])


@pytest.mark.parametrize("kw,want", [
    (dict(Hk=0), 1), (dict(D=-1), 1), (dict(bs=0), 1), (dict(T=-1), 1), (dict(dtype=5), 1),
    (dict(layout=2), 1), (dict(ks=-8), 1), (dict(D=4), 2), (dict(ks=250), 2), (dict(vs=4), 2),
    (dict(Hk=1 << 20), 2), (dict(T=0), 0), (dict(kn=None), 1), (dict(vc=P + 8), 1),
    (dict(slots=None), 1), (dict(slots=P + 4), 1), (dict(nb=0), 1),
])
def test_write_argument_checks(lib, kw, want):
    assert _write(lib, **kw) == want


def test_binding_refuses_tensors_off_the_device():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    slots, rows = torch.zeros(3, dtype=torch.int64), torch.zeros(3, 2, 64)
    caches = torch.zeros(4, 16, 2, 64)
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.pa_block_tables(i32(2), i32(3), i32(2, 4), slots, 16, num_blocks=4)
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.pa_cache_write_slots(rows, rows, caches, caches, slots, 16)
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.pa_forward_shared_prefix(torch.zeros(3, 4, 64), caches, caches, i32(2, 4), i32(2),
                                    i32(3), i32(2), i32(1), 4, 2, 64, 16, 0.1,
                                    torch.zeros(3, 4, 64), max_seq_len=64, max_prefix_len=32)


def test_binding_refuses_shapes_types_and_strides():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    slots, rows, caches = torch.zeros(3, dtype=torch.int64), torch.zeros(3, 2, 64), torch.zeros(4, 16, 2, 64)
    with pytest.raises(TypeError):
        pa.pa_block_tables(i32(2).long(), i32(3), i32(2, 4), slots, 16, num_blocks=4)
    with pytest.raises(ValueError):
        pa.pa_block_tables(i32(2), i32(2), i32(2, 4), slots, 16, num_blocks=4)
    with pytest.raises(ValueError):
        pa.pa_block_tables(i32(2), i32(3), i32(2, 4), slots, 16, num_blocks=4, free_start=i32(1))
    with pytest.raises(ValueError):
        pa.pa_block_tables(i32(2), i32(3), i32(4, 2).t(), slots, 16, num_blocks=4)
    with pytest.raises(TypeError):
        pa.pa_cache_write_slots(rows, rows, caches, caches, slots.int(), 16)
    with pytest.raises(TypeError):
        pa.pa_cache_write_slots(rows.half(), rows.half(), caches, caches, slots, 16)
    with pytest.raises(ValueError):
        pa.pa_cache_write_slots(rows, rows[:2], caches, caches, slots, 16)
    with pytest.raises(ValueError):
        pa.pa_cache_write_slots(rows, rows, caches, caches, slots, 32)
    args = [torch.zeros(3, 4, 64), caches, caches, i32(2, 4), i32(2), i32(3), i32(2), i32(1), 4, 2,
            64, 16, 0.1, torch.zeros(3, 4, 64)]
    for at, bad, err in ((0, torch.zeros(3, 64, 4).transpose(1, 2), ValueError),
                         (4, i32(2).long(), TypeError), (6, i32(3), ValueError),
                         (11, 32, ValueError), (13, torch.zeros(3, 4, 32), ValueError)):
        a = list(args)
        a[at] = bad
        with pytest.raises(err):
            pa.pa_forward_shared_prefix(*a, max_seq_len=64, max_prefix_len=32)
    with pytest.raises(TypeError):
        pa.pa_forward_shared_prefix(*args, max_seq_len=64, max_prefix_len=32, sinks=torch.zeros(3))

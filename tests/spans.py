"""Shared helpers of the tests of drafted trees and bounded caches: batches, the
oracle on them, and elementwise bounds derived from the arithmetic."""
import numpy as np
import torch

from oracle import oracle as orc
from paged_kv_attention_16_gb300 import inputs, pa


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def random_trees(rng, q_lens, chain=None):
    """Parents of every request's new tokens: a random earlier token or -1; `chain`:
    each the child of the one before."""
    return np.concatenate([np.arange(-1, n - 1) if chain else
                           np.array([rng.integers(-1, i) if i else -1 for i in range(n)], np.int64)
                           for n in q_lens] + [np.zeros(0, np.int64)]).astype(np.int64)


def random_mask(rng, q_lens, words, density=0.3):
    """Any mask at all, bits behind the last new token set too."""
    T = sum(q_lens)
    bits = rng.random((T, 64 * words)) < density
    return (bits.reshape(T, words, 64) << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64)


def to_words(mask):
    """uint64 words as the int64 tensor that the binding takes."""
    return torch.from_numpy(np.ascontiguousarray(mask).view(np.int64)).cuda()


def batch(q_lens, ctx_lens, H, Hk, D, bs, dtype="bf16", layout="nhd", seed=0, scale=None):
    b = inputs.paged_batch(q_lens, ctx_lens, H, Hk, D, bs, dtype=dtype, seed=seed, scale=scale)
    return inputs.as_hnd(b) if layout == "hnd" else b


def oracle(b, mask=None, sinks=None, values=True):
    return orc.span_attention(
        inputs.storage_array(b.q), inputs.storage_array(b.k_cache),
        inputs.storage_array(b.v_cache) if values else None, b.block_table.numpy(),
        b.seq_lens.numpy(), b.query_start_loc.numpy(), b.num_heads, b.num_kv_heads, b.head_dim,
        b.block_size, b.scale, mask=mask, sinks=sinks, kv_layout=b.kv_layout)


def weight_error(b, r, ctx):
    """Bound on the relative error of a softmax weight.  A score is a sum of D
    products in fp32 and its scaling (D + 4 roundings of 2^-24 on at most scale * dots,
    the query's scaling among them), in a difference of two (x 2); the base-2
    exponential 2^-22 and the reference's rounding 2^-24 on |scores| <= scale * dots,
    twice more; the sum of ctx weights and the partials' join ctx + 64 roundings."""
    u = 2.0 ** -24
    span = b.scale * r["dots"] + 1.0
    return 2 * (b.head_dim + 8) * u * span + 8 * u * (span + 64) + (ctx + 64) * u


def check_out(b, got, want, dtype):
    """got [T, H, D] float64 against the oracle's requests, element by element: the
    weights' error on sum p |v|, bf16 weights' rounding (2^-8) on it too, and the
    output's own rounding (2^-8 or 2^-24)."""
    qsl = b.query_start_loc.numpy()
    for s, r in enumerate(want):
        g = got[qsl[s]:qsl[s + 1]]
        if g.size == 0:
            continue
        assert np.isfinite(g).all(), f"request {s}: not finite"
        e = weight_error(b, r, int(b.seq_lens[s]))
        half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
        weights = half if dtype == "bf16" else 0.0
        # (the output is rounded from a value that is off already: half of either)
        tol = (1.01 * (e + weights) * r["mass"] + half * 1.01 * (np.abs(r["out"]) + 0.02 * r["mass"])
               + 1e-30)
        bad = np.abs(g - r["out"]) > tol
        assert not bad.any(), (f"request {s}: {bad.sum()} of {bad.size} off, by up to "
                               f"{(np.abs(g - r['out']) / tol).max():.2f} of the bound at "
                               f"{np.argwhere(bad)[:3].tolist()}")


def run_tree(b, mask, sinks=None, max_query_len=0, out=None, expect=0, stream=None, T=None, **kw):
    """pa_forward_tree on a CPU batch; out [T, H, D] float64."""
    d = pa.to_device(b)
    if out is None:
        out = torch.full_like(d.q, float("nan"))
    snk = None if sinks is None else torch.tensor(np.asarray(sinks), dtype=torch.float32).cuda()
    pa.pa_forward_tree(d.q, d.k_cache, d.v_cache, d.block_table, d.seq_lens, d.query_start_loc,
                       to_words(mask), b.num_heads, b.num_kv_heads, b.head_dim, b.block_size,
                       b.scale, out, stream, max_seq_len=b.max_seq_len, sinks=snk,
                       kv_layout=b.kv_layout, max_query_len=max_query_len, **kw)
    status = pa.pa_get_device_status()
    assert status == expect, f"device status {status:#x}, expected {expect:#x}"
    return out.float().cpu().numpy().astype(np.float64)


def slots_of(b, s):
    """(page, slot) of every position of request s."""
    at = np.arange(int(b.seq_lens[s]))
    return b.block_table.numpy()[s][at // b.block_size], at % b.block_size


def run_weights(b, weights, accumulate, output=True, sinks=None, max_query_len=0, expect=0, **kw):
    """pa_forward_weights on a CPU batch: (out or None, weights [nb, Hk, bs] float32)."""
    d = pa.to_device(b)
    out = torch.full_like(d.q, float("nan")) if output else None
    w = torch.tensor(weights, dtype=torch.float32).cuda()
    snk = None if sinks is None else torch.tensor(np.asarray(sinks), dtype=torch.float32).cuda()
    pa.pa_forward_weights(d.q, d.k_cache, d.v_cache if output else None, d.block_table, d.seq_lens,
                          d.query_start_loc, b.num_heads, b.num_kv_heads, b.head_dim, b.block_size,
                          b.scale, out, w, accumulate=accumulate, max_seq_len=b.max_seq_len,
                          sinks=snk, kv_layout=b.kv_layout, max_query_len=max_query_len, **kw)
    status = pa.pa_get_device_status()
    assert status == expect, f"device status {status:#x}, expected {expect:#x}"
    return (out.float().cpu().numpy().astype(np.float64) if output else None), w.cpu().numpy()


def check_weights(b, got, before, want, accumulate):
    """Every slot of the batch's positions against the oracle, every other slot as it
    was: the weights' error and the sum of rows on W, the accumulation's rounding."""
    expect, tol = before.astype(np.float64).copy(), np.zeros_like(before, np.float64)
    G = b.num_heads // b.num_kv_heads
    for s, r in enumerate(want):
        n = len(r["out"])
        if n == 0:
            continue
        page, slot = slots_of(b, s)
        ctx = len(page)
        e = weight_error(b, r, ctx) + (n * G + 2) * 2.0 ** -24
        for h in range(b.num_kv_heads):
            w = r["weights"][h].copy()
            t = e * w + 2.0 ** -24 * np.abs(w)
            if accumulate:
                old = before[page, h, slot][:ctx - n].astype(np.float64)
                w[:ctx - n] += old
                t[:ctx - n] += 2.0 ** -23 * np.abs(w[:ctx - n])
            expect[page, h, slot], tol[page, h, slot] = w, t + 1e-37
    bad = ~(np.abs(got - expect) <= tol)
    bad &= ~(np.isnan(got) & np.isnan(expect))
    assert not bad.any(), (f"{bad.sum()} of {bad.size} slots off at {np.argwhere(bad)[:4].tolist()}: "
                           f"{got[bad][:4]} for {expect[bad][:4]}")

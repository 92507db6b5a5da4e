"""Cases and plain forms of the operators for drafted trees of tokens and for bounded caches.

Three operators of a speculative decoding step, in the order in which the step calls them:

  masks    ancestor masks and rotary positions of the drafted tokens, from their parents
           (pa_tree_masks)
  tree     attention of the drafted tokens: each sees the cached positions, its ancestors and
           itself (pa_forward_tree)
  accept   the accepted path's K and V rows moved to the positions behind the cached ones, the
           new lengths and the pages that are free again (pa_cache_accept)

and two of a cache that is kept to a budget:

  weights  attention (its output is optional) that adds up the softmax weight that every cached
           position gets, KV head by KV head (pa_forward_weights)
  evict    each request and KV head keeps its first, its most recent and its heaviest positions;
           their rows move to the front (pa_cache_evict)

`own` chooses between the plain torch form of each and the framework's call.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the trees of a decode batch of 64: up to 16 drafted tokens each
        dict(name="masks_b64", op="masks", requests=64, nodes=16, words=1, cached=8192, pad=0,
             lens=11),
        # wide trees of a large batch, padded to a captured size
        dict(name="masks_large", op="masks", requests=256, nodes=250, words=4, cached=8192,
             pad=101, lens=12),
        # one user's step on a short context: the smallest call, where latency counts
        dict(name="tree_small", op="tree", heads=32, kv_heads=8, dim=128, block=16, dtype="bf16",
             layout="nhd", sinks=False, requests=1, nodes=8, words=1, cached=500, pad=0, lens=21),
        # a batch of 64 that verifies up to 16 drafted tokens a request
        dict(name="tree_b64", op="tree", heads=32, kv_heads=8, dim=128, block=16, dtype="bf16",
             layout="nhd", sinks=False, requests=64, nodes=16, words=1, cached=8192, pad=0,
             lens=22),
        # few requests with wide trees and long contexts, sinks on
        dict(name="tree_wide", op="tree", heads=64, kv_heads=4, dim=128, block=64, dtype="bf16",
             layout="hnd", sinks=True, requests=12, nodes=250, words=4, cached=16384, pad=37,
             lens=23),
        # the accepted paths of a decode batch of 64
        dict(name="accept_b64", op="accept", kv_heads=8, dim=128, block=16, dtype="bf16",
             layout="nhd", requests=64, nodes=16, path=8, cached=1000, lens=31),
        # long drafts of a large batch, most of them accepted; fp32 rows, head-major pages
        dict(name="accept_large", op="accept", kv_heads=4, dim=64, block=64, dtype="f32",
             layout="hnd", requests=500, nodes=250, path=200, cached=900, lens=32),
        # four decodes on short contexts
        dict(name="weights_decode_small", op="weights", heads=32, kv_heads=8, dim=128, block=16,
             dtype="bf16", layout="nhd", sinks=False, output=True, accumulate=True, requests=4,
             new=1, cached=1000, pad=0, lens=41),
        # a decode step of a batch of 64
        dict(name="weights_decode_b64", op="weights", heads=32, kv_heads=8, dim=128, block=16,
             dtype="bf16", layout="nhd", sinks=False, output=True, accumulate=True, requests=64,
             new=1, cached=8192, pad=0, lens=42),
        # the last 64 rows of each of 16 prompts vote on the prompt's positions; no output
        dict(name="weights_window", op="weights", heads=16, kv_heads=4, dim=64, block=64,
             dtype="bf16", layout="hnd", sinks=False, output=False, accumulate=False, requests=16,
             new=64, cached=16384, pad=0, lens=43),
        # prompts of a batch cut down to 2048 positions each
        dict(name="evict_b16", op="evict", kv_heads=8, dim=128, block=16, dtype="bf16",
             layout="nhd", requests=16, cached=8192, keep=2048, first=4, recent=256, lens=51),
        # very long documents, one KV head
        dict(name="evict_long", op="evict", kv_heads=1, dim=128, block=64, dtype="bf16",
             layout="nhd", requests=4, cached=131072, keep=16384, first=4, recent=1024, lens=52),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


HEADS = [(32, 8, 128), (64, 4, 128), (8, 1, 128), (16, 4, 64), (32, 8, 64), (8, 8, 128)]


def draw(rng):
    op = rng.choice(["masks", "tree", "tree", "accept", "weights", "weights", "evict"])
    lens = rng.randrange(1 << 30)
    if op == "masks":
        nodes = _log_int(rng, 1, 250)
        return dict(op=op, requests=_log_int(rng, 1, 256), nodes=nodes,
                    words=-(-nodes // 64) + rng.randrange(2), cached=_log_int(rng, 1, 8192),
                    pad=rng.choice([0, rng.randrange(1, 200)]), lens=lens)
    heads, kv_heads, dim = rng.choice(HEADS)
    case = dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim,
                block=rng.choice([16, 16, 32, 64, 128]),
                dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]),
                layout=rng.choice(["nhd", "hnd"]), lens=lens)
    if op == "accept":
        del case["heads"]
        nodes = _log_int(rng, 1, 250)
        return dict(case, requests=_log_int(rng, 1, 400), nodes=nodes, path=_log_int(rng, 1, nodes),
                    cached=_log_int(rng, 1, 900))
    if op == "evict":
        del case["heads"]
        cached = _log_int(rng, 16, 60000)
        keep = _log_int(rng, 1, cached)
        return dict(case, requests=_log_int(rng, 1, max(1, min(64, 130000 * 8 // (cached * kv_heads)))),
                    cached=cached, keep=keep, first=rng.choice([0, 1, 4, 64]),
                    recent=rng.choice([0, 1, _log_int(rng, 2, max(2, keep))]))
    cached = _log_int(rng, 1, 32768)
    if op == "tree":
        nodes = _log_int(rng, 1, 250)
        # the sizes that the listed cases have, in 32 bits a smaller share of them
        most = (1 << 30) // (1 if case["dtype"] == "bf16" else 8)
        requests = _log_int(rng, 1, max(1, min(128, most // ((cached + nodes) * nodes * heads),
                                               600000 // (cached + nodes))))
        return dict(case, sinks=rng.random() < 0.3, requests=requests, nodes=nodes,
                    words=-(-nodes // 64) + rng.randrange(2), cached=cached,
                    pad=rng.choice([0, rng.randrange(1, 50)]))
    new = rng.choice([1, 1, _log_int(rng, 2, 300)])
    most = (1 << 29) // (1 if case["dtype"] == "bf16" else 8)
    requests = _log_int(rng, 1, max(1, min(128, most // ((cached + new) * new * heads),
                                           600000 // (cached + new))))
    return dict(case, sinks=rng.random() < 0.3, output=rng.random() < 0.6,
                accumulate=rng.random() < 0.5, requests=requests, new=new, cached=cached,
                pad=rng.choice([0, rng.randrange(1, 50)]))


# ---------------------------------------------------------------------------
# lengths: from the case alone
# ---------------------------------------------------------------------------

def _lens(case):
    """(new tokens, length with them) of every request."""
    rng = random.Random(case["lens"])
    most = case.get("nodes", case.get("new", 0))
    new, total = [], []
    for _ in range(case["requests"]):
        n = rng.randint((most + 1) // 2, most)
        cached = rng.randint(case["cached"] // 16, case["cached"])
        new.append(n)
        total.append(max(1, n + cached))
    return new, total


def _path_lens(case):
    rng = random.Random(case["lens"] + 1)
    return [rng.randint(0, min(n, case["path"])) for n in _lens(case)[0]]


def _kept(case):
    """Length of every request before and behind an eviction to the budget."""
    total = _lens(case)[1]
    return total, [min(t, case["keep"]) for t in total]


def work(case):
    op = case["op"]
    new, total = _lens(case)
    T = sum(new) + case.get("pad", 0)
    if op == "masks":
        return {"bytes": 4 * T + 8 * len(new) + 8 * T * case["words"] + 4 * T, "flops": 0}
    es = 2 if case["dtype"] == "bf16" else 4
    row = case["kv_heads"] * case["dim"] * es
    if op == "accept":
        # (rows that stay where they are, or a path's first ones, are counted too)
        return {"bytes": 4 * row * sum(_path_lens(case)) + 20 * len(new), "flops": 0}
    if op == "evict":
        before, after = _kept(case)
        # the weights are read; a kept row moves unless it lies in the front part already. At
        # random, keep / length of the front's rows stay: those before the first evicted one,
        # hardly any, do not move.
        moved = sum(max(0, a - case["first"]) for b, a in zip(before, after) if b > a)
        return {"bytes": 4 * case["kv_heads"] * (sum(before) + sum(after)) + 4 * row * moved, "flops": 0}
    H, D = case["heads"], case["dim"]
    pairs = 0
    for n, t in zip(new, total):
        p = t - n
        pairs += n * p + n * (n + 1) // 2
    kv = sum(total)
    if op == "tree":
        return {"bytes": 2 * kv * row + 2 * sum(new) * H * D * es + 8 * sum(new) * case["words"],
                "flops": 4 * pairs * H * D}
    both = 2 if case["output"] else 1
    return {"bytes": both * (kv * row + sum(new) * H * D * es)
                     + 4 * case["kv_heads"] * kv * (2 if case["accumulate"] else 1),
            "flops": 2 * both * pairs * H * D}


# ---------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------

def _cum(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _i32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _trees(new, tokens, gen):
    """Parents of drafted tokens: token i of a request under a random one before it (or the last
    cached token, -1), every eighth request a plain chain."""
    n = torch.tensor(new + [tokens - sum(new)], dtype=torch.int64).cuda()
    i = torch.arange(tokens, device="cuda") - torch.repeat_interleave(torch.cumsum(n, 0) - n, n)
    s = torch.repeat_interleave(torch.arange(len(new) + 1, device="cuda"), n)
    at = torch.rand(tokens, generator=gen, device="cuda")
    parent = torch.floor(at * (i + 1)).long().clamp_max(i) - 1
    return torch.where(s % 8 == 7, i - 1, parent).to(torch.int32)


def _pages(case, total, gen):
    """Block table of the requests' pages, scattered over a pool that is a little larger."""
    bs = case["block"]
    pages = [-(-t // bs) for t in total]
    pool = sum(pages) + max(1, sum(pages) // 10)
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(total), max(pages)), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(max(pages), device="cuda")
    use = col[None, :] < _i32(pages)[:, None]
    table[use] = perm[:sum(pages)]
    return table, pool


def _caches(case, pool, gen):
    bs, Hk, D = case["block"], case["kv_heads"], case["dim"]
    shape = (pool, bs, Hk, D) if case["layout"] == "nhd" else (pool, Hk, bs, D)
    dt = DTYPES[case["dtype"]]
    return tuple(torch.randn(shape, generator=gen, device="cuda", dtype=dt) for _ in "kv")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    op = case["op"]
    new, total = _lens(case)
    S, n_max = len(new), max(new)
    T = sum(new) + case.get("pad", 0)
    st.update(seq_lens=_i32(total), starts=_i32(_cum(new)), max_seq=max(total), max_new=n_max)
    if op == "masks":
        st.update(parents=_trees(new, T, gen),
                  mask=torch.empty((T, case["words"]), dtype=torch.int64, device="cuda"),
                  positions=torch.empty(T, dtype=torch.int32, device="cuda"))
        return st
    table, pool = _pages(case, total, gen)
    k, v = _caches(case, pool, gen)
    st.update(table=table, k_cache=k, v_cache=v, pool=pool,
              new_lens=torch.empty(S, dtype=torch.int32, device="cuda"),
              freed=torch.full((table.numel(),), -1, dtype=torch.int32, device="cuda"),
              num_freed=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if op == "accept":
        lens = _i32(_path_lens(case))
        # an ascending choice of each request's nodes
        key = torch.rand((S, n_max), generator=gen, device="cuda")
        key[torch.arange(n_max, device="cuda")[None, :] >= _i32(new)[:, None]] = 2.0
        pick = torch.argsort(key, 1)[:, :case["path"]]
        if pick.shape[1] < case["path"]:
            pick = torch.nn.functional.pad(pick, (0, case["path"] - pick.shape[1]), value=n_max)
        col = torch.arange(case["path"], device="cuda")
        pick = torch.where(col[None, :] < lens[:, None], pick, 1 << 30).sort(1).values
        st.update(path=torch.where(pick < (1 << 30), pick, -1).to(torch.int32).contiguous(),
                  path_lens=lens)
        return st
    wshape = (pool, case["kv_heads"], case["block"])
    if op == "evict":
        # a few positions carry most of the weight
        weights = torch.exp(1.5 * torch.randn(wshape, generator=gen, device="cuda"))
        st.update(weights=weights, keep_lens=_i32([case["keep"]] * S),
                  weights_out=torch.zeros(wshape, device="cuda"))
        return st
    H, D = case["heads"], case["dim"]
    # scores of a few units' spread, so that some keys carry most of a row's weight
    q = (1.5 * torch.randn((T, H, D), generator=gen, device="cuda")).to(DTYPES[case["dtype"]])
    st.update(q=q, scale=1.0 / math.sqrt(D),
              sink=torch.randn(H, generator=gen, device="cuda") if case["sinks"] else None,
              out=torch.zeros_like(q))
    if op == "tree":
        mask = torch.zeros((T, case["words"]), dtype=torch.int64, device="cuda")
        seen = _ancestors(_trees(new, T, gen), st["starts"].long(), n_max)
        rows = torch.arange(n_max, device="cuda")[None, :] < _i32(new)[:, None]
        mask[:sum(new)] = _pack(seen, case["words"])[rows]
        st.update(mask=mask)
    else:
        # what some steps before have added up
        st.update(weights=torch.rand(wshape, generator=gen, device="cuda") * (8.0 * H / max(total)))
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(st):
    if own:
        return _OWN[st["op"]](st)
    return _PLAIN[st["op"]](st)


def _own_masks(st):
    from paged_kv_attention_16_gb300 import pa
    pa.pa_tree_masks(st["parents"], st["starts"], st["mask"], seq_lens=st["seq_lens"],
                     positions=st["positions"])
    return {"mask": st["mask"], "positions": st["positions"]}


def _own_tree(st):
    from paged_kv_attention_16_gb300 import pa
    pa.pa_forward_tree(st["q"], st["k_cache"], st["v_cache"], st["table"], st["seq_lens"],
                       st["starts"], st["mask"], st["heads"], st["kv_heads"], st["dim"],
                       st["block"], st["scale"], st["out"], max_seq_len=st["max_seq"],
                       sinks=st["sink"], kv_layout=st["layout"], max_query_len=st["max_new"])
    return {"out": st["out"]}


def _own_accept(st):
    from paged_kv_attention_16_gb300 import pa
    pa.pa_cache_accept(st["k_cache"], st["v_cache"], st["table"], st["seq_lens"], st["starts"],
                       st["path"], st["path_lens"], st["new_lens"], st["block"],
                       freed_pages=st["freed"], num_freed=st["num_freed"], kv_layout=st["layout"])
    return _kept_outputs(st)


def _own_weights(st):
    from paged_kv_attention_16_gb300 import pa
    out = st["out"] if st["output"] else None
    pa.pa_forward_weights(st["q"], st["k_cache"], st["v_cache"] if st["output"] else None,
                          st["table"], st["seq_lens"], st["starts"], st["heads"], st["kv_heads"],
                          st["dim"], st["block"], st["scale"], out, st["weights"],
                          accumulate=st["accumulate"], max_seq_len=st["max_seq"], sinks=st["sink"],
                          kv_layout=st["layout"], max_query_len=st["max_new"])
    return {"out": out, "weights": st["weights"]}


def _own_evict(st):
    from paged_kv_attention_16_gb300 import pa
    pa.pa_cache_evict(st["k_cache"], st["v_cache"], st["weights"], st["table"], st["seq_lens"],
                      st["keep_lens"], st["new_lens"], st["block"], weights_out=st["weights_out"],
                      num_first=st["first"], num_recent=st["recent"], freed_pages=st["freed"],
                      num_freed=st["num_freed"], max_seq_len=st["max_seq"], kv_layout=st["layout"])
    return dict(_kept_outputs(st), weights=st["weights_out"])


def _kept_outputs(st):
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"], "seq_lens": st["new_lens"],
            "freed": st["freed"], "num_freed": st["num_freed"]}


def _ancestors(parents, starts, n_max):
    """[requests, n_max, n_max]: whether token j is token i or an ancestor of it."""
    n = starts[1:] - starts[:-1]
    i = torch.arange(n_max, device=parents.device)
    real = i[None, :] < n[:, None]
    p = parents[(starts[:-1, None] + i).clamp_max(parents.shape[0] - 1)]
    p = torch.where(real, p.long(), -1)
    seen = ((p[:, :, None] == i) | (i[:, None] == i)).float()
    for _ in range(max(1, (n_max - 1).bit_length())):  # paths of twice the length each time
        seen = (torch.bmm(seen, seen) > 0).float()
    return (seen > 0) & real[:, :, None]


def _pack(seen, words):
    """Truth values [.., n] as 64-bit words [.., words]."""
    pad = torch.nn.functional.pad(seen, (0, 64 * words - seen.shape[-1]))
    bits = pad.view(*seen.shape[:-1], words, 64).long()
    return (bits << torch.arange(64, device=seen.device)).sum(-1)


def _plain_masks(st):
    starts, total, T = st["starts"].long(), st["seq_lens"].long(), st["parents"].shape[0]
    n = starts[1:] - starts[:-1]
    seen = _ancestors(st["parents"], starts, st["max_new"])
    tok = torch.arange(T, device="cuda")
    s = torch.searchsorted(starts[1:].contiguous(), tok, right=True)
    real = s < len(total)
    s = s.clamp_max(len(total) - 1)
    i = (tok - starts[s]).clamp_max(st["max_new"] - 1)
    words = torch.where(real[:, None], _pack(seen, st["words"])[s, i], 0)
    depth = seen.sum(-1)[s, i] - 1
    positions = torch.where(real, total[s] - n[s] + depth, 0)
    return {"mask": words, "positions": positions.to(torch.int32)}


def _rows(cache, layout, pages, at):
    """fp32 rows [..., kv_heads, dim] at (page, slot) of every index."""
    pages = pages.clamp_min(0).long()
    return (cache[pages, at] if layout == "nhd" else cache[pages, :, at]).float()


def _scores(st, seen):
    """Scaled scores [requests, kv_heads, t, group, positions], -inf where seen
    [requests, t, positions] is false, each row's maximum and sum (with its sink), and the rows'
    and positions' places."""
    q, bs, table = st["q"], st["block"], st["table"]
    T, H, D = q.shape
    Hk = st["kv_heads"]
    starts = st["starts"].long()
    at = (starts[:-1, None] + torch.arange(st["max_new"], device="cuda")).clamp_max(T - 1)
    pos = torch.arange(st["max_seq"], device="cuda")
    page = table.long()[:, pos // bs]
    slot = (pos % bs).expand(page.shape)
    k = _rows(st["k_cache"], st["layout"], page, slot)
    s = torch.einsum("ntkgd,npkd->nktgp", q.float().view(T, Hk, H // Hk, D)[at], k)
    s.mul_(st["scale"]).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    if st["sink"] is not None:
        m = torch.maximum(m, st["sink"].view(1, Hk, 1, H // Hk, 1))
    m.clamp_min_(torch.finfo(torch.float32).min)
    s.sub_(m).exp_()
    den = s.sum(-1, keepdim=True)
    if st["sink"] is not None:
        den = den + torch.exp(st["sink"].view(1, Hk, 1, H // Hk, 1) - m)
    return s, den, page, slot


def _values(st, w, den, page, slot):
    """The output [tokens, heads, dim] of weights w / den; rows behind the last request as they
    were."""
    T, H, D = st["q"].shape
    v = _rows(st["v_cache"], st["layout"], page, slot)
    o = torch.einsum("nktgp,npkd->ntkgd", w, v)
    o = o / den[..., 0].permute(0, 2, 1, 3)[..., None].clamp_min(1e-37)
    starts = st["starts"].long()
    tok = torch.arange(T, device="cuda")
    s = torch.searchsorted(starts[1:].contiguous(), tok, right=True)
    real = s < starts.shape[0] - 1
    s = s.clamp_max(starts.shape[0] - 2)
    rows = o[s, (tok - starts[s]).clamp_max(st["max_new"] - 1)].reshape(T, H, D)
    return torch.where(real[:, None, None], rows.to(st["q"].dtype), st["out"])


def _plain_tree(st):
    starts, total = st["starts"].long(), st["seq_lens"].long()
    n = starts[1:] - starts[:-1]
    prefix = (total - n)[:, None, None]
    i = torch.arange(st["max_new"], device="cuda")
    j = torch.arange(st["max_seq"], device="cuda") - prefix  # as a drafted token, < 0: cached
    words = st["mask"][(starts[:-1, None] + i).clamp_max(st["mask"].shape[0] - 1)]
    bit = j.clamp(0, 64 * st["words"] - 1).expand(-1, st["max_new"], -1)
    seen = (words.gather(2, bit // 64) >> (bit % 64)) & 1
    seen = ((j < 0) | (seen > 0)) & (j < n[:, None, None])
    w, den, page, slot = _scores(st, seen)
    return {"out": _values(st, w, den, page, slot)}


def _plain_weights(st):
    starts, total = st["starts"].long(), st["seq_lens"].long()
    n = starts[1:] - starts[:-1]
    prefix = (total - n)[:, None, None]
    i = torch.arange(st["max_new"], device="cuda")[None, :, None]
    pos = torch.arange(st["max_seq"], device="cuda")
    seen = pos <= prefix + i
    w, den, page, slot = _scores(st, seen)
    out = _values(st, w, den, page, slot) if st["output"] else None
    real = (i < n[:, None, None])[:, None, :, :, None]
    got = (w / den).masked_fill_(~real, 0.0).sum((2, 3))  # [requests, kv_heads, positions]
    there = (pos[None, :] < total[:, None])[:, None, :].expand_as(got)
    page, slot = page[:, None].expand_as(got), slot[:, None].expand_as(got)
    head = torch.arange(st["kv_heads"], device="cuda")[None, :, None].expand_as(got)
    if st["accumulate"]:  # a new token's weight starts here
        old = st["weights"][page.clamp_min(0), head, slot]
        got = got + torch.where((pos[None, :] < (total - n)[:, None])[:, None, :], old, 0.0)
    st["weights"][page[there], head[there], slot[there]] = got[there]
    return {"out": out, "weights": st["weights"]}


def _free_pages(st, after):
    """The pages that hold only positions from `after` on, request by request."""
    bs, table = st["block"], st["table"]
    col = torch.arange(table.shape[1], device="cuda")
    held = (st["seq_lens"].long() + bs - 1) // bs
    kept = (after + bs - 1) // bs
    gone = ((col >= kept[:, None]) & (col < held[:, None])).flatten()
    at = torch.cumsum(gone, 0)
    into = torch.cat([st["freed"], st["freed"][:1]])
    into[torch.where(gone, at - 1, len(st["freed"]))] = table.flatten()
    return {"seq_lens": after.to(torch.int32), "freed": into[:-1],
            "num_freed": at[-1:].to(torch.int32)}


def _move(st, cache, src, dst, real):
    """Rows at positions src of each request to positions dst where real; all [requests, kv_heads,
    n]. cache: [pages, block_size, kv_heads, ..] or, head-major, [pages, kv_heads, block_size, ..]."""
    bs, table = st["block"], st["table"].long()
    s = torch.arange(src.shape[0], device="cuda")[:, None, None].expand_as(src)
    h = torch.arange(src.shape[1], device="cuda")[None, :, None].expand_as(src)
    last = table.shape[1] * bs - 1
    src, dst = src.clamp(0, last), dst.clamp(0, last)
    a, b = table[s, src // bs][real], table[s, dst // bs][real]
    h, src, dst = h[real], (src % bs)[real], (dst % bs)[real]
    if cache.dim() == 4 and st["layout"] == "nhd":
        cache[b, dst, h] = cache[a, src, h]
    else:
        cache[b, h, dst] = cache[a, h, src]


def _plain_accept(st):
    starts, total = st["starts"].long(), st["seq_lens"].long()
    prefix = total - (starts[1:] - starts[:-1])
    path = st["path"].long()
    shape = (path.shape[0], st["kv_heads"], path.shape[1])
    k = torch.arange(path.shape[1], device="cuda")
    src = (prefix[:, None] + path)[:, None, :].expand(shape)
    dst = (prefix[:, None] + k)[:, None, :].expand(shape)
    real = (k < st["path_lens"][:, None])[:, None, :].expand(shape)
    _move(st, st["k_cache"], src, dst, real)
    _move(st, st["v_cache"], src, dst, real)
    return dict(_free_pages(st, prefix + st["path_lens"].long()), k_cache=st["k_cache"],
                v_cache=st["v_cache"])


def _plain_evict(st):
    bs, table, total = st["block"], st["table"].long(), st["seq_lens"].long()
    after = torch.minimum(total, st["keep_lens"].long())
    first = after.clamp_max(st["first"])
    recent = (after - first).clamp_max(st["recent"])
    pos = torch.arange(st["max_seq"], device="cuda")
    w = st["weights"][table[:, pos // bs].clamp_min(0), :, pos % bs].transpose(1, 2)
    rank = torch.where(torch.isnan(w), -math.inf, w).double()
    always = (pos < first[:, None]) | (pos >= (total - recent)[:, None])
    rank = torch.where(always[:, None, :], math.inf, rank)
    rank = torch.where((pos < total[:, None])[:, None, :], rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    n = min(st["keep"], st["max_seq"])
    i = torch.arange(n, device="cuda")
    real = (i < after[:, None])[:, None, :].expand(order.shape[0], order.shape[1], n)
    src = torch.where(real, order[..., :n], 1 << 40).sort(-1).values
    dst = i.expand_as(src)
    moves = real & (src != dst)
    _move(st, st["k_cache"], src, dst, moves)
    _move(st, st["v_cache"], src, dst, moves)
    s = torch.arange(src.shape[0], device="cuda")[:, None, None].expand_as(src)
    h = torch.arange(src.shape[1], device="cuda")[None, :, None].expand_as(src)
    st["weights_out"][table[s, dst // bs][real], h[real], (dst % bs)[real]] = w.gather(
        2, src.clamp_max(st["max_seq"] - 1))[real]
    return dict(_free_pages(st, after), k_cache=st["k_cache"], v_cache=st["v_cache"],
                weights=st["weights_out"])


_OWN = {"masks": _own_masks, "tree": _own_tree, "accept": _own_accept, "weights": _own_weights,
        "evict": _own_evict}
_PLAIN = {"masks": _plain_masks, "tree": _plain_tree, "accept": _plain_accept,
          "weights": _plain_weights, "evict": _plain_evict}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "masks":
        return None  # whole numbers: equal or not
    st = prepare(case, seed)
    new, total = _lens(case)
    bs, Hk, D, S = case["block"], case["kv_heads"], case["dim"], case["requests"]
    table = st["table"].cpu()

    def head_major(name):
        x = st[name].double()
        return x.transpose(1, 2).contiguous() if case["layout"] == "nhd" else x

    def stored(x):
        return x.transpose(1, 2).contiguous() if case["layout"] == "nhd" else x

    if op in ("accept", "evict"):
        k, v = head_major("k_cache"), head_major("v_cache")
        out_w = st["weights_out"].double() if op == "evict" else None
        path, path_lens = (st["path"].tolist(), st["path_lens"].tolist()) if op == "accept" else (None, None)
        for s in range(S):
            pages = table[s].long().cuda()
            if op == "accept":
                base = total[s] - new[s]
                keep = path[s][:path_lens[s]]
                src = (base + torch.tensor(keep, dtype=torch.int64).cuda()).expand(Hk, -1)
                dst = base + torch.arange(len(keep), device="cuda")
            else:
                base, n = 0, min(total[s], case["keep"])
                at = torch.arange(total[s], device="cuda")
                w = st["weights"][pages[at // bs], :, at % bs].double().t()
                f = min(case["first"], n)
                r = min(case["recent"], n - f)
                best = w.clone()
                best[:, :f] = math.inf
                best[:, total[s] - r:] = math.inf
                src = torch.argsort(best, dim=1, descending=True, stable=True)[:, :n].sort(1).values
                dst = torch.arange(n, device="cuda")
                h = torch.arange(Hk, device="cuda")[:, None]
                out_w[pages[dst // bs].expand(Hk, n), h, (dst % bs).expand(Hk, n)] = w.gather(1, src)
            h = torch.arange(Hk, device="cuda")[:, None].expand(src.shape)
            to = (pages[dst // bs].expand(src.shape), h, (dst % bs).expand(src.shape))
            for x in (k, v):
                x[to] = x[pages[src // bs], h, src % bs]
        both = {"k_cache": stored(k), "v_cache": stored(v), "seq_lens": None, "freed": None,
                "num_freed": None}
        return dict(both, weights=out_w) if op == "evict" else both

    H = case["heads"]
    G = H // Hk
    out = st["out"].double()
    weights = st["weights"].double() if op == "weights" else None
    start = 0
    for s in range(S):
        n, length = new[s], total[s]
        pages = table[s, :-(-length // bs)].long().cuda()

        def gather(cache):
            x = cache[pages].double()
            x = x.transpose(1, 2) if case["layout"] == "hnd" else x
            return x.reshape(-1, Hk, D)[:length].transpose(0, 1)

        k = gather(st["k_cache"])
        q = st["q"][start:start + n].double().view(n, Hk, G, D).permute(1, 0, 2, 3).reshape(Hk, n * G, D)
        w = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(D)
        if op == "tree":
            words = st["mask"][start:start + n].tolist()
            drafted = torch.tensor([[(words[i][j // 64] >> (j % 64)) & 1 for j in range(n)]
                                    for i in range(n)], dtype=torch.bool).view(n, n).cuda()
        else:
            drafted = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
        hidden = ~drafted.repeat_interleave(G, 0)
        w[:, :, length - n:] = w[:, :, length - n:].masked_fill(hidden, -math.inf)
        if st["sink"] is not None:
            sink = st["sink"].double().view(Hk, 1, G).expand(Hk, n, G).reshape(Hk, n * G, 1)
            w = torch.softmax(torch.cat([w, sink], -1), -1)[..., :-1]
        else:
            w = torch.softmax(w, -1)
        if op == "tree" or case["output"]:
            o = torch.matmul(w, gather(st["v_cache"])).view(Hk, n, G, D).permute(1, 0, 2, 3)
            out[start:start + n] = o.reshape(n, H, D)
        if op == "weights":
            got = w.sum(1)
            at = torch.arange(length, device="cuda")
            to = (pages[at // bs].expand(Hk, length),
                  torch.arange(Hk, device="cuda")[:, None].expand(Hk, length),
                  (at % bs).expand(Hk, length))
            if case["accumulate"]:
                got[:, :length - n] += weights[to][:, :length - n]
            weights[to] = got
        start += n
    if op == "tree":
        return {"out": out}
    return {"out": out if case["output"] else None, "weights": weights}

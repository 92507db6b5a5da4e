"""Cases and plain forms of the operators around a shared prompt prefix.

Three operators of a serving step, in the order in which the step calls them:

  tables  the block table rows and the slot map of a step's new tokens, from the request lengths
          and a list of free pages (pa_block_tables)
  write   the new tokens' K and V rows into the slots of that map (pa_cache_write_slots)
  attend  attention for a batch whose requests share long prefixes group by group, each prefix's
          keys and values read once for its whole group (pa_forward_shared_prefix)

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
        # one decode step of a batch of 64: one slot a request, a fresh page for a few of them
        dict(name="tables_decode_b64", op="tables", requests=64, new=1, cached=8192, block=16,
             pad=0, short=False, lens=11),
        # a step that admits prompts, padded to a captured size, and whose free pages run out
        dict(name="tables_prompts_short", op="tables", requests=37, new=4096, cached=1000, block=16,
             pad=333, short=True, lens=12),
        # a whole node's prompts at once
        dict(name="tables_prompts_large", op="tables", requests=512, new=2048, cached=8192,
             block=64, pad=0, short=False, lens=13),
        # the rows of one decode step, sliced out of a fused projection, three padded rows
        dict(name="write_decode_b64", op="write", tokens=64, kv_heads=8, dim=128, block=16,
             dtype="bf16", layout="nhd", fused=32, pad=3, lens=21),
        # fp32 rows, head-major pages, an odd number of tokens
        dict(name="write_extend_f32_hnd", op="write", tokens=4099, kv_heads=4, dim=64, block=64,
             dtype="f32", layout="hnd", fused=0, pad=0, lens=22),
        # a large prompt chunk of a fused projection
        dict(name="write_prompts_large", op="write", tokens=32749, kv_heads=8, dim=128, block=16,
             dtype="bf16", layout="nhd", fused=32, pad=19, lens=23),
        # four samples of one short prompt: the smallest call, where latency counts
        dict(name="attend_four_samples", op="attend", heads=32, kv_heads=8, dim=128, block=16,
             layout="nhd", sinks=False, groups=1, requests=4, prefix=1008, suffix=150, new=1,
             lens=31),
        # a decode batch of 64 under one system prompt
        dict(name="attend_decode_b64", op="attend", heads=32, kv_heads=8, dim=128, block=16,
             layout="nhd", sinks=False, groups=1, requests=64, prefix=8192, suffix=2048, new=1,
             lens=32),
        # several prompts, each sampled a few times, some of them short, sinks on
        dict(name="attend_many_prompts", op="attend", heads=64, kv_heads=4, dim=128, block=16,
             layout="nhd", sinks=True, groups=12, requests=90, prefix=6000, suffix=700, new=1,
             lens=33),
        # questions and decodes on one shared document: extends of many tokens, 64-wide heads
        dict(name="attend_questions", op="attend", heads=16, kv_heads=4, dim=64, block=64,
             layout="hnd", sinks=False, groups=2, requests=24, prefix=8192, suffix=900, new=512,
             lens=34),
        # a very long document, one KV head, few rows: the prefix has to be split
        dict(name="attend_long_document", op="attend", heads=8, kv_heads=1, dim=128, block=64,
             layout="nhd", sinks=False, groups=1, requests=48, prefix=131072, suffix=1500, new=1,
             lens=35),
        # a large batch on a long prompt: many rows for every key
        dict(name="attend_large_batch", op="attend", heads=64, kv_heads=4, dim=128, block=64,
             layout="nhd", sinks=False, groups=1, requests=256, prefix=32768, suffix=2048, new=1,
             lens=36),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["tables", "write", "attend", "attend"])
    if op == "tables":
        return dict(op=op, requests=_log_int(rng, 1, 512), new=rng.choice([1, _log_int(rng, 2, 2048)]),
                    cached=_log_int(rng, 1, 8192), block=rng.choice([16, 32, 64, 128]),
                    pad=rng.choice([0, rng.randrange(1, 400)]), short=rng.random() < 0.3,
                    lens=rng.randrange(1 << 30))
    if op == "write":
        tokens = _log_int(rng, 1, 32000)
        return dict(op=op, tokens=tokens, kv_heads=rng.choice([1, 2, 4, 8]),
                    dim=rng.choice([64, 128]), block=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), layout=rng.choice(["nhd", "hnd"]),
                    fused=rng.choice([0, 8, 32]), pad=rng.randrange(min(tokens, 20)),
                    lens=rng.randrange(1 << 30))
    heads, kv_heads, dim = rng.choice([(32, 8, 128), (64, 4, 128), (8, 1, 128), (16, 4, 64),
                                       (32, 8, 64), (8, 8, 128)])
    block = rng.choice([16, 16, 32, 64, 128])
    new = rng.choice([1, 1, _log_int(rng, 2, 400)])
    requests = _log_int(rng, 1, 200 if new == 1 else 20)
    groups = min(requests, rng.choice([1, 1, _log_int(rng, 2, 12)]))
    prefix = _log_int(rng, block, 32768 if groups == 1 and new == 1 else 8192) // block * block
    return dict(op="attend", heads=heads, kv_heads=kv_heads, dim=dim, block=block,
                layout=rng.choice(["nhd", "hnd"]), sinks=rng.random() < 0.3, groups=groups,
                requests=requests, prefix=max(prefix, block), suffix=_log_int(rng, 1, 2000),
                new=new, lens=rng.randrange(1 << 30))


# ---------------------------------------------------------------------------
# lengths: from the case alone
# ---------------------------------------------------------------------------

def _table_lens(case):
    """(new tokens, length with them) of every request."""
    rng = random.Random(case["lens"])
    new, total = [], []
    for _ in range(case["requests"]):
        n = 1 if case["new"] == 1 else rng.randint(0, case["new"])
        new.append(n)
        total.append(n + rng.randint(0, case["cached"]))
    return new, total


def _new_pages(case):
    bs = case["block"]
    return sum(-(-t // bs) - -(-(t - n) // bs) for n, t in zip(*_table_lens(case)))


def _attend_lens(case):
    """Group bounds, group prefixes, and each request's new tokens and own length behind the prefix."""
    rng = random.Random(case["lens"])
    S, G, bs = case["requests"], case["groups"], case["block"]
    bounds = [0] + sorted(rng.sample(range(1, S), G - 1)) + [S]
    prefix = [case["prefix"] // bs * bs]
    for _ in range(G - 1):
        prefix.append(0 if rng.random() < 0.15 else rng.randint(1, case["prefix"] // bs) * bs)
    new, own_len = [], []
    for _ in range(S):
        n = 1 if case["new"] == 1 or rng.random() < 0.5 else rng.randint(1, case["new"])
        new.append(n)
        own_len.append(rng.randint(n, max(n, case["suffix"])))
    return bounds, prefix, new, own_len


def work(case):
    if case["op"] == "tables":
        new, total = _table_lens(case)
        T, pages = sum(new) + case["pad"], _new_pages(case)
        # in: lengths, starts, a free page each; out: table entries, slots, positions, the count
        return {"bytes": 8 * len(new) + 4 + 8 * pages + 12 * T + 8, "flops": 0}
    if case["op"] == "write":
        row = case["kv_heads"] * case["dim"] * (2 if case["dtype"] == "bf16" else 4)
        return {"bytes": 4 * row * (case["tokens"] - case["pad"]) + 8 * case["tokens"], "flops": 0}
    bounds, prefix, new, own_len = _attend_lens(case)
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    kv = sum(prefix) + sum(own_len)
    pairs = 0
    for g, p in enumerate(prefix):
        for s in range(bounds[g], bounds[g + 1]):
            n, c = new[s], own_len[s]
            pairs += n * p + n * (c - n) + n * (n + 1) // 2
    return {"bytes": 4 * kv * Hk * D + 4 * sum(new) * H * D, "flops": 4 * pairs * H * D}


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    bs = case["block"]
    if case["op"] == "tables":
        new, total = _table_lens(case)
        S, T, pages = len(new), sum(new) + case["pad"], _new_pages(case)
        mbps = max(-(-max(total) // bs), 1) + 3
        held = [-(-(t - n) // bs) for n, t in zip(new, total)]
        pool = sum(held) + pages + 7
        perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((S, mbps), -1, dtype=torch.int32, device="cuda")
        first = _i32(_cum(held)[:-1])
        col = torch.arange(mbps, device="cuda", dtype=torch.int32)
        use = col[None, :] < _i32(held)[:, None]
        where = (first[:, None] + col[None, :]).clamp_max(pool - 1)
        table = torch.where(use, perm[where.long()], table)
        num_free = pages // 2 if case["short"] else pages + 5
        st.update(table=table, seq_lens=_i32(total), starts=_i32(_cum(new)), num_blocks=pool,
                  free=torch.cat([perm[:2], perm[sum(held):sum(held) + num_free]]).contiguous(),
                  free_start=_i32([2]), free_end=_i32([0]), tokens=T,
                  slots=torch.empty(T, dtype=torch.int64, device="cuda"),
                  positions=torch.empty(T, dtype=torch.int32, device="cuda"))
        return st
    if case["op"] == "write":
        T, Hk, D, dt = case["tokens"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
        n = T - case["pad"]
        blocks = -(-T // bs) + max(2, T // (8 * bs))
        rows = torch.randn((T, case["fused"] + 2 * Hk, D), generator=gen, device="cuda",
                           dtype=torch.float32).to(dt)
        if case["fused"] == 0:  # two tensors of their own
            k, v = rows[:, :Hk].contiguous(), rows[:, Hk:].contiguous()
        else:  # K and V behind the query heads of one projection
            k, v = rows[:, case["fused"]:case["fused"] + Hk], rows[:, case["fused"] + Hk:]
        shape = (blocks, bs, Hk, D) if case["layout"] == "nhd" else (blocks, Hk, bs, D)
        # runs of positions on scattered pages, as a step's requests have them
        page = torch.randperm(blocks, generator=gen, device="cuda")
        at = torch.arange(T, device="cuda") + int(torch.randint(bs, (1,), generator=gen, device="cuda"))
        slots = page[(at // bs) % blocks] * bs + at % bs
        slots[n:] = -1
        st.update(k=k, v=v, slots=slots, real=n, k_cache=torch.zeros(shape, dtype=dt, device="cuda"),
                  v_cache=torch.zeros(shape, dtype=dt, device="cuda"))
        return st
    bounds, prefix, new, own_len = _attend_lens(case)
    H, Hk, D, S = case["heads"], case["kv_heads"], case["dim"], case["requests"]
    T = sum(new)
    of = [g for g in range(case["groups"]) for _ in range(bounds[g], bounds[g + 1])]
    total = [prefix[of[s]] + own_len[s] for s in range(S)]
    mbps = max(-(-t // bs) for t in total)
    own_pages = [-(-c // bs) for c in own_len]
    used = sum(prefix) // bs + sum(own_pages)
    pool = used + max(1, used // 10)
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32).cpu()
    table, at = torch.full((S, mbps), -1, dtype=torch.int32), 0
    for g, p in enumerate(prefix):  # the shared pages stand in the group's first row alone
        table[bounds[g], :p // bs] = perm[at:at + p // bs]
        at += p // bs
    for s in range(S):
        p = prefix[of[s]] // bs
        table[s, p:p + own_pages[s]] = perm[at:at + own_pages[s]]
        at += own_pages[s]
    shape = (pool, bs, Hk, D) if case["layout"] == "nhd" else (pool, Hk, bs, D)
    # scores of a few units' spread, so that some keys carry most of a row's weight
    q = (1.5 * torch.randn((T, H, D), generator=gen, device="cuda")).to(torch.bfloat16)
    k = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    sinks = torch.randn(H, generator=gen, device="cuda") if case["sinks"] else None
    st.update(q=q, k_cache=k, v_cache=v, table=table.cuda(), seq_lens=_i32(total),
              starts=_i32(_cum(new)), group_starts=_i32(bounds), prefix_lens=_i32(prefix),
              sink=sinks, scale=1.0 / math.sqrt(D), out=torch.empty_like(q),
              # what a scheduler knows of the batch it built
              max_seq=max(total), max_prefix=max(prefix), max_new=max(new), max_own=max(own_len),
              max_rows=max(sum(new[bounds[g]:bounds[g + 1]]) for g in range(case["groups"])))
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(st):
    if st["op"] == "tables":
        return _run_tables(st) if own else _plain_tables(st)
    if st["op"] == "write":
        return _run_write(st) if own else _plain_write(st)
    return _run_attend(st) if own else _plain_attend(st)


def _run_tables(st):
    from paged_kv_attention_16_gb300 import pa
    pa.pa_block_tables(st["seq_lens"], st["starts"], st["table"], st["slots"], st["block"],
                       num_blocks=st["num_blocks"], free_pages=st["free"],
                       free_start=st["free_start"], free_end=st["free_end"],
                       positions=st["positions"])
    return {"table": st["table"], "slots": st["slots"], "positions": st["positions"],
            "free_end": st["free_end"]}


def _run_write(st):
    from paged_kv_attention_16_gb300 import pa
    pa.pa_cache_write_slots(st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"],
                            st["block"], kv_layout=st["layout"])
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _run_attend(st):
    from paged_kv_attention_16_gb300 import pa
    pa.pa_forward_shared_prefix(st["q"], st["k_cache"], st["v_cache"], st["table"], st["seq_lens"],
                                st["starts"], st["group_starts"], st["prefix_lens"], st["heads"],
                                st["kv_heads"], st["dim"], st["block"], st["scale"], st["out"],
                                max_seq_len=st["max_seq"], max_prefix_len=st["max_prefix"],
                                sinks=st["sink"], kv_layout=st["layout"],
                                max_query_len=st["max_new"])
    return {"out": st["out"]}


def _plain_tables(st):
    bs, T, table = st["block"], st["tokens"], st["table"]
    starts, total = st["starts"].long(), st["seq_lens"].long()
    q_len = starts[1:] - starts[:-1]
    held = (total - q_len + bs - 1) // bs
    need = (total + bs - 1) // bs - held
    begin = torch.cumsum(need, 0) - need
    avail = st["free"].shape[0] - st["free_start"].long()
    served = (need == 0) | (begin + need <= avail)
    taken = torch.where(served & (need > 0), begin + need, 0).amax()
    tok = torch.arange(T, device=table.device)
    real = tok < starts[-1]
    s = torch.searchsorted(starts[1:].contiguous(), tok, right=True).clamp_max(len(total) - 1)
    pos = total[s] - q_len[s] + tok - starts[s]
    page_at = pos // bs
    ok = real & served[s]
    fresh = ok & (page_at >= held[s])
    take = (st["free_start"].long() + begin[s] + page_at - held[s]).clamp(0, st["free"].shape[0] - 1)
    page_at = page_at.clamp(0, table.shape[1] - 1)
    page = torch.where(fresh, st["free"][take], table[s, page_at])
    table[s, page_at] = torch.where(fresh, page, table[s, page_at])
    slots = torch.where(ok, page.long() * bs + pos % bs, -1)
    positions = torch.where(real, pos, 0).to(torch.int32)
    return {"table": table, "slots": slots, "positions": positions,
            "free_end": (st["free_start"] + taken).to(torch.int32)}


def _plain_write(st):
    bs, n = st["block"], st["real"]
    page, at = st["slots"][:n] // bs, st["slots"][:n] % bs
    for cache, rows in ((st["k_cache"], st["k"]), (st["v_cache"], st["v"])):
        if st["layout"] == "nhd":
            cache[page, at] = rows[:n]
        else:
            cache[page, :, at] = rows[:n]
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _rows(cache, layout, pages, at):
    """fp32 rows [..., kv_heads, dim] at (page, slot) of every index."""
    pages = pages.clamp_min(0).long()
    return (cache[pages, at] if layout == "nhd" else cache[pages, :, at]).float()


def _partial(q, k, v, visible, scale):
    """Row maximum, weight sum and weighted values of queries [n, t, kv, g, d] on keys
    [n, p, kv, d]; visible [n, t, p]."""
    s = torch.einsum("ntkgd,npkd->nktgp", q, k).mul_(scale)
    s.masked_fill_(~visible[:, None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(m.clamp_min(torch.finfo(torch.float32).min)).exp_()
    l = s.sum(-1)
    o = torch.einsum("nktgp,npkd->ntkgd", s, v)
    return m[..., 0].permute(0, 2, 1, 3), l.permute(0, 2, 1, 3), o


def _plain_attend(st):
    q, bs, table, lay = st["q"], st["block"], st["table"], st["layout"]
    T, H, D = q.shape
    Hk = st["kv_heads"]
    dev = q.device
    starts, total = st["starts"].long(), st["seq_lens"].long()
    bounds, plen = st["group_starts"].long(), st["prefix_lens"].long()
    q32 = q.float().view(T, Hk, H // Hk, D)
    tok = torch.arange(T, device=dev)
    s_of = torch.searchsorted(starts[1:].contiguous(), tok, right=True)
    g_of_s = torch.searchsorted(bounds[1:].contiguous(), torch.arange(len(total), device=dev), right=True)
    g_of = g_of_s[s_of]
    # every group's rows against its prefix
    row0, row1 = starts[bounds[:-1]], starts[bounds[1:]]
    at = row0[:, None] + torch.arange(st["max_rows"], device=dev)
    pos = torch.arange(max(st["max_prefix"], 1), device=dev)
    page = table[bounds[:-1]][:, (pos // bs)]
    seen = (pos[None, None, :] < plen[:, None, None]) & (at < row1[:, None])[:, :, None]
    slot = (pos % bs).expand(page.shape)
    m, l, o = _partial(q32[at.clamp_max(T - 1)], _rows(st["k_cache"], lay, page, slot),
                       _rows(st["v_cache"], lay, page, slot), seen, st["scale"])
    local = tok - row0[g_of]
    m_p, l_p, o_p = m[g_of, local], l[g_of, local], o[g_of, local]
    del m, l, o
    # every request's rows against its own positions
    q_len = starts[1:] - starts[:-1]
    own_len = total - plen[g_of_s]
    at = starts[:-1, None] + torch.arange(st["max_new"], device=dev)
    i = torch.arange(st["max_new"], device=dev)
    j = torch.arange(st["max_own"], device=dev)
    pos = plen[g_of_s][:, None] + j
    page = table.gather(1, (pos // bs).clamp_max(table.shape[1] - 1))
    seen = j[None, None, :] <= (own_len - q_len)[:, None, None] + i[None, :, None]
    seen = seen & (j[None, None, :] < own_len[:, None, None])
    m, l, o = _partial(q32[at.clamp_max(T - 1)], _rows(st["k_cache"], lay, page, pos % bs),
                       _rows(st["v_cache"], lay, page, pos % bs), seen, st["scale"])
    local = tok - starts[s_of]
    m_o, l_o, o_o = m[s_of, local], l[s_of, local], o[s_of, local]
    top = torch.maximum(m_p, m_o)
    if st["sink"] is not None:
        sink = st["sink"].view(Hk, H // Hk)
        top = torch.maximum(top, sink)
    a, b = torch.exp(m_p - top), torch.exp(m_o - top)
    den = a * l_p + b * l_o
    if st["sink"] is not None:
        den = den + torch.exp(sink - top)
    out = (a[..., None] * o_p + b[..., None] * o_o) / den[..., None]
    return {"out": out.reshape(T, H, D).to(q.dtype)}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers: equal or not
    if case["op"] == "write":
        st = prepare(case, seed)
        out = {}
        for name in ("k", "v"):
            flat = st[name + "_cache"].double()
            if case["layout"] == "hnd":
                flat = flat.transpose(1, 2).contiguous()
            shape = flat.shape
            flat = flat.reshape(-1, *shape[2:])
            flat.index_copy_(0, st["slots"][:st["real"]], st[name][:st["real"]].double())
            flat = flat.view(shape)
            out[name + "_cache"] = flat.transpose(1, 2).contiguous() if case["layout"] == "hnd" else flat
        return out
    st = prepare(case, seed)
    bounds, prefix, new, own_len = _attend_lens(case)
    bs, Hk, G, D = case["block"], case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    table, start = st["table"].tolist(), 0
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")

    def gather(cache, pages):
        x = cache[torch.tensor(pages, device="cuda")].double()
        x = x if case["layout"] == "nhd" else x.transpose(1, 2)
        return x.reshape(-1, Hk, D).transpose(0, 1)

    for g, p in enumerate(prefix):
        shared = table[bounds[g]][:p // bs]
        for s in range(bounds[g], bounds[g + 1]):
            n, length = new[s], p + own_len[s]
            pages = shared + table[s][p // bs:-(-length // bs)]
            k, v = gather(st["k_cache"], pages)[:, :length], gather(st["v_cache"], pages)[:, :length]
            q = st["q"][start:start + n].double().view(n, Hk, G, D).permute(1, 0, 2, 3).reshape(Hk, n * G, D)
            w = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(D)
            last = torch.arange(length - n, length, device="cuda").repeat_interleave(G)
            w.masked_fill_(torch.arange(length, device="cuda")[None, :] > last[:, None], -math.inf)
            if st["sink"] is not None:
                sink = st["sink"].double().view(Hk, 1, G).expand(Hk, n, G).reshape(Hk, n * G, 1)
                w = torch.softmax(torch.cat([w, sink], -1), -1)[..., :-1]
            else:
                w = torch.softmax(w, -1)
            o = torch.matmul(w, v).view(Hk, n, G, D).permute(1, 0, 2, 3)
            out[start:start + n] = o.reshape(n, Hk * G, D)
            start += n
    return {"out": out}

"""The operators that the library adds beside plain paged decode, as cases to
measure: decode attention over a prefix that a batch shares, decode attention
that accumulates each cached token's attention weight, and the eviction of
tokens from a cache by that weight.

`own` false: the plain form, elementary torch operations in 32 bits on the
pages as they are stored.  `own` true: the library's calls.
"""
import math
import random

import torch

own = False

PAGE = 16
LOG_RANGE = 10  # ranges wider than this factor are drawn over their logarithm
# token t of an FP8 V page sits in slot RHO[t] of its row
RHO = [0, 1, 4, 5, 8, 9, 12, 13, 2, 3, 6, 7, 10, 11, 14, 15]
TYPES = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0), "bf16": (torch.bfloat16, None)}
NAMES = {"e4m3": "fp8_e4m3", "e5m2": "fp8_e5m2", "bf16": "bf16"}


# ---------------------------------------------------------------- the cases ---
def shared(name, batch, groups, prefix, lo, hi, kv_heads, group, head_dim, dtype):
    """A batch in `groups` groups, each after a prefix of its own (`prefix`
    tokens the longest), with lo .. hi tokens of its own per sequence."""
    return dict(name=name, kind="shared", batch=batch, groups=groups, prefix=prefix, lo=lo, hi=hi, kv_heads=kv_heads,
                group=group, head_dim=head_dim, dtype=dtype, per_token=False)


def weights(name, batch, lo, hi, kv_heads, group, head_dim, dtype, per_token=False, decay=1.0, window=-1):
    """One decode step over lo .. hi cached tokens per sequence."""
    return dict(name=name, kind="weights", batch=batch, lo=lo, hi=hi, kv_heads=kv_heads, group=group,
                head_dim=head_dim, dtype=dtype, per_token=per_token, decay=decay, window=window)


def evict(name, batch, lo, hi, keep, kv_heads, head_dim, dtype, per_token=False, sink=4, recent=64):
    """lo .. hi cached tokens per sequence cut to `keep` of them."""
    return dict(name=name, kind="evict", batch=batch, lo=lo, hi=hi, keep=keep, kv_heads=kv_heads, group=1,
                head_dim=head_dim, dtype=dtype, per_token=per_token, sink=sink, recent=recent)


def listed():
    return [
        # two requests right after one short prompt: latency
        shared("shared_tiny", 2, 1, 512, 1, 16, 1, 4, 64, "e4m3"),
        # a chat service's system prompt before 32 conversations
        shared("shared_chat_8k", 32, 1, 8192, 16, 1024, 8, 4, 128, "e4m3"),
        # many samples and questions over one long document, its length no multiple of a page
        shared("shared_document_32k", 128, 1, 32763, 128, 2048, 8, 4, 128, "e4m3"),
        # three prompts served in one batch, the other FP8 format, the wide head group
        shared("shared_three_prompts", 48, 3, 16384, 1, 777, 8, 8, 64, "e5m2"),
        # one short request
        weights("weights_tiny", 1, 512, 512, 1, 4, 64, "e4m3"),
        # eight requests of about 20K tokens
        weights("weights_batch8_20k", 8, 16384, 24576, 8, 4, 128, "e4m3"),
        # one request of 128K tokens
        weights("weights_128k", 1, 131072, 131072, 8, 4, 128, "e4m3", decay=0.99),
        # an unquantized layer with the wide head group
        weights("weights_bf16", 8, 1000, 4096, 8, 8, 64, "bf16"),
        # one short request cut to half
        evict("evict_tiny", 1, 512, 512, 256, 1, 64, "e4m3", recent=32),
        # eight requests of about 20K tokens cut to 8K
        evict("evict_batch8_20k", 8, 16384, 24576, 8192, 8, 128, "e4m3", recent=512),
        # one request of 128K tokens cut to an eighth: few tokens of a page survive
        evict("evict_128k", 1, 131072, 131072, 16384, 8, 128, "e4m3", recent=1024),
        # a light trim of a per-token-scaled cache
        evict("evict_trim_per_token", 8, 5000, 8192, 4999, 8, 64, "e4m3", per_token=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) if hi >= LOG_RANGE * lo else rng.randint(lo, hi)


def draw(rng):
    kind = rng.choice(["shared", "weights", "evict"])
    heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if kind == "shared":
        batch = _log(rng, 2, 128)
        hi = _log(rng, 1, 1500)
        return {k: v for k, v in shared("", batch, rng.randint(1, min(4, batch)), _log(rng, 100, 32000), rng.randint(0, hi), hi, heads,
                                        rng.randint(1, 4 if dim == 128 else 8), dim, rng.choice(["e4m3", "e5m2"])).items() if k != "name"}
    hi = _log(rng, 100, 60000)
    batch = _log(rng, 1, max(1, min(16, 131072 // hi)))
    lo = rng.randint(max(1, hi // 2), hi)
    dtype = rng.choice(["e4m3", "e4m3", "e5m2", "bf16"])
    per_token = dtype != "bf16" and rng.random() < 0.3
    if kind == "weights":
        return {k: v for k, v in weights("", batch, lo, hi, heads, rng.randint(1, 8), dim, dtype, per_token, rng.choice([1.0, 0.95]),
                                         rng.choice([-1, -1, rng.randint(1, hi)])).items() if k != "name"}
    keep = _log(rng, max(1, hi // 16), hi)
    return {k: v for k, v in evict("", batch, lo, hi, keep, heads, dim, dtype, per_token, rng.randint(0, 8), rng.randint(0, max(1, keep // 4))).items()
            if k != "name"}


def _lengths(case, n, lo, hi, what):
    r = random.Random("%s %d %d %d" % (what, n, lo, hi))
    return [r.randint(lo, hi) for _ in range(n)]


def _plan(case):
    """The lengths of a case: they are the case's, not the seed's."""
    seqs = _lengths(case, case["batch"], case["lo"], case["hi"], case["kind"])
    if case["kind"] != "shared":
        return seqs, [], []
    n = case["groups"]
    cuts = sorted(random.Random(n).sample(range(1, case["batch"]), n - 1))
    prefixes = [case["prefix"]] + _lengths(case, n - 1, case["prefix"] // 4, case["prefix"], "prefix")
    return seqs, prefixes, [0] + cuts + [case["batch"]]


def _pages(tokens):
    return -(-tokens // PAGE)


# ------------------------------------------------------------- page formats ---
def _row_order(row_bytes, device):
    """Chunk order of a K page as stored (its own inverse)."""
    n = row_bytes // 16
    order = []
    for t in range(PAGE):
        for j in range(n):
            order.append(t * n + (j ^ (t & 7) if n == 8 else j ^ ((t >> 1) & 3) if n == 4 else (j & 8) | ((j ^ t) & 7)))
    return torch.tensor(order, device=device)


def _bytes(x):
    return x.contiguous().view(torch.uint8)


def _k_page(k):
    """[..., 16, D] elements -> [..., page bytes]."""
    b = _bytes(k).flatten(-2)
    chunks = b.view(*b.shape[:-1], -1, 16)
    return chunks.index_select(-2, _row_order(b.shape[-1] // PAGE, b.device)).flatten(-2)


def _v_page(v):
    """[..., 16, D] elements -> [..., page bytes]: a row of token slots per dimension."""
    t = v.transpose(-1, -2)  # [..., D, 16]
    if v.element_size() == 1:
        back = torch.tensor([RHO.index(s) for s in range(PAGE)], device=v.device)
        return _bytes(t).index_select(-1, back).flatten(-2)
    t = t.unflatten(-1, (2, 8))
    swap = ((torch.arange(t.shape[-3], device=v.device) >> 2) & 1).bool()[:, None, None]
    return _bytes(torch.where(swap, t.flip(-2), t)).flatten(-3)


def _from_k_page(b, case):
    """[..., page bytes] -> [..., 16, D] elements."""
    size = TYPES[case["dtype"]][0].itemsize
    chunks = b.contiguous().unflatten(-1, (-1, 16)).index_select(-2, _row_order(case["head_dim"] * size, b.device))
    return chunks.flatten(-2).unflatten(-1, (PAGE, -1)).contiguous().view(TYPES[case["dtype"]][0])


def _from_v_page(b, case):
    dtype = TYPES[case["dtype"]][0]
    rows = b.contiguous().unflatten(-1, (case["head_dim"], -1))
    if dtype.itemsize == 1:
        return rows.index_select(-1, torch.tensor(RHO, device=b.device)).transpose(-1, -2).contiguous().view(dtype)
    t = rows.contiguous().view(dtype).unflatten(-1, (2, 8))
    swap = ((torch.arange(t.shape[-3], device=b.device) >> 2) & 1).bool()[:, None, None]
    return torch.where(swap, t.flip(-2), t).flatten(-2).transpose(-1, -2)


# ------------------------------------------------------------------- inputs ---
def _inputs(case, seed):
    """The logical contents: q, the pages' K and V as stored elements, scales, tables."""
    seqs, prefixes, starts = _plan(case)
    H, g, D, B = case["kv_heads"], case["group"], case["head_dim"], case["batch"]
    dtype, top = TYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    own_pages, pre_pages = [_pages(n) for n in seqs], [_pages(n) for n in prefixes]
    dst_pages = [_pages(min(n, case["keep"])) for n in seqs] if case["kind"] == "evict" else []
    used = sum(own_pages) + sum(pre_pages) + sum(dst_pages)
    blocks = used + used // 8 + 1
    order = torch.randperm(blocks, generator=gen, device="cuda").int()

    def table(counts, at):
        t = torch.zeros(len(counts), max(1, max(counts, default=1)), dtype=torch.int32)
        where = [(i, j) for i, c in enumerate(counts) for j in range(c)]
        if where:
            rows, cols = torch.tensor(where).T
            t[rows, cols] = torch.arange(at, at + len(where), dtype=torch.int32)
        t = t.cuda()
        return torch.where(torch.arange(t.shape[1], device="cuda")[None] < torch.tensor(counts, device="cuda")[:, None], order[t.long()], 0).int()

    own_table = table(own_pages, 0)
    pre_table = table(pre_pages, sum(own_pages)) if prefixes else None
    dst_table = table(dst_pages, sum(own_pages) + sum(pre_pages)) if dst_pages else None
    q = randn(B, H * g, D) * 1.2
    k, v = randn(blocks, H, PAGE, D), randn(blocks, H, PAGE, D)
    # the first token of a text draws weight from every query
    u = randn(H, D)
    q = (q + 0.5 * u.repeat_interleave(g, 0)).bfloat16()
    first = (pre_table if prefixes else own_table)[:, 0].long()
    k[first, :, 0] = 1.8 * u
    if dtype == torch.bfloat16:
        ks = vs = None
        k, v = k.bfloat16(), v.bfloat16()
    elif case["per_token"]:
        ks, vs = k.abs().amax(-1) / top, v.abs().amax(-1) / top  # [blocks, H, 16]
        k, v = (k / ks[..., None]).clamp(-top, top).to(dtype), (v / vs[..., None]).clamp(-top, top).to(dtype)
    else:
        ks, vs = ((a + 0.125 * torch.arange(H, device="cuda")) / top for a in (5.0, 4.5))
        k = (k / ks[:, None, None]).clamp(-top, top).to(dtype)
        v = (v / vs[:, None, None]).clamp(-top, top).to(dtype)
    d = dict(case=case, q=q, k=k, v=v, ks=ks, vs=vs, own_table=own_table, pre_table=pre_table, dst_table=dst_table, blocks=blocks,
             seqs=seqs, prefixes=prefixes, starts=starts, seq_lens=torch.tensor(seqs, dtype=torch.int32, device="cuda"))
    if prefixes:
        d["prefix_lens"] = torch.tensor(prefixes, dtype=torch.int32, device="cuda")
        d["group_starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    if case["kind"] != "shared":
        # what earlier steps have left: heavy tailed, and nothing yet for some tokens
        shape = (B, H, own_table.shape[1] * PAGE)
        w = torch.exp(1.5 * randn(*shape)) * (torch.rand(shape, generator=gen, device="cuda") > 0.1)
        w[..., 0] = 50.0
        d["weights"] = torch.where(torch.arange(shape[2], device="cuda") < d["seq_lens"][:, None, None], w, 0.0)
    if case["kind"] == "evict":
        cap = dst_table.shape[1] * PAGE
        d["keep"] = torch.tensor([min(n, case["keep"]) for n in seqs], dtype=torch.int32, device="cuda")
        d["dst_weights"] = torch.zeros(B, H, cap, device="cuda")
        d["kept"] = torch.zeros(B, H, cap, dtype=torch.int32, device="cuda")
        d["dst_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return d


def _tail(d):
    """The scale tail of each per-token V page, as bytes."""
    return _bytes(torch.cat([d["ks"], d["vs"]], -1))


def prepare(case, seed):
    """What a server holds before the step: the caches in the library's page
    format, tables, scales, the output and a workspace."""
    d = _inputs(case, seed)
    d["k_cache"] = _k_page(d.pop("k"))
    v = _v_page(d.pop("v"))
    d["v_cache"] = torch.cat([v, _tail(d)], -1).contiguous() if case["per_token"] else v
    d["out"] = torch.zeros_like(d["q"])
    d["workspace"] = None
    return d


# --------------------------------------------------------------- plain form ---
def _gathered(d, table):
    """K and V of a table's pages in 32 bits: [N, H, tokens, D]."""
    case = d["case"]
    at = table.long()
    page = PAGE * case["head_dim"] * TYPES[case["dtype"]][0].itemsize
    both = []
    for pages, back, scale, lo in ((d["k_cache"][at], _from_k_page, d["ks"], 0), (d["v_cache"][at], _from_v_page, d["vs"], 1)):
        x = back(pages[..., :page], case).float()  # [N, pages, H, 16, D]
        if case["per_token"]:
            tail = d["v_cache"][at][..., page:].contiguous().view(torch.float32)
            x = x * tail[..., lo * PAGE:(lo + 1) * PAGE, None]
        elif scale is not None:
            x = x * scale[:, None, None]
        both.append(x.transpose(1, 2).flatten(2, 3))
    return both


def _scores(q, k, lens, lo=None):
    """[N, H, rows, tokens] scores; -inf outside [lo, lens)."""
    at = torch.arange(k.shape[2], device=k.device)
    dead = at >= lens[:, None, None, None]
    if lo is not None:
        dead = dead | (at < lo[:, None, None, None])
    s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    return torch.where(dead, float("-inf"), s)


def _parts(s, v):
    """Maximum, sum and weighted V of one piece of a softmax; an empty row has a sum of zero."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    return m, p.sum(-1, keepdim=True), torch.matmul(p, v)


def _shared_plain(d):
    case = d["case"]
    B, H, g, D = case["batch"], case["kv_heads"], case["group"], case["head_dim"]
    q = d["q"].float().view(B, H, g, D)
    seq = torch.arange(B, device=q.device)
    group = torch.searchsorted(d["group_starts"][1:].long(), seq, right=True)
    place = seq - d["group_starts"].long()[group]
    most = max(b - a for a, b in zip(d["starts"], d["starts"][1:]))
    rows = torch.zeros(case["groups"], most, dtype=torch.long, device=q.device)
    rows[group, place] = seq
    k, v = _gathered(d, d["pre_table"])
    qg = q[rows].transpose(1, 2).flatten(2, 3)  # [G, H, most * g, D]
    first = [x.unflatten(2, (most, g)).transpose(1, 2)[group, place] for x in _parts(_scores(qg, k, d["prefix_lens"]), v)]
    k, v = _gathered(d, d["own_table"])
    second = _parts(_scores(q, k, d["seq_lens"]), v)
    m = torch.maximum(first[0], second[0])
    m = torch.where(m == float("-inf"), 0.0, m)
    a, b = torch.exp(first[0] - m), torch.exp(second[0] - m)
    total = a * first[1] + b * second[1]
    o = (a * first[2] + b * second[2]) / torch.where(total > 0, total, 1.0)
    d["out"].copy_(o.reshape(B, H * g, D))
    return d["out"]


def _weights_plain(d):
    case = d["case"]
    B, H, g, D = case["batch"], case["kv_heads"], case["group"], case["head_dim"]
    k, v = _gathered(d, d["own_table"])
    lo = (d["seq_lens"] - case["window"]).clamp(min=0) if case["window"] > 0 else None
    m, l, o = _parts(s := _scores(d["q"].float().view(B, H, g, D), k, d["seq_lens"], lo), v)
    l = torch.where(l > 0, l, 1.0)
    d["out"].copy_((o / l).reshape(B, H * g, D))
    p = torch.exp(s - torch.where(m == float("-inf"), 0.0, m)) / l
    live = torch.arange(k.shape[2], device=k.device) < d["seq_lens"][:, None, None]
    w = d["weights"]
    w.copy_(torch.where(live, case["decay"] * w + p.sum(2), w))
    return {"out": d["out"], "weights": w}


def _evict_plain(d):
    case = d["case"]
    w, L, n = d["weights"], d["seq_lens"].long(), d["keep"].long()
    n = torch.minimum(n, L)
    s = torch.clamp(n, max=case["sink"])
    r = torch.minimum(n - s, torch.full_like(n, case["recent"]))
    at = torch.arange(w.shape[-1], device=w.device)
    kept_anyway = (at < s[:, None]) | ((at >= (L - r)[:, None]) & (at < L[:, None]))
    score = torch.where(kept_anyway[:, None], float("inf"), torch.where((at < L[:, None])[:, None], w, float("-inf")))
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices  # ties: the lowest position first
    chosen = torch.zeros_like(w, dtype=torch.bool).scatter_(-1, best, (at < n[:, None])[:, None].expand_as(best))
    cap = d["kept"].shape[-1]
    source = torch.sort(torch.where(chosen, at, w.shape[-1]), dim=-1).values[..., :cap]
    live = torch.arange(cap, device=w.device) < n[:, None, None]
    source = torch.where(live, source, 0)
    d["kept"].copy_(torch.where(live, source.int(), d["kept"]))
    d["dst_weights"].copy_(torch.where(live, w.gather(-1, source), 0.0))
    d["dst_lens"].copy_(n)
    src, dst, page = d["own_table"].long(), d["dst_table"].long(), PAGE * case["head_dim"] * TYPES[case["dtype"]][0].itemsize
    put = torch.arange(dst.shape[1], device=w.device) < ((n + PAGE - 1) // PAGE)[:, None]

    def moved(x, old):  # tokens' values [B, pages, H, 16, ...]; the destination's unfilled slots stay
        x, old = (t.transpose(1, 2).flatten(2, 3) for t in (x, old))
        x = x.gather(2, source.view(*source.shape, *[1] * (x.dim() - 3)).expand(*source.shape, *x.shape[3:]))
        x = torch.where(live.view(*live.shape, *[1] * (x.dim() - 3)), x, old)
        return x.unflatten(2, (-1, PAGE)).transpose(1, 2)

    for name, back, forth in (("k_cache", _from_k_page, _k_page), ("v_cache", _from_v_page, _v_page)):
        cache = d[name]
        old, new = cache[src], cache[dst]
        kind = torch.uint8 if page == PAGE * case["head_dim"] else torch.int16
        x = forth(moved(back(old[..., :page], case).contiguous().view(kind), back(new[..., :page], case).contiguous().view(kind)))
        if case["per_token"] and name == "v_cache":
            tails = [t[..., page:].contiguous().view(torch.float32).unflatten(-1, (2, PAGE)).transpose(-1, -2) for t in (old, new)]
            x = torch.cat([x, _bytes(moved(*tails).transpose(-1, -2)).flatten(-2)], -1)
        cache[dst[put]] = x[put]


def _evicted(d):
    """The state after an eviction, its codes as the values they stand for."""
    case = d["case"]
    dtype, page = TYPES[case["dtype"]][0], PAGE * case["head_dim"]
    found = {"kept": d["kept"], "weights": d["dst_weights"], "lens": d["dst_lens"], "k": d["k_cache"].view(dtype)}
    if not case["per_token"]:
        return {**found, "v": d["v_cache"].view(dtype)}
    return {**found, "v": d["v_cache"][..., :page].view(dtype), "scales": d["v_cache"][..., page:].view(torch.float32)}


# ---------------------------------------------------------------------- run ---
def _own_workspace(d, size):
    """A program keeps its workspace from step to step."""
    if d["workspace"] is None:
        d["workspace"] = torch.empty(max(16, size()), dtype=torch.uint8, device="cuda")
    return d["workspace"]


def run(d):
    case = d["case"]
    if own:
        import fp8_kv_cache_reshape_gb300 as kvq

        B, H, D = case["batch"], case["kv_heads"], case["head_dim"]
        Hq, name = H * case["group"], NAMES[case["dtype"]]
        if case["kind"] == "shared":
            ws = _own_workspace(d, lambda: kvq.kvq_shared_prefix_workspace_size(
                B, case["groups"], Hq, H, D, d["pre_table"].shape[1], d["own_table"].shape[1]))
            return kvq.kvq_paged_decode_attention_shared_prefix(
                d["q"], d["k_cache"], d["v_cache"], d["ks"], d["vs"], d["pre_table"], d["prefix_lens"], d["group_starts"],
                d["own_table"], d["seq_lens"], d["out"], cache_dtype=name, workspace=ws)
        if case["kind"] == "weights":
            ws = _own_workspace(d, lambda: kvq.kvq_decode_weights_workspace_size(
                B, Hq, H, D, d["own_table"].shape[1], window=case["window"]))
            scales = (None, None) if case["per_token"] else (d["ks"], d["vs"])
            kvq.kvq_paged_decode_attention_weights(
                d["q"], d["k_cache"], d["v_cache"], *scales, d["own_table"], d["seq_lens"], d["out"], d["weights"],
                decay=case["decay"], window=case["window"], cache_dtype=name, per_token=case["per_token"], workspace=ws)
            return {"out": d["out"], "weights": d["weights"]}
        kvq.kvq_evict_tokens(
            d["weights"], d["k_cache"], d["v_cache"], d["own_table"], d["seq_lens"], d["keep"], d["dst_table"], d["dst_weights"],
            d["dst_lens"], d["kept"], head_dim=D, sink=case["sink"], recent=case["recent"], cache_dtype=name,
            per_token=case["per_token"])
        return _evicted(d)
    if case["kind"] == "shared":
        return _shared_plain(d)
    if case["kind"] == "weights":
        return _weights_plain(d)
    _evict_plain(d)
    return _evicted(d)


# --------------------------------------------------------------------- work ---
def work(case):
    seqs, prefixes, starts = _plan(case)
    H, g, D, B = case["kv_heads"], case["group"], case["head_dim"], case["batch"]
    token = 2 * D * TYPES[case["dtype"]][0].itemsize + (8 if case["per_token"] else 0)  # K and V of one head
    rows = 2 * B * H * g * D * 2  # q and the output
    if case["kind"] == "shared":
        keys = sum(seqs) + sum(n * (b - a) for n, a, b in zip(prefixes, starts, starts[1:]))
        return {"bytes": (sum(seqs) + sum(prefixes)) * H * token + rows, "flops": 4 * D * H * g * keys}
    if case["kind"] == "weights":
        seen = [min(n, case["window"]) if case["window"] > 0 else n for n in seqs]
        # where nothing decays, a token that is not attended to keeps its weight
        touched = seqs if case["decay"] != 1.0 else seen
        return {"bytes": sum(seen) * H * token + 8 * H * sum(touched) + rows, "flops": 4 * D * H * g * sum(seen)}
    kept = [min(n, case["keep"]) for n in seqs]
    # the weights once, the kept tokens once in and once out, their positions and weights out
    return {"bytes": H * (4 * sum(seqs) + sum(kept) * (2 * token + 8)), "flops": 0}


# -------------------------------------------------------------------- exact ---
def _softmax64(q, k, v):
    """Attention of q [rows, D] over k, v [tokens, D] in 64 bits: (probabilities, output)."""
    s = q @ k.T / math.sqrt(q.shape[1])
    p = torch.exp(s - torch.logsumexp(s, 1, keepdim=True))
    return p, p @ v


def exact(case, seed):
    d = _inputs(case, seed)
    H, g, D, B = case["kv_heads"], case["group"], case["head_dim"], case["batch"]
    if case["kind"] == "evict":
        return _exact_evicted(d)

    def tokens(table, n, h):  # one head's K and V of the first n tokens of a row of pages
        at = table[:_pages(n)].long()
        both = []
        for x, s in ((d["k"], d["ks"]), (d["v"], d["vs"])):
            y = x[at, h].double()
            if case["per_token"]:
                y = y * s[at, h, :, None].double()
            elif s is not None:
                y = y * s[h].double()
            both.append(y.reshape(-1, D)[:n])
        return both

    out = torch.zeros(B, H * g, D, dtype=torch.float64, device="cuda")
    acc = d["weights"].double() if case["kind"] == "weights" else None
    group = [i for i, (a, b) in enumerate(zip(d["starts"], d["starts"][1:])) for _ in range(b - a)]
    for h in range(H):
        prefix = [tokens(d["pre_table"][i], n, h) for i, n in enumerate(d["prefixes"])]
        for b, n in enumerate(d["seqs"]):
            k, v = tokens(d["own_table"][b], n, h)
            if prefix:
                k, v = (torch.cat([x, y]) for x, y in zip(prefix[group[b]], (k, v)))
            lo = max(0, n - case["window"]) if case.get("window", -1) > 0 else 0
            if not k.shape[0]:
                continue
            p, o = _softmax64(d["q"][b, h * g:(h + 1) * g].double(), k[lo:], v[lo:])
            out[b, h * g:(h + 1) * g] = o
            if acc is not None:
                acc[b, h, :n] *= case["decay"]
                acc[b, h, lo:n] += p.sum(0)
    return out if acc is None else {"out": out, "weights": acc}


def _exact_evicted(d):
    """Position by position on the host; the caches have no value in 64 bits."""
    case, w = d["case"], d["weights"].double().cpu()
    kept, moved = d["kept"].cpu(), d["dst_weights"].double().cpu()
    lens = []
    for b, L in enumerate(d["seqs"]):
        n = min(L, case["keep"])
        s = min(case["sink"], n)
        r = min(case["recent"], n - s)
        lens.append(n)
        for h in range(case["kv_heads"]):
            middle = w[b, h, s:L - r].tolist()
            best = sorted(range(len(middle)), key=lambda i: (-middle[i], i))[:n - s - r]
            at = torch.tensor(list(range(s)) + sorted(s + i for i in best) + list(range(L - r, L)), dtype=torch.long)
            kept[b, h, :n] = at.int()
            moved[b, h, :n] = w[b, h, at]
    return {"kept": kept, "weights": moved, "lens": torch.tensor(lens, dtype=torch.int32), "k": None, "v": None,
            **({"scales": None} if case["per_token"] else {})}

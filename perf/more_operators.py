"""The operators around the cache, as cases to measure: head norms and rotary
positions of queries and keys, the same written straight into the paged cache,
the 4-bit cache's write, reading tokens back out of a cache, and decode
attention over the 4-bit cache.

`own` false: the plain form, elementary torch operations in 32 bits (angles in
64).  `own` true: the library's calls.
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
NAMES = {"e4m3": "fp8_e4m3", "e5m2": "fp8_e5m2", "bf16": "bf16", "fp4": "fp4_e2m1"}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
EPS = 1e-6


# ---------------------------------------------------------------- the cases ---
def rotate(name, tokens, q_heads, kv_heads, head_dim, rot, axes=1, interleaved=False, norm=True, far=131072):
    """`tokens` tokens' queries and keys, `rot` of their head_dim dims rotated by
    positions of up to `far` along `axes` axes, after a norm of each head."""
    return dict(name=name, kind="rotate", tokens=tokens, seqs=1, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                rot=rot, axes=axes, interleaved=interleaved, norm=norm, far=far)


def append(name, tokens, seqs, q_heads, kv_heads, head_dim, rot, dtype, per_token=False, q8=False, axes=1, interleaved=False,
           norm=False, far=131072):
    """The new tokens of `seqs` sequences rotated and written into their pages,
    the queries beside them as bf16 or as E4M3 codes."""
    return dict(name=name, kind="append", tokens=tokens, seqs=seqs, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                rot=rot, dtype=dtype, per_token=per_token, q8=q8, axes=axes, interleaved=interleaved, norm=norm, far=far)


def fp4(name, tokens, seqs, kv_heads, head_dim):
    """New tokens into a 4-bit cache, and back as the values that attention will see."""
    return dict(name=name, kind="fp4", tokens=tokens, seqs=seqs, kv_heads=kv_heads, head_dim=head_dim, dtype="fp4",
                per_token=False, far=4096)


def gather(name, tokens, seqs, kv_heads, head_dim, dtype, per_token=False):
    """Cached tokens of `seqs` sequences back as bf16."""
    return dict(name=name, kind="gather", tokens=tokens, seqs=seqs, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype,
                per_token=per_token, far=64)


def decode(name, batch, lo, hi, kv_heads, group, head_dim, window=-1):
    """One decode step over lo .. hi tokens per sequence of a 4-bit cache."""
    return dict(name=name, kind="decode", batch=batch, lo=lo, hi=hi, kv_heads=kv_heads, group=group, head_dim=head_dim,
                window=window, dtype="fp4", per_token=False)


def listed():
    return [
        # one request's next token: latency
        rotate("rotate_one_token", 1, 32, 8, 128, 128),
        # a long video's patches: frame, row and column positions
        rotate("rotate_video_16k", 16383, 32, 8, 128, 128, axes=3, far=8192),
        # one decode step of a busy server
        append("append_step_64", 64, 64, 32, 8, 128, 128, "e4m3"),
        # a chunk of a long prompt, its queries for FP8 prefill
        append("append_chunk_4k", 4096, 1, 32, 8, 128, 128, "e4m3", q8=True, far=28672),
        # several short prompts into a per-token-scaled cache, half of each head rotated
        append("append_prompts_per_token", 1777, 5, 64, 8, 64, 32, "e5m2", per_token=True, interleaved=True),
        # a few requests' new tokens into a 4-bit cache
        fp4("fp4_step_24", 24, 24, 8, 128),
        # two prompts of a few thousand tokens
        fp4("fp4_prompts_8k", 8191, 2, 8, 128),
        # a short cached system prompt
        gather("gather_prompt_500", 500, 1, 4, 64, "bf16"),
        # a long conversation's context taken up again
        gather("gather_context_32k", 32763, 1, 8, 128, "e4m3"),
        # one short request
        decode("decode_fp4_tiny", 1, 512, 512, 1, 4, 64),
        # eight requests of about 20K tokens
        decode("decode_fp4_batch8_20k", 8, 16384, 24576, 8, 4, 128),
        # one request of 128K tokens
        decode("decode_fp4_128k", 1, 131072, 131072, 8, 4, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) if hi >= LOG_RANGE * lo else rng.randint(lo, hi)


def draw(rng):
    kind = rng.choice(["rotate", "append", "fp4", "gather", "decode"])
    heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if kind == "decode":
        hi = _log(rng, 1, 60000)
        batch = _log(rng, 1, max(1, min(64, 100000 // hi)))
        case = decode("", batch, rng.randint(0, hi), hi, heads, rng.randint(1, 8), dim, rng.choice([-1, -1, rng.randint(1, hi)]))
    elif kind == "fp4":
        tokens = _log(rng, 1, 8191)
        case = fp4("", tokens, _log(rng, 1, min(tokens, 64)), heads, dim)
    elif kind == "gather":
        dtype = rng.choice(["e4m3", "e5m2", "bf16", "fp4"])
        tokens = _log(rng, 1, 16000 if dtype == "bf16" else 32000)
        case = gather("", tokens, _log(rng, 1, min(tokens, 64)), heads, dim, dtype, dtype in ("e4m3", "e5m2") and rng.random() < 0.4)
    else:
        turn = dict(axes=rng.randint(1, 3), interleaved=rng.random() < 0.4, norm=rng.random() < 0.5, far=_log(rng, 1000, 1000000))
        if kind == "rotate":
            dim = rng.choice([64, 128, 256])
        rot = rng.choice([dim, dim, 16 * rng.randint(1, dim // 16)])
        q_heads = heads * rng.randint(1, 4)
        if kind == "rotate":
            case = rotate("", _log(rng, 1, 16000 if dim < 256 else 8000), q_heads, heads, dim, rot, **turn)
        else:
            dtype = rng.choice(["e4m3", "e4m3", "e5m2", "bf16"])
            tokens = _log(rng, 1, 4096)
            case = append("", tokens, _log(rng, 1, min(tokens, 64)), q_heads, heads, dim, rot, dtype,
                          dtype != "bf16" and rng.random() < 0.4, rng.random() < 0.4, **turn)
    return {k: v for k, v in case.items() if k != "name"}


def _plan(case):
    """(first position, new tokens) of each sequence; a decode case's lengths.
    They are the case's, not the seed's."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["kind"] == "decode":
        return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    n, T = case["seqs"], case["tokens"]
    cuts = [0] + sorted(r.sample(range(1, T), n - 1)) + [T]
    return [(r.randint(0, max(0, case["far"] - T)), b - a) for a, b in zip(cuts, cuts[1:])]


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
    dtype = TYPES[case["dtype"]][0]
    chunks = b.contiguous().unflatten(-1, (-1, 16)).index_select(-2, _row_order(case["head_dim"] * dtype.itemsize, b.device))
    return chunks.flatten(-2).unflatten(-1, (PAGE, -1)).contiguous().view(dtype)


def _from_v_page(b, case):
    dtype = TYPES[case["dtype"]][0]
    rows = b.contiguous().unflatten(-1, (case["head_dim"], -1))
    if dtype.itemsize == 1:
        return rows.index_select(-1, torch.tensor(RHO, device=b.device)).transpose(-1, -2).contiguous().view(dtype)
    t = rows.contiguous().view(dtype).unflatten(-1, (2, 8))
    swap = ((torch.arange(t.shape[-3], device=b.device) >> 2) & 1).bool()[:, None, None]
    return torch.where(swap, t.flip(-2), t).flatten(-2).transpose(-1, -2)


def _fp4_codes(y):
    """Nearest E2M1 code of each value, ties to the even code, beyond 6 to 6."""
    a = y.abs()
    code = torch.zeros(y.shape, dtype=torch.uint8, device=y.device)
    for i, (lo, hi) in enumerate(zip(E2M1, E2M1[1:])):
        middle = (lo + hi) / 2
        code += a >= middle if i % 2 else a > middle
    return code | (torch.signbit(y).to(torch.uint8) << 3)


def _fp4_quantise(x, scale):
    """[..., D] values and their head's scale -> codes [..., D], E4M3 block scales [..., D / 16]."""
    blocks = x.unflatten(-1, (-1, 16))
    top = blocks.abs().amax(-1)
    sb = (top / (6.0 * scale)[..., None]).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = (sb.float() * scale[..., None])[..., None]
    codes = _fp4_codes(torch.where(step > 0, blocks / step, 0.0))
    return codes.flatten(-2), sb


def _fp4_pages(codes, sb, v):
    """[..., 16, D] codes and [..., 16, D / 16] scales -> [..., page bytes] of a K or a V page."""
    pairs = codes[..., 0::2] | (codes[..., 1::2] << 4)  # [..., 16, D / 2]
    sb = sb.contiguous().view(torch.uint8)
    if not v:
        return torch.cat([pairs.flatten(-2), sb.flatten(-2)], -1)
    half = max(1, sb.shape[-1] // 4)
    x = pairs.unflatten(-1, (half, 4, 8)).unflatten(-4, (2, 4, 2))  # [..., hi, c, lo, h, db, r]
    s = sb.unflatten(-1, (half, 4)).unflatten(-3, (2, 4, 2))  # [..., hi, c, lo, h, db]
    lead = list(range(x.dim() - 6))
    at = len(lead)
    x = x.permute(*lead, at + 3, at + 5, at + 1, at + 4, at, at + 2)  # [h, r, c, db, hi, lo]
    s = s.permute(*lead, at + 3, at + 1, at + 4, at, at + 2)  # [h, c, db, hi, lo]
    return torch.cat([x.flatten(at), s.flatten(at)], -1)


def _fp4_unpacked(b, case, v):
    """[..., page bytes] -> codes [..., 16, D] and scales [..., 16, D / 16], as bytes."""
    D = case["head_dim"]
    pairs, sb = b[..., :PAGE * D // 2], b[..., PAGE * D // 2:]
    if v:
        h = D // 64
        x = pairs.unflatten(-1, (h, 8, 4, 4, 2, 2))
        s = sb.unflatten(-1, (h, 4, 4, 2, 2))
        lead = list(range(b.dim() - 1))
        at = len(lead)
        pairs = x.permute(*lead, at + 4, at + 2, at + 5, at, at + 3, at + 1).flatten(at + 3).flatten(at, at + 2)
        sb = s.permute(*lead, at + 3, at + 1, at + 4, at, at + 2).flatten(at + 3).flatten(at, at + 2)
    else:
        pairs, sb = pairs.unflatten(-1, (PAGE, -1)), sb.unflatten(-1, (PAGE, -1))
    return torch.stack([pairs & 15, pairs >> 4], -1).flatten(-2), sb.contiguous()


def _from_fp4_pages(b, case, v):
    """[..., page bytes] -> [..., 16, D] values without the head's scale."""
    codes, sb = _fp4_unpacked(b, case, v)
    values = torch.tensor(E2M1 + [-x for x in E2M1], device=b.device)[codes.int()]
    return (values.unflatten(-1, (-1, 16)) * sb.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


# ------------------------------------------------------------------- inputs ---
def _turns(case, plan):
    """Positions [axes, T] and the axis of each pair."""
    T, A, pairs = case["tokens"], case["axes"], case["rot"] // 2
    first = torch.cat([torch.arange(s, s + n) for s, n in plan])
    if A == 1:
        return first.cuda(), None
    at = torch.arange(T)
    wide = max(1, int(T ** (1 / A)))
    grid = [first[0] + at // wide ** (A - 1)] + [first[0] + at // wide ** (A - 1 - i) % wide for i in range(1, A)]
    axis = torch.arange(pairs) * A // pairs
    return torch.stack(grid).cuda(), axis.int().cuda()


def _cached(case, gen, blocks, first):
    """K and V of every page as stored elements [blocks, H, 16, D], and their
    scales; the tokens at `first` draw weight from every query."""
    H, D = case["kv_heads"], case["head_dim"]
    k, v = (torch.randn(blocks, H, PAGE, D, generator=gen, device="cuda") for _ in range(2))
    u = torch.randn(H, D, generator=gen, device="cuda")
    k[first, :, 0] = 1.8 * u
    if case["dtype"] == "fp4":
        ks, vs = ((a + 0.12917 * torch.arange(H, device="cuda")) / (6.0 * 448.0) for a in (5.0271, 4.5313))
        k, v = (_fp4_quantise(x, s[:, None]) for x, s in ((k, ks), (v, vs)))
        return k, v, ks, vs, u
    dtype, top = TYPES[case["dtype"]]
    if dtype == torch.bfloat16:
        return k.bfloat16(), v.bfloat16(), None, None, u
    if case["per_token"]:
        ks, vs = k.abs().amax(-1) / top, v.abs().amax(-1) / top  # [blocks, H, 16]
        return (k / ks[..., None]).clamp(-top, top).to(dtype), (v / vs[..., None]).clamp(-top, top).to(dtype), ks, vs, u
    ks, vs = ((a + 0.12917 * torch.arange(H, device="cuda")) / top for a in (5.0271, 4.5313))
    return (k / ks[:, None, None]).clamp(-top, top).to(dtype), (v / vs[:, None, None]).clamp(-top, top).to(dtype), ks, vs, u


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    plan = _plan(case)
    d = dict(case=case, plan=plan)
    D, H = case["head_dim"], case["kv_heads"]
    if case["kind"] in ("rotate", "append"):
        # a slice of what the projection of a layer has left: q, k and v of a token side by side
        T, Hq, pairs = case["tokens"], case["q_heads"], case["rot"] // 2
        qkv = torch.randn(T, (Hq + 2 * H) * D, generator=gen, device="cuda").bfloat16()
        d["q"], d["k"], d["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, H * D, H * D], 1))
        d["positions"], d["pair_axis"] = _turns(case, plan)
        d["inv_freq"] = (500000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().cuda()
        d["qw"], d["kw"] = ((1 + 0.3 * torch.randn(D, generator=gen, device="cuda")).bfloat16() if case["norm"] else None for _ in range(2))
        d["q_scale"] = torch.full((1,), 5.0271 / 448.0, device="cuda")
    elif case["kind"] == "fp4":
        d["k"], d["v"] = (torch.randn(case["tokens"], H, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    if case["kind"] in ("append", "fp4", "gather"):
        # each sequence's tokens start somewhere in a page, and its pages are anywhere
        spans = [(s % PAGE, _pages(s % PAGE + n)) for s, n in plan]
        used = sum(c for _, c in spans)
        blocks = used + used // 8 + 1
        order = torch.randperm(blocks, generator=gen, device="cuda")
        at = torch.cat([torch.arange(s % PAGE, s % PAGE + n) + sum(c for _, c in spans[:i]) * PAGE for i, (s, n) in enumerate(plan)]).cuda()
        d["slots"] = order[at // PAGE] * PAGE + at % PAGE
        d["k_in"], d["v_in"], d["ks"], d["vs"], _ = _cached(case, gen, blocks, order[:1])
    if case["kind"] == "decode":
        B, g = case["batch"], case["group"]
        counts = [_pages(n) for n in plan]
        used = sum(counts)
        blocks = used + used // 8 + 1
        order = torch.randperm(blocks, generator=gen, device="cuda").int()
        table = torch.zeros(B, max(1, max(counts)), dtype=torch.int32, device="cuda")
        live = torch.arange(table.shape[1], device="cuda") < torch.tensor(counts, device="cuda")[:, None]
        table[live] = order[:used]
        d["table"], d["seq_lens"] = table, torch.tensor(plan, dtype=torch.int32, device="cuda")
        d["k_in"], d["v_in"], d["ks"], d["vs"], u = _cached(case, gen, blocks, table[:, 0].long())
        q = 1.2 * torch.randn(B, H * g, D, generator=gen, device="cuda")
        d["q"] = (q + 0.5 * u.repeat_interleave(g, 0)).bfloat16()
    return d


def prepare(case, seed):
    """What a server holds before the step: activations, tables, caches in the
    library's page format, scales and outputs."""
    d = _inputs(case, seed)
    if "k_in" in d:
        k, v = d.pop("k_in"), d.pop("v_in")
        if case["dtype"] == "fp4":
            d["k_cache"], d["v_cache"] = _fp4_pages(*k, False), _fp4_pages(*v, True)
        else:
            d["k_cache"], d["v_cache"] = _k_page(k), _v_page(v)
            if case["per_token"]:
                d["v_cache"] = torch.cat([d["v_cache"], _bytes(torch.cat([d["ks"], d["vs"]], -1))], -1)
        d["k_cache"], d["v_cache"] = d["k_cache"].contiguous(), d["v_cache"].contiguous()
    D, T, H = case["head_dim"], case.get("tokens"), case["kv_heads"]
    if case["kind"] in ("rotate", "append"):
        d["q_out"] = torch.zeros(T, case["q_heads"], D, dtype=torch.uint8 if case.get("q8") else torch.bfloat16, device="cuda")
    if case["kind"] in ("rotate", "fp4", "gather"):
        d["k_out"], d["v_out"] = (torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if case["kind"] == "decode":
        d["out"] = torch.zeros_like(d["q"])
        d["workspace"] = None
    return d


# --------------------------------------------------------------- plain form ---
def _turned(x, weight, d):
    """Norm and rotation of [T, heads, D] in 32 bits, the angles in 64."""
    case = d["case"]
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.float()
    pos = d["positions"] if case["axes"] == 1 else d["positions"][d["pair_axis"].long()].T  # [T] or [T, pairs]
    angle = (pos[:, None] if case["axes"] == 1 else pos).double() * d["inv_freq"].double()
    cos, sin = (f(angle).float()[:, None] for f in (torch.cos, torch.sin))
    turn, rest = y[..., :case["rot"]], y[..., case["rot"]:]
    if case["interleaved"]:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turn.chunk(2, -1)
        turn = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turn, rest], -1)


def _stored(d, x, v):
    """Tokens [T, H, D] in 32 bits -> (their pages' elements, scales of a per-token cache)."""
    dtype, top = TYPES[d["case"]["dtype"]]
    if dtype == torch.bfloat16:
        return x.to(dtype), None
    if d["case"]["per_token"]:
        s = x.abs().amax(-1) / top
        s = torch.where(s > 0, s, 1.0)
        return (x / s[..., None]).clamp(-top, top).to(dtype), s
    s = (d["vs"] if v else d["ks"])[:, None]
    return (x / s).clamp(-top, top).to(dtype), None


def _write(d, k, v):
    """Puts tokens into the cache's pages: the pages out, the tokens in, the pages back."""
    case, slots = d["case"], d["slots"]
    block, off = slots // PAGE, slots % PAGE
    page = PAGE * case["head_dim"] * TYPES[case["dtype"]][0].itemsize
    for name, x, back, forth, lo in (("k_cache", k, _from_k_page, _k_page, 0), ("v_cache", v, _from_v_page, _v_page, 1)):
        cache = d[name]
        codes, scales = _stored(d, x, lo == 1)
        pages = back(cache[..., :page], case).clone()
        kind = torch.uint8 if codes.element_size() == 1 else torch.int16
        pages.view(kind)[block, :, off] = codes.view(kind)
        cache[..., :page] = forth(pages)
        if scales is not None:
            tail = d["v_cache"][..., page:].contiguous().view(torch.float32)
            tail[block, :, off + lo * PAGE] = scales
            d["v_cache"][..., page:] = _bytes(tail)


def _cache(d):
    """The caches, their codes as the values they stand for."""
    dtype, page = TYPES[d["case"]["dtype"]][0], PAGE * d["case"]["head_dim"]
    if not d["case"]["per_token"]:
        return {"k": d["k_cache"].view(dtype), "v": d["v_cache"].view(dtype)}
    return {"k": d["k_cache"].view(dtype), "v": d["v_cache"][..., :page].view(dtype), "scales": d["v_cache"][..., page:].view(torch.float32)}


def _append_plain(d):
    q = _turned(d["q"], d["qw"], d)
    if d["case"]["q8"]:
        d["q_out"].copy_((q / d["q_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    else:
        d["q_out"].copy_(q)
    _write(d, _turned(d["k"], d["kw"], d), d["v"].float())


def _appended(d):
    return {"q": d["q_out"].view(torch.float8_e4m3fn) if d["case"]["q8"] else d["q_out"], **_cache(d)}


def _gather_plain(d):
    case, slots = d["case"], d["slots"]
    block, off = slots // PAGE, slots % PAGE
    if case["dtype"] == "fp4":
        for name, v, scale, out in (("k_cache", False, "ks", "k_out"), ("v_cache", True, "vs", "v_out")):
            d[out].copy_(_from_fp4_pages(d[name], case, v)[block, :, off] * d[scale][:, None])
        return
    page = PAGE * case["head_dim"] * TYPES[case["dtype"]][0].itemsize
    for name, back, scale, out, lo in (("k_cache", _from_k_page, "ks", "k_out", 0), ("v_cache", _from_v_page, "vs", "v_out", 1)):
        x = back(d[name][..., :page], case)[block, :, off].float()
        if case["per_token"]:
            x = x * d["v_cache"][..., page:].contiguous().view(torch.float32)[block, :, off + lo * PAGE][..., None]
        elif d[scale] is not None:
            x = x * d[scale][:, None]
        d[out].copy_(x)


def _fp4_plain(d):
    block, off = d["slots"] // PAGE, d["slots"] % PAGE
    for name, v, scale, x in (("k_cache", False, "ks", "k"), ("v_cache", True, "vs", "v")):
        codes, sb = _fp4_unpacked(d[name], d["case"], v)
        codes[block, :, off], new = _fp4_quantise(d[x].float(), d[scale])
        sb[block, :, off] = new.view(torch.uint8)
        d[name].copy_(_fp4_pages(codes, sb, v))
    _gather_plain(d)


def _decode_plain(d):
    case = d["case"]
    B, H, g, D = case["batch"], case["kv_heads"], case["group"], case["head_dim"]
    at = d["table"].long()
    k, v = (_from_fp4_pages(d[n][at], case, w).transpose(1, 2).flatten(2, 3) * d[s][:, None, None]
            for n, w, s in (("k_cache", False, "ks"), ("v_cache", True, "vs")))
    s = torch.matmul(d["q"].float().view(B, H, g, D), k.transpose(-1, -2)) / math.sqrt(D)
    t = torch.arange(k.shape[2], device=k.device)
    dead = t >= d["seq_lens"][:, None]
    if case["window"] > 0:
        dead = dead | (t < (d["seq_lens"] - case["window"])[:, None])
    s = torch.where(dead[:, None, None], float("-inf"), s)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    d["out"].copy_(o.reshape(B, H * g, D))


# ---------------------------------------------------------------------- run ---
def run(d):
    case = d["case"]
    kind = case["kind"]
    if own:
        import fp8_kv_cache_reshape_gb300 as kvq

        name = NAMES.get(case.get("dtype"))
        scales = (None, None) if case.get("per_token") else (d.get("ks"), d.get("vs"))
        if kind in ("rotate", "append"):
            turn = dict(q_weight=d["qw"], k_weight=d["kw"], eps=EPS, pair_axis=d["pair_axis"], interleaved=case["interleaved"])
        if kind == "rotate":
            kvq.kvq_qk_norm_rope(d["q"], d["k"], d["positions"], d["inv_freq"], d["q_out"], d["k_out"], **turn)
            return {"q": d["q_out"], "k": d["k_out"]}
        if kind == "append":
            out = dict(q8=d["q_out"], q_scale=d["q_scale"]) if case["q8"] else dict(q_out=d["q_out"])
            kvq.kvq_rope_and_cache(d["q"], d["k"], d["v"], d["positions"], d["inv_freq"], d["slots"], d["k_cache"], d["v_cache"],
                                   *scales, cache_dtype=name, per_token=case["per_token"], **out, **turn)
            return _appended(d)
        if kind == "decode":
            if d["workspace"] is None:  # a program keeps its workspace from step to step
                size = kvq.kvq_decode_fp4_workspace_size(case["batch"], d["q"].shape[1], case["kv_heads"], case["head_dim"], d["table"].shape[1])
                d["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
            return kvq.kvq_paged_decode_attention_fp4(d["q"], d["k_cache"], d["v_cache"], *scales, d["table"], d["seq_lens"], d["out"],
                                                      window=case["window"], workspace=d["workspace"])
        if kind == "fp4":
            kvq.kvq_reshape_and_cache(d["k"], d["v"], d["slots"], d["k_cache"], d["v_cache"], *scales, cache_dtype=name)
        kvq.kvq_gather_cache(d["slots"], d["k_cache"], d["v_cache"], d["k_out"], d["v_out"], *scales, cache_dtype=name,
                             per_token=case["per_token"])
        return {"k": d["k_out"], "v": d["v_out"]}
    if kind == "rotate":
        d["q_out"].copy_(_turned(d["q"], d["qw"], d))
        d["k_out"].copy_(_turned(d["k"], d["kw"], d))
        return {"q": d["q_out"], "k": d["k_out"]}
    if kind == "append":
        _append_plain(d)
        return _appended(d)
    if kind == "decode":
        _decode_plain(d)
        return d["out"]
    (_fp4_plain if kind == "fp4" else _gather_plain)(d)
    return {"k": d["k_out"], "v": d["v_out"]}


# --------------------------------------------------------------------- work ---
def _token_bytes(case):
    """K and V of one token and head as stored."""
    D = case["head_dim"]
    if case["dtype"] == "fp4":
        return 2 * (D // 2 + D // 16)
    return 2 * D * TYPES[case["dtype"]][0].itemsize + (8 if case["per_token"] else 0)


def work(case):
    kind, D, H = case["kind"], case["head_dim"], case["kv_heads"]
    if kind == "decode":
        lens = _plan(case)
        seen = sum(min(n, case["window"]) if case["window"] > 0 else n for n in lens)
        Hq = H * case["group"]
        return {"bytes": seen * H * _token_bytes(case) + 2 * case["batch"] * Hq * D * 2, "flops": 4 * D * Hq * seen}
    T = case["tokens"]
    if kind in ("fp4", "gather"):
        # the bf16 tokens in (where they are written first) and out, the cache once
        return {"bytes": T * H * (_token_bytes(case) + (8 if kind == "fp4" else 4) * D), "flops": 0}
    Hq = case["q_heads"]
    turned = T * (Hq + H) * (3 * case["rot"] + (4 * D if case["norm"] else 0))
    if kind == "rotate":
        return {"bytes": T * ((Hq + H) * D * 4 + 8 * case["axes"]), "flops": turned}
    return {"bytes": T * (Hq * D * (3 if case["q8"] else 4) + 4 * H * D + H * _token_bytes(case) + 8 * case["axes"] + 8), "flops": turned}


# -------------------------------------------------------------------- exact ---
def _grid(y, bits, low, top):
    """Nearest number of `bits` mantissa bits, exponents from `low` on, up to `top`; ties to even."""
    y = y.clamp(-top, top)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** low))) - bits)
    return torch.round(y / step) * step


FORMAT = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}


def _turned64(x, weight, d):
    """The rotation as a product of complex numbers."""
    case = d["case"]
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.double()
    T, pairs, axes = y.shape[0], case["rot"] // 2, case["axes"]
    pos = d["positions"].double().view(axes, T)
    which = torch.zeros(pairs, dtype=torch.long, device=y.device) if axes == 1 else d["pair_axis"].long()
    unit = torch.polar(torch.ones(T, pairs, dtype=torch.float64, device=y.device), pos.index_select(0, which).T * d["inv_freq"].double())
    first = torch.arange(pairs, device=y.device) * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else pairs)
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * unit[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_appended(d):
    case, slots = d["case"], d["slots"]
    q, k, v = _turned64(d["q"], d["qw"], d), _turned64(d["k"], d["kw"], d), d["v"].double()
    if case["q8"]:
        q = _grid(q / d["q_scale"].double(), *FORMAT["e4m3"])
    cache = {}
    for name, x, pages, scale, old in (("k", k, _k_page, "ks", "k_in"), ("v", v, _v_page, "vs", "v_in")):
        dtype = TYPES[case["dtype"]][0]
        if case["dtype"] != "bf16":
            if case["per_token"]:
                s = x.abs().amax(-1) / FORMAT[case["dtype"]][2]
                cache[scale] = d[scale].double()
                cache[scale][slots // PAGE, :, slots % PAGE] = s
                s = s[..., None]
            else:
                s = d[scale].double()[:, None]
            x = _grid(x / s, *FORMAT[case["dtype"]])
        held = d[old].clone()
        kind = torch.uint8 if held.element_size() == 1 else torch.int16
        held.view(kind)[slots // PAGE, :, slots % PAGE] = x.to(dtype).view(kind)
        cache[name] = pages(held).view(dtype).double()
    if case["per_token"]:
        cache["scales"] = torch.cat([cache.pop("ks"), cache.pop("vs")], -1)
    return {"q": q, **cache}


def _exact_read(d):
    case, slots = d["case"], d["slots"]
    found = {}
    for name, scale in (("k", "ks"), ("v", "vs")):
        if case["kind"] == "fp4":
            x = d[name].double().unflatten(-1, (-1, 16))
            s = d[scale].double()[:, None, None]
            sb = _grid(x.abs().amax(-1, keepdim=True) / (6 * s), *FORMAT["e4m3"])
            step = sb * s
            found[name] = (torch.where(sb > 0, _grid(x / step, 1, 0, 6.0), 0.0) * step).flatten(-2)
            continue
        held = d[name + "_in"]
        if case["dtype"] == "fp4":
            codes, sb = (x[slots // PAGE, :, slots % PAGE] for x in (held[0], held[1].view(torch.uint8)))
            low = torch.bitwise_and(codes, 7).double()
            size = torch.where(low < 2, low / 2, torch.exp2(torch.floor(low / 2) - 1) * (1 + (low % 2) / 2))
            x = torch.where(codes > 7, -size, size).unflatten(-1, (-1, 16)) * sb.view(torch.float8_e4m3fn).double()[..., None]
            x = x.flatten(-2)
        else:
            kind = torch.uint8 if held.element_size() == 1 else torch.int16
            x = held.view(kind)[slots // PAGE, :, slots % PAGE].view(held.dtype).double()
        if case["per_token"]:
            x = x * d[scale][slots // PAGE, :, slots % PAGE].double()[..., None]
        elif d[scale] is not None:
            x = x * d[scale].double()[:, None]
        found[name] = x
    return found


def _exact_attended(d):
    """Sequence by sequence and head by head."""
    case = d["case"]
    g, D = case["group"], case["head_dim"]
    size = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64, device="cuda")
    out = torch.zeros(d["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(d["plan"]):
        lo = max(0, n - case["window"]) if case["window"] > 0 else 0
        at = d["table"][b, :_pages(n)].long()
        for h in range(case["kv_heads"] if n else 0):
            k, v = ((size[c[at, h].int()].unflatten(-1, (-1, 16)) * s[at, h].double()[..., None]).reshape(-1, D)[lo:n] * t[h].double()
                    for (c, s), t in ((d["k_in"], d["ks"]), (d["v_in"], d["vs"])))
            q = d["q"][b, h * g:(h + 1) * g].double()
            s = q @ k.T / math.sqrt(D)
            out[b, h * g:(h + 1) * g] = torch.exp(s - torch.logsumexp(s, 1, keepdim=True)) @ v
    return out


def exact(case, seed):
    d = _inputs(case, seed)
    if case["kind"] == "rotate":
        return {"q": _turned64(d["q"], d["qw"], d), "k": _turned64(d["k"], d["kw"], d)}
    if case["kind"] == "append":
        return _exact_appended(d)
    return _exact_attended(d) if case["kind"] == "decode" else _exact_read(d)

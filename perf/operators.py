"""What is measured of the attention block around the path selector: three
operators of the model that verifies a drafted block (and of the drafter's own
attention layers), each as a plain form in elementary torch operations and as
the calls a user makes of this package.

  norm_rope  per-head RMS norm and position rotation of queries and keys
  append     the same transform, with keys and values written to a paged cache
  attend     attention of each sequence's newest tokens over its paged cache

A case is a dict of plain values:
  op            "norm_rope", "append" or "attend"
  heads, kv_heads, head_dim, dtype ("bfloat16" or "float16")
  rotary, interleaved, norm       the transform (norm_rope, append)
  batch, new_min, new_max         sequences, and new tokens of each (ragged between the two)
  ctx_min, ctx_max                tokens a sequence has in the cache before its new ones
  page, fp8, head_major           page size, 8-bit cache, [page, head, slot] instead of [page, slot, head]
  with_q                          append only: the queries are transformed by the same call
  causal, window                  attend only
Lengths of the sequences follow from the case alone, so every seed has the same
work; all values follow from the seed.
"""
import math
import random

import torch

own = False

K_SCALE, V_SCALE = 0.03125, 0.015625  # what one step of an 8-bit cache stands for
EPS = 1e-6
MAX_POSITION = 1 << 18

#: no drawn case costs more than the largest listed ones
MOST_TOKENS = 16384 * 48 * 128      # values of a token's queries, keys and values times tokens
MOST_CACHE_BYTES = 536_000_000      # keys and values that an attention call reads
MOST_PAIRS = 1_000_000_000          # (query, key, head) triples of an attention call


def _norm_rope(name, tokens, heads, kv_heads, head_dim, dtype="bfloat16", rotary=None, interleaved=False, norm=True):
    return dict(name=name, op="norm_rope", tokens=tokens, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                dtype=dtype, rotary=head_dim if rotary is None else rotary, interleaved=interleaved, norm=norm)


def _append(name, batch, new, ctx, heads, kv_heads, head_dim, dtype="bfloat16", page=16, fp8=False, head_major=False,
            rotary=None, interleaved=False, norm=True, with_q=True):
    return dict(name=name, op="append", batch=batch, new_min=new[0], new_max=new[1], ctx_min=ctx[0], ctx_max=ctx[1],
                heads=heads, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, page=page, fp8=fp8,
                head_major=head_major, rotary=head_dim if rotary is None else rotary, interleaved=interleaved,
                norm=norm, with_q=with_q)


def _attend(name, batch, new, ctx, heads, kv_heads, head_dim, dtype="bfloat16", page=16, fp8=False, head_major=False,
            causal=True, window=0):
    return dict(name=name, op="attend", batch=batch, new_min=new[0], new_max=new[1], ctx_min=ctx[0], ctx_max=ctx[1],
                heads=heads, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, page=page, fp8=fp8,
                head_major=head_major, causal=causal, window=window)


def listed():
    return [
        # one sequence's block of 8 (the last verified token and 7 drafts) before a layer's attention: latency
        _norm_rope("norm_rope b1 block of 8", 8, 32, 8, 128),
        # 256 blocks of 16 at width 2560 (20 heads of 128): the stress batch
        _norm_rope("norm_rope b256 blocks of 16", 4096, 20, 4, 128),
        # a long prompt, half of each head rotated in adjacent pairs, an odd number of tokens
        _norm_rope("norm_rope 16001 tokens fp16", 16001, 32, 8, 64, dtype="float16", rotary=32, interleaved=True,
                   norm=False),
        # the block of one sequence goes into the cache, its queries are made by the same call: latency
        _append("append b1 block of 8", 1, (8, 8), (2041, 2041), 32, 8, 128),
        # 32 sequences with 1 to 16 tokens each, 8-bit cache: a mixed batch of single tokens and blocks
        _append("append b32 ragged fp8", 32, (1, 16), (100, 4000), 40, 8, 128, page=64, fp8=True),
        # the drafter's cache takes the keys and values of a prompt's features: no queries, pages by head
        _append("append 16384 tokens kv only", 1, (16384, 16384), (0, 0), 32, 8, 128, page=64, head_major=True,
                with_q=False),
        # one sequence's block verified over a short context: latency
        _attend("attend b1 block of 8 ctx 2041", 1, (8, 8), (2041, 2041), 32, 8, 128),
        # 32 sequences verify their blocks, ragged contexts: the memory-bound middle
        _attend("attend b32 blocks ragged", 32, (8, 8), (500, 7000), 32, 8, 128),
        # 128 sequences extend by a single token each, 8-bit cache
        _attend("attend b128 single token fp8", 128, (1, 1), (200, 3800), 32, 8, 128, page=64, fp8=True),
        # one block over a very long context, width 5120 (40 heads of 128): the work of few rows split over the GPU
        _attend("attend b1 block ctx 131065", 1, (8, 8), (131065, 131065), 40, 8, 128, page=64, head_major=True),
        # a chunk of a long prompt after 14 k tokens: bound by the tensor cores
        _attend("attend chunk 2048 after 14336", 1, (2048, 2048), (14336, 14336), 32, 8, 128, page=64),
        # drafter layers over several prompts at once: odd chunks, heads of 64, a sliding window
        _attend("attend b7 chunks window fp16", 7, (300, 1100), (0, 2500), 16, 2, 64, dtype="float16", window=1024),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = max(lo, min(hi, v))
    return v + 1 if v == 3072 else v


_HEADS = [(32, 8, 128), (20, 4, 128), (40, 8, 128), (10, 10, 128), (28, 4, 128), (64, 8, 64), (16, 2, 64), (12, 4, 64)]


def _draw_transform(rng, head_dim):
    return dict(rotary=rng.choice([head_dim, head_dim, head_dim // 2]), interleaved=rng.random() < 0.3,
                norm=rng.random() < 0.7)


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attend", "attend"])
    heads, kv_heads, head_dim = rng.choice(_HEADS)
    dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
    if op == "norm_rope":
        width = (heads + kv_heads) * head_dim
        c = _norm_rope("", _log_int(rng, 1, min(16384, MOST_TOKENS // width)), heads, kv_heads, head_dim, dtype,
                       **_draw_transform(rng, head_dim))
    elif op == "append":
        batch = _log_int(rng, 1, 256)
        most = min(16384, MOST_TOKENS // ((heads + 2 * kv_heads) * head_dim)) // batch
        new_max = _log_int(rng, 1, max(1, most))
        ctx_max = _log_int(rng, 1, max(1, min(8000, 200_000 // batch)))
        c = _append("", batch, (rng.randint(1, new_max), new_max), (rng.randint(0, ctx_max), ctx_max), heads,
                    kv_heads, head_dim, dtype, page=rng.choice([16, 32, 64]), fp8=rng.random() < 0.4,
                    head_major=rng.random() < 0.3, with_q=rng.random() < 0.7, **_draw_transform(rng, head_dim))
    else:
        fp8 = rng.random() < 0.35
        token = 2 * kv_heads * head_dim * (1 if fp8 else 2)
        if rng.random() < 0.6:  # single tokens and blocks
            batch = _log_int(rng, 1, 256)
            new_max = rng.choice([1, 4, 8, 8, 16])
            new_min = rng.choice([1, new_max])
        else:                   # chunks of prompts
            batch = _log_int(rng, 1, 16)
            new_max = _log_int(rng, 17, min(2048, int(math.sqrt(MOST_PAIRS / (batch * heads)))))
            new_min = rng.randint(1, new_max)
        most = min(MOST_CACHE_BYTES // (batch * token), MOST_PAIRS // (batch * new_max * heads)) - new_max
        ctx_max = _log_int(rng, 1, max(2, min(131072, most)))
        c = _attend("", batch, (new_min, new_max), (rng.randint(0, ctx_max), ctx_max), heads, kv_heads, head_dim,
                    dtype, page=rng.choice([16, 32, 64]), fp8=fp8, head_major=rng.random() < 0.3,
                    causal=rng.random() < 0.8, window=rng.choice([0, 0, 0, 1000]))
        if not c["causal"]:
            c["window"] = 0
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, cache length with them) of each sequence."""
    rng = random.Random("%(batch)d %(new_min)d %(new_max)d %(ctx_min)d %(ctx_max)d" % case)
    new = [rng.randint(case["new_min"], case["new_max"]) for _ in range(case["batch"])]
    ctx = [rng.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["batch"])]
    return new, [n + c for n, c in zip(new, ctx)]


def _visible(case, n, length):
    """Keys that the n newest of `length` tokens see, summed over them, and the keys that any of them sees."""
    if not case["causal"]:
        return n * length, length
    w = case["window"] or length
    return sum(min(length - n + i + 1, w) for i in range(n)), min(length, n - 1 + w)


def work(case):
    size = 2
    hq, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "norm_rope":
        t = case["tokens"]
        return {"bytes": t * (2 * (hq + hk) * d * size + 4 * case["rotary"] + 4), "flops": t * (hq + hk) * d * 7}
    new, lens = _lengths(case)
    t = sum(new)
    cell = 1 if case["fp8"] else size
    pages = sum(-(-n // case["page"]) for n in lens)
    if case["op"] == "append":
        q = 2 * hq * d * size if case["with_q"] else 0
        return {"bytes": t * (q + 2 * hk * d * (size + cell) + 4 * case["rotary"]) + 4 * (2 * len(lens) + t // case["page"]),
                "flops": t * ((hq if case["with_q"] else 0) + 2 * hk) * d * 7}
    pairs, keys = (sum(x) for x in zip(*(_visible(case, n, s) for n, s in zip(new, lens))))
    return {"bytes": 2 * t * hq * d * size + 4 * t * hq + 2 * keys * hk * d * cell + 4 * (2 * len(lens) + pages),
            "flops": 4 * pairs * hq * d}


def _rope_table(rotary, dev):
    """[positions, rotary] fp32: the cosines of a position's rotary / 2 angles, then the sines."""
    inv = 10000.0 ** (-torch.arange(0, rotary, 2, device=dev, dtype=torch.float64) / rotary)
    angle = torch.arange(MAX_POSITION, device=dev, dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


_tables = {}


def _transform(case, gen, dev, state):
    dt, d = getattr(torch, case["dtype"]), case["head_dim"]
    if case["rotary"] not in _tables:  # one table serves every layer and step of a program
        _tables[case["rotary"]] = _rope_table(case["rotary"], dev)
    state["table"] = _tables[case["rotary"]]
    for w in ("q_weight", "k_weight"):
        state[w] = (1 + 0.2 * torch.randn(d, device=dev, generator=gen)).to(dt) if case["norm"] else None


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = getattr(torch, case["dtype"])
    hq, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    s = {"case": case}
    if case["op"] == "norm_rope":
        t = case["tokens"]
        # a packed projection output [tokens, heads of q, k and v, head_dim]; q and k are slices of it
        qkv = (2 * torch.randn(t, hq + 2 * hk, d, device=dev, generator=gen)).to(dt)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], q_out=torch.empty(t, hq, d, device=dev, dtype=dt),
                 k_out=torch.empty(t, hk, d, device=dev, dtype=dt),
                 positions=torch.randint(0, MAX_POSITION, (t,), device=dev, generator=gen, dtype=torch.int32))
        _transform(case, gen, dev, s)
        if own:
            import speculative_decoding_draft_tcgen05_gb300 as pkg
            s["transform"] = pkg.QkTransform(s["table"], rotary_dim=case["rotary"], interleaved=case["interleaved"],
                                             q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
        return s

    new, lens = _lengths(case)
    t, b, page = sum(new), len(new), case["page"]
    cols = -(-max(lens) // page)
    pages = sum(-(-n // page) for n in lens)
    # pages in the order in which a busy allocator hands them out, a few of them free
    order = torch.randperm(pages + 3, device=dev, generator=gen)[:pages].to(torch.int32)
    need = torch.tensor([-(-n // page) for n in lens], device=dev)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(cols, device=dev)
    table = torch.where(col < need[:, None], order[(first[:, None] + col).clamp(max=pages - 1)], -1)
    s["page_table"] = table.to(torch.int32).contiguous()
    s["lens"] = torch.tensor(lens, device=dev, dtype=torch.int32)
    s["cu_tokens"] = torch.tensor([sum(new[:i]) for i in range(b + 1)], device=dev, dtype=torch.int32)
    s["max_tokens"], s["tokens"] = max(new), t
    shape = (pages + 3, hk, page, d) if case["head_major"] else (pages + 3, page, hk, d)
    for name, scale in (("k_cache", K_SCALE), ("v_cache", V_SCALE)):
        x = torch.randn(shape, device=dev, generator=gen, dtype=torch.float16)
        x = (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn) if case["fp8"] else x.to(dt)
        s[name] = x.transpose(1, 2) if case["head_major"] else x  # [page, slot, head, head_dim] either way
    if case["op"] == "append":
        qkv = (2 * torch.randn(t, hq + 2 * hk, d, device=dev, generator=gen)).to(dt)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:],
                 q_out=torch.empty(t, hq, d, device=dev, dtype=dt))
        _transform(case, gen, dev, s)
    else:
        s.update(q=(1.5 * torch.randn(t, hq, d, device=dev, generator=gen)).to(dt),
                 out=torch.empty(t, hq, d, device=dev, dtype=dt), lse=torch.empty(t, hq, device=dev))
    if own:
        import speculative_decoding_draft_tcgen05_gb300 as pkg
        s["layer"] = pkg.PagedAttention(heads=hq, kv_heads=hk, head_dim=d, page_size=page, dtype=dt,
                                        cache_dtype=s["k_cache"].dtype, max_batch=b)
        scales = dict(k_scale=K_SCALE, v_scale=V_SCALE) if case["fp8"] else {}
        s["cache"] = pkg.PagedCache(s["k_cache"], s["v_cache"], **scales)
        s["batch"] = pkg.PagedBatch(s["cu_tokens"], s["lens"], s["page_table"], max_tokens=s["max_tokens"])
        if case["op"] == "append":
            s["transform"] = pkg.QkTransform(s["table"], rotary_dim=case["rotary"], interleaved=case["interleaved"],
                                             q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
    return s


def run(s):
    op = s["case"]["op"]
    if op == "norm_rope":
        return _own_norm_rope(s) if own else _plain_norm_rope(s)
    if op == "append":
        return _own_append(s) if own else _plain_append(s)
    return _own_attend(s) if own else _plain_attend(s)


# ------------------------------------------------------------ the calls a user makes
def _own_norm_rope(s):
    import speculative_decoding_draft_tcgen05_gb300 as pkg
    pkg.dflash_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["transform"], s["positions"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_append(s):
    if s["case"]["with_q"]:
        s["layer"].append(s["cache"], s["batch"], s["k"], s["v"], s["transform"], q=s["q"], q_out=s["q_out"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    s["layer"].append(s["cache"], s["batch"], s["k"], s["v"], s["transform"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    s["layer"].attend(s["cache"], s["batch"], s["q"], s["out"], lse=s["lse"], causal=s["case"]["causal"],
                      window=s["case"]["window"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------ the plain forms
def _plain_transform(x, weight, table, positions, case):
    """RMS norm of each head of x [tokens, heads, head_dim], then the rotation of its first `rotary` values."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight.float()
    r = case["rotary"]
    row = table[positions.long()][:, None, :]
    cos, sin = row[..., :r // 2], row[..., r // 2:]
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., r:]], dim=-1)


def _plain_norm_rope(s):
    c = s["case"]
    return {"q": _plain_transform(s["q"], s["q_weight"], s["table"], s["positions"], c).to(s["q"].dtype),
            "k": _plain_transform(s["k"], s["k_weight"], s["table"], s["positions"], c).to(s["k"].dtype)}


def _token_places(s):
    """Of each new token: its sequence, its index within the sequence's new tokens, its place in the cache."""
    token = torch.arange(s["tokens"], device=s["lens"].device)
    cu = s["cu_tokens"].long()
    seq = torch.searchsorted(cu, token, right=True) - 1
    i = token - cu[seq]
    return seq, i, s["lens"].long()[seq] - (cu[seq + 1] - cu[seq]) + i


def _plain_append(s):
    c = s["case"]
    seq, _, at = _token_places(s)
    page = s["page_table"][seq, at // c["page"]].long()
    slot = at % c["page"]
    k = _plain_transform(s["k"], s["k_weight"], s["table"], at, c)
    for cache, x, scale in ((s["k_cache"], k, K_SCALE), (s["v_cache"], s["v"].float(), V_SCALE)):
        if c["fp8"]:
            x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            cache.view(torch.uint8)[page, slot] = x.view(torch.uint8)
        else:
            cache[page, slot] = x.to(cache.dtype)
    got = {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["with_q"]:
        got["q"] = _plain_transform(s["q"], s["q_weight"], s["table"], at, c).to(s["q"].dtype)
    return got


def _plain_attend(s):
    c = s["case"]
    hq, hk, d, g = c["heads"], c["kv_heads"], c["head_dim"], c["heads"] // c["kv_heads"]
    seq, i, at = _token_places(s)
    b, n = s["lens"].shape[0], s["max_tokens"]
    q = torch.zeros(b, n, hq, d, device=s["q"].device)
    q[seq, i] = s["q"].float()
    q = q.view(b, n, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * n, d)
    pages = s["page_table"].clamp(min=0).long()
    if c["fp8"]:
        k = s["k_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * K_SCALE
        v = s["v_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * V_SCALE
    else:
        k, v = s["k_cache"][pages].float(), s["v_cache"][pages].float()
    keys = pages.shape[1] * c["page"]
    k = k.reshape(b, keys, hk, d).permute(0, 2, 3, 1)
    v = v.reshape(b, keys, hk, d).permute(0, 2, 1, 3)
    score = torch.matmul(q, k).mul_(d ** -0.5).view(b, hk, g, n, keys)
    key = torch.arange(keys, device=q.device)
    place = torch.zeros(b, n, device=q.device, dtype=torch.long)
    place[seq, i] = at
    seen = (key < s["lens"].long()[:, None, None]).expand(b, n, keys)
    if c["causal"]:
        seen = seen & (key <= place[:, :, None])
    if c["window"]:
        seen = seen & (key > place[:, :, None] - c["window"])
    score = score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)  # a row that sees nothing
    p = score.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    lse = (total.log() + top).view(b, hq, n).permute(0, 2, 1)
    out = torch.matmul(p.view(b, hk, g * n, keys), v) / total.view(b, hk, g * n, 1).clamp(min=1e-30)
    out = out.view(b, hq, n, d).permute(0, 2, 1, 3)
    return {"out": out[seq, i].to(s["q"].dtype), "lse": lse[seq, i].contiguous()}


# ------------------------------------------------------------ the definitions in 64 bits
def _exact_transform(x, weight, positions, case):
    x, r = x.double().clone(), case["rotary"]
    if weight is not None:
        x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    half = torch.arange(r // 2, device=x.device, dtype=torch.float64)
    row = _tables[r][positions.long()].double()  # the angles' cosines and sines are an input
    turn = torch.complex(row[:, :r // 2], row[:, r // 2:])[:, None, :]
    first = (2 * half if case["interleaved"] else half).long()
    second = first + (1 if case["interleaved"] else r // 2)
    z = torch.complex(x[..., first], x[..., second]) * turn
    x[..., first], x[..., second] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return {"q": _exact_transform(s["q"], s["q_weight"], s["positions"], case),
                "k": _exact_transform(s["k"], s["k_weight"], s["positions"], case)}
    new, lens = _lengths(case)
    page, start = case["page"], 0
    if case["op"] == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        q = s["q"].double() if case["with_q"] else None
        for b, (n, length) in enumerate(zip(new, lens)):
            at = torch.arange(length - n, length, device=kc.device)
            where = (s["page_table"][b].long()[at // page], at % page)
            rows = slice(start, start + n)
            kc[where] = _exact_transform(s["k"][rows], s["k_weight"], at, case) / (K_SCALE if case["fp8"] else 1)
            vc[where] = s["v"][rows].double() / (V_SCALE if case["fp8"] else 1)
            if q is not None:
                q[rows] = _exact_transform(s["q"][rows], s["q_weight"], at, case)
            start += n
        if case["fp8"]:  # what the cache's 8 bits can hold
            kc, vc = kc.clamp(-448, 448), vc.clamp(-448, 448)
        got = {"k_cache": kc, "v_cache": vc}
        return got if q is None else {**got, "q": q}
    g = case["heads"] // case["kv_heads"]
    out = torch.empty(s["q"].shape, device=s["q"].device, dtype=torch.float64)
    lse = torch.empty(s["q"].shape[:2], device=out.device, dtype=torch.float64)
    for b, (n, length) in enumerate(zip(new, lens)):
        at = torch.arange(length, device=out.device)
        where = (s["page_table"][b].long()[at // page], at % page)
        place = at[length - n:, None]
        hidden = torch.zeros(n, length, dtype=torch.bool, device=out.device)
        if case["causal"]:
            hidden |= at > place
        if case["window"]:
            hidden |= at <= place - case["window"]
        for h in range(case["kv_heads"]):
            if case["fp8"]:
                k = s["k_cache"][:, :, h].double()[where] * K_SCALE
                v = s["v_cache"][:, :, h].double()[where] * V_SCALE
            else:
                k, v = s["k_cache"][:, :, h][where].double(), s["v_cache"][:, :, h][where].double()
            for j in range(h * g, (h + 1) * g):
                score = (s["q"][start:start + n, j].double() @ k.T / math.sqrt(case["head_dim"])).masked_fill(
                    hidden, -math.inf)
                total = torch.logsumexp(score, dim=1)
                lse[start:start + n, j] = total
                out[start:start + n, j] = (score - total[:, None]).exp() @ v
        start += n
    return {"out": out, "lse": lse}

"""What is measured of the rest of a verifying model's step: the operators
around its attention, each as a plain form in elementary torch operations and
as the calls a user makes of this package.

  pages   pages, positions and slots of a step's new tokens from the requests'
          lengths, and the pages of rejected tokens given back
  linear  y = residual + act(x W^T + bias)
  logits  the target's logits after penalties for repeated tokens, biases and
          a grammar's mask, as the accept checks take them: probabilities,
          the best tokens, or the logits themselves

A case is a dict of plain values:
  op           "pages", "linear" or "logits"
pages:
  requests, batch   requests the tables have rows for, and those with new tokens this step
  new_min, new_max  new tokens of each;  ctx_min, ctx_max  tokens that each holds before
  page, cols        page size, entries of a request's row of the page table
linear:
  m, n, k, dtype    x [m, k], W [n, k];  out  "same" or "float32"
  pad               extra columns of the buffer that x is a slice of
  bias, residual    truth values;  act  "none", "relu", "silu", "gelu" or "gelu_tanh"
logits:
  batch, rows, vocab, dtype     logits [batch, rows, vocab]: the positions of a drafted block
  hist_min, hist_max            tokens of a sequence so far, its prompt among them
  penalties, mask, temperature  truth values;  bias  entries of a sequence's list
  empty                         the first row's mask allows nothing
  want                          "argmax", "probs" or "logits" (of the type "dtype")
Lengths follow from the case alone, so every seed has the same work; all
values follow from the seed.
"""
import math
import random

import torch

own = False

#: no drawn case costs more than the largest listed ones
MOST_FLOPS = 430e9
MOST_WEIGHT = 151936 * 2560
MOST_LOGITS = 256 * 151936
MOST_TOKENS = 16384

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def _pages(name, requests, batch, new, ctx, page=16, cols=1024):
    return dict(name=name, op="pages", requests=requests, batch=batch, new_min=new[0], new_max=new[1], ctx_min=ctx[0],
                ctx_max=ctx[1], page=page, cols=cols)


def _linear(name, m, n, k, dtype="bfloat16", out="same", pad=0, bias=False, residual=False, act="none"):
    return dict(name=name, op="linear", m=m, n=n, k=k, dtype=dtype, out=out, pad=pad, bias=bias, residual=residual,
                act=act)


def _logits(name, batch, rows, vocab, hist, dtype="bfloat16", penalties=True, mask=True, bias=0, temperature=False,
            empty=False, want="argmax"):
    return dict(name=name, op="logits", batch=batch, rows=rows, vocab=vocab, hist_min=hist[0], hist_max=hist[1],
                dtype=dtype, penalties=penalties, mask=mask, bias=bias, temperature=temperature, empty=empty, want=want)


def listed():
    return [
        # one sequence's block of 8 (the last verified token and 7 drafts) gets its places: latency
        _pages("pages b1 block of 8", 1, 1, (8, 8), (2041, 2041)),
        # a server's step: 256 of 1024 requests, single tokens and blocks of 16 mixed, long rows of the page table
        _pages("pages b256 ragged of 1024", 1024, 256, (1, 16), (100, 16000)),
        # prompts come in: some 16 thousand tokens of 7 requests, pages of 64
        _pages("pages b7 prompts", 64, 7, (1200, 3500), (0, 900), page=64, cols=512),
        # the attention's output projection for one block, width 2560, with the residual: latency
        _linear("linear 8 rows 2560x2560 residual", 8, 2560, 2560, residual=True),
        # an up projection of 8 blocks, an odd number of rows, bias and activation
        _linear("linear 61 rows 10240x2560 gelu fp16", 61, 10240, 2560, dtype="float16", bias=True, act="gelu_tanh"),
        # the output head of one block: 778 MB of weights, logits in 32 bits
        _linear("linear 8 rows 151936x2560 to fp32", 8, 151936, 2560, out="float32"),
        # 32 blocks of 8 at width 5120, rows a slice of a wider buffer
        _linear("linear 256 rows 5120x5120", 256, 5120, 5120, pad=128, residual=True),
        # a long prompt through an up projection: bound by the tensor cores
        _linear("linear 8191 rows 10240x2560 silu", 8191, 10240, 2560, bias=True, act="silu"),
        # greedy verification of one sequence's block under a grammar, after 2000 tokens: latency
        _logits("logits b1 block of 8 argmax", 1, 8, 151936, (2000, 2000), bias=16),
        # single tokens of 48 sequences, odd vocabulary: the adjusted logits themselves
        _logits("logits b48 single token fp16", 48, 1, 32003, (1, 6000), dtype="float16", want="logits", mask=False,
                bias=5),
        # 32 sequences' blocks, ragged histories: probabilities for rejection sampling
        _logits("logits b32 blocks of 8 probs", 32, 8, 151936, (100, 8000), temperature=True, empty=True, want="probs"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "linear", "linear", "logits", "logits"])
    if op == "pages":
        batch = _log_int(rng, 1, 512)
        new_max = _log_int(rng, 1, MOST_TOKENS // batch)
        ctx_max = _log_int(rng, 1, max(2, min(16000, 2_000_000 // batch)))
        page = rng.choice([16, 32, 64])
        c = _pages("", batch + _log_int(rng, 1, 512) - 1, batch, (rng.randint(0, new_max), new_max),
                   (rng.randint(0, ctx_max), ctx_max), page=page,
                   cols=(new_max + ctx_max) // page + rng.randint(1, 200))
    elif op == "linear":
        k = 8 * _log_int(rng, 8, 2048)
        n = _log_int(rng, 64, 20480 if rng.random() < 0.8 else 151936)
        n = min(n, MOST_WEIGHT // k)
        if rng.random() < 0.7:  # widths of models are multiples of 64
            n = max(64, n // 64 * 64)
        m = _log_int(rng, 1, max(1, min(16384, int(MOST_FLOPS / (2.0 * n * k)))))
        c = _linear("", m, n, k, dtype=rng.choice(["bfloat16", "float16"]), out=rng.choice(["same", "same", "float32"]),
                    pad=rng.choice([0, 0, 8, 64]), bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    act=rng.choice(ACTS))
    else:
        rows = rng.choice([1, 1, 4, 8, 16])
        vocab = _log_int(rng, 1000, 151936)
        if rng.random() < 0.5:
            vocab = vocab // 8 * 8
        batch = _log_int(rng, 1, max(1, min(256, MOST_LOGITS // (rows * vocab))))
        hist_max = _log_int(rng, 1, 8000)
        c = _logits("", batch, rows, vocab, (rng.randint(0, hist_max), hist_max),
                    dtype=rng.choice(["bfloat16", "float16", "float32"]), penalties=rng.random() < 0.8,
                    mask=rng.random() < 0.6, bias=rng.choice([0, 0, 7, 300]), temperature=rng.random() < 0.5,
                    empty=rng.random() < 0.3, want=rng.choice(["argmax", "probs", "probs", "logits"]))
        c["empty"] = c["empty"] and c["mask"]
    del c["name"]
    return c


# ------------------------------------------------------------ lengths, work
def _page_lengths(case):
    """The batch's rows of the tables, new tokens and lengths before; tokens held by every request."""
    rng = random.Random("%(requests)d %(batch)d %(new_min)d %(new_max)d %(ctx_min)d %(ctx_max)d" % case)
    held = [rng.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["requests"])]
    rows = rng.sample(range(case["requests"]), case["batch"])
    new = [rng.randint(case["new_min"], case["new_max"]) for _ in rows]
    return rows, new, held


def _histories(case):
    """Tokens of each sequence, and those of its prompt."""
    rng = random.Random("%(batch)d %(hist_min)d %(hist_max)d" % case)
    total = [rng.randint(case["hist_min"], case["hist_max"]) for _ in range(case["batch"])]
    return total, [int(n * rng.uniform(0.2, 1)) for n in total]


def _ceil(a, b):
    return -(-a // b)


def work(case):
    if case["op"] == "pages":
        rows, new, held = _page_lengths(case)
        p = case["page"]
        entries = sum(_ceil(held[r] + n, p) for r, n in zip(rows, new))
        taken = sum(_ceil(held[r] + n, p) - _ceil(held[r], p) for r, n in zip(rows, new))
        # per sequence: row, new tokens, length in and out, cu_tokens, the batch's length, the length after the trim;
        # per entry of the batch's page table one read and one write; a page taken is written to its request's row and
        # back to the stack; a position and a slot for every token
        return {"bytes": 4 * (7 * len(rows) + 2 * entries + 3 * taken) + 12 * sum(new), "flops": 0}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        y = 4 if case["out"] == "float32" else 2
        return {"bytes": 2 * (m * k + n * k) + m * n * y * (2 if case["residual"] else 1) + (2 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    count = case["batch"] * case["rows"]
    values = count * case["vocab"]
    size = 4 if case["dtype"] == "float32" else 2
    read = values * size + (count * _ceil(case["vocab"], 32) * 4 if case["mask"] else 0)
    if case["penalties"]:
        read += 4 * sum(_histories(case)[0])
    read += 8 * case["batch"] * case["bias"]
    write = {"argmax": 4 * count, "probs": 4 * values, "logits": size * values}[case["want"]]
    return {"bytes": read + write, "flops": values * (8 if case["want"] == "probs" else 4)}


# ------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    make = {"pages": _prepare_pages, "linear": _prepare_linear, "logits": _prepare_logits}[case["op"]]
    s = make(case, gen, dev)
    s["case"] = case
    return s


def _prepare_pages(case, gen, dev):
    rows, new, held = _page_lengths(case)
    p, cols = case["page"], case["cols"]
    need = [_ceil(n, p) for n in held]
    taken = sum(_ceil(held[r] + n, p) - _ceil(held[r], p) for r, n in zip(rows, new))
    pages = sum(need) + taken + 5
    # pages in the order in which a busy allocator has handed them out
    order = torch.randperm(pages, device=dev, generator=gen).to(torch.int32)
    need_t = torch.tensor(need, device=dev)
    first = torch.cumsum(need_t, 0) - need_t
    col = torch.arange(cols, device=dev)
    table = torch.where(col < need_t[:, None], order[(first[:, None] + col).clamp(max=pages - 1)], -1)
    free = torch.full((pages,), -1, device=dev, dtype=torch.int32)
    free[:pages - sum(need)] = order[sum(need):]
    b, t = len(rows), sum(new)
    s = dict(page_table=table.to(torch.int32).contiguous(), lens=torch.tensor(held, device=dev, dtype=torch.int32),
             free=free, counters=torch.tensor([pages - sum(need), 0], device=dev, dtype=torch.int32),
             rows=torch.tensor(rows, device=dev, dtype=torch.int32), new=torch.tensor(new, device=dev, dtype=torch.int32),
             cu_tokens=torch.zeros(b + 1, device=dev, dtype=torch.int32), batch_lens=torch.zeros(b, device=dev, dtype=torch.int32),
             batch_table=torch.full((b, cols), -1, device=dev, dtype=torch.int32),
             positions=torch.zeros(t, device=dev, dtype=torch.int32), slots=torch.zeros(t, device=dev, dtype=torch.int64),
             taken=taken, entries=sum(_ceil(held[r] + n, p) for r, n in zip(rows, new)))
    if own:
        import speculative_decoding_draft_tcgen05_gb300 as pkg
        s["pool"] = pkg.PagePool(s["page_table"], s["lens"], s["free"], s["counters"], page_size=p)
        s["batch"] = pkg.PagedBatch(s["cu_tokens"], s["batch_lens"], s["batch_table"], max_tokens=max(new))
    return s


def _prepare_linear(case, gen, dev):
    m, n, k = case["m"], case["n"], case["k"]
    dt = getattr(torch, case["dtype"])
    yt = torch.float32 if case["out"] == "float32" else dt
    wide = torch.randn(m, k + case["pad"], device=dev, generator=gen, dtype=dt)
    s = dict(x=wide[:, :k], w=torch.randn(n, k, device=dev, generator=gen, dtype=dt).mul_(k ** -0.5),
             bias=torch.randn(n, device=dev, generator=gen, dtype=dt) if case["bias"] else None,
             residual=torch.randn(m, n, device=dev, generator=gen, dtype=yt) if case["residual"] else None,
             out=torch.empty(m, n, device=dev, dtype=yt))
    if own:
        import speculative_decoding_draft_tcgen05_gb300 as pkg
        s["layer"] = pkg.Linear(s["w"], s["bias"], activation=case["act"], out_dtype=yt)
    return s


def _prepare_logits(case, gen, dev):
    b, t, v = case["batch"], case["rows"], case["vocab"]
    dt = getattr(torch, case["dtype"])
    total, prompt = _histories(case)
    s = dict(logits=(2.5 * torch.randn(b, t, v, device=dev, generator=gen)).to(dt))

    def tokens(*shape):  # a few tokens are frequent, most are rare
        return (v * torch.rand(*shape, device=dev, generator=gen) ** 4).to(torch.int32).clamp(max=v - 1)

    def per_sequence(lo, hi):
        return lo + (hi - lo) * torch.rand(b, device=dev, generator=gen)
    s["tokens"], s["draft"] = tokens(b, max(max(total), 1)), tokens(b, t - 1) if t > 1 else None
    s["lens"], s["prompt_lens"] = (torch.tensor(x, device=dev, dtype=torch.int32) for x in (total, prompt))
    if case["penalties"]:
        s.update(repetition=per_sequence(0.9, 1.4), presence=per_sequence(-0.2, 0.8), frequency=per_sequence(0, 0.5))
    if case["bias"]:
        # entries of a list are distinct here: a random start and an odd step through the vocabulary
        first = torch.randint(0, v, (b, 1), device=dev, generator=gen)
        s["bias_ids"] = ((first + torch.arange(case["bias"], device=dev) * (v // case["bias"])) % v).to(torch.int32)
        s["bias_values"] = torch.randn(b, case["bias"], device=dev, generator=gen)
    if case["mask"]:
        words = _ceil(v, 32)
        s["mask"] = torch.randint(-2 ** 31, 2 ** 31, (b, t, words), device=dev, generator=gen, dtype=torch.int64).to(torch.int32)
        if case["empty"]:
            s["mask"][0, 0] = 0
    if case["temperature"]:
        s["temperature"] = per_sequence(0.5, 1.3)
    s["out"] = {"argmax": lambda: torch.empty(b, t, device=dev, dtype=torch.int32),
                "probs": lambda: torch.empty(b, t, v, device=dev),
                "logits": lambda: torch.empty(b, t, v, device=dev, dtype=dt)}[case["want"]]()
    if own:
        import speculative_decoding_draft_tcgen05_gb300 as pkg
        s["rules"] = pkg.LogitsRules(s["tokens"], s["lens"], s["prompt_lens"],
                                     **{name: s.get(name) for name in ("repetition", "presence", "frequency", "bias_ids",
                                                                       "bias_values", "temperature")})
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"pages": _own_pages, "linear": _own_linear, "logits": _own_logits}[op](s)
    return {"pages": _plain_pages, "linear": _plain_linear, "logits": _plain_logits}[op](s)


# ------------------------------------------------------------ the calls a user makes
def _own_pages(s):
    s["pool"].extend(s["batch"], s["new"], rows=s["rows"], positions=s["positions"], slots=s["slots"])
    s["pool"].trim(s["new"], rows=s["rows"])
    return {name: s[name] for name in ("cu_tokens", "batch_lens", "batch_table", "positions", "slots", "page_table", "lens",
                                       "free", "counters")}


def _own_linear(s):
    return s["layer"](s["x"], s["out"], residual=s["residual"])


def _own_logits(s):
    import speculative_decoding_draft_tcgen05_gb300 as pkg
    where = {"argmax": "argmax", "probs": "probs", "logits": "out"}[s["case"]["want"]]
    pkg.dflash_logits_adjust(s["logits"], s["rules"], draft=s["draft"], mask=s.get("mask"), **{where: s["out"]})
    return s["out"]


# ------------------------------------------------------------ the plain forms
def _plain_pages(s):
    """Enough pages are free in every case, so every sequence gets its tokens."""
    c, p = s["case"], s["case"]["page"]
    dev = s["lens"].device
    rows, new, old = s["rows"].long(), s["new"].long(), s["lens"].long()[s["rows"].long()]
    length = old + new
    held, pages = (old + p - 1) // p, (length + p - 1) // p
    take = pages - held
    count = s["counters"][0].long()
    # new pages, from the top of the stack in the order of the batch
    seq = torch.repeat_interleave(torch.arange(c["batch"], device=dev), take, output_size=s["taken"])
    i = torch.arange(s["taken"], device=dev)
    nth = i - (torch.cumsum(take, 0) - take)[seq]
    column = held[seq] + nth
    s["page_table"][rows[seq], column] = s["free"][count - 1 - i]
    s["lens"][rows] = length.to(torch.int32)
    s["counters"][0] -= s["taken"]
    # what the batch's calls take
    cu = torch.cumsum(new, 0)
    s["cu_tokens"][0] = 0
    s["cu_tokens"][1:] = cu.to(torch.int32)
    s["batch_lens"].copy_(length)
    entry = torch.arange(c["cols"], device=dev) < pages[:, None]
    s["batch_table"].copy_(torch.where(entry, s["page_table"][rows], s["batch_table"]))
    of = torch.repeat_interleave(torch.arange(c["batch"], device=dev), new, output_size=s["positions"].shape[0])
    at = old[of] + torch.arange(s["positions"].shape[0], device=dev) - (cu - new)[of]
    s["positions"].copy_(at)
    s["slots"].copy_(s["page_table"][rows[of], at // p].long() * p + at % p)
    # the step's tokens are given back: their pages return to the places that they were taken from
    back = s["lens"].long()[rows] - new
    gone = (length + p - 1) // p - (back + p - 1) // p
    count = s["counters"][0].long()
    s["free"][count + s["taken"] - 1 - i] = s["page_table"][rows[seq], (back + p - 1)[seq] // p + nth]
    s["lens"][rows] = back.to(torch.int32)
    s["counters"][0] += gone.sum()
    return {name: s[name] for name in ("cu_tokens", "batch_lens", "batch_table", "positions", "slots", "page_table", "lens",
                                       "free", "counters")}


def _plain_linear(s):
    c = s["case"]
    y = torch.matmul(s["x"].float(), s["w"].float().t())
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["act"] == "relu":
        y = torch.where(y < 0, torch.zeros_like(y), y)
    elif c["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif c["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * 0.5 ** 0.5))
    elif c["act"] == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh((2 / math.pi) ** 0.5 * (y + 0.044715 * y * y * y)))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return s["out"].copy_(y)


def _plain_logits(s):
    c = s["case"]
    b, t, v = c["batch"], c["rows"], c["vocab"]
    y = s["logits"].float()
    if c["penalties"]:
        dev = y.device
        place = torch.arange(s["tokens"].shape[1], device=dev)
        history = (place < s["lens"][:, None]).int()
        output = history * (place >= s["prompt_lens"][:, None]).int()
        ids = s["tokens"].long()
        seen = torch.zeros(b, v, device=dev, dtype=torch.int32).scatter_add_(1, ids, history)
        count = torch.zeros(b, v, device=dev, dtype=torch.int32).scatter_add_(1, ids, output)
        seen, count = seen[:, None].repeat(1, t, 1), count[:, None].repeat(1, t, 1)
        for j in range(t - 1):  # a position sees the drafts before it
            later = s["draft"][:, j].long()[:, None, None].expand(b, t - 1 - j, 1)
            one = torch.ones(later.shape, device=dev, dtype=torch.int32)
            seen[:, j + 1:].scatter_add_(2, later, one)
            count[:, j + 1:].scatter_add_(2, later, one)
        rho = s["repetition"][:, None, None]
        y = torch.where(seen > 0, torch.where(y > 0, y / rho, y * rho), y)
        y = y - s["frequency"][:, None, None] * count
        y = y - s["presence"][:, None, None] * (count > 0)
    if c["bias"]:
        y = y.scatter_add(2, s["bias_ids"].long()[:, None].expand(b, t, c["bias"]),
                          s["bias_values"][:, None].expand(b, t, c["bias"]))
    if c["mask"]:
        token = torch.arange(v, device=y.device)
        allowed = (s["mask"][:, :, token // 32] >> (token % 32)) & 1
        y = torch.where(allowed > 0, y, float("-inf"))
    if c["want"] == "logits":
        return s["out"].copy_(y)
    top = y.amax(dim=-1, keepdim=True)
    if c["want"] == "argmax":
        token = torch.arange(v, device=y.device)
        best = torch.where(y == top, token, v).amin(dim=-1)
        return s["out"].copy_(torch.where(top[..., 0] == float("-inf"), -1, best))
    if c["temperature"]:
        y, top = y / s["temperature"][:, None, None], top / s["temperature"][:, None, None]
    e = torch.exp(y - torch.where(top == float("-inf"), 0.0, top))
    total = e.sum(dim=-1, keepdim=True)
    return s["out"].copy_(e / torch.where(total == 0, 1.0, total))


# ------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"pages": _exact_pages, "linear": _exact_linear, "logits": _exact_logits}[case["op"]](s)


def _exact_pages(s):
    c, p = s["case"], s["case"]["page"]
    got = {name: s[name].cpu().clone() for name in ("cu_tokens", "batch_lens", "batch_table", "positions", "slots",
                                                    "page_table", "lens", "free", "counters")}
    stack = got["free"][:int(got["counters"][0])].tolist()
    token = 0
    for b, (r, n) in enumerate(zip(s["rows"].tolist(), s["new"].tolist())):
        length = int(got["lens"][r])
        row = got["page_table"][r].tolist()
        used = _ceil(length, p)
        for at in range(length, length + n):
            if at // p == used:
                row[used] = stack.pop()
                used += 1
            got["positions"][token], got["slots"][token] = at, row[at // p] * p + at % p
            token += 1
        got["page_table"][r] = torch.tensor(row, dtype=torch.int32)
        got["batch_table"][b, :used] = got["page_table"][r, :used]
        got["batch_lens"][b], got["cu_tokens"][b + 1] = length + n, token
    return got  # (the tokens are given back in the order that leaves lengths and stack as they were)


def _exact_linear(s):
    act = {"none": lambda z: z, "relu": lambda z: z.clamp(min=0), "silu": lambda z: z * torch.sigmoid(z),
           "gelu": lambda z: z * torch.special.ndtr(z),
           # 1/2 (1 + tanh(u)) = sigmoid(2 u)
           "gelu_tanh": lambda z: z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z.pow(3)))}[s["case"]["act"]]
    wt = s["w"].double().T
    out = torch.empty(s["out"].shape, device=wt.device, dtype=torch.float64)
    for i in range(0, out.shape[0], 1024):
        z = s["x"][i:i + 1024].double() @ wt
        if s["bias"] is not None:
            z += s["bias"].double()
        out[i:i + 1024] = act(z)
    return out if s["residual"] is None else out + s["residual"].double()


def _exact_logits(s):
    c = s["case"]
    want = c["want"]
    out = torch.empty(s["out"].shape, device=s["out"].device, dtype=torch.int32 if want == "argmax" else torch.float64)
    for b in range(c["batch"]):
        n, prompt = int(s["lens"][b]), int(s["prompt_lens"][b])
        for t in range(c["rows"]):
            z = s["logits"][b, t].double()
            if c["penalties"]:
                rho, alpha, beta = (float(s[name][b]) for name in ("repetition", "presence", "frequency"))
                drafts = s["draft"][b, :t] if t else s["tokens"][b, :0]
                answered = torch.cat([s["tokens"][b, prompt:n], drafts]).long()
                times = torch.bincount(answered, minlength=c["vocab"]).double()
                known = torch.cat([s["tokens"][b, :n], drafts]).long().unique()
                z[known] = torch.where(z[known] > 0, z[known] / rho, z[known] * rho)
                z -= beta * times + alpha * (times > 0)
            if c["bias"]:
                z[s["bias_ids"][b].long()] += s["bias_values"][b].double()
            if c["mask"]:
                bits = s["mask"][b, t].long()[:, None] >> torch.arange(32, device=z.device) & 1
                z[bits.view(-1)[:c["vocab"]] == 0] = -math.inf
            if want == "logits":
                out[b, t] = z
            elif want == "argmax":
                best = z.max()
                out[b, t] = -1 if best == -math.inf else int((z == best).nonzero()[0])
            elif z.max() == -math.inf:
                out[b, t] = 0
            else:
                out[b, t] = torch.softmax(z / (float(s["temperature"][b]) if c["temperature"] else 1.0), 0)
    return out

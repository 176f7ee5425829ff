"""The attention block's operators (per-head norm and rotation, append to a
paged cache, attention over it) against plain fp64 implementations, through
the C ABI. Tolerances are worst-case rounding bounds, written beside each."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP16, FP8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
UNIT = {t: torch.finfo(t).eps / 2 for t in (BF16, FP16)}  # largest relative error of one rounding
SCALES = dict(k_scale=0.05, v_scale=0.03)


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from speculative_decoding_draft_tcgen05_gb300 import build
    build.build()
    import speculative_decoding_draft_tcgen05_gb300 as p
    p.lib()
    return p


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rope_table(n, rotary, base=10000.0):
    inv = base ** (-torch.arange(0, rotary, 2, device="cuda", dtype=torch.float64) / rotary)
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def ref_transform(x, w, table, pos, rotary, interleaved, eps):
    """(the transform of x in fp64, the sum of the magnitudes that a result is made of)"""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    y, mag = x.clone(), x.abs()
    for i in range(rotary // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
        c, s = table[pos, i].double()[:, None], table[pos, rotary // 2 + i].double()[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
        mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, mag


def check_rounded(got, y, mag):
    # one rounding to 16 bits, fp32 arithmetic (mean of up to 256 squares, rsqrt, a few products) before it
    tol = UNIT[got.dtype] * y.abs() * 1.01 + 4e-6 * mag + 1e-7
    bad = (got.double() - y).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((got.double() - y).abs().max()):.3g}"


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("tokens,heads,kv_heads,d,dtype,rotary,inter,norm", [
    (1, 32, 8, 128, BF16, 128, False, True),
    (8, 32, 8, 128, BF16, 128, False, True),
    (257, 20, 4, 128, FP16, 64, False, True),
    (33, 5, 1, 64, BF16, 64, True, True),      # heads that fill no lane group evenly
    (100, 7, 7, 64, FP16, 32, True, False),
    (19, 1, 3, 128, BF16, 16, False, False),   # more key heads than query heads
    (41, 3, 2, 256, FP16, 256, False, True),
    (41, 3, 2, 256, BF16, 128, True, True),
    (65, 9, 2, 128, BF16, 0, False, True),     # norm alone
    (3000, 40, 8, 128, BF16, 128, False, True),
])
def test_norm_rope(pkg, tokens, heads, kv_heads, d, dtype, rotary, inter, norm):
    g = gen(tokens * 7 + heads)
    qkv = (2 * torch.randn(tokens, heads + 2 * kv_heads, d, device="cuda", generator=g)).to(dtype)
    q, k = qkv[:, :heads], qkv[:, heads:heads + kv_heads]  # strided slices of a packed projection
    wq, wk = ((1 + 0.3 * torch.randn(d, device="cuda", generator=g)).to(dtype) if norm else None for _ in range(2))
    table = rope_table(5000, rotary) if rotary else None
    pos = torch.randint(0, 5000, (tokens,), device="cuda", generator=g, dtype=torch.int32)
    tr = pkg.QkTransform(table, interleaved=inter, q_weight=wq, k_weight=wk, eps=1e-5)
    qo, ko = torch.empty(tokens, heads, d, device="cuda", dtype=dtype), torch.empty(tokens, kv_heads, d, device="cuda", dtype=dtype)
    pkg.dflash_qk_norm_rope(q, k, qo, ko, tr, pos)
    for x, w, o in ((q, wq, qo), (k, wk, ko)):
        check_rounded(o, *ref_transform(x, w, table, pos.long(), rotary, inter, 1e-5))
    before = qkv.clone()
    pkg.dflash_qk_norm_rope(q, k, q, k, tr, pos)  # in place, strided
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, heads + kv_heads:], before[:, heads + kv_heads:])
    ko2 = torch.empty_like(ko)
    pkg.dflash_qk_norm_rope(None, before[:, heads:heads + kv_heads], None, ko2, tr, pos)  # keys alone
    assert torch.equal(ko2, ko)


def test_norm_rope_special_values(pkg):
    d, table = 128, rope_table(16, 128)
    q = torch.zeros(4, 2, d, device="cuda", dtype=BF16)
    q[1, 0, 3] = float("inf")
    q[2, 1, 5] = float("nan")
    q[3] = 1e30                                        # squares overflow fp32: the norm becomes 0
    w = torch.ones(d, device="cuda", dtype=BF16)
    out = torch.empty_like(q)
    pos = torch.tensor([0, 1, -5, 400], device="cuda", dtype=torch.int32)  # the last two are clamped to the table
    pkg.dflash_qk_norm_rope(q, None, out, None, pkg.QkTransform(table, q_weight=w), pos)
    assert torch.equal(out[0], torch.zeros_like(out[0]))        # 0 / sqrt(0 + eps)
    assert torch.isnan(out[1, 0]).any() and torch.equal(out[1, 1], torch.zeros_like(out[1, 1]))
    assert torch.isnan(out[2, 1]).any() and torch.equal(out[2, 0], torch.zeros_like(out[2, 0]))
    x = torch.randn(2, 2, d, device="cuda").to(BF16)
    a, b = torch.empty_like(x), torch.empty_like(x)
    tr = pkg.QkTransform(table)
    pkg.dflash_qk_norm_rope(x, None, a, None, tr, torch.tensor([-5, 400], device="cuda", dtype=torch.int32))
    pkg.dflash_qk_norm_rope(x, None, b, None, tr, torch.tensor([0, 15], device="cuda", dtype=torch.int32))
    assert torch.equal(a, b)


# ------------------------------------------------------------------ a paged cache and its batch
class Paged:
    """Sequences with `new` new tokens that end at lengths `lens`, pages in random order; free pages and slots past
    a sequence's end hold NaN."""

    def __init__(self, pkg, new, lens, *, heads, kv_heads, d, dtype, cache=None, page=16, head_major=False, seed=0,
                 extra_cols=0, pad=0, poison=True):
        cache = dtype if cache is None else cache
        g = gen(seed)
        self.g, self.pkg, self.new, self.lens, self.page, self.d = g, pkg, new, lens, page, d
        self.heads, self.kv_heads, self.dtype, self.cache_dtype = heads, kv_heads, dtype, cache
        need = [-(-n // page) for n in lens]
        total = sum(need) + 3
        order = torch.randperm(total, device="cuda", generator=g).tolist()
        cols = max(max(need), 1) + extra_cols
        table = torch.full((len(lens), cols), -1, dtype=torch.int32)
        used, at = torch.zeros(total, page, dtype=torch.bool), 0
        for b, n in enumerate(need):
            pages = order[at:at + n]
            at += n
            table[b, :n] = torch.tensor(pages, dtype=torch.int32)
            for j, pg in enumerate(pages):
                used[pg, :min(page, lens[b] - j * page)] = True
        self.table, self.used = table.cuda(), used.cuda()
        shape = (total, kv_heads, page, d) if head_major else (total, page, kv_heads, d)
        self.raw = []
        for s in SCALES.values():
            x = torch.randn(shape, device="cuda", generator=g)
            if head_major:
                x = x.transpose(1, 2)
            if poison:
                x = torch.where(self.used[:, :, None, None], x, torch.full_like(x, math.nan))
            x = (x / s).to(FP8) if cache is FP8 else x.to(dtype)
            x = x.transpose(1, 2).contiguous().transpose(1, 2) if head_major else x.contiguous()
            self.raw.append(x)
        self.k, self.v = self.raw
        sc = SCALES if cache is FP8 else {}
        self.ks, self.vs = (sc.get("k_scale", 1.0), sc.get("v_scale", 1.0))
        self.tokens = sum(new) + pad
        self.cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], device="cuda", dtype=torch.int32)
        self.len_t = torch.tensor(lens, device="cuda", dtype=torch.int32)
        self.cache = pkg.PagedCache(self.k, self.v, **sc)
        self.batch = pkg.PagedBatch(self.cu, self.len_t, self.table, max_tokens=max(max(new), 1))
        self.layer = pkg.PagedAttention(heads=heads, kv_heads=kv_heads, head_dim=d, page_size=page, dtype=dtype,
                                        cache_dtype=cache, max_batch=len(lens))

    def rows(self, heads, std=1.0):
        return (std * torch.randn(self.tokens, heads, self.d, device="cuda", generator=self.g)).to(self.dtype)

    def gather(self, x, b, scale):
        n = self.lens[b]
        at = torch.arange(n, device="cuda")
        pg = self.table[b].long()[at // self.page]
        return x[pg, at % self.page].float().double() * scale

    def ref(self, q, causal, window, scale):
        """fp64: (out, lse, sum of weight * |v|, largest |v| * keys) of every row"""
        T, G = q.shape[0], self.heads // self.kv_heads
        out = torch.zeros(T, self.heads, self.d, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(out)
        lse = torch.full((T, self.heads), -math.inf, dtype=torch.float64, device="cuda")
        row = 0
        for b, n in enumerate(self.new):
            L = self.lens[b]
            place = torch.arange(L - n, L, device="cuda")[:, None]
            key = torch.arange(L, device="cuda")[None]
            see = torch.ones(n, L, dtype=torch.bool, device="cuda")
            if causal:
                see &= key <= place
            if window:
                see &= key > place - window
            if n and L:
                k, v = self.gather(self.k, b, f32(self.ks)), self.gather(self.v, b, f32(self.vs))
                for h in range(self.heads):
                    s = (q[row:row + n, h].double() @ k[:, h // G].T * scale).masked_fill(~see, -math.inf)
                    z = torch.logsumexp(s, 1)
                    w = torch.where(see, (s - torch.where(z.isinf(), 0.0, z)[:, None]).exp(), 0.0)
                    lse[row:row + n, h] = z
                    out[row:row + n, h] = w @ v[:, h // G]
                    mag[row:row + n, h] = w @ v[:, h // G].abs()
            row += n
        return out, lse, mag

    def check(self, q, causal=True, window=0, scale=None, lse=True):
        sc = self.d ** -0.5 if scale is None else scale
        out = torch.full((self.tokens, self.heads, self.d), 7.0, device="cuda", dtype=self.dtype)
        z = torch.full((self.tokens, self.heads), 7.0, device="cuda") if lse else None
        self.layer.attend(self.cache, self.batch, q, out, lse=z, causal=causal, window=window, scale=scale)
        self.layer.sync_status()
        ref, rl, mag = self.ref(q, causal, window, sc)
        n = sum(self.new)
        assert (out[n:] == 7).all()  # padding rows are not written
        # weights rounded to 16 bits, one rounding of the result, and fp32 scores (128 products of fp32 accuracy each):
        # 2 units and 5e-4 of the sum of the weighted magnitudes; fp16 weights below 2^-14 lose up to 2^-25 absolutely
        unit = UNIT[self.dtype]
        weight_unit = UNIT[FP16] if self.cache_dtype is FP8 else unit
        small = 2.0 ** -25 * max(self.lens) * 6 if weight_unit == UNIT[FP16] else 0.0
        tol = (weight_unit + 5e-4) * mag + unit * ref.abs() + small + 1e-6
        err = (out[:n].double() - ref[:n]).abs()
        bad = ~(err <= tol[:n])
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(err.max()):.3g}"
        if lse:
            assert (z[n:] == 7).all()
            gone = rl[:n].isinf()
            assert torch.equal(z[:n].isinf(), gone) and (z[:n][gone] < 0).all()
            # the score's fp32 error (<= D * 2^-24 * sum |q k| * scale < 2e-4 at these values)
            assert ((z[:n].double() - rl[:n]).abs()[~gone] <= 2e-4 + 1e-6 * rl[:n].abs()[~gone]).all()
        return out


def f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


KINDS = [(BF16, None), (FP16, None), (BF16, FP8), (FP16, FP8)]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens", [
    ([1], [1]),                                   # one token, one key
    ([1], [777]),
    ([8], [8]), ([8], [2049]),
    ([3], [65]), ([5], [64]),
    ([1, 8, 0, 4, 2], [16, 100, 50, 4, 333]),     # one sequence without new tokens
    ([1] * 40, list(range(1, 1200, 30))),
])
def test_attend_few_rows(pkg, dtype, cache, d, new, lens):
    s = Paged(pkg, new, lens, heads=8, kv_heads=2, d=d, dtype=dtype, cache=cache, seed=len(new) + lens[0])
    s.check(s.rows(8, 1.5))


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (6, 6), (7, 1), (40, 8), (33, 3), (64, 1)])
@pytest.mark.parametrize("page,head_major", [(16, False), (48, True), (256, False)])
def test_attend_heads_and_pages(pkg, heads, kv_heads, page, head_major):
    s = Paged(pkg, [4, 1, 7], [150, 31, 600], heads=heads, kv_heads=kv_heads, d=128, dtype=BF16, page=page,
              head_major=head_major, seed=heads, extra_cols=5)
    s.check(s.rows(heads))


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("d,heads,kv_heads", [(64, 4, 2), (128, 10, 2)])
@pytest.mark.parametrize("new,lens", [
    ([17], [17]), ([100], [100]), ([127, 129], [127, 400]), ([64, 1, 300], [1000, 513, 300]), ([513], [2000]),
])
def test_attend_chunks(pkg, dtype, cache, d, heads, kv_heads, new, lens):
    s = Paged(pkg, new, lens, heads=heads, kv_heads=kv_heads, d=d, dtype=dtype, cache=cache, page=32, seed=new[0])
    s.check(s.rows(heads, 1.5))
    s.check(s.rows(heads), causal=False, lse=False)


@pytest.mark.parametrize("cache", [None, FP8])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [1, 15, 64, 100, 5000])
@pytest.mark.parametrize("new,lens", [([8, 1, 3], [900, 300, 3]), ([200, 1], [700, 90])])
def test_attend_window(pkg, new, lens, window, causal, cache):
    s = Paged(pkg, new, lens, heads=8, kv_heads=2, d=128, dtype=BF16, cache=cache, seed=window)
    # pages that no row's window reaches have been given back: their entries are gone
    for b, (n, L) in enumerate(zip(new, lens)):
        s.table[b, :max(0, L - n + 1 - window) // s.page] = -1
    _windowed_check(s, s.rows(8), causal, window)


def _windowed_check(s, q, causal, window):
    """check() for a batch whose evicted pages have no table entry: the reference sees zeros there."""
    real, plain = s.gather, Paged.gather

    def gather(x, b, scale):
        t = s.table.clone()
        s.table[b] = t[b].clamp(min=0)
        got = plain(s, x, b, scale)
        s.table[:] = t
        at = torch.arange(s.lens[b], device="cuda") // s.page
        got[t[b].long()[at] < 0] = 0
        return got
    s.gather = gather
    try:
        s.check(q, causal=causal, window=window)
    finally:
        s.gather = real


@pytest.mark.parametrize("cache", [None, FP8])
@pytest.mark.parametrize("new,lens", [
    ([3, 2], [0, 0]),        # nothing in the cache: no row sees a key
    ([8, 1], [5, 64]),       # more new tokens than places: the first three rows see nothing
    ([40, 1], [7, 1]),
    ([300], [10]),
])
def test_attend_rows_that_see_nothing(pkg, new, lens, cache):
    s = Paged(pkg, new, lens, heads=8, kv_heads=2, d=64, dtype=FP16, cache=cache, seed=3)
    out = s.check(s.rows(8))
    seen = [max(0, L - n) for n, L in zip(new, lens)]
    assert (out[0] == 0).all() and all(x >= 0 for x in seen)
    if lens[0]:
        s.check(s.rows(8), causal=False)


@pytest.mark.parametrize("cache", [None, FP8])
@pytest.mark.parametrize("new", [4, 90])
def test_attend_scores_of_any_size(pkg, new, cache):
    """Rows whose scores span hundreds of powers of two, in both directions along the keys, and constant ones."""
    s = Paged(pkg, [new], [700], heads=4, kv_heads=4, d=64, dtype=BF16, cache=cache, seed=9, poison=False)
    ramp = torch.linspace(-1, 1, 700, device="cuda")
    at = torch.arange(700, device="cuda")
    kk = torch.zeros(700, 4, 64, device="cuda")
    kk[:, 0, 0], kk[:, 1, 0], kk[:, 2, 0] = ramp, -ramp, 1.0
    kk[350, 3, 0] = 1.0
    page = s.table[0].long()[at // 16]
    val = kk / (SCALES["k_scale"] if cache is FP8 else 1)
    s.k[page, at % 16] = val.to(s.k.dtype) if cache is None else val.to(FP8)
    q = torch.zeros(new, 4, 64, device="cuda", dtype=BF16)
    q[..., 0] = 2048.0
    s.check(q)
    q[..., 0] = 1e-30
    s.check(q)


def test_attend_no_contamination_between_sequences(pkg):
    """One sequence's NaN keys and values change no other sequence's rows."""
    s = Paged(pkg, [2, 2, 2], [100, 130, 90], heads=4, kv_heads=2, d=64, dtype=BF16, seed=1)
    q = s.rows(4)
    a = s.layer.attend(s.cache, s.batch, q)
    s.k[s.table[1, 2].long()] = math.nan
    s.v[s.table[1, 2].long()] = math.nan
    b = s.layer.attend(s.cache, s.batch, q)
    assert torch.equal(a[:2], b[:2]) and torch.equal(a[4:], b[4:]) and b[2:4].isnan().all()


@pytest.mark.parametrize("cache", [None, FP8])
@pytest.mark.parametrize("new,lens", [
    ([1, 2] * 300, [1 + 7 * i % 90 + 1 for i in range(600)]),          # more sequences than are planned in shared memory
    ([3] * 30 + [200, 0, 150] + [1] * 12, [40 + i for i in range(45)]),  # long ones among more than a warp of them;
                                                                         # some with more new tokens than places
    ([0, 0, 5, 0], [3, 0, 77, 9]),                                       # hardly any rows
])
def test_attend_many_sequences(pkg, new, lens, cache):
    s = Paged(pkg, new, lens, heads=4, kv_heads=2, d=64, dtype=BF16, cache=cache, seed=len(new), pad=5)
    q = s.rows(4)
    s.check(q)
    s.batch.c.max_tokens = 1  # by the other kernel
    s.check(q)


@pytest.mark.parametrize("heads", [40, 300])
@pytest.mark.parametrize("cache", [None, FP8])
def test_attend_wide_groups(pkg, heads, cache):
    """One key head for 40 and 300 query heads: rows of a token spread over several tiles."""
    s = Paged(pkg, [3, 1], [500, 70], heads=heads, kv_heads=1, d=64, dtype=FP16, cache=cache, seed=heads)
    s.check(s.rows(heads))
    s.check(s.rows(heads), window=33)


@pytest.mark.parametrize("cache", [None, FP8])
@pytest.mark.parametrize("heads,kv_heads", [(5, 5), (14, 7), (24, 12), (80, 40), (500, 500), (97, 97)])
def test_attend_numbers_of_key_heads(pkg, heads, kv_heads, cache):
    """Key heads that divide the grid, leave CTAs idle, are walked one after the other, or outnumber the CTAs; items
    of one CTA, of a few and of many."""
    s = Paged(pkg, [1, 4, 0, 2], [700, 90, 33, 4], heads=heads, kv_heads=kv_heads, d=64, dtype=BF16, cache=cache, seed=kv_heads)
    s.check(s.rows(heads))
    s.check(s.rows(heads), window=70)
    long = Paged(pkg, [2], [6000], heads=heads, kv_heads=kv_heads, d=64, dtype=FP16, cache=cache, seed=kv_heads + 1)
    long.check(long.rows(heads))


def test_attend_masked_keys_may_be_anything(pkg):
    """NaN and infinite keys at places that some tokens do not see leave those tokens alone; a value there must be finite."""
    for new in (6, 90):
        s = Paged(pkg, [new], [300], heads=4, kv_heads=2, d=64, dtype=BF16, seed=new, poison=False)
        q = s.rows(4)
        want = s.layer.attend(s.cache, s.batch, q)
        at = 300 - 2  # seen by the last two tokens only
        page = int(s.table[0, at // 16])
        s.k[page, at % 16] = math.nan
        got = s.layer.attend(s.cache, s.batch, q)
        assert torch.equal(got[:-2], want[:-2]) and got[-2:].isnan().all()
        s.k[page, at % 16] = math.inf
        got = s.layer.attend(s.cache, s.batch, q)
        assert torch.equal(got[:-2], want[:-2])


@pytest.mark.parametrize("new,length", [(8, 40000), (1, 70001), (300, 20000)])
def test_attend_long(pkg, new, length):
    """Long contexts: the keys of an item split over many CTAs."""
    s = Paged(pkg, [new], [length], heads=8, kv_heads=2, d=128, dtype=BF16, page=64, seed=5)
    s.check(s.rows(8, 1.5))


def test_attend_strides_streams_and_repeats(pkg):
    s = Paged(pkg, [8, 5, 70], [300, 5, 200], heads=8, kv_heads=2, d=128, dtype=BF16, seed=2, pad=6)
    packed = torch.randn(s.tokens, 12, 128, device="cuda").to(BF16)
    q = packed[:, 2:10]
    a = s.check(q)
    buf = torch.zeros(s.tokens, 3, 8, 128, device="cuda", dtype=BF16)
    s.layer.attend(s.cache, s.batch, q.contiguous(), buf[:, 1])
    n = sum(s.new)
    assert torch.equal(buf[:n, 1], a[:n]) and (buf[:, 0] == 0).all() and (buf[:, 2] == 0).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = s.layer.attend(s.cache, s.batch, q)
    side.synchronize()
    assert torch.equal(c[:n], a[:n])
    for _ in range(20):  # always the same bits, whatever order the CTAs run in
        assert torch.equal(s.layer.attend(s.cache, s.batch, q)[:n], a[:n])


def test_attend_in_a_graph_follows_the_lengths(pkg):
    s = Paged(pkg, [4, 4], [400, 400], heads=8, kv_heads=2, d=64, dtype=FP16, seed=4, poison=False)
    q, out = s.rows(8), torch.empty(8, 8, 64, device="cuda", dtype=FP16)
    s.layer.attend(s.cache, s.batch, q, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.layer.attend(s.cache, s.batch, q, out)
    for lens in ([400, 400], [37, 201], [4, 399]):
        s.lens = lens
        s.len_t.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = s.layer.attend(s.cache, s.batch, q)
        assert torch.equal(out, want)
        s.check(q)


def test_attend_hints_and_bad_places(pkg):
    """max_tokens below a sequence's new tokens changes no result; bad page ids and lengths are latched, never followed."""
    s = Paged(pkg, [40, 3], [300, 77], heads=8, kv_heads=2, d=64, dtype=BF16, seed=6)
    q = s.rows(8)
    s.batch.c.max_tokens = 1
    s.check(q)
    s.batch.c.max_tokens = 40
    s.check(q)
    good = s.table.clone()
    for value in (-1, 1 << 30):
        s.table[1, 1] = value
        s.layer.attend(s.cache, s.batch, q)
        with pytest.raises(pkg.DflashError) as e:
            s.layer.sync_status()
        assert e.value.status == pkg.DFLASH_ERR_DEVICE_CHECK
        s.table.copy_(good)
    s.len_t[1] = 1 << 30
    s.layer.attend(s.cache, s.batch, q)
    with pytest.raises(pkg.DflashError) as e:
        s.layer.sync_status()
    assert e.value.status == pkg.DFLASH_ERR_DEVICE_CHECK
    s.len_t[1] = 77
    s.check(q)  # and nothing is left of it


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("d,heads,kv_heads,rotary,inter,norm", [
    (128, 8, 2, 128, False, True), (64, 6, 3, 32, True, False), (128, 5, 1, 64, False, True), (64, 33, 11, 0, False, True)])
@pytest.mark.parametrize("new,lens,page,head_major", [
    ([1], [1], 16, False), ([8], [2049], 16, True), ([1, 8, 0, 15, 40], [33, 8, 9, 700, 41], 48, False),
    ([2] * 70, list(range(2, 142, 2)), 16, False)])
def test_append(pkg, dtype, cache, d, heads, kv_heads, rotary, inter, norm, new, lens, page, head_major):
    s = Paged(pkg, new, lens, heads=heads, kv_heads=kv_heads, d=d, dtype=dtype, cache=cache, page=page,
              head_major=head_major, seed=len(new), pad=3, poison=False)
    q, k, v = s.rows(heads, 2.0), s.rows(kv_heads, 2.0), s.rows(kv_heads, 2.0)
    wq, wk = ((1 + 0.3 * torch.randn(d, device="cuda", generator=s.g)).to(dtype) if norm else None for _ in range(2))
    table = rope_table(4096, rotary) if rotary else None
    tr = pkg.QkTransform(table, interleaved=inter, q_weight=wq, k_weight=wk)
    kc, vc = s.k.clone(), s.v.clone()
    qo = torch.full_like(q, 7.0)
    s.layer.append(s.cache, s.batch, k, v, tr, q=q, q_out=qo)
    s.layer.sync_status()
    n = sum(new)
    places = torch.cat([torch.arange(L - m, L) for m, L in zip(new, lens)]).cuda()
    owner = torch.cat([torch.full((m,), b) for b, m in enumerate(new)]).cuda().long()
    pg, slot = s.table[owner, places // page].long(), places % page
    check_rounded(qo[:n], *ref_transform(q[:n], wq, table, places, rotary, inter, 1e-6))
    assert (qo[n:] == 7).all()
    y, mag = ref_transform(k[:n], wk, table, places, rotary, inter, 1e-6)
    if cache is FP8:
        for c, want, m, sc in ((s.k, y, mag, SCALES["k_scale"]), (s.v, v[:n].double(), v[:n].double().abs(), SCALES["v_scale"])):
            want, got = (want / f32(sc)).clamp(-448, 448), c[pg, slot].float().double()
            # one rounding to e4m3: half a step, relative 2^-4 or 2^-10 below 2^-6; fp32 arithmetic before it
            assert ((got - want).abs() <= 2.0 ** -4 * want.abs() * 1.01 + 2.0 ** -10 + 4e-6 * m / f32(sc)).all()
    else:
        check_rounded(s.k[pg, slot], y, mag)
        assert torch.equal(s.v[pg, slot], v[:n])
    s.k.view(torch.uint8)[pg, slot] = kc.view(torch.uint8)[pg, slot]  # nothing else was touched
    s.v.view(torch.uint8)[pg, slot] = vc.view(torch.uint8)[pg, slot]
    assert torch.equal(s.k.view(torch.uint8), kc.view(torch.uint8)) and torch.equal(s.v.view(torch.uint8), vc.view(torch.uint8))


def test_append_positions_saturation_and_bad_places(pkg):
    s = Paged(pkg, [3, 2], [40, 20], heads=4, kv_heads=2, d=64, dtype=BF16, cache=FP8, seed=8, poison=False)
    k, v = s.rows(2), s.rows(2)
    v[0, 0, :4] = torch.tensor([1e6, -1e6, math.inf, math.nan], device="cuda").to(BF16)
    table = rope_table(64, 64)
    tr = pkg.QkTransform(table)
    pos = torch.tensor([5, 6, 7, 0, 63], device="cuda", dtype=torch.int32)
    s.layer.append(s.cache, s.batch, k, v, tr, positions=pos)
    s.layer.sync_status()
    got = s.v[s.table[0, 37 // 16].long(), 37 % 16, 0, :4].float()
    assert got[:3].tolist() == [448.0, -448.0, 448.0] and got[3].isnan()
    y, mag = ref_transform(k, None, table, pos.long(), 64, False, 0.0)
    got = s.k[s.table[1, 1].long(), 20 % 16 - 1].float().double()
    want = y[4] / f32(SCALES["k_scale"])
    assert ((got - want).abs() <= 2.0 ** -4 * want.abs() * 1.01 + 2.0 ** -10 + 1e-4).all()
    kc = s.k.clone()
    for spoil, mend in ((lambda: s.table.__setitem__((0, 2), -1), None), (lambda: s.len_t.__setitem__(0, 2), None),
                        (lambda: s.len_t.__setitem__(0, 1 << 30), None)):
        t, n = s.table.clone(), s.len_t.clone()
        spoil()
        s.layer.append(s.cache, s.batch, k, v)
        with pytest.raises(pkg.DflashError) as e:
            s.layer.sync_status()
        assert e.value.status == pkg.DFLASH_ERR_DEVICE_CHECK
        s.table.copy_(t)
        s.len_t.copy_(n)
    free = [p for p in range(s.k.shape[0]) if p not in s.table.flatten().tolist()]
    assert torch.equal(s.k[free].view(torch.uint8), kc[free].view(torch.uint8))


def test_offsets_beyond_32_bits(pkg):
    """A cache whose keys alone span 6.4 GB: the pages in use lie past 2^32 bytes and 2^31 values."""
    pages, page, hk, d = 12300, 64, 32, 128
    k, v = (torch.empty(pages, page, hk, d, device="cuda", dtype=BF16) for _ in range(2))
    new, L = 4, 200
    ids = [pages - 1, 3, pages - 2, 8200]
    x = torch.randn(2, L, hk, d, device="cuda").to(BF16)
    at = torch.arange(L, device="cuda")
    pg = torch.tensor(ids, device="cuda")[at // page]
    k[pg, at % page], v[pg, at % page] = x[0], x[1]
    k[pg[-new:], at[-new:] % page] = 0
    v[pg[-new:], at[-new:] % page] = 0
    layer = pkg.PagedAttention(heads=hk, kv_heads=hk, head_dim=d, page_size=page, dtype=BF16, max_batch=1)
    batch = pkg.PagedBatch(torch.tensor([0, new], device="cuda", dtype=torch.int32),
                           torch.tensor([L], device="cuda", dtype=torch.int32),
                           torch.tensor([ids], device="cuda", dtype=torch.int32), max_tokens=new)
    cache = pkg.PagedCache(k, v)
    layer.append(cache, batch, x[0, -new:].contiguous(), x[1, -new:].contiguous())
    assert torch.equal(k[pg, at % page], x[0]) and torch.equal(v[pg, at % page], x[1])
    q = torch.randn(new, hk, d, device="cuda").to(BF16)
    out = layer.attend(cache, batch, q)
    layer.sync_status()
    s = torch.einsum("thd,khd->thk", q.double(), x[0].double()) / math.sqrt(d)
    s = s.masked_fill(at[None, None] > (L - new + torch.arange(new, device="cuda"))[:, None, None], -math.inf)
    w = s.softmax(-1)
    want, mag = (torch.einsum("thk,khd->thd", w, z) for z in (x[1].double(), x[1].double().abs()))
    assert ((out.double() - want).abs() <= (UNIT[BF16] + 5e-4) * mag + UNIT[BF16] * want.abs() + 1e-6).all()


# ------------------------------------------------------------------ refusals
def test_refusals(pkg):
    ok = dict(heads=8, kv_heads=2, head_dim=64, page_size=16, dtype=BF16, max_batch=2)
    for change, status in ((dict(heads=7), 2), (dict(kv_heads=0), 2), (dict(heads=2048, kv_heads=2048), 2),
                           (dict(head_dim=96), 2), (dict(page_size=24), 2), (dict(page_size=0), 2),
                           (dict(dtype=torch.float32), 2), (dict(cache_dtype=FP16), 2), (dict(max_batch=0), 1)):
        with pytest.raises(pkg.DflashError) as e:
            pkg.PagedAttention(**{**ok, **change})
        assert e.value.status == status, change
    s = Paged(pkg, [4, 4], [30, 40], heads=8, kv_heads=2, d=64, dtype=BF16, seed=1)
    q, k, v = s.rows(8), s.rows(2), s.rows(2)

    def refused(status, f):
        with pytest.raises(pkg.DflashError) as e:
            f()
        assert e.value.status == status
    inv = pkg.DFLASH_ERR_INVALID_ARG
    refused(inv, lambda: s.layer.attend(s.cache, s.batch, q, q))                        # in place
    refused(inv, lambda: s.layer.attend(s.cache, s.batch, q, window=-1))
    refused(inv, lambda: s.layer.attend(s.cache, s.batch, q, scale=0.0))
    refused(inv, lambda: s.layer.attend(s.cache, s.batch, q, scale=math.nan))
    refused(inv, lambda: s.layer.attend(s.cache, s.batch, q, scale=1e-42))
    big = pkg.PagedBatch(torch.zeros(4, device="cuda", dtype=torch.int32), torch.zeros(3, device="cuda", dtype=torch.int32),
                         torch.zeros(3, 2, device="cuda", dtype=torch.int32), max_tokens=1)
    refused(inv, lambda: s.layer.attend(s.cache, big, q))                               # above max_batch
    off = torch.empty(8 * 8 * 64 + 1, device="cuda", dtype=BF16)[1:].view(8, 8, 64)
    refused(inv, lambda: s.layer.attend(s.cache, s.batch, off))                         # 2-byte alignment
    refused(inv, lambda: s.layer.append(s.cache, s.batch, k, v, q=q, q_out=off))
    wide = torch.empty(8, 8, 68, device="cuda", dtype=BF16)[..., :64]
    refused(inv, lambda: s.layer.attend(s.cache, s.batch, wide))                        # strides not of 16 bytes
    refused(inv, lambda: s.layer.append(s.cache, s.batch, k, v, pkg.QkTransform(rope_table(8, 24))))
    refused(inv, lambda: s.layer.append(s.cache, s.batch, k, v, pkg.QkTransform(rope_table(8, 80))))
    refused(inv, lambda: pkg.dflash_qk_norm_rope(q, k, q, k, pkg.QkTransform(rope_table(8, 64))))  # no positions
    refused(inv, lambda: s.layer.append(s.cache, s.batch, k, v, pkg.QkTransform(eps=math.nan)))
    odd = torch.empty(2, 2, 80, device="cuda", dtype=BF16)
    refused(pkg.DFLASH_ERR_UNSUPPORTED, lambda: pkg.dflash_qk_norm_rope(odd, None, odd, None, pkg.QkTransform()))
    f8 = Paged(pkg, [1], [5], heads=8, kv_heads=2, d=64, dtype=BF16, cache=FP8, seed=1)
    f8.cache.c.k_scale = 0.0
    refused(inv, lambda: f8.layer.attend(f8.cache, f8.batch, f8.rows(8)))
    for bad in (lambda: s.layer.attend(s.cache, s.batch, q.half()), lambda: s.layer.attend(f8.cache, s.batch, q),
                lambda: s.layer.attend(s.cache, s.batch, q[:, :4]), lambda: s.layer.append(s.cache, s.batch, k, v.half()),
                lambda: s.layer.append(s.cache, s.batch, k, v[:3]), lambda: s.layer.attend(s.cache, s.batch, q.transpose(1, 2)),
                lambda: s.layer.attend(s.cache, s.batch, q, lse=torch.empty(8, 8, device="cuda", dtype=BF16)),
                lambda: pkg.PagedCache(s.k, s.v[:1]), lambda: pkg.PagedCache(s.k.float(), s.v.float()),
                lambda: pkg.PagedBatch(s.cu.long(), s.len_t, s.table, max_tokens=1),
                lambda: pkg.PagedBatch(s.cu[:2], s.len_t, s.table, max_tokens=1),
                lambda: pkg.QkTransform(rope_table(8, 64).half()),
                lambda: s.layer.append(s.cache, s.batch, k, v, pkg.QkTransform(q_weight=torch.ones(64, device="cuda")))):
        with pytest.raises((TypeError, ValueError)):
            bad()
    # nothing to do: nothing launched, nothing written
    none = pkg.PagedBatch(torch.zeros(1, device="cuda", dtype=torch.int32), torch.zeros(0, device="cuda", dtype=torch.int32),
                          torch.zeros(0, 1, device="cuda", dtype=torch.int32), max_tokens=0)
    s.layer.attend(s.cache, none, q[:0])
    s.layer.append(s.cache, none, k[:0], v[:0])
    s.layer.sync_status()

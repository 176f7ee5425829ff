"""The attention block's operators where the order of the kernels' steps, the
range of the number formats or the limits of the arguments matter. Reference
and tolerances as in test_gpu_paged.py unless a test says otherwise."""
import math

import pytest
import torch

from test_gpu_paged import BF16, FP16, FP8, KINDS, UNIT, Paged, pkg  # noqa: F401  (pkg is a fixture)

pytestmark = pytest.mark.gpu

RAGGED = [70 + 37 * i % 59 for i in range(64)]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens", [
    ([256] * 32, [256] * 32),        # prompts from an empty cache: up to 7 items a CTA, one tile of keys in the first ones
    ([512] * 8, [512] * 8),          # 2 to 4 pieces a CTA, one-tile items after split ones
    (RAGGED, RAGGED),                # nothing but one-tile items, of 280 to 512 rows
    ([100 if i % 3 else 130 for i in range(48)], [100 if i % 3 else 700 + 90 * i for i in range(48)]),  # and between longer ones
])
def test_attend_many_pieces_of_a_cta(pkg, new, lens, d, dtype, cache):  # noqa: F811
    """CTAs of the many-row kernel walk several items one after the other; the size of the queries changes by powers of
    two between the row tiles and sequences, so that a row taken with another item's scale shows."""
    s = Paged(pkg, new, lens, heads=32, kv_heads=8, d=d, dtype=dtype, cache=cache, page=32, seed=len(new))
    size = torch.cat([2.0 ** (-3 * ((5 * b + torch.arange(n) // 64) % 4)) for b, n in enumerate(new)]).cuda()
    q = (s.rows(32, 1.5).float() * size[:, None, None]).to(dtype)
    out = s.check(q)
    for _ in range(5):
        assert torch.equal(s.layer.attend(s.cache, s.batch, q), out)


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("heads,new,batch,d", [
    (2, 1, 228, 64), (2, 8, 228, 128), (8, 4, 228, 64), (8, 8, 152, 128),  # few rows: 1, 8, 16 and 32 an item
    (2, 40, 76, 64), (2, 40, 76, 128), (8, 90, 76, 64), (8, 90, 76, 128)])  # many: one and two streams' rows
def test_attend_light_keys_of_a_long_context(pkg, heads, new, batch, d, dtype, cache):  # noqa: F811
    """100,000 keys of weight e^-18 = 2^-26 beside a few of weight 1, which alone have no value: what the light ones
    add up to is not lost. As many sequences as the items are walked whole, all over the same pages."""
    keys, page, kind = 100_000, 64, dtype if cache is None else cache
    heavy = [0, 16, 32, 48, 128]  # a key for each of the few-row kernel's warps and the many-row kernel's streams
    pages = -(-keys // page)
    k, v = torch.zeros(pages, page, 2, d, device="cuda"), torch.full((pages, page, 2, d), 4.0, device="cuda")
    for x in heavy:
        k[x // page, x % page, :, 0], v[x // page, x % page] = 12.0, 0.0
    k, v = k.to(kind), v.to(kind)  # (exact in every type)
    layer = pkg.PagedAttention(heads=heads, kv_heads=2, head_dim=d, page_size=page, dtype=dtype, cache_dtype=kind, max_batch=batch)
    b = pkg.PagedBatch(torch.arange(batch + 1, device="cuda", dtype=torch.int32) * new,
                       torch.full((batch,), keys, device="cuda", dtype=torch.int32),
                       torch.arange(pages, device="cuda", dtype=torch.int32).expand(batch, -1), max_tokens=new)
    q = torch.zeros(batch * new, heads, d, device="cuda", dtype=dtype)
    q[..., 0] = 12.0
    out = layer.attend(pkg.PagedCache(k, v), b, q, causal=False, scale=0.125)
    layer.sync_status()
    light = (keys - len(heavy)) * math.exp(-18.0)
    want = 4.0 * light / (len(heavy) + light)
    # fp16 weights are rounded at 2^-14 * 2^-7 of the largest one and below to steps of 2^-24 * 2^-7, above (and in bf16)
    # to their 11 (8) bits; fp32 scores of 18 are off by 18 * 2^-24 * log2(e) at most, and fp32 sums near 1 by 1e-4 (a
    # weight of 2^-26 itself is lost in one, a thread adds some thousands); the result is rounded once
    unit = UNIT[dtype]
    small = 4.0 * keys * 2.0 ** -32 / len(heavy) if cache is FP8 or dtype is FP16 else unit * want
    tol = small + 1e-4 * want + unit * want + 2.0 ** -25
    assert float((out.double() - want).abs().max()) <= tol


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("new,lens", [
    ([4, 2], [60, 3]), ([2, 1], [900, 16]), ([8], [9000]),            # few rows: whole items, joined by counters and by the merge
    ([70, 40], [70, 300]), ([60], [700]), ([200], [900]), ([64], [30000])])  # many rows
def test_attend_lse_of_rows_that_are_not_numbers(pkg, new, lens, dtype, cache):  # noqa: F811
    """A row whose every score is NaN has NaN results and a NaN logarithm, not that of a row that sees nothing."""
    s = Paged(pkg, new, lens, heads=8, kv_heads=2, d=64, dtype=dtype, cache=cache, seed=sum(new))
    q = s.rows(8)

    def run():
        lse = torch.full((s.tokens, 8), 7.0, device="cuda")
        out = s.layer.attend(s.cache, s.batch, q, lse=lse)
        s.layer.sync_status()
        return out, lse
    want, want_lse = run()
    token, head = s.tokens // 2, 5
    q[token, head, 3] = float("nan")
    out, lse = run()
    assert out[token, head].isnan().all() and lse[token, head].isnan()
    here = torch.zeros(s.tokens, 8, dtype=torch.bool, device="cuda")
    here[token, head] = True
    assert torch.equal(out[~here], want[~here]) and torch.equal(lse[~here], want_lse[~here])


@pytest.mark.parametrize("cache", [None, FP8])
@pytest.mark.parametrize("new,lens", [([8, 1], [5, 64]), ([40, 1], [7, 1]), ([300], [10])])
def test_attend_rows_that_see_nothing_exactly(pkg, new, lens, cache):  # noqa: F811
    """Exactly a sequence's first new - length tokens see no key: zeros and -inf there, even for queries that are not
    numbers, and ordinary results in all other rows."""
    s = Paged(pkg, new, lens, heads=8, kv_heads=2, d=64, dtype=BF16, cache=cache, seed=3)
    nothing = torch.cat([torch.arange(n) < n - L for n, L in zip(new, lens)]).cuda()
    assert nothing.any() and not nothing.all()
    q = s.rows(8)
    for x in (q, torch.where(nothing[:, None, None], torch.full_like(q, float("nan")), q)):
        lse = torch.full((s.tokens, 8), 7.0, device="cuda")
        out = s.layer.attend(s.cache, s.batch, x, lse=lse)
        s.layer.sync_status()
        assert (out[nothing] == 0).all() and (lse[nothing] == -math.inf).all()
        assert lse[~nothing].isfinite().all() and (out[~nothing] != 0).any(-1).all()


@pytest.mark.parametrize("new", [1, 4, 90])
@pytest.mark.parametrize("e", [-126, -118, -101, -99, 99, 107, 108, 120, 125])
def test_attend_queries_of_any_size(pkg, e, new):  # noqa: F811
    """bf16 queries of 2^e over an 8-bit cache, with scales that bring the scores back to ordinary sizes."""
    s = Paged(pkg, [new], [333], heads=4, kv_heads=2, d=64, dtype=BF16, cache=FP8, seed=new)
    for x in (s.k, s.v):
        x.copy_((0.125 * torch.randn(x.shape, device="cuda", generator=s.g)).to(FP8))
    q = (s.rows(4).clamp(-1.9, 1.9).double() * 2.0 ** e).to(BF16)
    # (scale * k_scale has to be an ordinary number; bf16 queries below 2^-126 keep few bits, which the reference reads as they are)
    k_scale, scale = 2.0 ** (-60 if e > 0 else 60), 2.0 ** ((60 if e > 0 else -60) - e)
    s.cache.c.k_scale, s.ks = k_scale, k_scale
    s.cache.c.v_scale, s.vs = 1.0, 1.0
    s.check(q, scale=scale)


def test_attend_makes_its_output_for_the_stream_of_the_call(pkg):  # noqa: F811
    """Without `out`, a call on another stream writes memory that no pending work of the current stream holds, and that
    is not handed out again while the current stream still reads it."""
    s = Paged(pkg, [8, 5], [300, 40], heads=8, kv_heads=2, d=64, dtype=BF16, seed=4)
    q = s.rows(8)
    want = s.layer.attend(s.cache, s.batch, q)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        x = torch.empty_like(q)
        torch.cuda._sleep(100_000_000)
        x.fill_(7)                       # pending on the current stream when its memory is given back
        del x
        out = s.layer.attend(s.cache, s.batch, q, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        out = s.layer.attend(s.cache, s.batch, q, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(100_000_000)
        got = out.clone()                # pending when the output is given back
        del out
        with torch.cuda.stream(side):
            other = [torch.full_like(q, 7) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(got, want) and len(other) == 4
    assert torch.equal(s.layer.attend(s.cache, s.batch, q, stream=torch.cuda.current_stream()), want)


def test_destroyed_handles_are_refused(pkg):  # noqa: F811
    s = Paged(pkg, [4, 4], [30, 40], heads=8, kv_heads=2, d=64, dtype=BF16, seed=1)
    q, k, v = s.rows(8), s.rows(2), s.rows(2)
    h = pkg.dflash_paged_init(heads=8, kv_heads=2, head_dim=64, page_size=16, dtype=BF16, max_batch=2)
    out = torch.empty_like(q)
    pkg.dflash_paged_attend(h, s.cache, s.batch, q, out)
    want = out.clone()
    pkg.dflash_paged_destroy(h)
    out.fill_(7)
    for call in (lambda: pkg.dflash_paged_attend(h, s.cache, s.batch, q, out),
                 lambda: pkg.dflash_paged_append(h, s.cache, s.batch, k, v), lambda: pkg.dflash_paged_sync_status(h)):
        with pytest.raises(pkg.DflashError) as e:
            call()
        assert e.value.status == pkg.DFLASH_ERR_INVALID_ARG
    pkg.dflash_paged_destroy(h)     # nothing left to free
    pkg.dflash_paged_destroy(None)
    assert (out == 7).all() and torch.equal(s.layer.attend(s.cache, s.batch, q), want)
    s.layer.close()
    for call in (lambda: s.layer.attend(s.cache, s.batch, q, out), lambda: s.layer.append(s.cache, s.batch, k, v)):
        with pytest.raises(pkg.DflashError):
            call()
    s.layer.close()


def test_new_handles_are_ready_for_any_stream(pkg):  # noqa: F811
    """A handle made behind pending work serves a call on another stream at once (items joined by its counters)."""
    s = Paged(pkg, [2, 1], [900, 16], heads=8, kv_heads=2, d=64, dtype=BF16, seed=4)
    q = s.rows(8)
    want = s.layer.attend(s.cache, s.batch, q)
    side, out = torch.cuda.Stream(), torch.full_like(q, 7)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    layer = pkg.PagedAttention(heads=8, kv_heads=2, head_dim=64, page_size=16, dtype=BF16, max_batch=2)
    layer.attend(s.cache, s.batch, q, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    layer.sync_status()


def test_scales_whose_reciprocal_is_infinite_are_refused(pkg):  # noqa: F811
    s = Paged(pkg, [2], [20], heads=4, kv_heads=2, d=64, dtype=BF16, cache=FP8, seed=1, poison=False)
    q, k, v = s.rows(4), torch.zeros_like(s.rows(2)), torch.zeros_like(s.rows(2))
    for name in ("k_scale", "v_scale"):
        for bad in (1e-40, 0.0, -1.0, math.inf, math.nan):
            good = getattr(s.cache.c, name)
            setattr(s.cache.c, name, bad)
            for call in (lambda: s.layer.append(s.cache, s.batch, k, v), lambda: s.layer.attend(s.cache, s.batch, q, scale=1e30)):
                with pytest.raises(pkg.DflashError) as e:
                    call()
                assert e.value.status == pkg.DFLASH_ERR_INVALID_ARG
            setattr(s.cache.c, name, good)
    s.cache.c.k_scale = s.cache.c.v_scale = 2.0 ** -126
    s.layer.append(s.cache, s.batch, k, v)
    s.layer.sync_status()
    at = s.table[0, 1].long()
    assert (s.k[at, 2:4].float() == 0).all() and (s.v[at, 2:4].float() == 0).all()

"""The operators around a step's attention where calls meet: logits that do not
arrive, outputs that lie in one buffer with inputs, two calls at once, changing
row counts, long sums."""
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, INT32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


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


# ------------------------------------------------------------ logits that do not arrive
@pytest.mark.parametrize("want,rank,at", [("argmax", 5, 2), ("argmax", 0, 1), ("argmax", 3, 0), ("probs", 5, 0), ("probs", 5, 2),
                                          ("greedy", 5, 1), ("out", 5, 1), ("all", 2, 3)])
def test_logits_that_do_not_arrive(pkg, want, rank, at):
    """A cluster of 16 CTAs has several positions of a sequence; the logits of one CTA do not come from position `at` on. No
    position is answered from what the other CTAs have, and no other sequence is touched."""
    B, T, V = 32, 8, 151936
    logits = torch.randn(B, T, V, device="cuda", generator=gen(1)).to(BF16)
    tokens = torch.randint(0, V, (B, 40), device="cuda", generator=gen(2), dtype=INT32)
    tau = torch.zeros(B, device="cuda") if want == "greedy" else torch.ones(B, device="cuda")
    rules = pkg.LogitsRules(tokens, torch.full((B,), 40, device="cuda", dtype=INT32), presence=torch.ones(B, device="cuda"), temperature=tau)

    def outputs():
        return dict(out=torch.zeros_like(logits) if want in ("out", "all") else None,
                    probs=torch.zeros(B, T, V, device="cuda") if want in ("probs", "greedy", "all") else None,
                    argmax=torch.zeros(B, T, device="cuda", dtype=INT32) if want in ("argmax", "all") else None)
    good, bad = outputs(), outputs()
    pkg.dflash_logits_adjust(logits, rules, **good)
    pkg.dflash_selftest_logits_lost(logits, rules, rank=rank, at=at, **bad)
    own = torch.arange(V, device="cuda") // 2048 % 16 == rank
    for name, y in good.items():
        if y is None:
            continue
        x = bad[name]
        assert torch.equal(x[1:], y[1:])
        for t in range(at - 1 if name == "argmax" else at):
            assert torch.equal(x[0, t], y[0, t])
        if name == "argmax":
            assert int(x[0, at]) == -1
            assert at == 0 or int(x[0, at - 1]) in (-1, int(y[0, at - 1]))
        elif name == "probs":
            assert torch.isnan(x[0, at]).all()
        else:
            assert torch.isnan(x[0, at, own]).all()
            assert torch.equal(x[0, at, ~own], y[0, at, ~own]) or torch.isnan(x[0, at]).all()
        for t in range(at + 1, T):  # given up too, or another cluster's
            if name == "argmax":
                assert int(x[0, t]) in (-1, int(y[0, t]))
            else:
                assert torch.isnan(x[0, t, own]).all() or torch.equal(x[0, t], y[0, t])
    pkg.dflash_logits_adjust(logits, rules, **bad)  # the next call is whole again
    assert all(y is None or torch.equal(bad[name], y) for name, y in good.items())


def test_the_self_test_refuses_what_does_not_fit(pkg):
    logits, best = torch.zeros(2, 3, 64, device="cuda"), torch.zeros(2, 3, device="cuda", dtype=INT32)
    lose = pkg.dflash_selftest_logits_lost
    for x, kw in ((logits[0], {}), (logits[:, ::2], {}), (logits.cpu(), {}), (logits, dict(argmax=best[:1])), (logits, dict(argmax=best.long())),
                  (logits, dict(out=logits.half())), (logits, dict(probs=torch.zeros(2, 3, 65, device="cuda"))),
                  (logits, dict(argmax=best, rules=pkg.LogitsRules(temperature=torch.ones(1, device="cuda"))))):
        with pytest.raises(ValueError):
            lose(x, rank=0, at=0, **kw)
    with pytest.raises(pkg.DflashError, match="rank"):
        lose(logits, argmax=best, rank=-1, at=0)
    lose(logits, argmax=best, rank=3, at=0)  # (no such CTA: nothing is lost)
    assert not best.any()


# ------------------------------------------------------------ logits and outputs in one buffer
@pytest.mark.parametrize("V", [512, 515])
def test_logits_into_other_slices_of_their_buffer(pkg, V):
    """Rows that pass one another are answered, rows that share values are refused."""
    B, T = 3, 4
    mask = torch.randint(-2 ** 31, 2 ** 31, (B, T, -(-V // 32)), device="cuda", generator=gen(3)).to(INT32)

    def buffer(*shape):
        return torch.randn(*shape, device="cuda", generator=gen(4)).to(BF16)
    for x, y in ((b := buffer(B, T, 2, V), b[:, :, 0], b[:, :, 1])[1:], (b := buffer(B, 2 * T, V), b[:, T:], b[:, :T])[1:],
                 (b := buffer(2 * B, T, V), b[B:], b[:B])[1:], (b := buffer(B, T, 2 * V + 5), b[..., 1:V + 1], b[..., V + 1:2 * V + 1])[1:],
                 (b := buffer(2 * B, 2 * T, V), b[::2, ::2], b[1::2, 1::2])[1:],
                 (buffer(B, T, V), buffer(T, B, V).transpose(0, 1))):
        want = torch.empty(B, T, V, device="cuda", dtype=BF16)
        pkg.dflash_logits_adjust(x.contiguous(), out=want, mask=mask)
        before = x.clone()
        pkg.dflash_logits_adjust(x, out=y, mask=mask)
        assert torch.equal(y, want) and torch.equal(x, before)
    b = buffer(B + 1, T + 1, V + 8)
    for x, y in ((b[:B, :T, :V], b[1:, :T, :V]), (b[:B, :T, :V], b[:B, 1:, :V]), (b[:B, 1:, :V], b[1:, :T, :V]), (b[:B, :T, :V], b[:B, :T, 8:]),
                 (b[:1, :T, :V], b[:1, 1:, :V])):
        before = b.clone()
        with pytest.raises(pkg.DflashError, match="overlap"):
            pkg.dflash_logits_adjust(x, out=y)
        assert torch.equal(b, before)


# ------------------------------------------------------------ pages and their pool
@pytest.mark.parametrize("B", [3, 300, 3000])
def test_counts_that_are_the_pools_lengths(pkg, B):
    """An entry's number may be its own request's length: as many tokens again, then all of them dropped."""
    pool = pkg.PagePool.empty(requests=B, cols=6, num_pages=6 * B, page_size=4)
    start = torch.randint(0, 12, (B,), device="cuda", generator=gen(B), dtype=INT32)
    pool.extend(None, start)
    pool.extend(None, pool.lens)
    assert torch.equal(pool.lens, 2 * start)
    assert pool.counters.tolist() == [6 * B - int(((2 * start + 3) // 4).sum()), 0]
    pool.trim(pool.lens)
    assert not pool.lens.any() and sorted(pool.free_pages.tolist()) == list(range(6 * B))
    with pytest.raises(pkg.DflashError, match="overlap"):
        pool.trim(pool.lens, rows=torch.arange(B, device="cuda", dtype=INT32))
    batch = pkg.PagedBatch(torch.zeros(B, device="cuda", dtype=INT32), pool.lens[1:], torch.zeros(B - 1, 6, device="cuda", dtype=INT32), max_tokens=4)
    with pytest.raises(pkg.DflashError, match="overlap"):
        pool.extend(batch, start[1:].clone())
    assert not pool.lens.any()


def test_a_batch_in_the_columns_beside_the_pools(pkg):
    """The batch's page table may lie in the same rows of a buffer as the pool's."""
    wide = torch.full((4, 20), -1, device="cuda", dtype=INT32)
    empty = pkg.PagePool.empty(requests=4, cols=8, num_pages=32, page_size=16)
    pool = pkg.PagePool(wide[:, :8], empty.lens, empty.free_pages, empty.counters, page_size=16)
    batch = pkg.PagedBatch(torch.zeros(5, device="cuda", dtype=INT32), torch.zeros(4, device="cuda", dtype=INT32), wide[:, 8:16], max_tokens=100)
    pool.extend(batch, torch.tensor([100, 0, 17, 1], device="cuda", dtype=INT32))
    assert wide[0].tolist() == [0, 1, 2, 3, 4, 5, 6, -1, 0, 1, 2, 3, 4, 5, 6, -1, -1, -1, -1, -1]
    assert wide[2, :3].tolist() == [7, 8, -1] and wide[2, 8:11].tolist() == [7, 8, -1] and (wide[1] == -1).all()
    with pytest.raises(pkg.DflashError, match="overlap"):
        pool.extend(pkg.PagedBatch(batch.tensors[0], batch.tensors[1], wide[:, 7:15], max_tokens=1), torch.ones(4, device="cuda", dtype=INT32))


@pytest.mark.parametrize("B", [5, 200, 2500])
def test_a_batch_padded_with_a_request_that_it_has(pkg, B):
    """Entries without new tokens, and those that lose none, may name the request of another entry: it keeps what that one does."""
    pool = pkg.PagePool.empty(requests=B, cols=4, num_pages=4 * B, page_size=16)
    pool.extend(None, torch.full((B,), 20, device="cuda", dtype=INT32))
    for real in (0, B // 2, B - 1):  # one entry does something, before, between or behind those that pad
        rows = torch.full((B,), 3, device="cuda", dtype=INT32)
        counts = torch.zeros(B, device="cuda", dtype=INT32)
        counts[real] = 17
        positions = torch.full((17,), -1, device="cuda", dtype=INT32)
        for _ in range(20):
            pool.extend(None, counts, rows=rows, positions=positions)
            assert int(pool.lens[3]) == 37 and positions.tolist() == list(range(20, 37)) and pool.counters.tolist() == [2 * B - 1, 0]
            pool.trim(counts, rows=rows)
            assert int(pool.lens[3]) == 20 and pool.counters.tolist() == [2 * B, 0]


# ------------------------------------------------------------ row counts that change from call to call
def test_a_handle_with_changing_row_counts(pkg):
    """Results are those of a handle that has seen no other row count (rows 5, 261, 517, .. share a remembered plan's place)."""
    w = (torch.randn(136, 1032, device="cuda", generator=gen(1)) / 32).to(BF16)
    x = torch.randn(2053, 1032, device="cuda", generator=gen(2)).to(BF16)
    with pkg.Linear(w, activation="silu") as layer:
        for rows in (5, 261, 517, 5, 2053, 1, 257, 256, 512, 5, 261, 130, 33, 1, 2053):
            with pkg.Linear(w, activation="silu") as other:
                assert torch.equal(layer(x[:rows]), other(x[:rows]))


def test_changing_row_counts_cost_no_search(pkg):
    """The host's time of a call: 40 to 90 us more where each call looked through the plans (128 features of 8192 columns)."""
    w = torch.zeros(128, 8192, device="cuda", dtype=BF16)
    xs = [torch.zeros(rows, 8192, device="cuda", dtype=BF16) for rows in (256, 255)]
    ys = [torch.zeros(rows, 128, device="cuda", dtype=BF16) for rows in (256, 255)]
    with pkg.Linear(w) as layer:
        def host(order):
            best = 1.0
            for _ in range(12):
                torch.cuda.synchronize()
                t = time.perf_counter()
                for i in order * 20:
                    layer(xs[i], ys[i])
                best = min(best, time.perf_counter() - t)
            torch.cuda.synchronize()
            return best / (20 * len(order))
        host([0, 1])
        same, changing = host([0, 0]), host([0, 1])
        assert changing < same + 15e-6, (same, changing)


# ------------------------------------------------------------ long sums of the matrix product
def signed(g, sign, *shape, dtype):
    v = torch.rand(*shape, device="cuda", generator=g) if sign == "one sign" else torch.randn(*shape, device="cuda", generator=g) / 2
    return (v * 2.0 ** -4).to(dtype)


@pytest.mark.parametrize("rows", [8, 300])
@pytest.mark.parametrize("k", [16384, 32760])
@pytest.mark.parametrize("dtype,sign", [(BF16, "one sign"), (BF16, "both signs"), (FP16, "one sign"), (FP16, "both signs")])
def test_fp32_results_are_summed_in_short_pieces(pkg, rows, k, dtype, sign):
    """The accumulator of up to 512 columns takes 32 steps of 16 products. A step drops less than 2^-23 of the sum so far, and of
    each product what lies 2^-25 below the sum: nothing of a bf16 one (16 bits, at most 2^9 below the sum of 512), up to 2^-25 of
    the sum of an fp16 one (22 bits). Over the steps of one sign that is at most (1 + .. + 32) / 32 = 16.5 times as much, of both
    signs (sums that grow like the root) 21.6 times the sum's own part while the products' parts cancel; half of it on
    average, and 2^-23 for the sums of the pieces. One accumulator for 2048 columns, an eighth of k, would be off by more than that."""
    g = gen(k + rows)
    x, w = signed(g, sign, rows, k, dtype=dtype), signed(g, sign, 520, k, dtype=dtype)
    z = x.double() @ w.double().T
    with pkg.Linear(w, out_dtype=FP32) as layer:
        off = float((layer(x).double() - z).norm() / z.norm())
    step = 2.0 ** -23 if sign == "both signs" or dtype is BF16 else 2.0 ** -23 + 16 * 2.0 ** -25
    bound = (21.6 if sign == "both signs" else 16.5) * step / 2 + 2.0 ** -23
    assert off <= bound, (off, bound)


@pytest.mark.parametrize("rows,n,k", [(1, 200, 65544), (16, 129, 262144), (300, 128, 262144), (70, 513, 70000)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_long_sums_of_one_sign(pkg, rows, n, k, dtype):
    """Results in 16 bits are within their rounding however long the sum: 256 steps of an accumulator of 4096 columns drop at most
    (1 + .. + 256) / 256 = 128.5 times what one drops (2^-23 of the sum so far, and 2^-25 of it for each of 16 products), and 2^-23 for each sum of the pieces of a part."""
    g = gen(k + rows)
    x, w, bias, residual = (signed(g, "one sign", *shape, dtype=dtype) for shape in ((rows, k), (n, k), (n,), (rows, n)))
    z = (x.double() @ w.double().T + bias.double()).clamp(min=0) + residual.double()
    with pkg.Linear(w, bias, activation="relu") as layer:
        y = layer(x, residual=residual).double()
    off = ((y - z).abs() / z).max()
    assert float(off) <= torch.finfo(dtype).eps / 2 * 1.001 + 128.5 * (2 ** -23 + 16 * 2 ** -25) + (k / 4096 + 12) * 2 ** -23


@pytest.mark.parametrize("rows,n,k", [(1, 1, 8), (3, 129, 16384), (8, 520, 70000), (65, 300, 4096), (300, 513, 2568), (700, 128, 33000), (4097, 640, 328)])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (FP16, FP16), (BF16, FP32), (FP16, FP32)])
def test_whole_numbers_are_exact(pkg, rows, n, k, dtype, out):
    """Sums of products of -1, 0 and 1 fit any accumulator, so that a column that is lost or taken twice shows."""
    g = gen(rows + k)
    x, w = (torch.randint(-1, 2, shape, device="cuda", generator=g).to(dtype) for shape in ((rows, k), (n, k)))
    with pkg.Linear(w, out_dtype=out) as layer:
        assert torch.equal(layer(x), (x.double() @ w.double().T).to(out))


# ------------------------------------------------------------ calls at the same time
def test_clusters_of_several_calls_at_the_same_time(pkg):
    """Pairs, clusters that share k, single CTAs and the logits' clusters of 16 on four streams: each as if alone."""
    g = gen(9)

    def product(rows, n, k, **kw):
        x, w = torch.randn(rows, k, device="cuda", generator=g).to(BF16), (torch.randn(n, k, device="cuda", generator=g) / 50).to(BF16)
        layer = pkg.Linear(w, **kw)
        y = torch.empty(rows, n, device="cuda", dtype=kw.get("out_dtype") or BF16)
        return (lambda stream: layer(x, y, stream=stream)), y, layer
    logits = torch.randn(2, 8, 151936, device="cuda", generator=g).to(BF16)
    tokens = torch.randint(0, 151936, (2, 500), device="cuda", generator=g, dtype=INT32)
    rules = pkg.LogitsRules(tokens, torch.full((2,), 500, device="cuda", dtype=INT32), repetition=torch.full((2,), 1.3, device="cuda"))
    probs = torch.empty(2, 8, 151936, device="cuda")
    work = [product(300, 5120, 2560), product(256, 2560, 2560), product(8, 2560, 2560), product(200, 128, 640, out_dtype=FP32),
            (lambda stream: pkg.dflash_logits_adjust(logits, rules, probs=probs, stream=stream), probs, None), product(2000, 1280, 640, activation="silu"),
            product(40, 20000, 512), product(16, 64, 4096)]
    want = []
    for call, y, _ in work:
        call(None)
        want.append(y.clone())
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for turn in range(30):
        for i, (call, _, _) in enumerate(work):
            call(streams[i % 4])
    torch.cuda.synchronize()
    for (_, y, layer), z in zip(work, want):
        assert torch.equal(y, z)
        if layer is not None:
            layer.sync_status()


def in_threads(*calls):
    """Runs every call in a thread of its own, all at once; raises what the first of them raised."""
    raised = []

    def one(call):
        try:
            call()
        except BaseException as e:
            raised.append(e)
    threads = [threading.Thread(target=one, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if raised:
        raise raised[0]


def test_a_threads_first_use_of_the_gpu(pkg):
    """A thread that has not used the GPU calls operators that make tensor maps."""
    w, x = torch.randn(128, 64, device="cuda").to(BF16), torch.randn(40, 64, device="cuda").to(BF16)
    y = torch.zeros(40, 128, device="cuda", dtype=BF16)
    cache = pkg.PagedCache(*(torch.randn(8, 16, 2, 64, device="cuda").to(BF16) for _ in range(2)))
    batch = pkg.PagedBatch(torch.tensor([0, 40], device="cuda", dtype=INT32), torch.tensor([100], device="cuda", dtype=INT32),
                           torch.arange(8, device="cuda", dtype=INT32).view(1, 8), max_tokens=40)
    q = torch.randn(40, 4, 64, device="cuda").to(BF16)
    a = torch.zeros_like(q)
    with pkg.Linear(w) as layer, pkg.PagedAttention(heads=4, kv_heads=2, head_dim=64, page_size=16, dtype=BF16, max_batch=1) as attention:
        torch.cuda.synchronize()
        in_threads(lambda: layer(x, y), lambda: attention.attend(cache, batch, q, a))
        torch.cuda.synchronize()
        assert torch.equal(y, layer(x)) and torch.equal(a, attention.attend(cache, batch, q))


def test_one_handle_by_two_threads(pkg):
    """Two threads call one handle with row counts of their own, each on its stream."""
    w = (torch.randn(640, 1280, device="cuda", generator=gen(1)) / 36).to(BF16)
    x = torch.randn(520, 1280, device="cuda", generator=gen(2)).to(BF16)
    counts = ((1, 257, 33, 513, 5), (256, 1, 512, 7, 261))
    with pkg.Linear(w) as layer:
        want = {n: layer(x[:n]) for c in counts for n in c}
        torch.cuda.synchronize()
        wrong = []

        def calls(mine):
            stream = torch.cuda.Stream()
            outs = []
            for _ in range(40):
                for n in mine:
                    outs.append((n, layer(x[:n], torch.empty(n, 640, device="cuda", dtype=BF16), stream=stream)))
            stream.synchronize()
            wrong.extend(n for n, y in outs if not torch.equal(y, want[n]))
        in_threads(*(lambda c=c: calls(c) for c in counts))
        assert not wrong


# ------------------------------------------------------------ the ends of the sizes
@pytest.mark.parametrize("n,k", [(1, 1), (5, 1), (130, 3), (1, 7), (64, 65)])
@pytest.mark.parametrize("rows", [1, 9, 70])
def test_products_of_few_columns(pkg, rows, n, k):
    """Rows of x and W that start on 16 bytes, with fewer columns than that or an odd number of them."""
    x, w = (torch.randint(-4, 5, (m, 72), device="cuda", generator=gen(m)).to(BF16)[:, :k] for m in (rows, n))
    for out in (BF16, FP32):
        with pkg.Linear(w, out_dtype=out) as layer:
            assert torch.equal(layer(x), (x.double() @ w.double().T).to(out))


def test_results_beyond_31_bits(pkg):
    rows, n = 47000, 46000  # 2.16e9 values
    x, w = (torch.randint(-2, 3, (m, 64), device="cuda", generator=gen(m)).to(BF16) for m in (rows, n))
    with pkg.Linear(w) as layer:
        y = layer(x)
        for part in (slice(0, 300), slice(rows // 2 - 1, rows // 2 + 200), slice(rows - 500, rows)):
            assert torch.equal(y[part], (x[part].double() @ w.double().T).to(BF16))
        z = torch.ones_like(y)
        layer(x, z, residual=z)
        for part in (slice(0, 300), slice(rows - 500, rows)):
            assert torch.equal(z[part], ((x[part].double() @ w.double().T) + 1).to(BF16))


def test_logits_beyond_31_bits(pkg):
    B, V = 14200, 151936  # 2.16e9 values
    logits = torch.zeros(B, 1, V, device="cuda", dtype=BF16)
    at = torch.randint(0, V, (B,), device="cuda", generator=gen(1))
    logits[torch.arange(B, device="cuda"), 0, at] = 1
    best = torch.empty(B, 1, device="cuda", dtype=INT32)
    tokens = at.to(INT32).view(B, 1)
    pkg.dflash_logits_adjust(logits, argmax=best)
    assert torch.equal(best.view(-1), at.to(INT32))
    rules = pkg.LogitsRules(tokens, torch.ones(B, device="cuda", dtype=INT32), presence=torch.full((B,), 3.0, device="cuda"))
    pkg.dflash_logits_adjust(logits, rules, out=logits, argmax=best)  # in place: the one token falls to -2
    assert torch.equal(best.view(-1), (at == 0).to(INT32))
    assert (logits[torch.arange(B, device="cuda"), 0, at] == -2).all() and not logits[-1, 0, : int(at[-1])].any()


def test_the_largest_batch_of_pages(pkg):
    B, page = 65536, 3
    pool = pkg.PagePool.empty(requests=B + 7, cols=4, num_pages=3 * B, page_size=page)
    rows = torch.randperm(B + 7, device="cuda", generator=gen(1))[:B].to(INT32)
    new = torch.randint(0, 2 * page + 1, (B,), device="cuda", generator=gen(2), dtype=INT32)
    total = int(new.sum())
    positions, slots = torch.full((total,), -1, device="cuda", dtype=INT32), torch.full((total,), -1, device="cuda", dtype=torch.int64)
    batch = pkg.PagedBatch(torch.zeros(B + 1, device="cuda", dtype=INT32), torch.zeros(B, device="cuda", dtype=INT32),
                           torch.full((B, 4), -1, device="cuda", dtype=INT32), max_tokens=2 * page)
    granted = torch.zeros(B, device="cuda", dtype=INT32)
    pool.extend(batch, new, rows=rows, positions=positions, slots=slots, granted=granted)
    take = (new + page - 1) // page
    cu = torch.cumsum(new, 0)
    assert granted.all() and torch.equal(batch.tensors[0][1:], cu.to(INT32)) and torch.equal(pool.lens[rows.long()], new)
    of = torch.repeat_interleave(torch.arange(B, device="cuda"), new.long())
    at = torch.arange(total, device="cuda") - (cu - new)[of]
    first = torch.cumsum(take, 0) - take  # (pages are taken from 0 on)
    assert torch.equal(positions.long(), at) and torch.equal(slots, (first[of] + at // page) * page + at % page)
    assert pool.counters.tolist() == [3 * B - int(take.sum()), 0]
    pool.trim(new, rows=rows)
    assert not pool.lens.any() and pool.counters.tolist() == [3 * B, 0]
    assert torch.equal(pool.free_pages, torch.arange(3 * B - 1, -1, -1, device="cuda", dtype=INT32))

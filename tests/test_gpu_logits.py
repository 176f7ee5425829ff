"""Penalties, biases and masks on logits, and what is made of them
(dflash_logits_adjust), against fp64, through the C ABI. Tolerances are
worst-case rounding bounds, written at check()."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
INF = float("inf")


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


def reference(logits, r, draft=None, mask=None):
    """(x in fp64, the magnitudes that it is made of) of every position; r: LogitsRules' tensors by name."""
    B, T, V = logits.shape
    x, mag = logits.double().clone(), logits.double().abs()
    for b in range(B):
        n = min(max(int(r["lens"][b]), 0), r["tokens"].shape[1]) if "tokens" in r else 0
        prompt = int(r["prompt_lens"][b]) if "prompt_lens" in r else 0
        past = r["tokens"][b, :n].tolist() if n else []
        for t in range(T):
            drafts = draft[b, :t].tolist() if draft is not None else []
            seen = {v for v in past + drafts if 0 <= v < V}
            times = torch.zeros(V, dtype=torch.float64)
            for v in past[max(prompt, 0):] + drafts:
                if 0 <= v < V:
                    times[v] += 1
            times = times.cuda()
            ids = torch.tensor(sorted(seen), device="cuda", dtype=torch.long)
            rho = float(r["repetition"][b]) if "repetition" in r else 1.0
            z = x[b, t]
            z[ids] = torch.where(z[ids] > 0, z[ids] / rho, z[ids] * rho)
            mag[b, t] = torch.maximum(mag[b, t], z.abs())
            for name, amount in (("frequency", times), ("presence", (times > 0).double())):
                if name in r:
                    z -= float(r[name][b]) * amount
                    mag[b, t] += abs(float(r[name][b])) * amount
            if "bias_ids" in r:
                last = {int(v): float(w) for v, w in zip(r["bias_ids"][b], r["bias_values"][b]) if 0 <= int(v) < V}
                for v, w in last.items():
                    z[v] += w
                    mag[b, t, v] += abs(w)
            if mask is not None:
                bits = (mask[b, t].long()[:, None] >> torch.arange(32, device="cuda")) & 1
                z[bits.reshape(-1)[:V] == 0] = -INF
                mag[b, t][bits.reshape(-1)[:V] == 0] = 0
    return x, mag


def check(pkg, logits, r, draft=None, mask=None, in_place=False):
    B, T, V = logits.shape
    x, mag = reference(logits, r, draft, mask)
    rules = pkg.LogitsRules(r.get("tokens"), r.get("lens"), r.get("prompt_lens"),
                            **{k: v for k, v in r.items() if k not in ("tokens", "lens", "prompt_lens")})
    probs, best = torch.full((B, T, V), -7.0, device="cuda"), torch.full((B, T), -7, device="cuda", dtype=torch.int32)
    out = torch.full_like(logits, -7.0)
    alone = [torch.empty_like(logits), torch.empty_like(probs), torch.empty_like(best)]
    kw = dict(draft=draft, mask=mask)
    pkg.dflash_logits_adjust(logits, rules, out=alone[0], **kw)
    pkg.dflash_logits_adjust(logits, rules, probs=alone[1], **kw)
    pkg.dflash_logits_adjust(logits, rules, argmax=alone[2], **kw)
    target = logits if in_place else out
    pkg.dflash_logits_adjust(logits, rules, out=target, probs=probs, argmax=best, **kw)
    for a, c in zip(alone, (target, probs, best)):
        assert torch.equal(a.nan_to_num(nan=-3), c.nan_to_num(nan=-3))
    # five operations, each rounded to fp32 (half of 2^-23 of at most the magnitudes), then once to the output's type
    err = 5 * 2 ** -24 * mag
    fin = torch.isfinite(x)
    tol = err + torch.finfo(logits.dtype).eps / 2 * x.abs() * 1.01 + (2 ** -25 if logits.dtype is FP16 else 1e-40)
    over = x.abs() > torch.finfo(logits.dtype).max  # (rounds to an infinity, or to the largest number)
    got = target.double()
    bad = fin & ~over & ~((got - x).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} logits off"
    assert torch.equal(got[~fin].nan_to_num(nan=-3), x[~fin].nan_to_num(nan=-3))
    # the best token: no other may be better by more than both errors; -1 where there is none
    number = torch.where(torch.isnan(x), -INF, x)
    top = number.amax(-1)
    for b in range(B):
        for t in range(T):
            i = int(best[b, t])
            if top[b, t] == -INF:
                assert i == -1
            elif top[b, t] == INF:
                assert i == int((number[b, t] == INF).nonzero()[0])
            else:
                assert 0 <= i < V and number[b, t, i] >= top[b, t] - err[b, t, i] - err[b, t][number[b, t] == top[b, t]].max()
    # the probabilities: the exponent is off by the logit's error and three roundings of itself, over tau; the sum alike
    tau = (r["temperature"] if "temperature" in r else torch.ones(B, device="cuda")).double()[:, None, None]
    for b in range(B):
        for t in range(T):
            z, p = x[b, t], probs[b, t].double()
            if top[b, t] == -INF and not torch.isnan(z).any():
                assert (p == 0).all()
            elif float(tau[b]) == 0:
                assert float(p.sum()) == 1 and float(p[int(best[b, t])]) == 1
            elif torch.isnan(z).any() or (z == INF).any():
                assert torch.isnan(p).all()
            else:
                q = torch.softmax(z / tau[b, 0], 0)
                d = (z - top[b, t]).clamp(min=-1e4).abs()
                rel = (err[b, t].max() * 2 + 4 * 2 ** -24 * d) / tau[b, 0] + 16 * 2 ** -23
                assert ((p - q).abs() <= q * (rel.clamp(max=50).exp() - 1) + 1e-37).all()


def rules_for(g, B, V, hist, names):
    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand(B, device="cuda", generator=g)
    r = {}
    if hist:
        r["tokens"] = (V * torch.rand(B, hist, device="cuda", generator=g) ** 3).to(torch.int32)
        r["lens"] = torch.randint(0, hist + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
        r["lens"][0] = hist
        r["prompt_lens"] = (r["lens"] * torch.rand(B, device="cuda", generator=g)).to(torch.int32)
    make = dict(repetition=(0.7, 1.5), presence=(-0.5, 1.5), frequency=(-0.1, 0.6), temperature=(0.3, 2.0))
    for n in names:
        r[n] = uniform(*make[n])
    return r


ALL = ("repetition", "presence", "frequency", "temperature")
CASES = [  # batch, rows, vocab, history, rules, biases, mask
    (1, 1, 1, 3, ALL, 1, True),
    (2, 1, 7, 0, (), 0, False),
    (3, 4, 33, 20, ALL, 5, True),
    (2, 8, 256, 100, ALL, 0, True),
    (5, 1, 1000, 50, ("repetition",), 3, False),
    (2, 3, 4097, 700, ("presence", "temperature"), 20, True),
    (4, 2, 32003, 2500, ALL, 300, True),
    (3, 16, 32000, 40, ("frequency",), 0, False),
    (1, 8, 151936, 2000, ALL, 16, True),
    (2, 2, 151937, 9, ALL, 2, True),
    (70, 1, 5000, 30, ALL, 4, True),
    (40, 8, 1024, 64, ALL, 0, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:4]))
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_rules(pkg, case, dtype):
    B, T, V, hist, names, bias, mask = case
    g = gen(V + B)
    logits = (3 * torch.randn(B, T, V, device="cuda", generator=g)).to(dtype)
    r = rules_for(g, B, V, hist, names)
    if bias:
        r["bias_ids"] = torch.randint(-1, V + 1, (B, bias), device="cuda", generator=g, dtype=torch.int32)  # twice, outside
        r["bias_values"] = torch.randn(B, bias, device="cuda", generator=g)
    m = None
    if mask:
        m = torch.randint(-2 ** 31, 2 ** 31, (B, T, -(-V // 32)), device="cuda", generator=g).to(torch.int32)
        m[0, 0] = 0 if V > 1 else m[0, 0]
    draft = torch.randint(0, min(V, 50), (B, T - 1), device="cuda", generator=g, dtype=torch.int32) if T > 1 else None
    check(pkg, logits, r, draft, m, in_place=B % 2 == 0)


def test_repeated_tokens_and_biases(pkg):
    V = 500
    logits = torch.ones(1, 3, V, device="cuda")
    r = dict(tokens=torch.tensor([[4, 4, 9, 4, -1, V, 2 ** 31 - 1, 4]], device="cuda", dtype=torch.int32),
             lens=torch.tensor([99], device="cuda", dtype=torch.int32),  # cut to the row
             prompt_lens=torch.tensor([2], device="cuda", dtype=torch.int32),
             repetition=torch.tensor([2.0], device="cuda"), presence=torch.tensor([0.25], device="cuda"),
             frequency=torch.tensor([0.125], device="cuda"),
             bias_ids=torch.tensor([[9, 9, 7, 9, -5]], device="cuda", dtype=torch.int32),
             bias_values=torch.tensor([[1.0, 2.0, 3.0, 4.0, 5.0]], device="cuda"))
    draft = torch.tensor([[4, 7]], device="cuda", dtype=torch.int32)
    out = torch.empty_like(logits)
    pkg.dflash_logits_adjust(logits, pkg.LogitsRules(**r), out=out, draft=draft)
    want = torch.ones(3, V)
    want[:, 4] = 0.5 - 0.25 - torch.tensor([2, 3, 3]) * 0.125
    want[:, 9] = 0.5 - 0.25 - 0.125 + 4                    # the last bias listed
    want[:, 7] = torch.tensor([4.0, 4.0, 0.5 - 0.25 - 0.125 + 3])
    assert torch.equal(out[0].cpu(), want)
    check(pkg, logits, r, draft)


def test_a_long_history_of_one_token(pkg):
    n, V = 70001, 1000
    r = dict(tokens=torch.full((2, n), 3, device="cuda", dtype=torch.int32), lens=torch.tensor([n, 0], device="cuda", dtype=torch.int32),
             frequency=torch.tensor([2.0 ** -10, 5.0], device="cuda"))
    logits = torch.zeros(2, 1, V, device="cuda")
    out = torch.empty_like(logits)
    pkg.dflash_logits_adjust(logits, pkg.LogitsRules(**r), out=out)
    assert out[0, 0, 3] == -n / 1024 and out[0, 0].abs().sum() == n / 1024 and (out[1] == 0).all()


@pytest.mark.parametrize("hist", [30000, 36000])
@pytest.mark.parametrize("V", [40000, 40001])
def test_most_of_the_vocabulary_has_occurred(pkg, hist, V):
    """More tokens than a list holds, with counts in 16 and in 32 bits."""
    g = gen(hist)
    logits = torch.randn(2, 3, V, device="cuda", generator=g).to(BF16)
    r = rules_for(g, 2, V, 1, ALL)
    r["tokens"] = torch.stack([torch.randperm(V, device="cuda", generator=g)[:hist] for _ in range(2)]).to(torch.int32)
    r["lens"] = torch.tensor([hist, hist - 11], device="cuda", dtype=torch.int32)
    r["bias_ids"] = torch.randint(0, V, (2, 9), device="cuda", generator=g, dtype=torch.int32)
    r["bias_values"] = torch.randn(2, 9, device="cuda", generator=g)
    check(pkg, logits, r, torch.randint(0, V, (2, 2), device="cuda", generator=g, dtype=torch.int32))


def test_drafts_that_fill_a_list(pkg):
    """Lists that the positions of one sequence fill to 2048 tokens of the first ones (which one CTA has) and beyond."""
    B, T, V = 40, 6, 65536
    g = gen(3)
    logits = torch.randn(B, T, V, device="cuda", generator=g).to(BF16)
    r = rules_for(g, B, V, 2050, ("repetition", "presence", "frequency"))
    r["tokens"] = torch.arange(2050, device="cuda", dtype=torch.int32).repeat(B, 1)
    r["lens"] = 2044 + torch.arange(B, device="cuda", dtype=torch.int32) % 6
    r["prompt_lens"] = torch.full((B,), 700, device="cuda", dtype=torch.int32)
    late = torch.tensor([2047, 65535, 2046, 5, 32768, 2045, 2047, 16384, 16385, 900], device="cuda", dtype=torch.int32)
    draft = late[(torch.arange(B, device="cuda")[:, None] + torch.arange(T - 1, device="cuda")) % len(late)].contiguous()
    check(pkg, logits, r, draft)


@pytest.mark.parametrize("n", [1536, 2048])
def test_drafts_that_fill_one_ctas_list(pkg, n):
    """Lists that the positions of one sequence fill to n tokens of one CTA (of up to 8, which take turns at 2048) and beyond."""
    B, T, V = 40, 6, 65536
    g = gen(3)
    logits = torch.randn(B, T, V, device="cuda", generator=g).to(BF16)
    r = rules_for(g, B, V, 2050, ("repetition", "presence", "frequency"))
    own = torch.arange(65536 // 8, device="cuda", dtype=torch.int32)
    own = (own >> 11 << 14) + (own & 2047)
    r["tokens"] = own[:n + 2].repeat(B, 1)
    r["lens"] = n - 4 + torch.arange(B, device="cuda", dtype=torch.int32) % 6
    r["prompt_lens"] = torch.full((B,), 700, device="cuda", dtype=torch.int32)
    late = own[[n - 1, 8191, n - 2, 5, n, n - 3, n - 1, 3000, 3001, 900]].clone()
    late[3] = 65535  # (another CTA's)
    draft = late[(torch.arange(B, device="cuda")[:, None] + torch.arange(T - 1, device="cuda")) % len(late)].contiguous()
    check(pkg, logits, r, draft)


@pytest.mark.parametrize("V,n,hist,dtype", [(40, 200, 0, BF16), (40, 200, 300, BF16), (5000, 6000, 0, BF16), (5000, 6000, 300, FP16),
                                            (70000, 40000, 0, BF16), (70000, 40000, 300, BF16), (262144, 8192, 33000, FP32)])
def test_many_biases(pkg, V, n, hist, dtype):
    """More biases than tokens, each several times; more than 16 bits count."""
    g = gen(n)
    logits = torch.randn(2, 2, V, device="cuda", generator=g).to(dtype)
    r = rules_for(g, 2, V, hist, ALL if hist else ())
    r["bias_ids"] = torch.randint(-1, V + 1, (2, n), device="cuda", generator=g, dtype=torch.int32)
    r["bias_values"] = torch.randn(2, n, device="cuda", generator=g)
    check(pkg, logits, r, torch.randint(0, V, (2, 1), device="cuda", generator=g, dtype=torch.int32) if hist else None)


@pytest.mark.parametrize("V,dtype,hist", [(262144, FP32, 40000), (1700000, BF16, 0), (1100001, FP16, 0)])
def test_largest_vocabularies(pkg, V, dtype, hist):
    g = gen(V)
    logits = (3 * torch.randn(1, 2, V, device="cuda", generator=g)).to(dtype)
    r = rules_for(g, 1, V, hist, ALL if hist else ("temperature",))
    if hist:
        r["bias_ids"] = torch.randint(0, V, (1, 300), device="cuda", generator=g, dtype=torch.int32)
        r["bias_values"] = torch.randn(1, 300, device="cuda", generator=g)
    mask = torch.randint(-2 ** 31, 2 ** 31, (1, 2, -(-V // 32)), device="cuda", generator=g).to(torch.int32)
    check(pkg, logits, r, torch.full((1, 1), V - 1, device="cuda", dtype=torch.int32), mask)


@pytest.mark.parametrize("V", [40, 20000, 32001])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_rows_without_a_choice_and_values_that_are_no_numbers(pkg, V, dtype):
    g = gen(V)
    logits = torch.randn(3, 4, V, device="cuda", generator=g).to(dtype)
    mask = torch.full((3, 4, -(-V // 32)), -1, device="cuda", dtype=torch.int32)
    logits[0, 0] = -INF                       # nothing above -inf
    mask[0, 1] = 0                            # nothing allowed
    mask[0, 2] = 0
    mask[0, 2, (V - 1) // 32] = -2 ** 31 if V % 32 == 0 else 1 << ((V - 1) % 32)  # the last token alone
    logits[0, 3, 5] = float("nan")            # masked: does not count
    mask[0, 3, 0] = ~(1 << 5)
    logits[1, 0, 7] = float("nan")            # not masked
    logits[1, 1, 30] = INF
    logits[1, 2, 2:9] = INF
    mask[1, 2, 0] = ~((1 << 9) - 4)           # infinities, masked
    logits[1, 3] = float("nan")
    logits[2, 0] = torch.finfo(dtype).min     # a mask of the lowest value
    logits[2, 0, 11] = 0.5
    logits[2, 1] = torch.finfo(dtype).min
    logits[2, 2] = torch.finfo(dtype).max
    mask[2, 3, 1:] = 0
    r = dict(temperature=torch.tensor([0.5, 1.0, 0.0], device="cuda"))
    check(pkg, logits, r, mask=mask)
    check(pkg, logits, {}, mask=mask)


def test_ties_go_to_the_lowest_token(pkg):
    for V, ids in ((64, (3, 60)), (20000, (19999, 255, 256, 8000)), (151936, (151935, 9496, 77777)), (9001, (9000, 31, 32))):
        logits = torch.zeros(2, 1, V, device="cuda", dtype=BF16)
        logits[0, 0, list(ids)] = 2.0
        logits[1, 0, 0] = -0.0                # equal to 0
        best, probs = torch.empty(2, 1, device="cuda", dtype=torch.int32), torch.empty(2, 1, V, device="cuda")
        pkg.dflash_logits_adjust(logits, argmax=best)
        assert best.view(-1).tolist() == [min(ids), 0]
        pkg.dflash_logits_adjust(logits, pkg.LogitsRules(temperature=torch.zeros(2, device="cuda")), probs=probs)
        assert probs.argmax(-1).view(-1).tolist() == [min(ids), 0] and (probs.sum(-1) == 1).all()


def test_temperatures_at_their_ends(pkg):
    logits = torch.tensor([[[1.0, 2.0, 2.5, -3.0]]], device="cuda").expand(4, 1, 4).contiguous()
    tau = torch.tensor([0.0, 1e-40, 1e30, INF], device="cuda")
    probs = torch.empty(4, 1, 4, device="cuda")
    pkg.dflash_logits_adjust(logits, pkg.LogitsRules(temperature=tau), probs=probs)
    best = torch.tensor([0.0, 0, 1, 0], device="cuda")
    assert torch.equal(probs[0, 0], best) and torch.equal(probs[1, 0], best)
    assert (probs[2:] == 0.25).all()


@pytest.mark.parametrize("V,pad", [(1000, 24), (1000, 3), (1001, 7)])
def test_strides_and_shared_masks(pkg, V, pad):
    B, T, g = 3, 4, gen(pad)
    wide = (2 * torch.randn(B, T + 1, V + pad, device="cuda", generator=g)).to(BF16)
    logits = wide[:, 1:, :V]
    words = -(-V // 32)
    masks = torch.randint(-2 ** 31, 2 ** 31, (B, words + 2), device="cuda", generator=g).to(torch.int32)
    mask = masks[:, None, :words].expand(B, T, words)       # a sequence's mask for all of its positions
    r = rules_for(g, B, V, 30, ALL)
    r["tokens"] = torch.cat([r["tokens"], r["tokens"]], 1)[:, :30]   # rows further apart
    draft = torch.randint(0, V, (B, T + 2), device="cuda", generator=g, dtype=torch.int32)[:, :T - 1]
    before = wide.clone()
    check(pkg, logits, r, draft, mask)
    assert torch.equal(wide.nan_to_num(), before.nan_to_num())
    check(pkg, logits, r, draft, mask, in_place=True)
    assert torch.equal(wide[:, 0], before[:, 0]) and torch.equal(wide[..., V:], before[..., V:])
    one = masks[:1, None, :words].expand(B, T, words)       # one mask for all
    check(pkg, logits.clone(), r, draft, one)


def test_captured_and_replayed_and_on_another_stream(pkg):
    g, V = gen(1), 6000
    logits = torch.randn(2, 3, V, device="cuda", generator=g)
    r = rules_for(g, 2, V, 40, ALL)
    rules = pkg.LogitsRules(**r)
    draft = torch.zeros(2, 2, device="cuda", dtype=torch.int32)
    probs, best = torch.empty(2, 3, V, device="cuda"), torch.empty(2, 3, device="cuda", dtype=torch.int32)
    pkg.dflash_logits_adjust(logits, rules, probs=probs, argmax=best, draft=draft)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.dflash_logits_adjust(logits, rules, probs=probs, argmax=best, draft=draft)
    for seed in (1, 2):
        logits.copy_(torch.randn(2, 3, V, device="cuda", generator=gen(seed)))
        r["tokens"].random_(0, V)
        r["lens"].random_(0, 41)
        draft.random_(0, V)
        graph.replay()
        p, i = torch.empty_like(probs), torch.empty_like(best)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        pkg.dflash_logits_adjust(logits, rules, probs=p, argmax=i, draft=draft, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(p, probs) and torch.equal(i, best)
        check(pkg, logits.clone(), r, draft)


def test_into_the_accept_checks(pkg):
    """Probabilities as dflash_verify_rejection takes them, best tokens as dflash_verify_prefix does; an empty row's -1 and
    zeros end a block with -1 in both."""
    B, L, K, V, g = 4, 7, 16, 3001, gen(9)
    logits = torch.randn(B, L + 1, V, device="cuda", generator=g).to(BF16)
    mask = torch.full((B, L + 1, -(-V // 32)), -1, device="cuda", dtype=torch.int32)
    mask[3] = 0
    probs, best = torch.empty(B, L + 1, V, device="cuda"), torch.empty(B, L + 1, device="cuda", dtype=torch.int32)
    pkg.dflash_logits_adjust(logits, probs=probs, argmax=best, mask=mask)
    path = best[:, :L].clamp(min=0).contiguous()
    path[1, 3] = (path[1, 3] + 1) % V
    accept, emitted = torch.empty(B, device="cuda", dtype=torch.int32), torch.empty(B, L + 1, device="cuda", dtype=torch.int32)
    pkg.dflash_verify_prefix(path, best, accept, emitted)
    assert accept.tolist() == [7, 3, 7, 0] and emitted[3].tolist() == [-1] * 8
    ids = (path[:, :, None] + torch.arange(K, device="cuda", dtype=torch.int32)) % V
    q = torch.zeros(B, L, K, device="cuda")
    q[:, :, 0] = 1
    ones = torch.full((B, L), 0.0, device="cuda")
    pkg.dflash_verify_rejection(path, ids, q, probs, ones, torch.full((B,), 0.5, device="cuda"), accept, emitted)
    assert accept.tolist() == [7, 7, 7, 0] and int(emitted[3, 0]) == -1 and bool((emitted[:3] >= 0).all())


def test_refusals(pkg):
    x = torch.zeros(2, 3, 64, device="cuda")
    best = torch.zeros(2, 3, device="cuda", dtype=torch.int32)
    adjust = pkg.dflash_logits_adjust
    with pytest.raises(pkg.DflashError, match="one of out"):
        adjust(x)
    with pytest.raises(pkg.DflashError, match="dtype"):
        adjust(x.double(), argmax=best)
    for kw in (dict(argmax=best.long()), dict(argmax=best[:1]), dict(probs=torch.zeros(2, 3, 65, device="cuda")),
               dict(probs=torch.zeros(2, 3, 128, device="cuda")[..., :64]), dict(argmax=best, draft=best),
               dict(argmax=best, mask=torch.zeros(2, 3, 1, device="cuda", dtype=torch.int32)), dict(out=x.half()),
               dict(argmax=best, rules=pkg.LogitsRules(temperature=torch.ones(3, device="cuda")))):
        with pytest.raises((TypeError, ValueError)):
            adjust(x, **kw)
    with pytest.raises(pkg.DflashError, match="strides"):
        adjust(x[:, :2], out=x.view(-1)[:256].view(2, 2, 64))
    with pytest.raises(ValueError):
        adjust(x[..., ::2], argmax=best)
    for kw in (dict(tokens=best), dict(bias_ids=best), dict(bias_ids=best, bias_values=torch.zeros(2, 2, device="cuda"))):
        with pytest.raises(ValueError):
            pkg.LogitsRules(**kw)
    with pytest.raises(TypeError):
        pkg.LogitsRules(temperature=torch.ones(2, device="cuda").half())
    huge = torch.empty(1, 1, 2_000_000, device="cuda")
    with pytest.raises(pkg.DflashError, match="vocabulary"):
        adjust(huge, pkg.LogitsRules(best[:1], torch.zeros(1, device="cuda", dtype=torch.int32), presence=torch.ones(1, device="cuda")),
               argmax=torch.empty(1, 1, device="cuda", dtype=torch.int32))
    adjust(torch.empty(0, 3, 64, device="cuda"), argmax=torch.empty(0, 3, device="cuda", dtype=torch.int32))

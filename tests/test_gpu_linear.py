"""The matrix product with bias, activation and residual (dflash_linear_*)
against fp64, through the C ABI. Tolerances are worst-case rounding bounds,
written at check()."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
ACT = {
    None: lambda z: z,
    "relu": lambda z: z.clamp(min=0),
    "silu": lambda z: z * torch.sigmoid(z),
    "gelu": lambda z: z * torch.special.ndtr(z),
    "gelu_tanh": lambda z: z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z.pow(3))),
}


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


def randn(g, *shape, dtype):
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


def check(got, x, w, bias=None, residual=None, act=None):
    k = x.shape[1]
    z = x.double() @ w.double().T
    mag = x.double().abs() @ w.double().abs().T
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    y = ACT[act](z)
    # every 16 products join the fp32 accumulator by one truncation (2^-23 of what is there, at most mag), a few more
    # where sums of parts are joined; activations have slopes below 1.2 and errors of a few 2^-22 of their argument
    tol = 1.2 * (k / 16 + 16) * 2 ** -23 * mag + 2 ** -19 * z.abs()
    if residual is not None:
        y = y + residual.double()
    tol = tol + 2 ** -23 * y.abs() + torch.finfo(got.dtype).eps / 2 * y.abs() * 1.01 + 1e-30
    if got.dtype is FP16:
        tol = tol + 2 ** -25  # half of the smallest number
    bad = ~((got.double() - y).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((got.double() - y).abs().max()):.3g}"


SHAPES = [(1, 1, 8), (1, 129, 64), (2, 128, 72), (8, 2560, 2560), (16, 127, 136), (17, 513, 1000), (61, 1024, 512),
          (64, 300, 4096), (65, 256, 64), (129, 1000, 328), (255, 640, 2560), (256, 5120, 512), (257, 129, 8), (300, 20000, 64),
          (1000, 2560, 640), (4097, 1281, 640), (33, 1100, 16384), (700, 33, 1280)]


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (FP16, FP16), (BF16, FP32), (FP16, FP32)])
def test_product(pkg, i, shape, dtype, out):
    rows, n, k = shape
    g = gen(rows + n + k)
    x, w = randn(g, rows, k, dtype=dtype), (randn(g, n, k, dtype=FP32) * k ** -0.5).to(dtype)
    act = list(ACT)[i % 5]
    bias = randn(g, n, dtype=dtype) if i % 2 else None
    residual = randn(g, rows, n, dtype=out) if i % 3 else None
    with pkg.Linear(w, bias, activation=act, out_dtype=out) as layer:
        y = layer(x, residual=residual)
        layer.sync_status()
        assert y.dtype is out and tuple(y.shape) == (rows, n)
        check(y, x, w, bias, residual, act)
        assert torch.equal(y, layer(x, residual=residual))  # (no sum depends on timing)


@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("rows", [5, 200])
def test_activations(pkg, act, rows):
    g = gen(3)
    x, w, bias = randn(g, rows, 64, dtype=BF16), randn(g, 200, 64, dtype=BF16), randn(g, 200, dtype=BF16)  # |z| up to 35
    with pkg.Linear(w, bias, activation=act, out_dtype=FP32) as layer:
        check(layer(x), x, w, bias, None, act)


@pytest.mark.parametrize("rows", [1, 7, 40, 150, 600])
@pytest.mark.parametrize("pad", [1, 3, 4, 8])  # rows of y that start anywhere, on 4 values, on 16 bytes
def test_strides(pkg, rows, pad):
    g, n, k = gen(rows + pad), 261, 200
    wide, wbuf = randn(g, rows, 2 * k + 16, dtype=BF16), randn(g, n, k + 24, dtype=BF16)
    x, w = wide[:, 8:8 + k], wbuf[:, 16:16 + k]
    for out in (BF16, FP32):
        buf, res = torch.full((rows + 1, n + pad), 7.0, device="cuda", dtype=out), randn(g, rows, n + 2 * pad, dtype=out)
        y, r = buf[:rows, pad:], res[:, :n]
        with pkg.Linear(w, activation="silu", out_dtype=out) as layer:
            layer(x, y, residual=r)
        check(y, x, w, None, r, "silu")
        assert (buf[:, :pad] == 7).all() and (buf[rows] == 7).all()  # nothing beside or behind the rows is written


def test_column_slices_of_one_buffer(pkg):
    g = gen(5)
    buf, w = randn(g, 40, 512, dtype=BF16), randn(g, 128, 256, dtype=BF16)
    x = buf[:, :256].clone()
    with pkg.Linear(w) as layer:
        layer(buf[:, :256], buf[:, 256:384])
        check(buf[:, 256:384], x, w)
        assert torch.equal(buf[:, :256], x)


@pytest.mark.parametrize("rows,n,k", [(3, 300, 2560), (130, 520, 640), (2000, 1000, 128)])
def test_residual_in_place(pkg, rows, n, k):
    g = gen(rows)
    for out in (BF16, FP32):
        x, w, y = randn(g, rows, k, dtype=BF16), (randn(g, n, k, dtype=FP32) * k ** -0.5).to(BF16), randn(g, rows, n, dtype=out)
        r = y.clone()
        with pkg.Linear(w, activation="gelu", out_dtype=out) as layer:
            layer(x, y, residual=y)
        check(y, x, w, None, r, "gelu")


def test_a_row_that_is_no_number_stays_in_its_row(pkg):
    g = gen(6)
    for rows in (9, 300):
        x, w = randn(g, rows, 136, dtype=FP16), randn(g, 140, 136, dtype=FP16)
        clean = x.clone()
        x[1, 5], x[4, 0] = float("nan"), float("inf")
        with pkg.Linear(w) as layer:
            y, z = layer(x), layer(clean)
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[4]).any()
        keep = [i for i in range(rows) if i not in (1, 4)]
        assert torch.equal(y[keep], z[keep])
        big = torch.full_like(x, 200.0)
        with pkg.Linear(torch.full_like(w, 200.0)) as layer:
            assert torch.isinf(layer(big)).all()  # 136 * 40000 is beyond fp16


def test_activations_at_their_ends(pkg):
    x = torch.zeros(8, 8, device="cuda", dtype=BF16)
    x[:, 0] = torch.tensor([-1e30, -200, -88.5, -1, 0, 88.5, 200, 1e30])
    w = torch.eye(8, device="cuda", dtype=BF16)
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        with pkg.Linear(w, activation=act, out_dtype=FP32) as layer:
            y = layer(x)[:, 0].double()
        z = x[:, 0].double()
        want = torch.where(z < -80, torch.zeros_like(z), torch.where(z > 80, z, ACT[act](z)))
        assert ((y - want).abs() <= 2 ** -19 * want.abs() + 1e-30).all(), (act, y, want)


def test_no_rows(pkg):
    w = torch.zeros(16, 64, device="cuda", dtype=BF16)
    with pkg.Linear(w) as layer:
        assert layer(torch.empty(0, 64, device="cuda", dtype=BF16)).shape == (0, 16)


@pytest.mark.parametrize("rows", [8, 100, 1500])
def test_captured_and_replayed(pkg, rows):
    g = gen(7)
    x, w = randn(g, rows, 640, dtype=BF16), (randn(g, 300, 640, dtype=FP32) / 25).to(BF16)
    first, second = pkg.Linear(w, activation="silu"), pkg.Linear((randn(g, 200, 296, dtype=FP32) / 17).to(BF16))
    h, y = torch.empty(rows, 300, device="cuda", dtype=BF16), torch.empty(rows, 200, device="cuda", dtype=BF16)
    hh = torch.empty(rows, 304, device="cuda", dtype=BF16)[:, :300]  # rows on whole 16 bytes, as the second takes them
    first(x, hh), second(hh[:, :296], y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first(x, hh)
        second(hh[:, :296], y)
    for seed in (1, 2):
        x.copy_(randn(gen(seed), rows, 640, dtype=BF16))
        graph.replay()
        first(x, h)
        assert torch.equal(h, hh)
        check(y, hh[:, :296], second._weights[0])


def test_one_handle_on_two_streams(pkg):
    g = gen(8)
    w = (randn(g, 2000, 1280, dtype=FP32) / 36).to(BF16)
    xs = [randn(g, 24, 1280, dtype=BF16) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    with pkg.Linear(w) as layer:
        want = [layer(x) for x in xs]
        torch.cuda.synchronize()
        outs = [torch.empty_like(y) for y in want]
        for _ in range(20):
            for x, y, s in zip(xs, outs, streams):
                layer(x, y, stream=s)
        torch.cuda.synchronize()
        for y, z in zip(outs, want):
            assert torch.equal(y, z)
        made = layer(xs[0], stream=streams[1])  # an output of the call's own, on that stream
        torch.cuda.synchronize()
        assert torch.equal(made, want[0])
        layer.sync_status()


def test_refusals(pkg):
    w = torch.zeros(32, 64, device="cuda", dtype=BF16)
    x, y = torch.zeros(4, 64, device="cuda", dtype=BF16), torch.zeros(4, 32, device="cuda", dtype=BF16)
    with pytest.raises(pkg.DflashError, match="dtype"):
        pkg.Linear(w.float())
    with pytest.raises(pkg.DflashError, match="out_dtype"):
        pkg.Linear(w, out_dtype=FP16)
    with pytest.raises(pkg.DflashError, match="aligned"):
        pkg.Linear(torch.zeros(32, 65, device="cuda", dtype=BF16))
    with pytest.raises(ValueError, match="activation"):
        pkg.Linear(w, activation="tanh")
    with pytest.raises(ValueError, match="bias"):
        pkg.Linear(w, torch.zeros(31, device="cuda", dtype=BF16))
    with pytest.raises(ValueError, match="CUDA"):
        pkg.Linear(w.cpu())
    layer = pkg.Linear(w)
    for bad in (x.half(), x[:, :56], torch.zeros(4, 128, device="cuda", dtype=BF16)[:, ::2]):
        with pytest.raises((TypeError, ValueError)):
            layer(bad, y)
    with pytest.raises(ValueError):
        layer(x, y[:3])
    with pytest.raises(ValueError):
        layer(x, y, residual=y[:3])
    with pytest.raises(pkg.DflashError, match="x must"):
        layer(torch.zeros(4, 68, device="cuda", dtype=BF16)[:, 1:65], y)  # not on 16 bytes
    with pytest.raises(pkg.DflashError, match="x must"):
        layer(torch.zeros(4, 66, device="cuda", dtype=BF16)[:, :64], y)   # rows 132 bytes apart
    with pytest.raises(pkg.DflashError, match="overlap"):
        layer(x, x[:, :32])
    buf = torch.zeros(5, 32, device="cuda", dtype=BF16)
    with pytest.raises(pkg.DflashError, match="overlap"):
        layer(x, buf[1:], residual=buf[:4])
    square = torch.zeros(64, 64, device="cuda", dtype=BF16)
    with pytest.raises(pkg.DflashError, match="overlap"):
        pkg.Linear(square)(x, square[:4])
    layer.close()
    with pytest.raises(pkg.DflashError, match="handle"):
        layer(x, y)

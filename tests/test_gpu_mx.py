"""GPU parity of the microscaled quantisation and product through the public calls, against the fp64 reference
(oracle/mx.py).

Quantisation is exact: codes and scale bytes must be equal.  The product's tolerance: the K exact products are added
in fp32, in any order and with truncation (each of the at most K additions is off by at most 2^-23 of the running sum
of magnitudes), so |err| <= K 2^-23 sum|x w|, plus half a step of the result's type.  Integer data (every partial sum
a whole number below 2^24) must come out exact."""
import numpy as np
import pytest
import torch

from oracle import mx

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module")
def dbf():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from binary_factorized_weight_b200 import build

    build.build()
    import binary_factorized_weight_b200 as mod

    mod.load_library()
    return mod


def host(t):
    return t.detach().double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def held(v, fmt):
    """A matrix in the library's buffers, made by the reference: (codes, scales) on the GPU."""
    code, byte = mx.quantize(v, fmt)
    return (torch.from_numpy(mx.pack_codes(code, fmt)).cuda(),
            torch.from_numpy(mx.pack_scales(byte, *v.shape)).cuda())


def assert_held(codes, scales, v, fmt):
    rows, cols = v.shape
    code, byte = mx.quantize(v, fmt)
    np.testing.assert_array_equal(mx.unpack_scales(host(scales), rows, cols), byte)
    np.testing.assert_array_equal(mx.unpack_codes(host(codes), rows, cols, fmt), code)


def source(rows, cols, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-12, 12, (rows, 1), generator=g).float())
    return v.to(TYPES[kind]).cuda()


@pytest.mark.parametrize("fmt", [mx.E2M1, mx.E4M3])
@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (3, 31), (130, 33), (257, 520), (64, 1000), (127, 129)])
def test_quantize_is_exact(dbf, rows, cols, kind, fmt):
    v = source(rows, cols, kind)
    codes, scales = dbf.dbf_mx_quantize(v, fmt)
    assert_held(codes, scales, host(v), fmt)
    codes, scales = dbf.dbf_mx_quantize(v, fmt, transpose=True)
    assert_held(codes, scales, np.ascontiguousarray(host(v).T), fmt)


@pytest.mark.parametrize("fmt", [mx.E2M1, mx.E4M3])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_borders_and_special_values(dbf, fmt, transpose):
    rng = np.random.default_rng(3)
    grid = mx.values(fmt)
    mid = (grid[1:] + grid[:-1]) / 2
    near = np.concatenate([grid, mid, np.nextafter(mid.astype(np.float32), np.float32(0)).astype(np.float64),
                           np.nextafter(mid.astype(np.float32), np.float32(9e9)).astype(np.float64)])
    rows = [rng.permutation(np.resize(near, 320)) * rng.choice([-1, 1], 320) * 2.0 ** e
            for e in (-126, -100, -20, 0, 3, 100, 110)]
    rows += [np.resize(2.0 ** -149 * np.arange(9), 320), np.zeros(320), np.full(320, -0.0), np.full(320, 3.4028234e38)]
    v = np.array(rows).astype(np.float32)
    v[2, 40] = np.nan
    v[3, 70] = np.inf
    v[4, 319] = -np.inf
    t = torch.from_numpy(v).cuda()
    codes, scales = dbf.dbf_mx_quantize(t.t().contiguous() if transpose else t, fmt, transpose=transpose)
    assert_held(codes, scales, v.astype(np.float64), fmt)
    back = host(dbf.dbf_mx_dequantize(codes, scales, *v.shape, fmt))
    code, byte = mx.quantize(v, fmt)
    np.testing.assert_array_equal(back, mx.dequantize(code, byte, 320, fmt))


@pytest.mark.parametrize("fmt", [mx.E2M1, mx.E4M3])
@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 100), (130, 256), (129, 1001)])
def test_dequantize(dbf, rows, cols, kind, fmt):
    v = host(source(rows, cols, "fp32", seed=1))
    got = dbf.dbf_mx_dequantize(*held(v, fmt), rows, cols, fmt, dtype=TYPES[kind])
    want = torch.from_numpy(mx.dequantize(*mx.quantize(v, fmt), cols, fmt)).float().to(TYPES[kind])
    assert got.dtype == TYPES[kind] and torch.equal(got.cpu(), want)


def test_every_code(dbf):
    codes = np.arange(256).reshape(2, 128)
    byte = np.array([[0, 1, 127, 253], [255, 130, 120, 64]])
    got = host(dbf.dbf_mx_dequantize(torch.from_numpy(codes.astype(np.uint8)).cuda().view(-1),
                                     torch.from_numpy(mx.pack_scales(byte, 2, 128)).cuda(), 2, 128, mx.E4M3))
    with np.errstate(over="ignore"):
        want = mx.dequantize(codes, byte, 128, mx.E4M3).astype(np.float32).astype(np.float64)
    np.testing.assert_array_equal(got, want)


def product(dbf, X, W, xf, wf, kind, **more):
    return dbf.dbf_mx_forward(*held(X, xf), *held(W, wf), W.shape[0], W.shape[1], X.shape[0], x_fmt=xf, w_fmt=wf,
                              y_dtype=TYPES[kind], **more)


def assert_product(y, X, W, xf, wf, kind):
    x = mx.dequantize(*mx.quantize(X, xf), X.shape[1], xf)
    w = mx.dequantize(*mx.quantize(W, wf), W.shape[1], wf)
    want = x @ w.T
    tol = X.shape[1] * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T) + STEP[kind] * np.abs(want) + 2.0 ** -25
    assert (np.abs(host(y) - want) <= tol).all(), np.max(np.abs(host(y) - want) / tol)


FORMATS = [(mx.E2M1, mx.E2M1), (mx.E4M3, mx.E2M1), (mx.E4M3, mx.E4M3), (mx.E2M1, mx.E4M3)]
SHAPES = [(1, 128, 128), (1, 1, 1), (3, 100, 33), (16, 256, 512), (17, 130, 640), (33, 1000, 300), (64, 129, 1111),
          (65, 257, 700), (100, 64, 4096), (200, 300, 520), (1, 4096, 4096), (130, 96, 129)]


@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("batch,n,m_in", SHAPES)
def test_integer_product_is_exact(dbf, batch, n, m_in, xf, wf):
    rng = np.random.default_rng(batch + n + m_in)
    X = rng.choice([0.0, 1, 2, 3, 4, 6, -1, -2, -6], (batch, m_in))
    W = rng.choice([0.0, 1, -1, 2, -3, 6], (n, m_in)) * 2.0 ** rng.integers(-1, 3, (n, 1))
    X[:, 0::32] = 6  # every block's largest value: nothing is lost
    W[:, 0::32] = 6
    assert (mx.dequantize(*mx.quantize(X, xf), m_in, xf) == X).all()
    y = product(dbf, X, W, xf, wf, "fp32")
    w = mx.dequantize(*mx.quantize(W, wf), m_in, wf)
    np.testing.assert_array_equal(host(y), X @ w.T)


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("batch,n,m_in", [(1, 300, 1000), (16, 1024, 4096), (77, 501, 1111), (300, 640, 1500), (2, 77, 5000)])
def test_product(dbf, batch, n, m_in, xf, wf, kind):
    rng = np.random.default_rng(n)
    X = rng.standard_normal((batch, m_in)) * np.where(rng.random(m_in) < 0.01, 30, 1)
    W = rng.standard_normal((n, m_in)) * 0.05
    assert_product(product(dbf, X, W, xf, wf, kind), X, W, xf, wf, kind)


@pytest.mark.parametrize("kind", ["fp16", "fp32"])
@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("batch,n,m_in", [(2048, 2504, 384), (1000, 4737, 130), (260, 14336, 256), (65, 19001, 100),
                                          (1024, 2400, 2100)])
def test_many_tiles(dbf, batch, n, m_in, xf, wf, kind):
    rng = np.random.default_rng(9)
    X, W = rng.standard_normal((batch, m_in)), rng.standard_normal((n, m_in)) * 0.05
    whole = torch.full((batch * n + 64,), 7.0, dtype=TYPES[kind], device="cuda")
    y = product(dbf, X, W, xf, wf, kind, y=whole[: batch * n].view(batch, n))
    assert_product(y, X, W, xf, wf, kind)
    assert (whole[batch * n:] == 7).all()


@pytest.mark.parametrize("xf,wf", FORMATS)
def test_many_tiles_integer_exact(dbf, xf, wf):
    """Several tiles per CTA pair, every row and column with a scale of its own."""
    rng = np.random.default_rng(10)
    batch, n, m_in = 1100, 5000, 700
    X = rng.choice([0.0, 1, 2, 3, -1, -2, -6], (batch, m_in)) * 2.0 ** rng.integers(-2, 3, (batch, 1))
    W = rng.choice([0.0, 1, -1, 2, -3], (n, m_in)) * 2.0 ** rng.integers(-2, 3, (n, 1))
    x, w = mx.dequantize(*mx.quantize(X, xf), m_in, xf), mx.dequantize(*mx.quantize(W, wf), m_in, wf)
    np.testing.assert_array_equal(host(product(dbf, X, W, xf, wf, "fp32")), x @ w.T)


@pytest.mark.parametrize("batch", [1, 40, 300])
@pytest.mark.parametrize("xf,wf", FORMATS)
def test_nan_blocks_stay_in_their_rows(dbf, batch, xf, wf):
    rng = np.random.default_rng(2)
    X, W = rng.standard_normal((batch, 300)), rng.standard_normal((600, 300))
    X[batch // 2, 290] = np.inf
    W[7, 3] = np.nan
    y = host(product(dbf, X, W, xf, wf, "fp32"))
    bad = np.zeros((batch, 600), bool)
    bad[batch // 2] = True
    bad[:, 7] = True
    np.testing.assert_array_equal(np.isnan(y), bad)
    assert np.isfinite(y[~bad]).all()


@pytest.mark.parametrize("xf,wf", FORMATS)
def test_scale_range(dbf, xf, wf):
    """Blocks whose scales lie far apart: the sum is exact where one block carries it all."""
    X, W = np.zeros((2, 128)), np.zeros((3, 128))
    X[:, :] = 2.0 ** -60
    W[:, :] = 2.0 ** -50
    X[1, 32:64] = 2.0 ** 60
    W[2, 32:64] = 2.0 ** 50
    y = host(product(dbf, X, W, xf, wf, "fp32"))
    x, w = X.astype(np.float64), W.astype(np.float64)
    np.testing.assert_allclose(y, x @ w.T, rtol=2.0 ** -20)


def test_one_long_token(dbf):
    """m_in at a million.  Normal data: the running sum stays below about 4 sqrt(K) = 2^12, an addition for each 32 of K
    loses at most 2^-23 of it: 2^15 2^-23 2^12 = 2^4; the bound allows four times that, 2^-14 |x| |w| = 2^6."""
    rng = np.random.default_rng(4)
    X, W = rng.standard_normal((2, 1 << 20)), rng.standard_normal((5, 1 << 20))
    for xf, wf in FORMATS[:2]:
        x, w = mx.dequantize(*mx.quantize(X, xf), 1 << 20, xf), mx.dequantize(*mx.quantize(W, wf), 1 << 20, wf)
        y = host(product(dbf, X, W, xf, wf, "fp32"))
        assert (np.abs(y - x @ w.T) <= 2.0 ** -14 * np.sqrt((x * x).sum(1)[:, None] * (w * w).sum(1)[None, :])).all()


@pytest.mark.parametrize("batch", [1, 20, 100, 300])
def test_nothing_outside_y_is_written(dbf, batch):
    rng = np.random.default_rng(8)
    n, m_in = 333, 200
    X, W = rng.standard_normal((batch, m_in)), rng.standard_normal((n, m_in))
    whole = torch.full((batch * n + 64,), 7.0, dtype=torch.float32, device="cuda")
    product(dbf, X, W, mx.E4M3, mx.E2M1, "fp32", y=whole[: batch * n].view(batch, n))
    assert (whole[batch * n:] == 7).all()


def test_streams_graph_and_shared_workspace(dbf):
    """Calls on two streams and in replayed graphs share one workspace; results equal the plain call's."""
    rng = np.random.default_rng(1)
    n, m_in = 700, 900
    W = held(rng.standard_normal((n, m_in)), mx.E2M1)
    ws = dbf.dbf_mx_new_workspace(n, m_in, 8)
    xs = [held(rng.standard_normal((8, m_in)), mx.E4M3) for _ in range(2)]
    call = lambda x, **k: dbf.dbf_mx_forward(*x, *W, n, m_in, 8, workspace=ws, flags=dbf.DBF_FWD_WEIGHTS_STATIC, **k)  # noqa: E731
    want = [call(x).clone() for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [call(x, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(x))
        graphs.append(g)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert dbf.dbf_workspace_status(ws) == 0


def test_results_repeat_bit_for_bit(dbf):
    rng = np.random.default_rng(12)
    for batch in (1, 16, 128, 600):
        X, W = held(rng.standard_normal((batch, 2000)), mx.E4M3), held(rng.standard_normal((1500, 2000)), mx.E2M1)
        first = dbf.dbf_mx_forward(*X, *W, 1500, 2000, batch, y_dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(first, dbf.dbf_mx_forward(*X, *W, 1500, 2000, batch, y_dtype=torch.float32))


def test_refusals_of_the_binding(dbf):
    x = torch.zeros(4, 64, device="cuda")
    codes, scales = dbf.dbf_mx_quantize(x, mx.E2M1)
    with pytest.raises(ValueError):
        dbf.dbf_mx_quantize(x.t(), mx.E2M1)  # not contiguous
    with pytest.raises(ValueError):
        dbf.dbf_mx_quantize(x, 5)
    with pytest.raises(ValueError):
        dbf.dbf_mx_dequantize(codes, scales, 5, 64, mx.E2M1)  # buffers too small
    with pytest.raises(ValueError):
        dbf.dbf_mx_forward(codes, scales, codes, scales, 4, 64, 4, x_fmt=mx.E4M3, w_fmt=mx.E2M1)
    with pytest.raises(TypeError):
        dbf.dbf_mx_forward(codes, scales, codes, scales, 4, 64, 4, x_fmt=0, w_fmt=0, y_dtype=torch.float64)
    with pytest.raises(dbf.DBFError):
        dbf.dbf_mx_forward(codes, scales, codes, scales, 4, 64, 4, x_fmt=0, w_fmt=0, flags=1 << 5)


def test_offsets_past_32_bits(dbf):
    """Matrices of more than 2^31 elements: their last rows equal those rows handled alone."""
    rows, cols = 70000, 32768
    src = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    tail = src[-3:].contiguous()
    for fmt in (mx.E2M1, mx.E4M3):
        codes, scales = dbf.dbf_mx_quantize(src, fmt)
        want = dbf.dbf_mx_dequantize(*dbf.dbf_mx_quantize(tail, fmt), 3, cols, fmt, dtype=torch.bfloat16)
        whole = dbf.dbf_mx_dequantize(codes, scales, rows, cols, fmt, dtype=torch.bfloat16)
        assert torch.equal(whole[-3:], want)
        del codes, scales, whole
    codes, scales = dbf.dbf_mx_quantize(src, mx.E2M1, transpose=True)
    back = dbf.dbf_mx_dequantize(codes, scales, cols, rows, mx.E2M1, dtype=torch.bfloat16)
    want = dbf.dbf_mx_dequantize(*dbf.dbf_mx_quantize(src[:, -5:].t().contiguous(), mx.E2M1), 5, rows, mx.E2M1,
                                 dtype=torch.bfloat16)
    assert torch.equal(back[-5:], want)
    del codes, scales, back
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    y, _ = dbf.dbf_rmsnorm_forward(src, w, 1e-5)
    assert torch.equal(y[-3:], dbf.dbf_rmsnorm_forward(tail, w, 1e-5)[0])
    dx, _ = dbf.dbf_rmsnorm_backward(y, src, w, 1e-5, dx=y)
    assert torch.equal(dx[-3:], dbf.dbf_rmsnorm_backward(dbf.dbf_rmsnorm_forward(tail, w, 1e-5)[0], tail, w, 1e-5)[0])


@pytest.mark.parametrize("n", [60000, 60001])
def test_results_past_32_bits(dbf, n):
    batch, m_in = 40000, 130
    g = torch.Generator(device="cuda").manual_seed(3)
    X, W = (torch.randn(r, m_in, generator=g, device="cuda") for r in (batch, n))
    x, w = dbf.dbf_mx_quantize(X, mx.E4M3), dbf.dbf_mx_quantize(W, mx.E2M1)
    y = dbf.dbf_mx_forward(*x, *w, n, m_in, batch)
    xs, ws = host(X)[-300:], host(W)[-500:]
    assert_product(y[-300:, -500:], xs, ws, mx.E4M3, mx.E2M1, "fp16")
    assert_product(y[:5, :300], host(X)[:5], host(W)[:300], mx.E4M3, mx.E2M1, "fp16")


@pytest.mark.parametrize("seed", range(24))
def test_random_sizes(dbf, seed):
    """Sizes, formats and result types at random, the split and the pair kernel among them."""
    rng = np.random.default_rng(100 + seed)
    size = lambda low, high: int(round(low * (high / low) ** rng.random()))  # noqa: E731
    batch, n, m_in = size(1, 2000), size(1, 6000), size(1, 3000)
    xf, wf = FORMATS[rng.integers(4)]
    kind = ["fp16", "bf16", "fp32"][rng.integers(3)]
    X, W = rng.standard_normal((batch, m_in)), rng.standard_normal((n, m_in)) * 0.1
    assert_product(product(dbf, X, W, xf, wf, kind), X, W, xf, wf, kind)


def test_a_call_behind_one_that_writes_its_operands(dbf):
    """Quantisation and product back to back on one stream, without the static flag: the product waits for the weights."""
    rng = np.random.default_rng(21)
    src = [torch.from_numpy(rng.standard_normal((2048, 1024))).to(torch.bfloat16).cuda() for _ in range(2)]
    X = held(rng.standard_normal((16, 1024)), mx.E4M3)
    codes, scales = (torch.empty_like(t) for t in dbf.dbf_mx_quantize(src[0], mx.E2M1))
    ws = dbf.dbf_mx_new_workspace(2048, 1024, 16)
    want = [dbf.dbf_mx_forward(*X, *dbf.dbf_mx_quantize(s, mx.E2M1), 2048, 1024, 16) for s in src]
    torch.cuda.synchronize()
    for i in range(40):
        dbf.dbf_mx_quantize(src[i % 2], mx.E2M1, codes=codes, scales=scales)
        y = dbf.dbf_mx_forward(*X, codes, scales, 2048, 1024, 16, workspace=ws)
        assert torch.equal(y, want[i % 2])


def test_bench_mode_runs():
    """bench.py --mx prints one JSON line with every layer shape of the set.  The relative error against the dense
    layer is the formats' own: e2m1 rounds a normal weight block by about 0.11 rms, e4m3 its input by 0.03."""
    import json
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "bench.py", "--mx"], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    rows = json.loads(out.stdout.strip().splitlines()[-1])["mx"]
    assert {(r["n"], r["m_in"]) for r in rows} == {(1024, 4096), (4096, 4096), (14336, 4096), (4096, 14336)}
    for r in rows:
        for b in (1, 16, 128, 2048):
            assert r[f"product_us_b{b}"] > 0 and 0.05 < r[f"rel_error_b{b}"] < 0.2


def test_first_calls_inside_a_capture(dbf):
    """A process whose first calls of every operator are captured: nothing needs a call before."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch
import binary_factorized_weight_b200 as dbf
W = torch.randn(4096, 512, device="cuda"); x = torch.randn(600, 512, device="cuda"); w = torch.ones(512, device="cuda")
ws = dbf.dbf_mx_new_workspace(4096, 512, 600)
torch.cuda.synchronize()
def run():
    q = dbf.dbf_mx_quantize(W, 0)
    t = dbf.dbf_mx_quantize(W, 1, transpose=True)
    c, s, h = dbf.dbf_rmsnorm_mx_forward(x, w, 1e-5, 1, residual=x)
    y = dbf.dbf_mx_forward(c, s, *q, 4096, 512, 600, workspace=ws, y_dtype=torch.float32)
    few = dbf.dbf_mx_quantize(x[:5].contiguous(), 1)
    z = dbf.dbf_mx_forward(*few, *q, 4096, 512, 5, workspace=ws, y_dtype=torch.float32)
    dx, dw = dbf.dbf_rmsnorm_backward(x, h, w, 1e-5)
    return y, z, dx, dw, dbf.dbf_mx_dequantize(*t, 512, 4096, 1), dbf.dbf_rmsnorm_forward(x, w, 1e-5)[0]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = run()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, run())) and dbf.dbf_workspace_status(ws) == 0
print("same")
"""
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=200)
    assert out.returncode == 0 and out.stdout.strip().endswith("same"), out.stderr[-2000:]


def test_a_product_longer_than_the_limit_of_a_wait(dbf):
    """8.6e14 operations, about 0.3 s: a bounded wait (0.2 s) covers a step or an item of a kernel, never all of it.
    Ones with a scale for each row (of 128 in turn), so that y is known exactly: 2^17 times two powers of two."""
    n, m_in = 57344, 1 << 17
    row = torch.arange(128, device="cuda")
    at = torch.arange(512, device="cuda")  # the tile's byte 16 (r % 32) + 4 (r / 32) + k belongs to row r
    row_of = at // 16 + 32 * (at % 16 // 4)

    def operand(fmt, exponent):
        codes = torch.full((dbf.dbf_mx_code_bytes(n, m_in, fmt),), 0x22 if fmt == mx.E2M1 else 0x38, dtype=torch.uint8,
                           device="cuda")
        tiles = (127 + exponent[row_of]).to(torch.uint8)
        return codes, tiles.repeat(dbf.dbf_mx_scale_bytes(n, m_in) // 512)

    ex, ew = row % 7 - 3, row % 5 - 2
    x, w = operand(mx.E4M3, ex), operand(mx.E2M1, ew)
    y = torch.zeros(n, n, dtype=torch.bfloat16, device="cuda")
    ws = dbf.dbf_mx_new_workspace(n, m_in, n)
    want = torch.exp2((17 + ex[:, None] + ew[None, :]).double()).to(torch.bfloat16)
    for _ in range(2):
        dbf.dbf_mx_forward(*x, *w, n, m_in, n, y=y, workspace=ws)
    assert dbf.dbf_workspace_status(ws) == 0
    assert (y.view(n // 128, 128, n // 128, 128) == want[None, :, None, :]).all()


def test_out_of_memory_is_torchs_error(dbf):
    """y of 2^40 elements from small operands: the allocator's error comes through as it is."""
    codes, scales = dbf.dbf_mx_quantize(torch.zeros(1 << 20, 1, dtype=torch.float16, device="cuda"), mx.E2M1)
    with pytest.raises(torch.OutOfMemoryError):
        dbf.dbf_mx_forward(codes, scales, codes, scales, 1 << 20, 1, 1 << 20, x_fmt=mx.E2M1, w_fmt=mx.E2M1)
    dbf.dbf_mx_quantize(torch.zeros(2, 2, device="cuda"), mx.E2M1)


def test_calls_release_the_interpreter(dbf):
    """A launch may wait for room in the GPU's queue; other Python threads run meanwhile.  In place of the entry points
    stands a function that answers whether its thread holds the interpreter's lock (as a status: 0, no)."""
    import ctypes

    binding, lib = dbf._binding(), dbf.load_library()
    entries = [lib.dbf_mx_quantize, lib.dbf_mx_dequantize, lib.dbf_mx_forward, lib.dbf_rmsnorm_forward,
               lib.dbf_rmsnorm_mx_forward, lib.dbf_rmsnorm_backward]
    sizes = [lib.dbf_mx_code_bytes, lib.dbf_mx_scale_bytes, lib.dbf_mx_forward_workspace_bytes,
             lib.dbf_rmsnorm_backward_workspace_bytes]
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    c, s = dbf.dbf_mx_quantize(x, mx.E4M3)
    binding.init(dbf._raise_status, *[address(ctypes.pythonapi.PyGILState_Check)] * 6, *map(address, sizes))
    try:
        dbf.dbf_mx_quantize(x, mx.E4M3)
        dbf.dbf_mx_dequantize(c, s, 4, 64, mx.E4M3)
        dbf.dbf_mx_forward(c, s, c, s, 4, 64, 4, w_fmt=mx.E4M3)
        dbf.dbf_rmsnorm_forward(x, w, 1e-5)
        dbf.dbf_rmsnorm_mx_forward(x, w, 1e-5)
        dbf.dbf_rmsnorm_backward(x, x, w, 1e-5)
    finally:
        binding.init(dbf._raise_status, *map(address, entries + sizes))


def test_calls_from_two_threads(dbf):
    """Two threads at once, each on its own stream, with a workspace between them: every result is the single call's."""
    import threading

    rng = np.random.default_rng(30)
    sizes = [(1, 640, 900), (40, 640, 900), (300, 1000, 900)]
    W = {n: held(rng.standard_normal((n, 900)), mx.E2M1) for _, n, _ in sizes}
    X = {b: torch.from_numpy(rng.standard_normal((b, 900))).half().cuda() for b, _, _ in sizes}
    g = torch.ones(900, dtype=torch.float16, device="cuda")
    ws = dbf.dbf_mx_new_workspace(1000, 900, 300)

    def run(b, n, m_in):
        codes, scales, _ = dbf.dbf_rmsnorm_mx_forward(X[b], g, 1e-5, residual=X[b])
        y = dbf.dbf_mx_forward(codes, scales, *W[n], n, m_in, b, workspace=ws, y_dtype=torch.float32)
        return y, dbf.dbf_rmsnorm_backward(X[b], X[b], g, 1e-5)[1]

    want = [run(*s) for s in sizes]
    torch.cuda.synchronize()
    wrong = []

    def thread():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(60):
                    got = [run(*s) for s in sizes]
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for p, q in zip(got, want) for a, b in zip(p, q)):
                        wrong.append("another result")
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    threads = [threading.Thread(target=thread) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and dbf.dbf_workspace_status(ws) == 0


@pytest.mark.parametrize("fmt", [mx.E2M1, mx.E4M3])
def test_quantize_at_the_largest_shapes(dbf, fmt):
    """One row or column of 2^24: a long row equals the same blocks as many rows, a column its rows by themselves, and
    the transposed forms each other."""
    size = 1 << 24
    g = torch.Generator(device="cuda").manual_seed(51)
    v = torch.randn(size, generator=g, device="cuda").to(torch.bfloat16)
    row, column, table = v.view(1, size), v.view(size, 1), v.view(size // 4096, 4096)
    q = dbf.dbf_mx_quantize(row, fmt)
    want = dbf.dbf_mx_dequantize(*dbf.dbf_mx_quantize(table, fmt), *table.shape, fmt)
    assert torch.equal(dbf.dbf_mx_dequantize(*q, 1, size, fmt).view(-1), want.view(-1))
    t = dbf.dbf_mx_quantize(column, fmt, transpose=True)
    assert torch.equal(t[0], q[0])
    assert torch.equal(dbf.dbf_mx_dequantize(*t, 1, size, fmt).view(-1), want.view(-1))
    c = dbf.dbf_mx_quantize(column, fmt)
    back = dbf.dbf_mx_dequantize(*c, size, 1, fmt).view(-1)
    some = torch.cat([torch.arange(300, device="cuda"), torch.arange(size - 300, size, device="cuda")])
    few = dbf.dbf_mx_dequantize(*dbf.dbf_mx_quantize(column[some].contiguous(), fmt), 600, 1, fmt).view(-1)
    assert torch.equal(back[some], few)
    t = dbf.dbf_mx_quantize(row, fmt, transpose=True)
    assert torch.equal(t[0], c[0]) and torch.equal(dbf.dbf_mx_dequantize(*t, size, 1, fmt).view(-1), back)


@pytest.mark.parametrize("xf,wf", [(mx.E2M1, mx.E2M1), (mx.E4M3, mx.E2M1)])
@pytest.mark.parametrize("batch,n", [(1, 1 << 24), (70, 1 << 24), (1 << 24, 3), (1 << 24, 300)])
def test_product_at_the_largest_shapes(dbf, batch, n, xf, wf):
    """2^24 weight rows or tokens: whole numbers, exact at both ends and at random places between."""
    m_in = 33
    g = torch.Generator(device="cuda").manual_seed(52)
    pick = lambda rows: torch.tensor([0.0, 1, 2, 3, -1, -2, -6], device="cuda")[  # noqa: E731
        torch.randint(0, 7, (rows, m_in), generator=g, device="cuda")].to(torch.bfloat16)
    X, W = pick(batch), pick(n)
    y = dbf.dbf_mx_forward(*dbf.dbf_mx_quantize(X, xf), *dbf.dbf_mx_quantize(W, wf), n, m_in, batch, x_fmt=xf, w_fmt=wf,
                           y_dtype=torch.float32 if n < 300 or batch == 1 else torch.float16)
    X, W = (dbf.dbf_mx_dequantize(*dbf.dbf_mx_quantize(t, f), t.shape[0], m_in, f) for t, f in ((X, xf), (W, wf)))

    def some(size):
        if size < 1000:
            return torch.arange(size, device="cuda")
        return torch.cat([torch.arange(300, device="cuda"), torch.arange(size - 300, size, device="cuda"),
                          torch.randint(0, size, (1000,), generator=g, device="cuda")])

    i, j = some(batch), some(n)
    assert torch.equal(y[i][:, j].double(), X[i].double() @ W[j].double().t())


@pytest.mark.parametrize("batch", [1, 20, 100, 300])
@pytest.mark.parametrize("xf,wf", FORMATS)
def test_what_lay_in_the_buffers_reaches_no_result(dbf, batch, xf, wf):
    """Codes and scales written into buffers of 0xFF (NaN scales, which rows behind the last one keep): the matrices and
    their product are those of fresh buffers, bit for bit, from the quantisation, its transpose and the norm."""
    n, m_in = 333, 200
    g = torch.Generator(device="cuda").manual_seed(60)
    X, W = torch.randn(batch, m_in, generator=g, device="cuda"), torch.randn(n, m_in, generator=g, device="cuda")
    weight = torch.ones(m_in, device="cuda")

    def used(rows, fmt):
        full = lambda size: torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # noqa: E731
        return dict(codes=full(dbf.dbf_mx_code_bytes(rows, m_in, fmt)), scales=full(dbf.dbf_mx_scale_bytes(rows, m_in)))

    kw = dict(x_fmt=xf, w_fmt=wf, y_dtype=torch.float32)
    w = dbf.dbf_mx_quantize(W, wf)
    want = dbf.dbf_mx_forward(*dbf.dbf_mx_quantize(X, xf), *w, n, m_in, batch, **kw)
    assert torch.isfinite(want).all()
    dirty = dbf.dbf_mx_quantize(X.t().contiguous(), xf, transpose=True, **used(batch, xf))
    for other in (dbf.dbf_mx_quantize(W, wf, **used(n, wf)),
                  dbf.dbf_mx_quantize(W.t().contiguous(), wf, transpose=True, **used(n, wf))):
        assert torch.equal(other[0], w[0])
        assert torch.equal(dbf.dbf_mx_forward(*dirty, *other, n, m_in, batch, **kw), want)
    clean = dbf.dbf_rmsnorm_mx_forward(X, weight, 1e-5, xf)
    normed = dbf.dbf_rmsnorm_mx_forward(X, weight, 1e-5, xf, **used(batch, xf))
    assert torch.equal(normed[0], clean[0])
    assert torch.equal(dbf.dbf_mx_forward(*normed[:2], *w, n, m_in, batch, **kw),
                       dbf.dbf_mx_forward(*clean[:2], *w, n, m_in, batch, **kw))

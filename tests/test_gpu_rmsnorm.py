"""GPU parity of the RMS norm (dense and microscaled output) and of its gradients through the public calls, against
the fp64 reference (oracle/mx.py).

Tolerances.  u = 2^-24.  A thread adds at most 16 squares of a row that fits the block (cols / 1024 + 8 of a wider
one), two warp sums add five more each, the wide reading's rounds included in L = 26 + cols / 1024; all terms are
positive, so the sum is off by at most L u relative, its root by half of that; mean, eps, root, quotient and the two
products add a rounding each: |y err| <= (L / 2 + 8) u |y|, and half a step of the type.  Quantised outputs must lie
between the quantised ends of that interval (rounding is monotone)."""
import numpy as np
import pytest
import torch

from oracle import mx
from test_gpu_mx import STEP, TYPES, dbf, host  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134, "fp32": 2.0 ** -150}  # half the smallest step
SHAPES = [(1, 1), (1, 32), (2, 64), (3, 100), (1, 4096), (5, 4097), (200, 256), (129, 1000), (17, 8192), (4, 8200),
          (3, 16384), (2, 16385), (2, 40000), (1000, 512),
          (3, 65536), (2, 65537), (300, 700), (80, 9008)]


def rel(cols):
    return ((26 + cols / 1024) / 2 + 8) * U


def data(rows, cols, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[kind]
    x, r = (torch.randn(rows, cols, generator=g).to(t).cuda() for _ in range(2))
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(t).cuda()
    return x, r, w


def assert_dense(y, h, w, eps, kind):
    want = mx.rmsnorm(host(h), host(w), eps)
    tol = rel(h.shape[1]) * np.abs(want) + STEP[kind] * np.abs(want) * (1 + rel(h.shape[1])) + TINY[kind]
    assert (np.abs(host(y) - want) <= tol).all(), np.max(np.abs(host(y) - want) / tol)


def assert_quantised(codes, scales, h, w, eps, fmt):
    rows, cols = h.shape
    y = mx.rmsnorm(host(h), host(w), eps)
    byte = mx.unpack_scales(host(scales), rows, cols)
    got = mx.dequantize(mx.unpack_codes(host(codes), rows, cols, fmt), byte, cols, fmt)
    d = rel(cols)
    amax = np.abs(mx.blocks(y)).max(2)
    low, high = mx.scale_byte(amax * (1 - d), fmt), mx.scale_byte(amax * (1 + d), fmt)
    assert ((byte == low) | (byte == high)).all()
    f = np.repeat(mx.factor(byte), 32, axis=1)[:, :cols]
    grid = mx.values(fmt)
    least, most = (grid[mx.round_codes(np.abs(y) * s / f, fmt)] * f for s in (1 - d, 1 + d))
    assert ((np.abs(got) >= least) & (np.abs(got) <= most)).all()
    assert ((np.sign(got) == np.sign(y)) | (got == 0)).all()
    pads = mx.unpack_codes(host(codes), rows, cols, fmt)[:, cols:]
    assert (pads == 0).all() and (byte[:, -(-cols // 32):] == 0).all()


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(dbf, rows, cols, kind):
    x, r, w = data(rows, cols, kind)
    y, h = dbf.dbf_rmsnorm_forward(x, w, EPS)
    assert h is x
    assert_dense(y, x, w, EPS, kind)
    y, h = dbf.dbf_rmsnorm_forward(x, w, EPS, residual=r)
    assert torch.equal(h.cpu(), (x.float() + r.float()).to(TYPES[kind]).cpu())
    assert_dense(y, h, w, EPS, kind)


@pytest.mark.parametrize("fmt", [mx.E2M1, mx.E4M3])
@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantised_forward(dbf, rows, cols, kind, fmt):
    x, r, w = data(rows, cols, kind, seed=1)
    codes, scales, h = dbf.dbf_rmsnorm_mx_forward(x, w, EPS, fmt)
    assert_quantised(codes, scales, x, w, EPS, fmt)
    codes, scales, h = dbf.dbf_rmsnorm_mx_forward(x, w, EPS, fmt, residual=r)
    assert torch.equal(h.cpu(), (x.float() + r.float()).to(TYPES[kind]).cpu())
    assert_quantised(codes, scales, h, w, EPS, fmt)


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("in_place", ["x", "residual"])
def test_in_place(dbf, kind, in_place):
    for rows, cols in ((4, 4096), (3, 77), (2, 20000)):
        x, r, w = data(rows, cols, kind)
        want_y, want_h = dbf.dbf_rmsnorm_forward(x, w, EPS, residual=r)
        y, h = dbf.dbf_rmsnorm_forward(x, w, EPS, residual=r, h=x if in_place == "x" else r)
        assert torch.equal(y, want_y) and torch.equal(h, want_h) and h.data_ptr() in (x.data_ptr(), r.data_ptr())


def test_special_rows(dbf):
    """Rows of zeros, of large values and with an infinity or NaN, beside ordinary ones."""
    x, _, w = data(6, 256, "fp32")
    x[0] = 0
    x[1] *= 1e15
    x[2] *= 1e-18
    x[3, 5] = float("nan")
    x[4, 6] = float("inf")
    y, _ = dbf.dbf_rmsnorm_forward(x, w, EPS)
    codes, scales, _ = dbf.dbf_rmsnorm_mx_forward(x, w, EPS, mx.E4M3)
    assert (host(y)[0] == 0).all() and np.isnan(host(y)[3]).all()
    assert np.isnan(host(y)[4, 6]) and (np.delete(host(y)[4], 6) == 0).all()  # inf / inf, and values over inf
    keep = [0, 1, 2, 5]
    assert_dense(y[keep], x[keep], w, EPS, "fp32")
    v = host(dbf.dbf_mx_dequantize(codes, scales, 6, 256, mx.E4M3))
    assert np.isnan(v[3]).all() and np.isnan(v[4, :32]).all() and (v[4, 32:] == 0).all() and (v[0] == 0).all()
    assert np.isfinite(v[keep]).all()


def test_unaligned_rows(dbf):
    """Tensors that start inside an allocation: aligned to their element only."""
    x, r, w = data(3, 512, "fp16")
    shift = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
    y, h = dbf.dbf_rmsnorm_forward(shift(x), shift(w), EPS, residual=shift(r))
    assert_dense(y, h, w, EPS, "fp16")
    dx, dw = dbf.dbf_rmsnorm_backward(shift(r), shift(x), shift(w), EPS)
    assert_grads(dx, dw, r, x, w, None, "fp16")
    codes, scales = dbf.dbf_mx_quantize(shift(x), mx.E2M1)
    assert torch.equal(codes, dbf.dbf_mx_quantize(x, mx.E2M1)[0])
    out = torch.zeros(3 * 512 + 1, dtype=torch.float16, device="cuda")[1:].view(3, 512)
    dbf.dbf_mx_dequantize(codes, scales, 3, 512, mx.E2M1, dst=out)
    assert torch.equal(out, dbf.dbf_mx_dequantize(codes, scales, 3, 512, mx.E2M1, dtype=torch.float16))


# ---------------------------------------------------------------- gradients
def assert_grads(dx, dw, dy, h, w, dh, kind):
    """dx: every product and sum rounds once, the two row sums lose L u of the sum of magnitudes; dweight: each of its
    terms carries the same and is added in at most rows + 320 steps."""
    rows, cols = h.shape
    a, b, c = host(dy), host(h), host(w)
    want_dx, want_dw = mx.rmsnorm_grads(a, b, c, EPS, None if dh is None else host(dh))
    r = 1 / np.sqrt((b * b).mean(1, keepdims=True) + EPS)
    g, d = np.abs(a * c), 4 * rel(cols)
    size = r * g + np.abs(b) * r ** 3 * (g * np.abs(b)).mean(1, keepdims=True)
    tol = 2 * d * size + STEP[kind] * np.abs(want_dx) + TINY[kind] + (0 if dh is None else U * np.abs(host(dh)) + U * size)
    tol = tol * (1 + STEP[kind])
    assert (np.abs(host(dx) - want_dx) <= tol).all(), np.max(np.abs(host(dx) - want_dx) / tol)
    tol = ((rows + 320) * U + d) * (np.abs(a * b) * r).sum(0)
    assert dw.dtype == torch.float32 and (np.abs(host(dw) - want_dw) <= tol).all()


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(dbf, rows, cols, kind):
    h, dy, w = data(rows, cols, kind, seed=2)
    dh = data(rows, cols, kind, seed=3)[0]
    for extra in (None, dh):
        dx, dw = dbf.dbf_rmsnorm_backward(dy, h, w, EPS, dh=extra)
        assert dx.dtype == TYPES[kind]
        assert_grads(dx, dw, dy, h, w, extra, kind)


def test_backward_against_differences(dbf):
    """Along random directions the gradients give the fp64 norm's central difference (error: step^2 of its third
    derivative, about 1e-8 here; the fp32 gradients' own is about 1e-5 of the sum of magnitudes)."""
    h, dy, w = data(4, 333, "fp32", seed=5)
    dx, dw = (host(t) for t in dbf.dbf_rmsnorm_backward(dy, h, w, EPS))
    rng = np.random.default_rng(0)
    H, W, D = host(h), host(w), host(dy)
    for _ in range(5):
        u, v = rng.standard_normal(H.shape), rng.standard_normal(W.shape)
        f = lambda s: (D * mx.rmsnorm(H + s * u, W + s * v, EPS)).sum()  # noqa: E731
        num = (f(1e-4) - f(-1e-4)) / 2e-4
        assert abs(num - (dx * u).sum() - (dw * v).sum()) < 1e-5 * ((np.abs(dx * u)).sum() + np.abs(dw * v).sum())


@pytest.mark.parametrize("alias", ["dh", "dy"])
def test_backward_in_place(dbf, alias):
    for rows, cols in ((7, 512), (3, 9000)):
        h, dy, w = data(rows, cols, "bf16", seed=2)
        dh = data(rows, cols, "bf16", seed=3)[0]
        want = dbf.dbf_rmsnorm_backward(dy, h, w, EPS, dh=dh)
        dx, dw = dbf.dbf_rmsnorm_backward(dy, h, w, EPS, dh=dh, dx=dh if alias == "dh" else dy)
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_backward_repeats_and_replays(dbf):
    """Bit for bit the same again, on another stream, and in a replayed graph with new inputs."""
    h, dy, w = data(700, 1024, "bf16", seed=7)
    first = dbf.dbf_rmsnorm_backward(dy, h, w, EPS)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    again = dbf.dbf_rmsnorm_backward(dy, h, w, EPS, stream=s)
    s.synchronize()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    ws = dbf.dbf_rmsnorm_backward_new_workspace(700, 1024)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dx, dw = dbf.dbf_rmsnorm_backward(dy, h, w, EPS, workspace=ws)
    g.replay()
    assert torch.equal(dx, first[0]) and torch.equal(dw, first[1])
    dy.copy_(data(700, 1024, "bf16", seed=8)[1])
    want = dbf.dbf_rmsnorm_backward(dy, h, w, EPS)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("batch", [1, 16, 130, 600])
@pytest.mark.parametrize("wf", [mx.E2M1, mx.E4M3])
def test_norm_feeds_the_product(dbf, batch, wf):
    """The run of a layer: residual and norm into codes, the product, and its result back into the next norm."""
    n, m_in = 640, 1000
    x, r, w = data(batch, m_in, "bf16", seed=4)
    rng = np.random.default_rng(4)
    W = torch.from_numpy(rng.standard_normal((n, m_in)) * 0.05).to(torch.bfloat16).cuda()
    wc, wsc = dbf.dbf_mx_quantize(W, wf)
    codes, scales, h = dbf.dbf_rmsnorm_mx_forward(x, w, EPS, mx.E4M3, residual=r)
    y = dbf.dbf_mx_forward(codes, scales, wc, wsc, n, m_in, batch, x_fmt=mx.E4M3, w_fmt=wf, y_dtype=torch.bfloat16,
                           flags=dbf.DBF_FWD_WEIGHTS_STATIC)
    z, _ = dbf.dbf_rmsnorm_forward(y, torch.ones(n, dtype=torch.bfloat16, device="cuda"), EPS)
    a = mx.dequantize(mx.unpack_codes(host(codes), batch, m_in, mx.E4M3), mx.unpack_scales(host(scales), batch, m_in),
                      m_in, mx.E4M3)
    b = mx.dequantize(*mx.quantize(host(W), wf), m_in, wf)
    tol = m_in * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T) + STEP["bf16"] * np.abs(a @ b.T)
    assert (np.abs(host(y) - a @ b.T) <= tol).all()
    assert_dense(z, y, torch.ones(n, dtype=torch.bfloat16), EPS, "bf16")


def test_gradients_of_a_layer_by_transposed_operands(dbf):
    """dX = dY W and dW = dY^T X as products of transposed quantised operands."""
    rng = np.random.default_rng(11)
    b, n, m = 96, 200, 160
    dY, X, W = (torch.from_numpy(rng.standard_normal(s)).float().cuda() for s in ((b, n), (b, m), (n, m)))
    q = lambda t, tr=False: dbf.dbf_mx_quantize(t, mx.E4M3, transpose=tr)  # noqa: E731
    deq = lambda t: mx.dequantize(*mx.quantize(host(t), mx.E4M3), t.shape[1], mx.E4M3)  # noqa: E731
    kw = dict(x_fmt=mx.E4M3, w_fmt=mx.E4M3, y_dtype=torch.float32)
    dX = dbf.dbf_mx_forward(*q(dY), *q(W, True), m, n, b, **kw)
    dW = dbf.dbf_mx_forward(*q(dY, True), *q(X, True), m, b, n, **kw)
    for got, left, right, k in ((dX, deq(dY), deq(W.t()), n), (dW, deq(dY.t()), deq(X.t()), b)):
        tol = k * 2.0 ** -23 * (np.abs(left) @ np.abs(right).T) + STEP["fp32"] * np.abs(left @ right.T)
        assert (np.abs(host(got) - left @ right.T) <= tol).all()


def test_refusals_of_the_binding(dbf):
    x, r, w = data(2, 64, "fp16")
    for bad in (lambda: dbf.dbf_rmsnorm_forward(x, w.float(), EPS), lambda: dbf.dbf_rmsnorm_forward(x, w[:32], EPS),
                lambda: dbf.dbf_rmsnorm_forward(x, w, EPS, residual=r[:1]),
                lambda: dbf.dbf_rmsnorm_forward(x, w, EPS, h=torch.empty_like(x)),
                lambda: dbf.dbf_rmsnorm_forward(x[:, ::2], w[:32], EPS),
                lambda: dbf.dbf_rmsnorm_mx_forward(x, w, EPS, 3),
                lambda: dbf.dbf_rmsnorm_backward(r.float(), x, w, EPS),
                lambda: dbf.dbf_rmsnorm_backward(r, x, w, EPS, dweight=torch.empty(64, dtype=torch.float16, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dbf.dbf_rmsnorm_forward(x, w, 0.0), lambda: dbf.dbf_rmsnorm_forward(x[:0], w, EPS),
                lambda: dbf.dbf_rmsnorm_backward(r, x, w, EPS, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(dbf.DBFError):
            bad()


@pytest.mark.parametrize("seed", range(16))
def test_random_sizes(dbf, seed):
    rng = np.random.default_rng(200 + seed)
    size = lambda low, high: int(round(low * (high / low) ** rng.random()))  # noqa: E731
    rows, cols, kind = size(1, 400), size(1, 20000), ["fp16", "bf16", "fp32"][rng.integers(3)]
    x, r, w = data(rows, cols, kind, seed=seed)
    y, h = dbf.dbf_rmsnorm_forward(x, w, EPS, residual=r)
    assert_dense(y, h, w, EPS, kind)
    fmt = [mx.E2M1, mx.E4M3][rng.integers(2)]
    codes, scales, _ = dbf.dbf_rmsnorm_mx_forward(x, w, EPS, fmt, residual=r)
    assert_quantised(codes, scales, h, w, EPS, fmt)
    dx, dw = dbf.dbf_rmsnorm_backward(y, h, w, EPS, dh=r)
    assert_grads(dx, dw, y, h, w, r, kind)


# ---------------------------------------------------------------- the ends of the range
# Few rows (one cluster), a warp's rows (aligned and not), a block's, a cluster's, and rows of any width.
GRAD_FORMS = [(5, 256), (5, 4095), (40, 512), (40, 333), (40, 4096), (40, 1000), (40, 9008), (24, 20001), (5, 65537)]


@pytest.mark.parametrize("eps", [1e-5, 1e-30, 1.2e-38])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", GRAD_FORMS)
def test_backward_of_special_rows(dbf, rows, cols, kind, eps):
    """Rows of zeros, of large and of small values, at every eps that the calls take.  The tolerance is assert_grads':
    it counts relative roundings only, so it holds as long as no intermediate leaves the normal range, and here the
    squares (up to 65537 * 2^4 * 1e30 < 1e37) and quotients (1 / sqrt(1.2e-38) < 1e20) are far from its ends."""
    h, dy, w = data(rows, cols, kind, seed=12)
    dh = data(rows, cols, kind, seed=13)[0]
    h[0] = 0
    h[1] *= 1e15
    h[2] *= 1e-18
    h[3] *= 1e13
    a, b, c = host(dy), host(h), host(w)
    r = 1 / np.sqrt((b * b).mean(1, keepdims=True) + eps)
    g, d = np.abs(a * c), 4 * rel(cols)
    size = r * g + r * np.abs(b * r) * (g * np.abs(b * r)).mean(1, keepdims=True)
    for extra in (None, dh):
        dx, dw = dbf.dbf_rmsnorm_backward(dy, h, w, eps, dh=extra)
        want_dx, want_dw = mx.rmsnorm_grads(a, b, c, eps, None if extra is None else host(extra))
        tol = 2 * d * size + STEP[kind] * np.abs(want_dx) + TINY[kind]
        tol = (tol + (0 if extra is None else U * np.abs(host(extra)) + U * size)) * (1 + STEP[kind])
        assert (np.abs(host(dx) - want_dx) <= tol).all(), np.nanmax(np.abs(host(dx) - want_dx) / tol, axis=1)[:5]
        tol = ((rows + 320) * U + d) * (np.abs(a * b) * r).sum(0)
        assert (np.abs(host(dw) - want_dw) <= tol).all()


@pytest.mark.parametrize("rows,cols", GRAD_FORMS)
def test_backward_of_rows_with_nan_and_infinity(dbf, rows, cols):
    """They make their own rows and, through the sum over rows, dweight NaN; the other rows are as without them."""
    h, dy, w = data(rows, cols, "fp32", seed=14)
    want, _ = dbf.dbf_rmsnorm_backward(dy, h, w, EPS)
    h[1, cols // 2] = float("nan")
    h[3, cols - 1] = float("inf")
    dx, dw = dbf.dbf_rmsnorm_backward(dy, h, w, EPS)
    assert torch.isnan(dx[[1, 3]]).all() and torch.isnan(dw).all()
    keep = [i for i in range(rows) if i not in (1, 3)]
    assert torch.equal(dx[keep], want[keep])


@pytest.mark.parametrize("fmt", [mx.E2M1, mx.E4M3])
@pytest.mark.parametrize("rows,cols", [(6, 33), (6, 16), (200, 528), (6, 1000), (200, 1001), (6, 17000), (6, 40001), (6, 40016)])
def test_padding_behind_rows_with_nan(dbf, rows, cols, fmt):
    """Blocks that lie wholly behind the last column are zero, with a NaN in the row (its own blocks are NaN, as
    dbf_mx_quantize makes them) or an infinity less an infinity."""
    x, r, w = data(rows, cols, "fp32", seed=15)
    x[1, cols // 3] = float("nan")
    x[3, 2], r[4, 2], x[4, 2] = float("inf"), float("-inf"), float("inf")
    for residual in (None, r):
        codes, scales, _ = dbf.dbf_rmsnorm_mx_forward(x, w, EPS, fmt, residual=residual)
        own = -(-cols // 32)
        byte, code = mx.unpack_scales(host(scales), rows, cols), mx.unpack_codes(host(codes), rows, cols, fmt)
        assert (byte[:, own:] == 0).all() and (code[:, cols:] == 0).all()
        bad = [1] if residual is None else [1, 4]
        assert (byte[bad, :own] == 255).all() and (byte[[0, 2, 5], :own] < 255).all()


@pytest.mark.parametrize("batch", [1, 16, 130])
def test_dense_norm_feeds_the_factorised_layer(dbf, batch):
    """Residual and norm into a DBF layer's x and its result back into the residual stream, on one stream without a
    synchronisation between, plain and replayed: the norm against its reference, the layer against the oracle on the
    norm's own output (bars of test_gpu_parity)."""
    import test_gpu_parity as parity

    n, k, m_in = 512, 384, 768
    layer = parity.random_layer(dbf, n, k, m_in, batch, seed=40)
    ws = dbf.dbf_new_workspace(n, k, m_in, batch)
    x, r, w = data(batch, m_in, "fp16", seed=41)
    one = torch.ones(n, dtype=torch.float16, device="cuda")
    z = torch.zeros(batch, n, dtype=torch.float16, device="cuda")

    def run():
        y, h = dbf.dbf_rmsnorm_forward(x, w, EPS, residual=r)
        out = dbf.dbf_forward(y, layer.pA, layer.pB, layer.a, layer.mid, layer.b, n, k, m_in, workspace=ws)
        return y, h, out, *dbf.dbf_rmsnorm_forward(out, one, EPS, residual=z)

    plain = run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        replayed = run()
    g.replay()
    for y, h, out, last, stream in (plain, replayed):
        assert_dense(y, h, w, EPS, "fp16")
        L = layer.np
        want = parity.oracle.forward_staged(host(y), L["A"], L["B"], L["a"], L["mid"], L["b"])
        parity.assert_fp16_close(host(out), want)
        assert torch.equal(stream, out)
        assert_dense(last, stream, one, EPS, "fp16")


@pytest.mark.parametrize("alias", ["dh", "dy"])
@pytest.mark.parametrize("rows,cols", GRAD_FORMS)
def test_backward_in_place_in_every_form(dbf, rows, cols, alias):
    for kind in ("bf16", "fp32"):
        h, dy, w = data(rows, cols, kind, seed=2)
        dh = data(rows, cols, kind, seed=3)[0]
        want = dbf.dbf_rmsnorm_backward(dy, h, w, EPS, dh=dh)
        dx, dw = dbf.dbf_rmsnorm_backward(dy, h, w, EPS, dh=dh, dx=dh if alias == "dh" else dy)
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("rows,cols", [(1 << 24, 1), (2, 1 << 20), (1, (1 << 20) - 1)])
def test_largest_shapes(dbf, rows, cols):
    """The ends of the shape contract against the formulas in fp64 on the GPU (tolerances as above; a row that fits no
    block adds cols / 1024 squares a thread, which rel() counts)."""
    g = torch.Generator(device="cuda").manual_seed(50)
    h, dy = (torch.randn(rows, cols, generator=g, device="cuda") for _ in range(2))
    w = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    H, D, W = h.double(), dy.double(), w.double()
    r = 1 / torch.sqrt((H * H).mean(1, keepdim=True) + EPS)
    d = rel(cols)
    y, _ = dbf.dbf_rmsnorm_forward(h, w, EPS)
    assert ((y - H * r * W).abs() <= (d + U * (1 + d)) * (H * r * W).abs() + TINY["fp32"]).all()
    codes, scales, _ = dbf.dbf_rmsnorm_mx_forward(h, w, EPS, mx.E4M3)
    back = dbf.dbf_mx_dequantize(codes, scales, rows, cols, mx.E4M3)
    # e4m3: off by 2^-4 of the value, by (512 - 448) / 512 = 2^-3 where a block's largest saturates, and by half of the
    # smallest step, 2^-10 of a scale of 2^-8 of the top at most
    top = (H * r * W).abs()
    top = top if cols == 1 else torch.nn.functional.pad(top, (0, -cols % 32)).view(rows, -1, 32).amax(2).repeat_interleave(
        32, 1)[:, :cols]
    assert ((back - H * r * W).abs() <= (1 + 2 * d) * (2.0 ** -3 * (H * r * W).abs() + 2.0 ** -18 * top)).all()
    dx, dw = dbf.dbf_rmsnorm_backward(dy, h, w, EPS)
    size = r * (D * W).abs() + r * (H * r).abs() * (D * W * H * r).abs().mean(1, keepdim=True)
    m = (D * W * H * r).mean(1, keepdim=True)
    assert ((dx - (r * D * W - r * H * r * m)).abs() <= 2 * 4 * d * size + 2 * U * size + TINY["fp32"]).all()
    # 2^24 rows: a warp adds 2^24 / (8 * 296) of them one after another, then eight and 296 sums
    assert ((dw - (D * H * r).sum(0)).abs() <= (rows / 2368 + 320 + 1) * U * (D * H * r).abs().sum(0) * (1 + 4 * d) + 4 * d * (
        D * H * r).abs().sum(0)).all()

"""GPU parity of the 8-bit rows: int8_quantize / int8_dequantize, int8_matmul and its
gradient, and the layer's backward from an 8-bit checkpoint, against 64-bit forms.

Tolerances follow from the stated roundings: half a unit in the last place of each output type
(bf16 2^-8 of the value at most, fp16 2^-11, fp32 2^-24), plus what each comment counts."""
import numpy as np
import pytest
import torch

import int8_reference as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def f64(t):
    return t.detach().double().cpu().numpy()


def rand(seed, *shape, dtype="bf16", scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(DT[dtype]).cuda()


def check_rows(q8, x):
    codes, scales = ref.quantize(f64(x))
    assert np.array_equal(q8.scales.cpu().numpy(), scales, equal_nan=True)
    assert np.array_equal(q8.codes.cpu().numpy(), codes)


# ------------------------------------------------------------------------------ rows
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 64), (2, 255), (65, 1000), (2, 4099), (5, 8192),
                                       (1, 28672), (2, 33000), (700, 40)])
def test_quantize_exact(qlib, rows, cols, dtype):
    x = rand(rows * 31 + cols, rows, cols, dtype=dtype, scale=3.0)
    check_rows(qlib.int8_quantize(x), x)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_quantize_ties(qlib, dtype):
    """Scale 2^-3 exactly: every half-odd multiple of it is a tie and goes to the even code; in
    fp32, the neighbours of each tie go to their own side."""
    s = 2.0 ** -3
    k = torch.arange(-126, 126, dtype=torch.float64) + 0.5
    vals = torch.cat([k * s, torch.tensor([127 * s, -127 * s, 0.0, 126.5 * s])])
    x = vals.to(DT[dtype])[None].repeat(3, 1)
    if dtype == "fp32":
        x[1] = torch.nextafter(x[0], torch.full_like(x[0], 1e9))
        x[2] = torch.nextafter(x[0], torch.full_like(x[0], -1e9))
        x[1:, 252:254] = x[0, 252:254]
    x = x.cuda()
    check_rows(qlib.int8_quantize(x), x)


def test_quantize_near_ties_odd_scales(qlib):
    """Values one fp32 step around (k + 1/2) s for scales with all 24 bits in use."""
    g = torch.Generator().manual_seed(5)
    top = (1 + torch.rand(64, generator=g)) * 10.0 ** torch.randint(-20, 20, (64,), generator=g)
    s = top.float() / torch.tensor(127.0)
    mid = ((torch.arange(0, 127).double() + 0.5)[None] * s.double()[:, None]).float()
    x = torch.cat([top.float()[:, None], mid, torch.nextafter(mid, mid * 2), -torch.nextafter(mid, mid * 0)], 1).cuda()
    check_rows(qlib.int8_quantize(x), x)


def test_quantize_extremes(qlib):
    """Zero rows, subnormal rows (a scale of 0 too), rows next to the largest finite value."""
    x = torch.zeros(8, 40)
    x[1] = torch.linspace(-1, 1, 40) * 1e-43           # scale subnormal
    x[2, 3] = 2.0 ** -149                              # scale rounds to 0
    x[3] = torch.linspace(-190, 190, 40) * 2.0 ** -149  # quotients past 127 are cut
    x[4] = torch.linspace(-1, 1, 40) * 3.4e38
    x[5] = torch.linspace(-1, 1, 40) * 2.0 ** -121
    x[6, 0] = -5.0
    check_rows(qlib.int8_quantize(x.cuda()), x.cuda())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols,stride", [(2000, 2048, 2048), (1000, 4099, 4104), (700, 20000, 20000),
                                              (900, 3001, 3001), (3000, 1000, 1000), (400, 300, 301), (901, 1024, 2048),
                                              (641, 9000, 9008), (1200, 2055, 2055), (50, 20001, 20001)])
def test_quantize_many_rows(qlib, rows, cols, stride, dtype):
    """Persistent CTAs, a warp a row and a CTA a row; among the rows: zero, tiny, huge and non-finite
    ones, scales that a / 127 gives exactly (a = 127 m 2^e, quotients of k + 1/2 among them), ties."""
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, stride, generator=g)
    x[5] = 0
    x[6] *= 1e-6 if dtype == "fp16" else 1e-37
    x[7] *= 1e3 if dtype == "fp16" else 1e37
    x[8, 3] = float("inf")
    x[9, cols - 1] = float("nan")
    k = torch.arange(stride) % 253
    for i, m in enumerate((1, 2, 3, 5, 7, 9, 11, 13, 15)):
        x[20 + i] = (k - 126 + 0.5) * m * 2.0 ** (i % 3 - 1) / 2      # k + 1/2 steps, where the type holds them
        x[20 + i, 0] = 127 * m * 2.0 ** (i % 3 - 1) / 2
    x = x.to(DT[dtype]).cuda()[:, :cols]
    out = qlib.Int8Rows(torch.full((rows + 1, (cols + 31) // 16 * 16), 77, dtype=torch.int8, device="cuda")[:rows, :cols],
                        torch.empty(rows, device="cuda"))
    check_rows(qlib.int8_quantize(x, out=out), x)
    assert (out.codes.as_strided((rows, 16), out.codes.stride(), out.codes.storage_offset() + cols) == 77).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_quantize_nonfinite(qlib, dtype, bad):
    x = rand(3, 6, 100, dtype=dtype)
    x[2, 17] = bad
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q8 = qlib.int8_quantize(x, status=status)
    check_rows(q8, x)
    assert int(status.item()) == qlib.STATUS_NONFINITE
    w = qlib.int8_quantize(rand(4, 24, 100, dtype="fp32"))
    y = qlib.int8_matmul(x, w)
    assert torch.isnan(y[2]).all() and torch.isfinite(torch.cat([y[:2], y[3:]])).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize_strided_and_out(qlib, dtype):
    """Rows inside a wider matrix, at odd offsets too; only cols bytes of a row of `out` are written."""
    wide = rand(9, 20, 333, dtype=dtype)
    for lo, hi in ((0, 333), (8, 264), (3, 200), (5, 6)):
        x = wide[:, lo:hi]
        buf = torch.full((22, 352), 99, dtype=torch.int8, device="cuda")
        sc = torch.full((22,), 7.0, device="cuda")
        out = qlib.Int8Rows(buf[1:21, :hi - lo], sc[1:21])
        assert qlib.int8_quantize(x, out=out) is out
        check_rows(out, x)
        assert (buf[0] == 99).all() and (buf[21] == 99).all() and (buf[:, hi - lo:] == 99).all()
        assert sc[0] == 7 and sc[21] == 7


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows", [3, 600])
def test_rows_at_every_offset(qlib, dtype, rows):
    """Rows that start anywhere between two 16-byte borders, from none to several whole vectors inside
    them, the largest value at either end; the input gradient's rows likewise."""
    size = 4 if dtype == "fp32" else 2
    for lo in range(16 // size):
        for cols in (1, 2, 7, 8, 9, 15, 16, 17, 22, 23, 24, 25, 31, 33, 40, 263, 1030):
            x = rand(lo + cols, rows * cols + lo + 1, dtype=dtype)[lo:lo + rows * cols].view(rows, cols)
            x[0, 0], x[1, cols - 1] = 9.0, -9.0
            check_rows(qlib.int8_quantize(x), x)
            if dtype == "fp32" or rows > 3 and cols not in (23, 1030):
                continue
            w = qlib.Int8Rows(torch.zeros(cols, 16, dtype=torch.int8, device="cuda"), torch.ones(cols, device="cuda"))
            w.codes[0, 0] = w.codes[cols - 1, 1] = w.codes[cols // 2, 2] = 1
            dx = qlib.int8_matmul_backward(x, w)
            want = torch.zeros(rows, 16, dtype=torch.float64, device="cuda")
            for j, c in enumerate((0, cols - 1, cols // 2)):
                want[:, j] += x[:, c].double()
            # 0.51 of a step of the row's fixed point, then the type's own rounding
            step = x.double().abs().amax(1, keepdim=True) / 32639
            assert ((dx.double() - want).abs() <= 0.51 * step + (HALF[DT[dtype]] + 2.0 ** -23) * want.abs()).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 17), (64, 4096), (5, 1003)])
def test_dequantize_exact(qlib, rows, cols, dtype):
    q8 = qlib.int8_quantize(rand(rows + cols, rows, cols, dtype="fp32"))
    v = ref.values(q8.codes.cpu().numpy(), q8.scales.cpu().numpy()).astype(np.float32)
    got = qlib.int8_dequantize(q8, DT[dtype])
    assert torch.equal(got.cpu(), torch.from_numpy(v).to(DT[dtype]))


# ------------------------------------------------------------------------------ product
MATMUL = [(1, 1, 1), (1, 64, 8), (1, 4096, 256), (2, 100, 130), (16, 4096, 1000), (17, 999, 77), (33, 257, 511),
          (64, 512, 384), (130, 1000, 264), (256, 640, 129), (257, 333, 128), (300, 128, 1001), (1000, 2048, 520),
          (5, 131072, 8), (2049, 100, 16), (512, 4096, 4096), (700, 1500, 2504), (384, 96, 5000),
          # many tokens: one tile a CTA pair and several, reductions shorter and longer than the ring
          (1100, 200, 5000), (2600, 1500, 2504), (513, 96, 9999), (700, 5000, 333), (2100, 2053, 40),
          (1200, 40, 3000), (1000, 24, 2504), (600, 16, 11008), (950, 33, 2500), (620, 200, 25000), (1501, 8, 8192),
          (3001, 16, 11001), (1500, 2000, 3001), (900, 6000, 5001), (1600, 3001, 2000), (2100, 3010, 1500),
          (1030, 2500, 4100),
          (4100, 640, 3000), (4100, 200, 3001), (2100, 3000, 700), (9300, 130, 1000),
          # a few tokens: quantized by the product's own CTAs or before it, rows in one wave and several
          (3, 1000, 2500), (8, 2048, 9500), (4, 513, 5000), (7, 12000, 33), (1, 28672, 100), (2, 8192, 5003),
          (1, 16385, 3000), (6, 15, 20000)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K,N", MATMUL)
def test_matmul(qlib, M, K, N, dtype):
    """Exact integer sums and stated fp32 steps: the result before its last rounding is known to the
    bit, so y is that value's nearest in its type."""
    x = rand(M + K, M, K, dtype=dtype)
    w = qlib.int8_quantize(rand(N + K, N, K, dtype="fp32", scale=0.02))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x8 = qlib.Int8Rows.empty(M, K)
    y = qlib.int8_matmul(x, w, x8_out=x8, status=status)
    check_rows(x8, x)
    assert int(status.item()) == 0
    acc = x8.codes.double() @ w.codes.double().t()      # exact: far below 2^53
    want = (acc.float() * x8.scales[:, None]) * w.scales[None]
    assert torch.equal(y, want.to(DT[dtype]))
    # rows that are in 8 bits already, into an `out` between guards
    buf = torch.full((M + 2, N), 5.0, dtype=DT[dtype], device="cuda")
    y2 = qlib.int8_matmul(x8, w, out=buf[1:M + 1])
    assert torch.equal(y2, y) and (buf[0] == 5).all() and (buf[M + 1] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K,N", [(1, 96, 40), (19, 500, 333), (600, 256, 1024)])
def test_matmul_bias(qlib, M, K, N, dtype):
    """One fma after the fp32 product: half a unit of fp32 before the type's own half unit."""
    x = rand(M, M, K, dtype=dtype)
    w = qlib.int8_quantize(rand(N, N, K, dtype="fp32"))
    bias = rand(7, N, dtype=dtype, scale=20.0)
    y = f64(qlib.int8_matmul(x, w, bias=bias))
    x8 = qlib.int8_quantize(x)
    want = ref.matmul32(x8.codes.cpu().numpy(), x8.scales.cpu().numpy(), w.codes.cpu().numpy(),
                        w.scales.cpu().numpy(), f64(bias)).astype(np.float64)
    assert (np.abs(y - want) <= (HALF[DT[dtype]] + 2.0 ** -23) * np.abs(want) + TINY[DT[dtype]]).all()


def test_matmul_largest_sums(qlib):
    """Every code 127: the sums reach 131072 * 127^2 = 2.11e9 without wrapping."""
    for K in (131072, 100000):
        x8 = qlib.Int8Rows(torch.full((3, K), 127, dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda"))
        w8 = qlib.Int8Rows(torch.full((130, K), -127, dtype=torch.int8, device="cuda"), torch.ones(130, device="cuda"))
        y = qlib.int8_matmul(x8, w8, dtype=torch.float32)
        assert (y == float(np.float32(-127 * 127 * K))).all()


def test_matmul_zero_rows_and_tokens(qlib):
    x = rand(1, 40, 200)
    x[7] = 0
    w0 = rand(2, 60, 200, dtype="fp32")
    w0[3] = 0
    w = qlib.int8_quantize(w0)
    y = qlib.int8_matmul(x, w, bias=rand(3, 60))
    assert torch.equal(y[7], rand(3, 60)) and torch.equal(y[:, 3], rand(3, 60)[3].expand(40))
    for dt in DT.values():
        assert qlib.int8_matmul(x[:0], w, dtype=dt).shape == (0, 60)
    assert qlib.int8_matmul_backward(y[:0], w).shape == (0, 200)
    assert qlib.int8_matmul(x, qlib.Int8Rows(w.codes[:0], w.scales[:0])).shape == (40, 0)


# ------------------------------------------------------------------------------ input gradient
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,N", [m for m in MATMUL if m[1] < 131072] + [(3, 40, 131072)])
def test_input_gradient(qlib, M, K, N, dtype):
    """dX is within (step / 2) sum_n |cw| of the exact product: 0.51 of a step a value counts the fp32
    roundings of dY sw and of its quotient (32639 * 2^-23 < 0.004 step each) too; then two fp32
    roundings (2^-23 of the value) and the type's own."""
    dt = DT[dtype]
    w = qlib.int8_quantize(rand(N + K, N, K, dtype="fp32", scale=0.05))
    dy = rand(M + N, M, N, dtype=dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    buf = torch.full((M + 2, K), 5.0, dtype=dt, device="cuda")
    dx = qlib.int8_matmul_backward(dy, w, out=buf[1:M + 1], status=status)
    assert int(status.item()) == 0 and (buf[0] == 5).all() and (buf[M + 1] == 5).all()
    cw, sw = w.codes.double(), w.scales.double()
    D = dy.double() * sw
    want = D @ cw
    step = D.abs().amax(1, keepdim=True) / 32639
    tol = 0.51 * step * cw.abs().sum(0)[None] + (HALF[dt] + 2.0 ** -23) * want.abs() + TINY[dt]
    assert ((dx.double() - want).abs() <= tol).all()


def test_input_gradient_is_the_products(qlib):
    """Against differences of the straight-through forward: <dX, v> = <dY, (v W^T)> for directions v."""
    M, K, N = 9, 160, 72
    w = qlib.int8_quantize(rand(1, N, K, dtype="fp32"))
    dy = rand(2, M, N, dtype="fp16")
    dx = f64(qlib.int8_matmul_backward(dy, w))
    Wt = ref.values(w.codes.cpu().numpy(), w.scales.cpu().numpy())
    g = np.random.default_rng(0)
    for _ in range(4):
        v = g.standard_normal((M, K))
        h = 0.5
        loss = lambda z: float((f64(dy) * (z @ Wt.T)).sum())   # noqa: E731
        diff = (loss(h * v) - loss(-h * v)) / (2 * h)
        # fp16 dX: half a unit (2^-11) of each term, and the fixed point's 1e-4 of a row
        assert abs(float((dx * v).sum()) - diff) <= (2.0 ** -11 + 1e-4) * np.abs(dx * v).sum()


def test_input_gradient_rows_of_any_size(qlib):
    """Rows of very different sizes, a zero row, subnormal and huge rows, a NaN: each on its own."""
    N, K = 90, 64
    w = qlib.Int8Rows(qlib.int8_quantize(rand(1, N, K, dtype="fp32")).codes, torch.ones(N, device="cuda"))
    dy = rand(5, 7, N, dtype="bf16")
    dy[1] = 0
    dy[2] *= 1e-30
    dy[3] *= 1e30
    dy[4] = 0
    dy[4, 5] = 1e-38
    dy[5, 3] = float("nan")
    dx = qlib.int8_matmul_backward(dy, w)
    want = dy.double() @ w.codes.double()
    assert torch.isnan(dx[5]).all()
    for m in (0, 1, 2, 3, 4, 6):
        step = float(dy[m].double().abs().max()) / 32639
        tol = 0.51 * step * w.codes.double().abs().sum(0) + (2.0 ** -8 + 2.0 ** -22) * want[m].abs() + 2.0 ** -133
        assert ((dx[m].double() - want[m]).abs() <= tol).all(), m


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("K,N", [(1000, 3000), (512, 4096)])
def test_tokens_do_not_depend_on_their_batch(qlib, K, N, dtype):
    """The same bits for a token alone, in a few, in some and in many (four kernels and every split)."""
    x = rand(1, 4000, K, dtype=dtype)
    w = qlib.int8_quantize(rand(2, N, K, dtype="fp32"))
    dy = rand(3, 4000, N, dtype=dtype)
    y, dx = qlib.int8_matmul(x, w), qlib.int8_matmul_backward(dy, w)
    for m in (1, 2, 4, 5, 16, 40, 130, 400, 1100):
        assert torch.equal(qlib.int8_matmul(x[:m], w), y[:m]), m
        assert torch.equal(qlib.int8_matmul_backward(dy[:m], w), dx[:m]), m


def test_nonfinite_and_zero_weight_rows(qlib):
    """A channel with a NaN gives NaN in its column and, through its scale, in every input gradient;
    a zero channel gives zeros."""
    w0 = rand(1, 70, 96, dtype="fp32")
    w0[5, 3] = float("nan")
    w0[6] = 0
    w = qlib.int8_quantize(w0)
    for M in (1, 30, 700):
        y = qlib.int8_matmul(rand(2, M, 96), w)
        assert torch.isnan(y[:, 5]).all() and not y[:, 6].any() and torch.isfinite(y[:, 7:]).all()
    assert torch.isnan(qlib.int8_matmul_backward(rand(3, 4, 70), w)).all()
    v = qlib.int8_dequantize(w)
    assert torch.isnan(v[5]).all() and not v[6].any()


def test_refusals_on_the_device(qlib):
    x, w8 = rand(1, 4, 64), qlib.int8_quantize(rand(2, 16, 64, dtype="fp32"))
    x8, dy = qlib.int8_quantize(x), rand(3, 4, 16)
    E = qlib.Int8Rows
    for call in (lambda: qlib.int8_quantize(x.double()), lambda: qlib.int8_quantize(x[0]),
                 lambda: qlib.int8_matmul(x.int(), w8), lambda: qlib.int8_matmul(x, w8, dtype=torch.float64),
                 lambda: qlib.int8_matmul(x, w8, bias=torch.zeros(16, device="cuda")),
                 lambda: qlib.int8_matmul(x, w8, out=torch.zeros(4, 16, device="cuda"), dtype=torch.bfloat16),
                 lambda: qlib.int8_matmul_backward(dy.float(), w8), lambda: qlib.int8_matmul(x, w8.codes),
                 lambda: qlib.int8_matmul(E(x8.codes.short(), x8.scales), w8),
                 lambda: qlib.int8_matmul(E(x8.codes, x8.scales.cpu()), w8),
                 lambda: qlib.Int8LinearFn.apply(x.float(), w8),
                 lambda: qlib.int8_dequantize(x8, torch.int8)):
        with pytest.raises((TypeError, AttributeError)):
            call()
    for call in (lambda: qlib.int8_quantize(x.t()), lambda: qlib.int8_quantize(x[:, :0]),
                 lambda: qlib.int8_quantize(x[:1].expand(4, 64)), lambda: qlib.int8_quantize(x, out=w8),
                 lambda: qlib.int8_matmul(x[:, :32], w8), lambda: qlib.int8_matmul(x, w8, out=dy[:2]),
                 lambda: qlib.int8_matmul(x, w8, bias=dy[0, :8]), lambda: qlib.int8_matmul(x8, w8, x8_out=x8),
                 lambda: qlib.int8_matmul(x, w8, x8_out=w8), lambda: qlib.int8_matmul_backward(dy[:, :8].contiguous(), w8),
                 lambda: qlib.int8_matmul(E(x8.codes[:, 1:33], x8.scales), w8),
                 lambda: qlib.int8_matmul(E(x8.codes, x8.scales[:3]), w8),
                 lambda: qlib.int8_matmul(E(x8.codes.t().contiguous().t(), x8.scales), w8)):
        with pytest.raises(ValueError):
            call()
    w, x, A, B, dy = layer_case(qlib, 20, 128, 64, 4, 1, "bf16")
    x8 = qlib.int8_quantize(x)
    bad8 = qlib.int8_quantize(x[:19])
    for call in (lambda: qlib.backward(bad8, dy, w, A, B, 8.0), lambda: qlib.backward(x8, dy, w, A[:64], B, 8.0),
                 lambda: qlib.backward(x8, dy, w, A, B[:, :32].contiguous(), 8.0),
                 lambda: qlib.backward(x8, dy, w, A, B, 8.0, T=torch.zeros(20, 3, device="cuda")),
                 lambda: qlib.backward(x8, dy, w, A, B, 8.0, pool_group=2)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        qlib.backward(x8, dy.half(), w, A, B, 8.0)
    with pytest.raises(qlib.QLoRAError):
        qlib.backward(x8, dy, w, A, B, float("inf"))


# ------------------------------------------------------------------------------ checkpoint
def layer_case(qlib, M, K, N, r, g, dtype, seed=0):
    w = qlib.quantize(rand(seed + 1, N, K, dtype="fp32", scale=0.02), compute_dtype=DT[dtype])
    x = rand(seed + 2, M, K, dtype=dtype)
    A = rand(seed + 3, K // g, r, dtype=dtype, scale=r ** -0.5)
    B = rand(seed + 4, r, N, dtype=dtype, scale=0.05)
    dy = rand(seed + 5, M, N, dtype=dtype)
    return w, x, A, B, dy


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,N,r,g", [(1, 64, 8, 1, 1), (5, 192, 200, 8, 1), (16, 256, 296, 16, 1), (17, 320, 72, 3, 1),
                                       (100, 1024, 264, 64, 1), (129, 128, 1000, 85, 1), (300, 704, 520, 256, 1),
                                       (1000, 2048, 200, 24, 1), (33, 512, 136, 8, 64), (260, 4096, 88, 40, 64),
                                       (2, 64, 8, 1, 64), (90, 192, 64, 256, 64), (700, 9024, 264, 17, 64)])
def test_checkpoint_backward(qlib, M, K, N, r, g, dtype):
    """dX is qlora_backward's to the bit; dA, dB and a recomputed T against the formulas of the 8-bit
    input.  Bounds: G's fp32 accumulation (N terms, 2^-23 each, of the sum of magnitudes), 0.51 of the
    24-bit step of G's column (over a token's scale), fp32 roundings; in dB, T's terms (three of bf16,
    two of fp16: 2^-22, or an fp16 subnormal's 2^-25) and the M fp32 terms of its sums."""
    alpha = 16.0
    w, x, A, B, dy = layer_case(qlib, M, K, N, r, g, dtype)
    x8 = qlib.int8_quantize(x)
    _, T = qlib.forward(x, w, A, B, alpha, g)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx0, _, _ = qlib.backward(x, dy, w, A, B, alpha, g, T=T)
    dx, da, db = qlib.backward(x8, dy, w, A, B, alpha, g, T=T, status=status)
    assert int(status.item()) == 0
    assert torch.equal(dx, dx0)
    pool = lambda z: z.reshape(M, K // g, g).mean(2)   # noqa: E731
    xs = x8.scales.double()[:, None]
    xh = x8.codes.double() * xs
    p, pabs, pcodes = pool(xh), pool(xh.abs()), pool(x8.codes.double().abs())
    s = alpha / r
    G, Gabs = dy.double() @ B.double().t(), dy.double().abs() @ B.double().abs().t()
    want = s * p.t() @ G
    eG = N * 2.0 ** -23 * Gabs + 2.0 ** -23 * G.abs()
    step = (xs * (G.abs() + eG)).amax(0, keepdim=True) / 8355711
    tol = s * (pabs.t() @ eG + 0.51 * step * pcodes.sum(0)[:, None]) + 2.0 ** -22 * want.abs() + 1e-30
    assert ((da.double() - want).abs() <= tol).all()

    def check_db(db, T, eT):
        wantB = s * T.t() @ dy.double()
        eT = eT + (2.0 ** -22 + M * 2.0 ** -23) * T.abs() + (2.0 ** -25 if dtype == "fp16" else 0)
        assert ((db.double() - wantB).abs() <= s * eT.t() @ dy.double().abs() + 2.0 ** -22 * wantB.abs() + 1e-30).all()

    check_db(db, T.double(), 0)
    # T from the checkpoint: exact sums of the codes with A's columns in 24 bits, and fp32 roundings
    _, _, db2 = qlib.backward(x8, dy, w, A, B, alpha, g, need_dx=False, need_dA=False)
    Th = p @ A.double()
    check_db(db2, Th, 0.51 * A.double().abs().amax(0) / 8355711 * pabs.sum(1, keepdim=True) + 2.0 ** -22 * Th.abs())


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -10, 2.0 ** -20])
def test_checkpoint_small_activations(qlib, scale):
    """T far below fp16's normal range (2^-14), where its second 16-bit term would be lost: dB to 2e-6
    in the 2-norm.  T's two terms leave 2^-23 of each value; sums in the tensor cores' accumulator lose
    7e-7 of their magnitudes at most, three times the 2-norm of a sum of M = 300 random signs' terms,
    rarely in one direction.  The second term is kept 2^11 up, so its own subnormals end at 2^-24 / 2^11:
    half of that a value of T at most, over the sum ||E^T dy|| <= ||E|| ||dy||, ||E|| <= sqrt(M r) 2^-36
    (4e-7 here, which counts at the smallest scale only; without the 2^11 the error there is 3e-5)."""
    M, K, N, r = 300, 256, 264, 8
    w, x, A, B, dy = layer_case(qlib, M, K, N, r, 1, "fp16")
    A = (A.float() * scale).half()
    x8 = qlib.int8_quantize(x)
    T = (x8.codes.double() * x8.scales.double()[:, None] @ A.double()).float()
    _, _, db = qlib.backward(x8, dy, w, A, B, 16.0, 1, T=T, need_dx=False, need_dA=False)
    want = 16.0 / r * T.double().t() @ dy.double()
    floor = 16.0 / r * (M * r) ** 0.5 * 2.0 ** -36 * dy.double().norm()
    assert (db.double() - want).norm() <= 2e-6 * want.norm() + floor


def test_checkpoint_gradient_against_differences(qlib):
    """The loss <dY, y(x^, A, B)> is linear in A and in B: central differences of the fp64 layer."""
    M, K, N, r, g = 20, 128, 64, 4, 1
    w, x, A, B, dy = layer_case(qlib, M, K, N, r, g, "fp16", seed=40)
    x8 = qlib.int8_quantize(x)
    _, da, db = qlib.backward(x8, dy, w, A, B, 8.0, g)
    Wt = f64(qlib.dequantize(w, dtype=torch.float16))
    xh = ref.values(x8.codes.cpu().numpy(), x8.scales.cpu().numpy())
    rng = np.random.default_rng(1)
    dA_, dB_ = rng.standard_normal(A.shape), rng.standard_normal(B.shape)
    loss = lambda a, b: float((f64(dy) * ref.layer(xh, Wt, a, b, 8.0, g)).sum())   # noqa: E731
    h = 0.25
    num = (loss(f64(A) + h * dA_, f64(B)) - loss(f64(A) - h * dA_, f64(B))) / (2 * h)
    assert abs(float((f64(da) * dA_).sum()) - num) <= 1e-4 * np.abs(f64(da) * dA_).sum()
    num = (loss(f64(A), f64(B) + h * dB_) - loss(f64(A), f64(B) - h * dB_)) / (2 * h)
    assert abs(float((f64(db) * dB_).sum()) - num) <= 1e-4 * np.abs(f64(db) * dB_).sum()


def test_checkpoint_parts_and_empty(qlib):
    w, x, A, B, dy = layer_case(qlib, 50, 128, 64, 4, 1, "bf16")
    x8 = qlib.int8_quantize(x)
    full = qlib.backward(x8, dy, w, A, B, 8.0)
    for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 0, 0)):
        got = qlib.backward(x8, dy, w, A, B, 8.0, need_dx=need[0], need_dA=need[1], need_dB=need[2])
        for n, a, b in zip(need, got, full):
            assert (a is None) == (not n) and (a is None or torch.equal(a, b))
    e = qlib.Int8Rows(x8.codes[:0], x8.scales[:0])
    dx, da, db = qlib.backward(e, dy[:0], w, A, B, 8.0)
    assert dx.shape == (0, 128) and not da.any() and not db.any()


# ------------------------------------------------------------------------------ together
def test_shared_checkpoint_autograd(qlib):
    """Three layers read one x and share one checkpoint; gradients against the fp64 formulas, with the
    layer parity bounds (5e-3 relative Frobenius) used for bf16 outputs elsewhere."""
    M, K, r, alpha = 70, 256, 8, 16.0
    x = rand(1, M, K).requires_grad_()
    x8 = qlib.int8_quantize(x.detach())
    xh = ref.values(x8.codes.cpu().numpy(), x8.scales.cpu().numpy())
    total, dxs = 0, 0
    leaves = []
    for i, N in enumerate((128, 64, 200)):
        w, _, A, B, dy = layer_case(qlib, M, K, N, r, 1, "bf16", seed=10 * i)
        A.requires_grad_(), B.requires_grad_()
        y = qlib.QLoRALinear8BitInputFn.apply(x, A, B, w, alpha, 1, x8)
        total = total + (y.float() * dy.float()).sum()
        leaves.append((w, A, B, dy))
    total.backward()
    rel = lambda a, b: np.linalg.norm(a - b) / np.linalg.norm(b)   # noqa: E731
    for w, A, B, dy in leaves:
        Wt = f64(qlib.dequantize(w))
        # T was saved by the forward, from x itself
        gx, ga, gb = ref.layer_backward(xh, f64(dy), Wt, f64(A), f64(B), alpha, 1, T=f64(x) @ f64(A))
        dxs = dxs + gx
        assert rel(f64(A.grad), ga) <= 5e-3 and rel(f64(B.grad), gb) <= 5e-3
    assert rel(f64(x.grad), dxs) <= 8e-3    # three bf16 sums more


def test_merge_then_eight_bits(qlib):
    """The deployment path: merge, quantize the merged weight, multiply; and a frozen 8-bit layer's
    gradient.  Codes are off by at most half a scale each, so y by what that bounds."""
    M, K, N = 40, 512, 192
    w, x, A, B, dy = layer_case(qlib, M, K, N, 8, 1, "bf16")
    W = qlib.merge(w, A, B, 16.0)
    w8 = qlib.int8_quantize(W)
    check_rows(w8, W)
    xg = x.clone().requires_grad_()
    y = qlib.Int8LinearFn.apply(xg, w8)
    y.backward(dy)
    exact = x.double() @ W.double().t()
    x8 = qlib.int8_quantize(x)
    ex, ew = 0.5 * x8.scales.double()[:, None], 0.5 * w8.scales.double()[None]
    tol = ex * W.double().abs().sum(1)[None] + x.double().abs().sum(1, keepdim=True) * ew + K * ex * ew
    assert ((y.double() - exact).abs() <= tol + 2.0 ** -8 * (exact.abs() + tol)).all()
    assert torch.equal(xg.grad, qlib.int8_matmul_backward(dy, w8))


def test_autograd_captured(qlib):
    """Forward and backward of both autograd functions in one graph, replayed on new inputs."""
    M, K, N = 30, 256, 128
    w, x, A, B, dy = layer_case(qlib, M, K, N, 8, 1, "bf16")
    w8 = qlib.int8_quantize(qlib.dequantize(w, dtype=torch.float32))

    def step(x, A, B, dy):
        x, A, B = (t.detach().requires_grad_() for t in (x, A, B))
        y = qlib.QLoRALinear8BitInputFn.apply(x, A, B, w, 16.0)
        z = qlib.Int8LinearFn.apply(x, w8)
        return torch.autograd.grad((y, z), (x, A, B), (dy, dy))

    xs, dys = x.clone(), dy.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(xs, A, B, dys)
    torch.cuda.current_stream().wait_stream(s)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = step(xs, A, B, dys)
    for seed in (50, 51):
        x2, dy2 = rand(seed, M, K), rand(seed + 9, M, N)
        xs.copy_(x2)
        dys.copy_(dy2)
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step(x2, A, B, dy2)))


def test_two_streams_at_once(qlib):
    """Calls in flight on two streams, each with its own buffers, from two host threads."""
    import threading
    w = qlib.int8_quantize(rand(1, 1500, 700, dtype="fp32"))
    xs = [rand(2 + i, 300 + 100 * i, 700) for i in range(2)]
    want = [(qlib.int8_matmul(x, w), qlib.int8_matmul_backward(rand(9, x.shape[0], 1500), w)) for x in xs]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            st = torch.cuda.Stream()
            dy = rand(9, xs[i].shape[0], 1500)
            torch.cuda.synchronize()
            with torch.cuda.stream(st):
                for _ in range(20):
                    got[i] = (qlib.int8_matmul(xs[i], w), qlib.int8_matmul_backward(dy, w))
            st.synchronize()
        except Exception as e:   # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    assert all(torch.equal(a, b) for g, v in zip(got, want) for a, b in zip(g, v))


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second GPU")
def test_other_device_than_the_current_one(qlib):
    x, w0 = rand(1, 20, 128).to("cuda:1"), rand(2, 64, 128, dtype="fp32").to("cuda:1")
    w = qlib.int8_quantize(w0)
    assert w.device.index == 1 and torch.equal(qlib.int8_matmul(x, w).cpu(),
                                               qlib.int8_matmul(x.to("cuda:0"), qlib.int8_quantize(w0.to("cuda:0"))).cpu())
    with pytest.raises(ValueError):
        qlib.int8_matmul(x.to("cuda:0"), w)


def test_streams_graphs_and_repeats(qlib):
    """On a stream of its own, captured (two graphs with one workspace, replayed in turn) and repeated:
    the same bits, from the inputs at replay."""
    M, K, N = 24, 640, 320
    w, x, A, B, dy = layer_case(qlib, M, K, N, 8, 1, "bf16")
    w8 = qlib.int8_quantize(qlib.dequantize(w, dtype=torch.float32))
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")

    def step(x, dy):
        x8 = qlib.int8_quantize(x)
        y = qlib.int8_matmul(x, w8)
        dx = qlib.int8_matmul_backward(dy, w8, workspace=ws)
        return (y, dx) + qlib.backward(x8, dy, w, A, B, 16.0, workspace=ws)

    x2, dy2 = rand(70, M, K), rand(71, M, N)
    want, want2 = step(x, dy), step(x2, dy2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(x, dy)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    xs, dys = x.clone(), dy.clone()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(xs, dys))
        graphs.append(gr)
    for i in range(4):
        xs.copy_(x if i < 2 else x2)
        dys.copy_(dy if i < 2 else dy2)
        graphs[i & 1].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[i & 1], want if i < 2 else want2))

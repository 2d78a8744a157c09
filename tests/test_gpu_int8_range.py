"""8-bit rows where their fixed point and their sums are pressed hardest.

Tolerances: half a step of each output type (bf16 2^-8 of the value at most, fp16 2^-11), plus what
each comment counts."""
import pytest
import torch

from test_gpu_int8 import DT, HALF, layer_case, rand

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ input gradient
def head(qlib, N, K, mean, seed=1):
    """A weight of N channels whose values have a mean, in units of their deviation."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(N, K, generator=g, device="cuda") + mean
    return qlib.int8_quantize(0.02 * w)


def loss_rows(M, N, dtype, spread, seed=2):
    """softmax(logits) - onehot, as the cross entropy leaves it in the logits' gradient."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    p = torch.softmax(spread * torch.randn(M, N, generator=g, device="cuda"), 1)
    p[torch.arange(M), torch.randint(N, (M,), generator=g, device="cuda")] -= 1
    return p.to(DT[dtype])


def row_errors(dx, dy, w):
    """2-norm of each row's error over the row's own 2-norm, against 64 bits."""
    want = (dy.double() * w.scales.double()) @ w.codes.double()
    return (dx.double() - want).norm(dim=1) / want.norm(dim=1)


# The fixed point may take as much as the output's own rounding: half a step of the type each
# (a quarter of that in noise, half of it in errors of one direction, for weights whose mean is at
# most their deviation).
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("mean", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("spread", [0.0, 1.0, 4.0])
@pytest.mark.parametrize("M,N,K", [(3, 32000, 256), (5, 4096, 512), (200, 32000, 128), (700, 5003, 136), (3, 128256, 64),
                                   (2, 1000, 64), (70, 131072, 24)])
def test_input_gradient_of_a_loss(qlib, M, N, K, spread, mean, dtype):
    if dtype == "fp16" and spread == 0 and N > 32000:
        pytest.skip("1 / N is an fp16 subnormal there: nothing more than the case of 32000")
    w = head(qlib, N, K, mean)
    dy = loss_rows(M, N, dtype, spread)
    assert row_errors(qlib.int8_matmul_backward(dy, w), dy, w).max() <= 2 * HALF[DT[dtype]]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K,large", [(4, 28672, 256, 3000.0), (300, 11008, 512, 1000.0), (40, 4096, 100, 300.0),
                                         (600, 28672, 64, 3000.0), (9, 4099, 72, 60000.0)])
def test_input_gradient_of_rows_with_one_large_value(qlib, M, N, K, large, dtype):
    """Every third row has a value far above the others, where its channel has few codes: what the
    large value leaves of the others decides the result in most columns."""
    w = head(qlib, N, K, 0.3)
    w.codes[7, :K // 2] = 0
    dy = rand(4, M, N, dtype="fp32")
    dy[::3, 7] = large
    dy = dy.to(DT[dtype])
    dx = qlib.int8_matmul_backward(dy, w)
    want = (dy.double() * w.scales.double()) @ w.codes.double()
    err = (dx.double() - want)[:, :K // 2].norm(dim=1) / want[:, :K // 2].norm(dim=1)
    # these columns hold none of the large value: the fixed point's share of the row's norm, which
    # that value makes up to `ratio` times theirs, counts against them
    D = dy.double() * w.scales.double()
    rest = D.clone()
    rest[:, 7] = 0
    ratio = D.norm(dim=1) / rest.norm(dim=1)
    half = HALF[DT[dtype]]
    assert (err <= half + half * ratio).all()
    assert row_errors(dx, dy, w).max() <= 2 * half


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_input_gradient_of_equal_values(qlib, dtype):
    """Values that all lie the same fraction of a step off: their errors have one sign."""
    N, K = 1000, 64
    w = qlib.Int8Rows(torch.randint(1, 100, (N, K), dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda"))
    dy = torch.full((3, N), -1e-3, device="cuda")
    dy[0, 5], dy[1, 900], dy[2, 0] = 1.0, 1.0, 1.0
    dy = dy.to(DT[dtype])
    assert row_errors(qlib.int8_matmul_backward(dy, w), dy, w).max() <= 2 * HALF[DT[dtype]]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("N,K", [(3000, 264), (4099, 130)])
def test_peaked_tokens_do_not_depend_on_their_batch(qlib, N, K, dtype):
    """Peaked, ordinary, sparse, zero and NaN rows next to one another: each row's bits are its own."""
    M = 2100
    w = head(qlib, N, K, 0.5)
    dy = rand(3, M, N, dtype=dtype)
    dy[::5] = loss_rows(M // 5, N, dtype, 1.0)
    dy[1::5] *= (torch.rand(M // 5, N, device="cuda", generator=torch.Generator(device="cuda").manual_seed(8)) < 0.1)
    dy[2] = 0
    dy[3, 17] = float("nan")
    dy[700:1400] = rand(6, 700, N, dtype=dtype)     # a long run of ordinary rows
    dx = qlib.int8_matmul_backward(dy, w)
    assert torch.isnan(dx[3]).all() and not dx[2].any()
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[2:4] = False
    assert row_errors(dx[keep], dy[keep], w).max() <= 2 * HALF[DT[dtype]]
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))   # noqa: E731
    for m in (1, 2, 5, 40, 65, 130, 400, 900, 1500):
        assert same(qlib.int8_matmul_backward(dy[:m], w), dx[:m]), m
    for lo, hi in ((700, 1400), (1399, 1402), (5, 6), (650, 1405)):
        assert same(qlib.int8_matmul_backward(dy[lo:hi].contiguous(), w), dx[lo:hi]), (lo, hi)


@pytest.mark.parametrize("M,N,K", [(30, 2000, 320), (300, 3000, 520), (1100, 3000, 264)])
def test_peaked_tokens_at_replay(qlib, M, N, K):
    """One captured call (one launch of four planes, two launches, passes of tiles) on a stream of its own
    takes its tokens' fixed point from the values at replay, with one workspace for two graphs."""
    w = head(qlib, N, K, 0.3)
    plain, peaked = rand(3, M, N), loss_rows(M, N, "bf16", 1.0)
    mixed = plain.clone()
    mixed[M // 2] = peaked[0]
    want = [qlib.int8_matmul_backward(d, w) for d in (plain, peaked, mixed)]
    need = 4 * M * ((N + 127) // 128 * 128) + 8 * M + 4096
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    dy = plain.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(qlib.int8_matmul_backward(dy, w, workspace=ws), want[0])
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(qlib.int8_matmul_backward(dy, w, workspace=ws))
        graphs.append(g)
    for i, d in enumerate((plain, peaked, mixed, plain, mixed, peaked)):
        dy.copy_(d)
        graphs[i & 1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i & 1], want[(0, 1, 2, 0, 2, 1)[i]]), i


def test_peaked_rows_at_every_offset_and_size(qlib):
    """Peaked rows that start off 16-byte borders, with tiny and huge levels, guards around the result."""
    for N, K, lo in ((1003, 40, 1), (2051, 33, 3), (17, 16, 5), (9001, 64, 7)):
        w = head(qlib, N, K, 0.5)
        M = 70
        dy = torch.zeros(M * N + 16, dtype=torch.bfloat16, device="cuda")[lo:lo + M * N].view(M, N)
        dy.copy_(loss_rows(M, N, "bf16", 2.0))
        dy[1] *= 2.0 ** -90
        dy[2] *= 2.0 ** 90
        dy[3] *= 2.0 ** -118
        buf = torch.full((M + 2, K), 5.0, dtype=torch.bfloat16, device="cuda")
        dx = qlib.int8_matmul_backward(dy, w, out=buf[1:M + 1])
        assert (buf[0] == 5).all() and (buf[M + 1] == 5).all()
        # row 3's products of dY and the scale lie at 2^-129: fp32's unit there is 2^-149, 2^-20 of them
        err = row_errors(dx, dy, w)
        assert err.max() <= 2 * 2.0 ** -8, N


# ------------------------------------------------------------------------------ the code -128
@pytest.mark.parametrize("M,N", [(1, 40), (2, 9), (3, 40), (130, 300), (700, 264)])
def test_largest_sums_of_the_lowest_code(qlib, M, N):
    """Rows made elsewhere may hold -128: 131072 terms of 2^14 are 2^31, one past a 32-bit integer."""
    K = 131072
    x8 = qlib.Int8Rows(torch.full((M, K), -128, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda"))
    w8 = qlib.Int8Rows(torch.full((N, K), -128, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda"))
    w8.codes[N // 2, 5] = 127
    y = qlib.int8_matmul(x8, w8, dtype=torch.float32)
    want = torch.full((M, N), 2.0 ** 31, device="cuda")
    want[:, N // 2] = 2.0 ** 31 - 128 * 255
    assert torch.equal(y, want)


def test_largest_digit_sums_of_the_lowest_code(qlib):
    """The same in the digits' products: M = 131072 tokens of codes -128 under equal gradients."""
    M, K, N, r = 131072, 64, 8, 4
    w, _, A, B, _ = layer_case(qlib, 1, K, N, r, 1, "bf16")
    x8 = qlib.Int8Rows(torch.full((M, K), -128, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda"))
    dy = rand(7, 1, N).expand(M, N).contiguous()
    _, da, _ = qlib.backward(x8, dy, w, A, B, 8.0, need_dx=False, need_dB=False)
    G = dy[:1].double() @ B.double().t()
    want = (8.0 / r * -128.0 * M * G).expand(K, r)
    # G's eight fp32 terms, half a 24-bit step, fp32 roundings
    assert ((da.double() - want).abs() <= 2.0 ** -20 * (dy[:1].double().abs() @ B.double().abs().t()) * 128 * M * 8 / r).all()


# ------------------------------------------------------------------------------ the checkpoint
def checkpoint_formulas(x8, dy, A, B, alpha, T=None):
    """(dA, dB) of an unpooled layer in 64 bits."""
    s = alpha / A.shape[1]
    xh = x8.codes.double() * x8.scales.double()[:, None]
    T = xh @ A.double() if T is None else T.double()
    G = dy.double() @ B.double().t()
    return s * xh.t() @ G, s * T.t() @ dy.double()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,N,r", [(4096, 256, 11008, 16), (4096, 256, 11008, 64), (4096, 192, 11000, 24),
                                     (4000, 128, 11008, 64), (3136, 64, 24576, 40), (4096, 64, 11008, 85),
                                     (2048, 64, 28672, 256), (9000, 128, 1024, 24), (20000, 64, 2048, 8),
                                     (12288, 64, 11008, 16)])
def test_checkpoint_long_reductions(qlib, M, K, N, r, dtype):
    """More k-tiles in a split of G and of dB than one accumulator takes (12), exact multiples of it and
    others; ranks past 64; tokens past what the columns' digits keep.  dA and dB in the 2-norm: an
    accumulator that rounds toward zero loses 1.3e-8 of the sum in each of 12 x 4 steps (6.3e-7), the sums
    over turns and splits, up to 40 fp32 roundings in one chain, 2^-24 each at random (sqrt(40) 2^-24 =
    3.8e-7), T's terms and the fixed point 2^-23 (1.2e-7): 1.2e-6.  An accumulator that is not taken out
    loses 1.4e-6 (22 k-tiles) to 2.3e-6 (35) in one direction; a stale or lost one, the whole result."""
    w, x, A, B, dy = layer_case(qlib, M, K, N, r, 1, dtype, seed=M + r)
    x8 = qlib.int8_quantize(x)
    T = (x8.codes.double() * x8.scales.double()[:, None] @ A.double()).float()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, da, db = qlib.backward(x8, dy, w, A, B, 16.0, 1, T=T, need_dx=False, status=status)
    assert int(status.item()) == 0
    wantA, wantB = checkpoint_formulas(x8, dy, A, B, 16.0, T)
    assert (da.double() - wantA).norm() <= 1.2e-6 * wantA.norm()
    assert (db.double() - wantB).norm() <= 1.2e-6 * wantB.norm()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,r", [(40, 9024, 16), (300, 16448, 40), (17, 28672, 8)])
def test_checkpoint_recomputes_T_of_long_rows(qlib, M, K, r, dtype):
    """Unpooled inputs past the 8192 rows of A that its columns' digits keep in shared memory.  In the
    2-norm: A's columns within half a 24-bit step (6e-8 of their maximum, under 3e-7 of a normal
    column's values), four fp32 roundings in a chain, dB's and G's short sums (5 k-tiles: 2.6e-7)."""
    N = 136
    w, x, A, B, dy = layer_case(qlib, M, K, N, r, 1, dtype, seed=K)
    x8 = qlib.int8_quantize(x)
    _, da, db = qlib.backward(x8, dy, w, A, B, 16.0, 1, need_dx=False)
    wantA, wantB = checkpoint_formulas(x8, dy, A, B, 16.0)
    assert (da.double() - wantA).norm() <= 1.2e-6 * wantA.norm()
    assert (db.double() - wantB).norm() <= 1.2e-6 * wantB.norm()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,r", [(4096, 11008, 16), (512, 4096, 85)])
def test_checkpoint_dx_of_long_reductions(qlib, M, N, r, dtype):
    """dX differs from qlora_backward's by G's summation alone: s G rounded the other way for a few of its
    values (one step, two halves of it) and the result's own rounding the other way."""
    w, x, A, B, dy = layer_case(qlib, M, 128, N, r, 1, dtype)
    x8 = qlib.int8_quantize(x)
    dx0, _, _ = qlib.backward(x, dy, w, A, B, 16.0, need_dA=False, need_dB=False)
    dx, _, _ = qlib.backward(x8, dy, w, A, B, 16.0, need_dA=False, need_dB=False)
    half = HALF[DT[dtype]]
    sG = 16.0 / r * (dy.double() @ B.double().t()).abs()
    assert ((dx.double() - dx0.double()).abs() <= 2 * half * (sG @ A.double().abs().t()) + 2 * half * dx0.double().abs()).all()
    assert torch.isfinite(dx).all()


@pytest.mark.parametrize("level", [0, -70, -105, -118])
@pytest.mark.parametrize("seed", range(3))
def test_column_digits_within_half_a_step(qlib, seed, level):
    """dA of one token is its column's fixed point times codes of 1: within 0.51 of the step max / 8355711
    and one fp32 rounding (2^-24 of the value, 2^-150), for G = dY exactly (B the identity); of columns
    below 2^-100 the step is a power of two, at most max / 2^21."""
    M, K, N, r = 8000, 8192, 8, 8
    w, _, A, _, _ = layer_case(qlib, 1, K, N, r, 1, "bf16")
    x8 = qlib.Int8Rows(torch.zeros(M, K, dtype=torch.int8, device="cuda"),
                       torch.rand(M, generator=torch.Generator().manual_seed(seed)).cuda() + 0.5)
    x8.scales.mul_(2.0 ** level)
    k = torch.arange(M, device="cuda")
    x8.codes[k, k] = 1                                 # feature k reads token k alone
    dy = rand(seed, M, N)
    B = torch.eye(N, device="cuda").bfloat16()
    _, da, _ = qlib.backward(x8, dy, w, A, B, float(r), need_dx=False, need_dB=False)
    want = dy.float() * x8.scales[:, None]             # the product in fp32, as it is cut
    step = want.double().abs().amax(0) / (8355711 if level > -100 else 2 ** 21)
    assert ((da[:M].double() - want.double()).abs() <= 0.51 * step + 2.0 ** -24 * want.double().abs() + 2.0 ** -150).all()


# ------------------------------------------------------------------------------ autograd
def test_bias_that_wants_a_gradient_is_refused(qlib):
    """The frozen bias gets no gradient: one that asks for it must not go without in silence."""
    w8 = qlib.int8_quantize(rand(2, 16, 64, dtype="fp32"))
    x, bias = rand(1, 4, 64).requires_grad_(), rand(3, 16).requires_grad_()
    with torch.no_grad():
        y = qlib.Int8LinearFn.apply(x, w8, bias)
    assert torch.equal(qlib.Int8LinearFn.apply(x, w8, bias.detach()), y)
    with pytest.raises(RuntimeError, match="bias"):
        qlib.Int8LinearFn.apply(x, w8, bias).sum().backward()
    z = qlib.Int8LinearFn.apply(x, w8, bias.detach())
    z.sum().backward()
    assert torch.equal(x.grad, qlib.int8_matmul_backward(torch.ones_like(z), w8))

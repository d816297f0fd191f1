"""GPU parity of the row quantiser and of the scaled int8 product with plain
64-bit numpy forms of their definitions.

Tolerance of the product, with e = 2^-24 and S = |P| + |beta C| + |bias|
(P the scaled product): the sum's rounding to fp32, the three multiplications,
beta * C and the two additions are seven roundings of at most e relative to
values of at most S (to first order; 1 % covers the rest), so
  |err| <= L * 7.1 e S + r * |ref| + tiny,
L the activation's slope (1, or 1.13 for GELU, whose own error is at most
2.2e-7 * max(1, |x|)) and r half a step of the output type (fp32 2^-24, fp16
2^-11, bf16 2^-8; r acts on the value before the rounding, 1.01 covers that);
tiny = 2^-25 is half of fp16's smallest step.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import dense_mixed_precision_tiled_amd as lg
from gpu_util import log

pytestmark = pytest.mark.gpu

R, C = lg.GEMM_ROW_MAJOR, lg.GEMM_COL_MAJOR
F32, F16, BF16 = lg.GEMM_F32, lg.GEMM_F16, lg.GEMM_BF16
TORCH = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
HALF_STEP = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
PAD8, PADD = -128, 12288.0  # exact in every output type


def stream():
    return torch.cuda.current_stream().cuda_stream


def stored(x, layout, ld, fill):
    """Matrix x in a buffer of the given layout and leading dimension, padding filled."""
    rows, cols = x.shape
    outer, inner = (rows, cols) if layout == R else (cols, rows)
    buf = np.full((outer, ld), fill, dtype=x.dtype)
    buf[:, :inner] = x if layout == R else x.T
    return buf


def gelu(x):
    return x * 0.5 * np.vectorize(math.erfc)(-x / math.sqrt(2.0))


class Scaled:
    """One seeded call of gemm_run_scaled and its 64-bit reference."""

    def __init__(self, M, N, K, la=R, lb=C, lc=R, ld=R, out=BF16, pad=16, alpha=1.0, beta=1.0,
                 bias=False, act=0, c=False, inplace=False, sa=True, sb=True, satf=0, seed=0,
                 offset=0):
        g = np.random.default_rng(seed + 1000 * M + 100 * N + K)
        self.__dict__.update(M=M, N=N, K=K, la=la, lb=lb, lc=lc, ld=ld, out=out, alpha=alpha,
                             beta=beta, act=act, inplace=inplace, satf=satf)
        self.A = g.integers(-128, 128, (M, K), dtype=np.int8)
        self.B = g.integers(-128, 128, (K, N), dtype=np.int8)
        self.sA = g.uniform(0.5, 2.0, M).astype(np.float32) / 127 if sa else None
        self.sB = g.uniform(0.5, 2.0, N).astype(np.float32) / (64 * max(1, K) ** 0.5) if sb else None
        self.bias = g.normal(size=N).astype(np.float32) if bias else None
        self.C = torch.from_numpy(g.normal(size=(M, N)).astype(np.float32)).to(TORCH[out]) \
            if (c or inplace) else None

        def ldim(inner):
            return (max(inner, 1) + 15) // 16 * 16 + pad if pad % 16 == 0 else max(inner, 1) + pad

        self.lda = ldim(K if la == R else M)
        self.ldb = ldim(N if lb == R else K)
        self.ldd = (N if ld == R else M) + (4 if pad % 16 == 0 else 3)
        self.ldc = self.ldd if inplace else (N if lc == R else M) + 5
        self.offset = offset

    def device(self):
        def dev8(x, layout, ldx):
            buf = torch.from_numpy(stored(x, layout, ldx, PAD8)).reshape(-1)
            store = torch.full((buf.numel() + self.offset,), PAD8, dtype=torch.int8)
            store[self.offset:] = buf
            return store.cuda()[self.offset:]

        def matrix(x, layout, ldx, dtype):
            rows, cols = self.M, self.N
            outer, inner = (rows, cols) if layout == R else (cols, rows)
            buf = torch.full((outer, ldx), PADD, dtype=dtype)
            if x is not None:
                buf[:, :inner] = x if layout == R else x.T
            return buf.cuda()

        f = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
        self.dA, self.dB = dev8(self.A, self.la, self.lda), dev8(self.B, self.lb, self.ldb)
        self.dsA, self.dsB, self.dbias = f(self.sA), f(self.sB), f(self.bias)
        self.dD = matrix(self.C if self.inplace else None, self.ld, self.ldd, TORCH[self.out])
        self.dC = self.dD if self.inplace else (
            None if self.C is None else matrix(self.C, self.lc, self.ldc, TORCH[self.out]))

    def call(self, s=None):
        ptr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
        epi = lg.GemmEpilogue(self.alpha, self.beta, ptr(self.dbias), self.act,
                              self.ld if self.inplace else self.lc, self.ld)
        st = lg.gemm_run_scaled(self.M, self.N, self.K, ptr(self.dA), self.lda, self.la,
                                ptr(self.dB), self.ldb, self.lb, ptr(self.dsA), ptr(self.dsB),
                                ptr(self.dC), self.ldc, ptr(self.dD), self.ldd, lg.GEMM_I8,
                                lg.GEMM_I32, self.out, self.satf, epi, stream() if s is None else s)
        assert st == 0, lg.gemm_status_string(st)

    def result(self):
        """(M x N values as float64, padding)."""
        d = self.dD.cpu()
        inner = self.N if self.ld == R else self.M
        v = d[:, :inner].double().numpy()
        return (v if self.ld == R else v.T), d[:, inner:].float().numpy()

    def reference(self):
        n = self.A.astype(np.float64) @ self.B.astype(np.float64)
        one = np.float64(1.0)
        P = n * (one if self.sA is None or self.K == 0 else self.sA.astype(np.float64)[:, None])
        P = P * (one if self.sB is None or self.K == 0 else self.sB.astype(np.float64)) * self.alpha
        size = np.abs(P)
        x = P
        if self.C is not None and self.beta != 0:
            bc = self.beta * self.C.double().numpy()
            x, size = x + bc, size + np.abs(bc)
        if self.bias is not None:
            x, size = x + self.bias.astype(np.float64), size + np.abs(self.bias)
        slope, own = 1.0, 0.0
        if self.act == lg.GEMM_ACT_RELU:
            y = np.maximum(x, 0)
        elif self.act == lg.GEMM_ACT_GELU:
            y, slope, own = gelu(x), 1.13, 2.2e-7 * np.maximum(1, np.abs(x))
        else:
            y = x
        tol = slope * 7.1 * 2.0 ** -24 * size + own + 1.01 * HALF_STEP[self.out] * np.abs(y) + 2.0 ** -25
        return y, tol

    def check(self, label=""):
        log("case: scaled %dx%dx%d %s" % (self.M, self.N, self.K, label))
        self.device()
        self.call()
        got, pad = self.result()
        ref, tol = self.reference()
        err = np.abs(got - ref)
        worst = np.unravel_index(np.argmax(err - tol), err.shape)
        assert (err <= tol).all(), "%s: at %s got %r ref %r tol %r" % (
            label, worst, got[worst], ref[worst], tol[worst])
        assert (pad == PADD).all(), "padding written"
        return got


LAYOUTS = [(R, C), (R, R), (C, C), (C, R)]
# one token to a large tile, odd and ragged sizes, sizes next to a tile's edge
SHAPES = [(1, 1, 1), (1, 100, 64), (3, 257, 130), (16, 130, 513), (17, 64, 640), (33, 500, 100),
          (64, 1031, 257), (65, 190, 300), (257, 129, 128), (1000, 1300, 200)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("la,lb", LAYOUTS)
@pytest.mark.parametrize("pad", [16, 3])
def test_layouts_and_sizes(M, N, K, la, lb, pad):
    """pad 16: the vector loads (padding lines hold -128); pad 3: element loads."""
    for out in (BF16, F32):
        Scaled(M, N, K, la, lb, out=out, pad=pad, bias=out == F32).check(
            "A%d B%d pad %d out %d" % (la, lb, pad, out))


# the eight-wave and four-wave 256x256 tiles: 192 tiles and more on 256 CUs
@pytest.mark.parametrize("la,lb", LAYOUTS)
@pytest.mark.parametrize("K", [256, 300])
def test_large_tiles(la, lb, K):
    Scaled(3500, 3600, K, la, lb, out=F16, bias=True, c=True, beta=0.5).check("large")


# sizes that the pipelined kernel's tiles of 32x32 to 128x128 each take on 256 CUs,
# with whole and ragged K-tiles, fewer K-tiles than stages, and odd edges
@pytest.mark.parametrize("M,N", [(40, 500), (127, 4090), (250, 4090), (499, 4096), (1000, 4001)])
@pytest.mark.parametrize("K", [16, 128, 200, 1152])
def test_pipelined_tiles(M, N, K):
    Scaled(M, N, K, out=BF16, bias=True).check("pipelined")
    Scaled(M, N, K, out=F32, c=True, beta=0.5, act=lg.GEMM_ACT_RELU).check("pipelined, C")


@pytest.mark.parametrize("M", [3, 40])
def test_operand_past_4_gib(M):
    """B of 4.6 GB: its columns past 2^32 bytes, and those next to where the call
    takes the next part, in the result's first and last rows."""
    N, K = 70000, 65536
    g = torch.Generator(device="cuda").manual_seed(9)
    A = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    B = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    sB = torch.rand(N, device="cuda", generator=g) + 0.5
    bias = torch.randn(N, device="cuda", generator=g)
    D = torch.zeros(M, N, device="cuda")
    st = lg.gemm_run_scaled(M, N, K, A.data_ptr(), K, R, B.data_ptr(), K, C, 0, sB.data_ptr(), 0, N,
                            D.data_ptr(), N, lg.GEMM_I8, lg.GEMM_I32, F32, 0,
                            lg.GemmEpilogue(bias=bias.data_ptr()), stream())
    assert st == 0
    cols = [0, 1, 65023, 65024, 65279, 65280, 65535, 65536, 69999]
    want = A.double() @ B[cols].double().T
    ref = (want * sB[cols].double() + bias[cols].double()).cpu()
    assert ((D[:, cols].double().cpu() - ref).abs() <= 4 * 2.0 ** -24 * (ref.abs() + 8)).all()


@pytest.mark.parametrize("swap", [False, True])
def test_longest_line(swap):
    """2^31 - 1 outputs of one row or one column, from one product each."""
    n = 2 ** 31 - 1
    g = torch.Generator(device="cuda").manual_seed(5)
    long = torch.randint(-128, 128, (n,), dtype=torch.int8, device="cuda", generator=g)
    one = torch.tensor([-7], dtype=torch.int8, device="cuda")
    D = torch.zeros(n + 1, dtype=torch.float16, device="cuda")
    M, N, A, B = (n, 1, long, one) if swap else (1, n, one, long)
    log("case: scaled %d x %d x 1" % (M, N))
    st = lg.gemm_run_scaled(M, N, 1, A.data_ptr(), 1, R, B.data_ptr(), 1, C, 0, 0, 0, N,
                            D.data_ptr(), N, lg.GEMM_I8, lg.GEMM_I32, F16, 0, None, stream())
    assert st == 0 and D[n] == 0
    for i in range(0, n, 2 ** 28):
        part = long[i:i + 2 ** 28]
        assert torch.equal(D[i:i + part.numel()], part.to(torch.float16) * -7), i


@pytest.mark.parametrize("la,lb", LAYOUTS)
def test_medium_tiles(la, lb):
    Scaled(1500, 1600, 384, la, lb, out=BF16, bias=True).check("medium")


@pytest.mark.parametrize("M", [1, 5, 16, 40, 64, 200])
@pytest.mark.parametrize("out", [F32, F16, BF16])
@pytest.mark.parametrize("act", [lg.GEMM_ACT_NONE, lg.GEMM_ACT_RELU, lg.GEMM_ACT_GELU])
def test_epilogue(M, out, act):
    for kw in (dict(alpha=1.5, bias=True), dict(alpha=-0.75, beta=2.0, c=True, bias=True),
               dict(c=True, inplace=True), dict(c=True, beta=0.0), dict(sa=False, alpha=2.0 ** -13),
               dict(sb=False, alpha=2.0 ** -9)):
        Scaled(M, 203, 264, out=out, act=act, **kw).check("out %d act %d %s" % (out, act, kw))


@pytest.mark.parametrize("M", [1, 30, 64, 130])
@pytest.mark.parametrize("la,lb", LAYOUTS)
def test_column_major_c_and_d(M, la, lb):
    """A column-major D runs as its transpose: scales and bias change sides with it."""
    for lc, ld in ((C, R), (R, C), (C, C)):
        Scaled(M, 75, 160, la, lb, lc, ld, out=BF16, c=True, bias=True).check("C%d D%d" % (lc, ld))
    # few columns: the transposed product has few rows
    Scaled(300, M, 160, la, lb, R, C, out=F32, bias=True).check("transposed, %d columns" % M)


@pytest.mark.parametrize("M", [1, 9, 64, 100])
def test_unit_scales_are_exact(M):
    """Without scales and with sums below 2^24 the fp32 output is the integer sum."""
    p = Scaled(M, 70, 1000, out=F32, sa=False, sb=False)
    got = p.check("unit scales")
    assert np.array_equal(got, p.A.astype(np.int64) @ p.B.astype(np.int64))


@pytest.mark.parametrize("M", [2, 64, 70])
def test_long_k_reaches_the_int32_range(M):
    """K = 2^17 - 1 of -128 * -128: the largest sum, just under 2^31."""
    p = Scaled(M, 20, 2 ** 17 - 1, out=F32, sa=False, sb=False)
    p.A[:], p.B[:] = -128, -128
    got = p.check("longest")
    assert (got == float(np.float32((2 ** 17 - 1) * 2 ** 14))).all()


def test_empty_operations():
    Scaled(5, 7, 0, out=F32, bias=True, c=True).check("K = 0")
    for M, N in ((0, 5), (5, 0)):
        st = lg.gemm_run_scaled(M, N, 3, 0, 3, R, 0, 3, C, 0, 0, 0, 5, 0, 5, lg.GEMM_I8,
                                lg.GEMM_I32, F32, 0, None, stream())
        assert st == 0


@pytest.mark.parametrize("M", [4, 100])
def test_scales_that_are_nan_inf_zero_or_tiny(M):
    """A NaN row scale (a row that could not be quantised) gives a NaN row, zero
    scales zeros, and two tiny scales whose product underflows still meet a
    large sum first; satf turns NaN into 0 and Inf into the largest value."""
    p = Scaled(M, 40, 512, out=F32, seed=5)
    p.B[:] = np.abs(p.B.astype(np.int16)).clip(0, 127)
    p.A[:] = np.abs(p.A.astype(np.int16)).clip(1, 127)
    p.B[0] = 1
    p.sA[0], p.sA[1], p.sA[2] = np.nan, 0.0, 1e-30
    p.sB[0], p.sB[1] = np.inf, 1e-12
    for satf in (0, 1):
        p.satf = satf
        p.device()
        p.call()
        got, _ = p.result()
        n = p.A.astype(np.float64) @ p.B.astype(np.float64)
        with np.errstate(invalid="ignore"):
            ref = n * p.sA.astype(np.float64)[:, None] * p.sB.astype(np.float64)
        if satf:
            assert (got[0] == 0).all() and got[1, 0] == 0 and (got[3:, 0] > 3.4e38).all()
        else:
            assert np.isnan(got[0]).all() and np.isnan(got[1, 0]) and np.isinf(got[3:, 0]).all()
        assert (got[1, 1:] == 0).all()
        fine = np.isfinite(ref)
        fine[0] = False
        # 1e-30 * 1e-12 * sum is below fp32's normal range only by its last bits
        assert np.allclose(got[fine], ref[fine], rtol=2.0 ** -20, atol=2.0 ** -148)


def test_rows_and_columns_of_padding_never_reach_the_result():
    """Operands that start 16 bytes into their buffer, padding of -128 around them."""
    for M in (3, 64, 90):
        Scaled(M, 100, 72, offset=16, out=F32).check("offset 16")
        Scaled(M, 100, 72, offset=5, out=F32).check("offset 5")


# ------------------------------------------------------------------ quantiser
def quant_reference(x):
    """int8 values and fp32 scales of float64 rows; a row that is not finite
    (a value past fp16's range became Inf) has zeros and the scale NaN."""
    bad = ~np.isfinite(x).all(axis=1)
    x = np.where(bad[:, None], 0.0, x)
    a = np.abs(x).max(axis=1, initial=0.0)
    q = np.rint(127 * x / np.where(a > 0, a, 1.0)[:, None])
    s = a.astype(np.float32) / np.float32(127)
    return q.astype(np.int8), np.where(bad, np.float32(np.nan), s)


def quantize(x, pad_x=8, pad_q=16, offset=0):
    """x: a torch matrix on the CPU; (Q, scales, Q's padding) of the GPU."""
    M, K = x.shape
    ldx, ldq = max(1, K) + pad_x, max(1, K) + pad_q
    X = torch.full((M * ldx + offset,), float("nan"), dtype=x.dtype)
    X[offset:].view(M, ldx)[:, :K] = x
    X = X.cuda()[offset:]
    Q = torch.full((M, ldq), 77, dtype=torch.int8, device="cuda")
    s = torch.full((M + 1,), -1.0, device="cuda")
    code = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}[x.dtype]
    st = lg.gemm_quantize_rows(M, K, X.data_ptr(), ldx, code, Q.data_ptr(), ldq, s.data_ptr(),
                               stream())
    assert st == 0, lg.gemm_status_string(st)
    Q, s = Q.cpu().numpy(), s.cpu().numpy()
    assert s[M] == -1.0 and (Q[:, K:] == 77).all(), "written past the rows"
    return Q[:, :K], s[:M]


DTYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 16), (2, 7), (5, 100), (3, 2048), (4, 2049),
                                 (7, 4096), (2, 8200), (3, 16384), (1, 40001), (300, 33),
                                 (1000, 512)])
@pytest.mark.parametrize("aligned", [True, False])
def test_quantize_is_exact(dtype, M, K, aligned):
    """Bit for bit the rounded exact quotient, whatever the type and alignment."""
    log("case: quantize %dx%d %s aligned %s" % (M, K, dtype, aligned))
    g = torch.Generator().manual_seed(M + 7 * K)
    x = (torch.randn(M, K, generator=g) * torch.exp(3 * torch.randn(M, 1, generator=g))).to(dtype)
    up = lambda n: (n + 15) // 16 * 16 - n  # noqa: E731
    Q, s = quantize(x, up(K) if aligned else 1, up(K) + 16 if aligned else 3, 0 if aligned else 1)
    q, t = quant_reference(x.double().numpy())
    assert np.array_equal(Q, q) and np.array_equal(s, t, equal_nan=True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_ties_go_to_even(dtype):
    """Rows whose largest value is 127 units hold every half of a step."""
    for unit in (1.0, 2.0 ** -6, 2.0 ** 7):
        x = torch.cat([torch.arange(-126.5, 127, 1.0), torch.tensor([127.0])]) * unit
        x = x.to(dtype)
        if not torch.equal(x.double(), (torch.cat([torch.arange(-126.5, 127, 1.0),
                                                   torch.tensor([127.0])]) * unit).double()):
            # bf16 holds halves up to 63.5 only
            x = torch.cat([torch.arange(-63.5, 64, 1.0), torch.tensor([127.0])]).mul(unit).to(dtype)
        Q, s = quantize(x.reshape(1, -1))
        q, t = quant_reference(x.double().numpy().reshape(1, -1))
        assert np.array_equal(Q, q) and np.array_equal(s, t) and (q[0, :-1] % 2 == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_special_rows(dtype):
    """Zeros, one value, the smallest and the largest magnitudes, Inf and NaN."""
    fi = torch.finfo(dtype)
    tiny = fi.smallest_normal * fi.eps
    x = torch.zeros(9, 50, dtype=torch.float64)
    x[1, 3] = -2.0
    x[2] = torch.linspace(-60, 60, 50, dtype=torch.float64).round() * tiny
    x[3, 7], x[3, 8] = fi.max, -fi.max
    x[4] = torch.linspace(-1, 1, 50, dtype=torch.float64) * fi.smallest_normal
    x[5, 49], x[6, 0], x[7, 20] = float("inf"), float("nan"), -float("inf")
    x[8, 0] = tiny
    x = x.to(dtype)
    Q, s = quantize(x)
    q, t = quant_reference(torch.nan_to_num(x.double(), 0.0, 0.0, 0.0).numpy())
    for i in range(9):
        if i in (5, 6, 7):
            assert np.isnan(s[i]) and (Q[i] == 0).all(), i
        else:
            assert np.array_equal(Q[i], q[i]) and s[i] == t[i], i


def test_quantize_more_rows_than_a_grid_holds():
    """2^24 + 3 rows of one value, element by element: 2^32 threads and more."""
    M = 2 ** 24 + 3
    g = torch.Generator(device="cuda").manual_seed(4)
    X = torch.randn(M, generator=g, device="cuda").half()
    X[::1000] = 0
    Q = torch.full((M + 1,), 77, dtype=torch.int8, device="cuda")
    s = torch.full((M + 1,), -1.0, device="cuda")
    st = lg.gemm_quantize_rows(M, 1, X.data_ptr(), 1, F16, Q.data_ptr(), 1, s.data_ptr(), stream())
    assert st == 0
    assert Q[M] == 77 and s[M] == -1.0
    assert torch.equal(Q[:M], (X.sign() * 127).to(torch.int8))
    assert torch.equal(s[:M].double(), (X.double().abs() / 127).float().double())


def test_quantize_without_columns():
    s = torch.full((3,), 5.0, device="cuda")
    assert lg.gemm_quantize_rows(3, 0, 0, 1, F16, 0, 1, s.data_ptr(), stream()) == 0
    assert (s.cpu() == 0).all()


# --------------------------------------------------------- the layer as a whole
def linear_buffers(M, N, K, out, seed):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(M, K, generator=g).to(TORCH[out])
    W = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8)
    sB = torch.rand(N, generator=g) / (64 * K ** 0.5)
    bias = torch.randn(N, generator=g)
    return [t.cuda() for t in (X, W, sB, bias)] + [
        torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"),
        torch.empty(M, N, dtype=TORCH[out], device="cuda")]


def linear(b, out, s):
    X, W, sB, bias, Q, sA, D = b
    (M, K), N = X.shape, W.shape[0]
    st = lg.gemm_quantize_rows(M, K, X.data_ptr(), K, out, Q.data_ptr(), K, sA.data_ptr(), s)
    assert st == 0
    epi = lg.GemmEpilogue(bias=bias.data_ptr(), activation=lg.GEMM_ACT_GELU)
    st = lg.gemm_run_scaled(M, N, K, Q.data_ptr(), K, R, W.data_ptr(), K, C, sA.data_ptr(),
                            sB.data_ptr(), 0, N, D.data_ptr(), N, lg.GEMM_I8, lg.GEMM_I32, out, 0,
                            epi, s)
    assert st == 0
    return D


@pytest.mark.parametrize("M", [1, 33, 200])
@pytest.mark.parametrize("out", [F16, BF16])
def test_linear_layer(M, out):
    """Quantiser and product in a row: the reference quantises the same rows in
    64 bits (the int8 values agree exactly), the fp32 scale is rounded once more
    (2^-24) than the product's own seven roundings."""
    N, K = 333, 1024
    b = linear_buffers(M, N, K, out, 11 + M)
    got = linear(b, out, stream()).double().cpu().numpy()
    X, W, sB, bias = [t.double().cpu().numpy() for t in b[:4]]
    q, _ = quant_reference(X)
    P = q.astype(np.float64) @ W.T * (np.abs(X).max(1) / 127)[:, None] * sB
    ref = gelu(P + bias)
    tol = 1.13 * 8.1 * 2.0 ** -24 * (np.abs(P) + np.abs(bias)) + \
        2.2e-7 * np.maximum(1, np.abs(P + bias)) + 1.01 * HALF_STEP[out] * np.abs(ref) + 2.0 ** -25
    assert (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("M", [1, 48, 300])
def test_linear_layer_in_a_graph(M):
    """Captured once, replayed on new activations, with eager work on another
    stream between the replays: every replay equals the eager result."""
    b, other = linear_buffers(M, 640, 512, BF16, 3), linear_buffers(M, 640, 512, BF16, 4)
    linear(b, BF16, stream())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        linear(b, BF16, stream())
    side = torch.cuda.Stream()
    for seed in range(3):
        new = linear_buffers(M, 640, 512, BF16, 20 + seed)
        want = linear(new, BF16, stream()).clone()
        b[0].copy_(new[0])
        for dst, src in zip(b[1:4], new[1:4]):
            dst.copy_(src)
        b[6].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            linear(other, BF16, side.cuda_stream)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b[6], want)


# --------------------------------------- the large tiles without C or activation
@pytest.mark.parametrize("out", [F32, F16, BF16])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("K", [256, 300])
@pytest.mark.parametrize("M,N", [(3501, 3601), (4203, 4111)])
def test_large_tiles_without_c(M, N, K, bias, out):
    """The four-wave tile (K = 256) and the eight-wave one (300), at 14 x 15 tiles and
    with 17 x 17, more tiles than CUs, in the staggered order; odd edges."""
    Scaled(M, N, K, out=out, bias=bias).check("large, out %d bias %d" % (out, bias))


@pytest.mark.parametrize("la,lb", [(R, R), (C, C), (C, R)])
@pytest.mark.parametrize("out", [F32, BF16])
def test_large_tiles_without_c_in_other_layouts(la, lb, out):
    Scaled(3501, 3601, 200, la, lb, out=out, bias=True).check("large, A%d B%d" % (la, lb))
    Scaled(3501, 3601, 72, la, lb, out=out, pad=3).check("large, A%d B%d elements" % (la, lb))


@pytest.mark.parametrize("out", [F32, F16, BF16])
@pytest.mark.parametrize("M,N,K,lb", [(8, 203, 264, C), (40, 500, 200, C), (100, 200, 96, R),
                                      (3500, 3600, 256, C), (3500, 3600, 300, C)])
def test_satf_in_every_type(M, N, K, lb, out):
    """Rows that overflow the output type and one of NaN: with satf the largest finite
    value and 0, without it Inf and NaN; the rows between them as ever."""
    p = Scaled(M, N, K, lb=lb, out=out, bias=True)
    p.sA[2::3] = 1e30 if out == F16 else 3e38
    p.sA[1] = np.nan
    top = torch.finfo(TORCH[out]).max
    rest = np.ones(M, bool)
    rest[1], rest[2::3] = False, False
    for satf in (0, 1):
        p.satf = satf
        p.device()
        p.call()
        got, pad = p.result()
        log("case: scaled %dx%dx%d satf %d out %d" % (M, N, K, satf, out))
        with np.errstate(invalid="ignore", over="ignore"):
            ref, tol = p.reference()
        assert (np.abs(got[rest] - ref[rest]) <= tol[rest]).all()
        big, sign = got[2::3], np.sign(ref[2::3])
        over = np.abs(ref[2::3]) > 2 * top
        assert over.any()
        want = sign * (top if satf else np.inf)
        assert (big[over] == want[over]).all()
        assert (got[1] == 0).all() if satf else np.isnan(got[1]).all()
        assert (pad == PADD).all()


@pytest.mark.parametrize("swap", [False, True])
def test_strided_operand_past_4_gib(swap):
    """A row-major B (or column-major A) of 4.6 GB, read element by element."""
    N, K, M = 70000, 65536, 3
    g = torch.Generator(device="cuda").manual_seed(10)
    few = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    many = torch.randint(-127, 128, (K, N), dtype=torch.int8, device="cuda", generator=g)
    scale = torch.rand(N, device="cuda", generator=g) + 0.5
    D = torch.zeros(N, M, device="cuda") if swap else torch.zeros(M, N, device="cuda")
    log("case: strided operand past 4 GiB, swap %d" % swap)
    if swap:  # A(i, k) = many[k][i], B(k, j) = few[j][k]
        st = lg.gemm_run_scaled(N, M, K, many.data_ptr(), N, C, few.data_ptr(), K, C,
                                scale.data_ptr(), 0, 0, M, D.data_ptr(), M, lg.GEMM_I8, lg.GEMM_I32,
                                F32, 0, None, stream())
    else:
        st = lg.gemm_run_scaled(M, N, K, few.data_ptr(), K, R, many.data_ptr(), N, R, 0,
                                scale.data_ptr(), 0, N, D.data_ptr(), N, lg.GEMM_I8, lg.GEMM_I32,
                                F32, 0, None, stream())
    assert st == 0
    cols = [0, 1, 30000, 65535, 65536, 69999]
    ref = (few.double() @ many[:, cols].double()) * scale[cols].double()
    got = (D.t() if swap else D)[:, cols].double()
    # the sum's rounding and one multiplication
    assert ((got - ref).abs() <= 2.02 * 2.0 ** -24 * ref.abs()).all()

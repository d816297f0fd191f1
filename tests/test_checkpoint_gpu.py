"""GPU parity of the checkpoint calls with their definitions in 64 bits.

pack and unpack are compared exactly.  With e = 2^-24 and r half a step of the output's
type (fp16 2^-11, bf16 2^-8, fp32 2^-24):

act_grad: the slope is within s = 1e-6 absolutely (its exponential's and polynomial's
errors, see the header), times |g|, rounded once: r |y| + (1 + r) s |g| + |g| e; plus
half of the type's smallest subnormal.

wgrad: the products are exact; their fp32 sum of M terms (in up to 64 parts) is off by
at most (M + 70) e sum|g x|; C is added in fp32 (e of the result) and the result rounded
once: r |d|.  Integer-valued inputs whose sums stay below 2^24 are exact.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import checkpoint_util as ck
import dense_mixed_precision_tiled_amd as lg

pytestmark = pytest.mark.gpu

F32, F16, BF16 = lg.GEMM_F32, lg.GEMM_F16, lg.GEMM_BF16
TORCH = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
HALF_STEP = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F32: 2.0 ** -150, F16: 2.0 ** -25, BF16: 2.0 ** -134}
SENTINEL = 77


def stream():
    return torch.cuda.current_stream().cuda_stream


def ok(st):
    assert st == 0, lg.gemm_status_string(st)


class Lines:
    """A matrix on the device with lines of `ld` elements, `shift` elements into its
    buffer; everything outside the matrix holds a sentinel."""

    def __init__(self, rows, cols, dtype, ld=None, shift=0, fill=None):
        self.rows, self.cols, self.ld, self.shift = rows, cols, ld or max(cols, 1), shift
        self.buf = torch.full((shift + (rows + 1) * self.ld + 16,), SENTINEL, dtype=dtype,
                              device="cuda")
        self.view = self.buf[shift:shift + rows * self.ld].view(rows, self.ld)[:, :cols]
        if fill is not None:
            self.view.copy_(fill)

    @property
    def ptr(self):
        return self.buf.data_ptr() + self.shift * self.buf.element_size()

    def get(self):
        host = self.buf.cpu().clone()
        out = host[self.shift:self.shift + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols].clone()
        host[self.shift:self.shift + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = SENTINEL
        assert (host == SENTINEL).all(), "written outside the matrix"
        return out


def activations(M, K, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + M * 1000 + K)
    x = torch.randn(M, K, generator=g) * torch.exp(2 * torch.randn(M, 1, generator=g))
    x[torch.rand(M, K, generator=g) < 0.02] *= 50
    x[torch.rand(M, K, generator=g) < 0.1] = 0.0
    return x.to(TORCH[dtype])


def layout(K, dtype, how):
    """(ldx, ldq, lds, shift of X, shift of Q)"""
    per = 4 if dtype == F32 else 8
    up = lambda n, m: (n + m - 1) // m * m  # noqa: E731
    if how == "vec":
        return up(K, per), up(K, 16), (K + 31) // 32, 0, 0
    if how == "vec_wide":
        return up(K, per) + 2 * per, up(K, 16) + 32, (K + 31) // 32 + 3, per, 16
    return K + 3, K + 5, (K + 31) // 32 + 1, 1, 3  # odd


SHAPES = [(1, 1), (1, 8), (3, 31), (5, 32), (7, 33), (4, 63), (2, 100), (300, 40), (1025, 96),
          (17, 1000), (3, 4104), (33, 4096)]


def run_pack(X, dtype, how):
    M, K = X.shape
    ldx, ldq, lds, sx, sq = layout(K, dtype, how)
    dX = Lines(M, K, TORCH[dtype], ldx, sx, X)
    dQ, dS = Lines(M, K, torch.int8, ldq, sq), Lines(M, (K + 31) // 32, torch.uint8, lds, sq)
    ok(lg.gemm_checkpoint_pack(M, K, dX.ptr, ldx, dtype, dQ.ptr, ldq, dS.ptr, lds, stream()))
    dX.get()
    return dQ, dS


@pytest.mark.parametrize("how", ["vec", "vec_wide", "odd"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("M,K", SHAPES)
def test_pack_and_unpack(M, K, dtype, how):
    X = activations(M, K, dtype)
    dQ, dS = run_pack(X, dtype, how)
    Q, S = ck.pack(X.double().numpy())
    assert np.array_equal(dS.get().numpy(), S)
    assert np.array_equal(dQ.get().numpy(), Q)
    V = ck.values(Q, S)
    for out in (F32, F16, BF16):
        ldd, _, _, sd, _ = layout(K, out, how)
        dD = Lines(M, K, TORCH[out], ldd, sd)
        ok(lg.gemm_checkpoint_unpack(M, K, dQ.ptr, dQ.ld, dS.ptr, dS.ld, dD.ptr, ldd, out, stream()))
        want = torch.from_numpy(V).to(TORCH[out])  # exact; fp16 rounds once
        assert torch.equal(dD.get(), want)


@pytest.mark.parametrize("how", ["vec", "odd"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_special_values(dtype, how):
    t = torch.finfo(TORCH[dtype])
    small = t.smallest_normal * t.eps
    rows = [[0.0, -0.0] * 16, [t.max, -t.max, 1.0] * 10, [small] * 32, [small, 3 * small, -7 * small] * 10,
            [t.smallest_normal, small] * 16, [float("inf")] + [1.0] * 31, [float("nan")] + [1.0] * 31,
            [-float("inf"), float("nan")] * 16, [1.0, 1.984375, 1.9921875, 2.0 - t.eps] * 8,
            # ties: odd multiples of half a step
            [1.0, 0.5 / 64, 1.5 / 64, 2.5 / 64, -0.5 / 64, -1.5 / 64, 63.5 / 64, 62.5 / 64] * 4,
            [1.0] * 31 + [float("nan")], [1e-30] * 16 + [1e30 if dtype != F16 else 6e4] * 16]
    K = 96  # each row's values in its first, second or third block, the others ordinary
    X = torch.ones(len(rows) * 3, K)
    for i, r in enumerate(rows):
        for b in range(3):
            X[3 * i + b, 32 * b:32 * b + len(r)] = torch.tensor(r)
    X = X.to(TORCH[dtype])
    dQ, dS = run_pack(X, dtype, how)
    Q, S = ck.pack(X.double().numpy())
    assert np.array_equal(dS.get().numpy(), S) and np.array_equal(dQ.get().numpy(), Q)
    dD = Lines(X.shape[0], K, TORCH[dtype])
    ok(lg.gemm_checkpoint_unpack(X.shape[0], K, dQ.ptr, dQ.ld, dS.ptr, dS.ld, dD.ptr, K, dtype, stream()))
    got, want = dD.get().double().numpy(), ck.values(Q, S)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(want).any()
    fin = ~np.isnan(want)
    assert np.array_equal(got[fin], want[fin])


def test_pack_many_rows():
    """More items than one launch holds would need 2^31; rows and lanes past 2^16 here."""
    M, K = 70001, 33
    X = activations(M, K, BF16, seed=5)
    dQ, dS = run_pack(X, BF16, "odd")
    Q, S = ck.pack(X.double().numpy())
    assert np.array_equal(dS.get().numpy(), S) and np.array_equal(dQ.get().numpy(), Q)


def test_pack_more_than_one_launch():
    """2^31 items of 8 values and more: the rows on both sides of the launches' border."""
    M, K = (1 << 29) + 5, 1  # four items for each row
    X = torch.ones(M, dtype=torch.bfloat16, device="cuda")
    edge = 0x7fffffff // 4
    X[edge - 2:edge + 2] = torch.tensor([3.0, -0.25, 0.0, 96.0], dtype=torch.bfloat16)
    X[-1] = -1.75
    Q = torch.zeros(M, dtype=torch.int8, device="cuda")
    S = torch.zeros(M, dtype=torch.uint8, device="cuda")
    ok(lg.gemm_checkpoint_pack(M, K, X.data_ptr(), 1, BF16, Q.data_ptr(), 1, S.data_ptr(), 1, stream()))
    assert Q[edge - 2:edge + 2].tolist() == [96, -64, 0, 96] and Q[-1].item() == -112
    assert S[edge - 2:edge + 2].tolist() == [128, 125, 0, 133] and S[-1].item() == 127
    assert int((Q == 64).sum()) == M - 5 and int((S == 127).sum()) == M - 4


def slope64(x, a):
    if a == lg.GEMM_ACT_RELU:
        return np.where(np.isnan(x), x, (x > 0) * 1.0)
    if a == lg.GEMM_ACT_GELU:
        return 0.5 * np.vectorize(math.erfc)(-x / math.sqrt(2.0)) + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-x))
    return s + x * s * (1 - s)


def function64(x, a):
    if a == lg.GEMM_ACT_RELU:
        return np.maximum(x, 0)
    if a == lg.GEMM_ACT_GELU:
        return x * 0.5 * np.vectorize(math.erfc)(-x / math.sqrt(2.0))
    return x / (1 + np.exp(-x))


ACTS = [lg.GEMM_ACT_RELU, lg.GEMM_ACT_GELU, lg.GEMM_ACT_SILU]


@pytest.mark.parametrize("a", ACTS)
def test_slopes_are_differences(a):
    x = np.concatenate([np.linspace(-9, 9, 721), [-0.3, 1e-3]])
    x = x[np.abs(x) > 1e-4] if a == lg.GEMM_ACT_RELU else x
    h = 1e-5
    num = (function64(x + h, a) - function64(x - h, a)) / (2 * h)
    assert np.abs(num - slope64(x, a)).max() <= 1e-9


@pytest.mark.parametrize("a", ACTS)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("M,K,how", [(1, 1, "vec"), (5, 33, "odd"), (64, 128, "vec"), (9, 1000, "vec_wide"),
                                     (40, 200, "odd"), (300, 72, "vec")])
def test_act_grad(M, K, how, dtype, a):
    rng = np.random.default_rng(M + K)
    X = rng.normal(size=(M, K)) * np.exp(rng.normal(size=(M, 1)))
    X[0, 0] = -0.0
    Q, S = ck.pack(X)
    V = ck.values(Q, S)
    G = activations(M, K, dtype, seed=1)
    ldx, ldq, lds, sx, sq = layout(K, dtype, how)
    dQ, dS = Lines(M, K, torch.int8, ldq, sq, torch.from_numpy(Q)), \
        Lines(M, S.shape[1], torch.uint8, lds, sq, torch.from_numpy(S))
    dG, dD = Lines(M, K, TORCH[dtype], ldx, sx, G), Lines(M, K, TORCH[dtype], ldx, sx)
    ok(lg.gemm_checkpoint_act_grad(M, K, dQ.ptr, ldq, dS.ptr, lds, dG.ptr, ldx, a, dD.ptr, ldx,
                                   dtype, stream()))
    got, g = dD.get().double().numpy(), G.double().numpy()
    want = g * slope64(V, a)
    r = HALF_STEP[dtype]
    tol = r * np.abs(want) + (1 + r) * (1e-6 + 2.0 ** -24) * np.abs(g) + TINY[dtype]
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) - tol)
    # in place, the same bits
    first = dD.get()
    ok(lg.gemm_checkpoint_act_grad(M, K, dQ.ptr, ldq, dS.ptr, lds, dG.ptr, ldx, a, dG.ptr, ldx,
                                   dtype, stream()))
    assert torch.equal(dG.get(), first)


@pytest.mark.parametrize("a", ACTS)
def test_act_grad_extremes(a):
    """The largest and smallest values of the format, and blocks that stand for NaN."""
    M = 256
    Q = np.tile(np.array([0, 1, -1, 127, -127, 64, -64, 5], np.int8), (M, 4))
    S = np.arange(M, dtype=np.uint8).reshape(M, 1)
    V = ck.values(Q, S)
    dQ, dS = Lines(M, 32, torch.int8, fill=torch.from_numpy(Q)), Lines(M, 1, torch.uint8, fill=torch.from_numpy(S))
    dG, dD = Lines(M, 32, torch.float32, fill=torch.ones(M, 32)), Lines(M, 32, torch.float32)
    ok(lg.gemm_checkpoint_act_grad(M, 32, dQ.ptr, 32, dS.ptr, 1, dG.ptr, 32, a, dD.ptr, 32, F32, stream()))
    got = dD.get().double().numpy()
    assert np.isnan(got[255]).all()
    with np.errstate(over="ignore", invalid="ignore"):
        v = np.clip(V[:255], -300, 300)  # the slope is 0 or 1 past that
        want = slope64(v, a)
    assert (np.abs(got[:255] - want) <= 1e-6 + 2.0 ** -23).all()


# ------------------------------------------------------------------ wgrad

class Wgrad:
    def __init__(self, M, N, K, i=BF16, o=F32, add=False, how="vec", ints=False, seed=0):
        self.__dict__.update(M=M, N=N, K=K, i=i, o=o)
        rng = np.random.default_rng(seed + M + 7 * N + 13 * K)
        if ints:
            X = rng.integers(-3, 4, size=(M, K)).astype(np.float64)
            G = rng.integers(-3, 4, size=(M, N)).astype(np.float64)
        else:
            X = rng.normal(size=(M, K)) * np.exp(rng.normal(size=(M, 1)))
            X[rng.random(size=(M, K)) < 0.02] *= 20
            G = rng.normal(size=(M, N)) / max(M, 1) ** 0.5
        self.Q, self.S = ck.pack(X) if M else (np.zeros((0, K), np.int8), np.zeros((0, (K + 31) // 32), np.uint8))
        self.V = ck.values(self.Q, self.S) if M else np.zeros((0, K))
        if ints:
            assert np.array_equal(self.V, X)
        self.G = torch.from_numpy(G).to(TORCH[i])
        self.C = None
        if add:
            self.C = torch.from_numpy(rng.integers(-9, 10, size=(N, K)) * 1.0 if ints else rng.normal(size=(N, K))).to(TORCH[o])
        _, ldq, lds, _, sq = layout(K, i, how)
        ldg, _, _, sg, _ = layout(N, i, how)
        ldd, _, _, sd, _ = layout(K, o, how)
        self.dQ = Lines(M, K, torch.int8, ldq, sq, torch.from_numpy(self.Q))
        self.dS = Lines(M, self.S.shape[1], torch.uint8, lds, sq, torch.from_numpy(self.S))
        self.dG = Lines(M, N, TORCH[i], ldg, sg, self.G)
        self.dC = None if self.C is None else Lines(N, K, TORCH[o], ldd, sd, self.C)
        self.dD = Lines(N, K, TORCH[o], ldd, sd)
        self.size = lg.gemm_checkpoint_wgrad_workspace(M, N, K)
        assert self.size >= 0
        self.ws = torch.full((self.size + 64,), 255, dtype=torch.uint8, device="cuda")

    def call(self, D=None, s=None):
        D = self.dD if D is None else D
        ok(lg.gemm_checkpoint_wgrad(self.M, self.N, self.K, self.dG.ptr, self.dG.ld, self.dQ.ptr, self.dQ.ld,
                                    self.dS.ptr, self.dS.ld, 0 if self.dC is None else self.dC.ptr, D.ld, D.ptr,
                                    D.ld, self.i, self.o, self.ws.data_ptr() if self.size else 0, self.size,
                                    stream() if s is None else s))
        return self

    def reference(self):
        g = self.G.double().numpy()
        d = g.T @ self.V
        mag = np.abs(g).T @ np.abs(self.V)
        if self.C is not None:
            d = d + self.C.double().numpy()
        r = HALF_STEP[self.o]
        return d, (self.M + 70) * 2.0 ** -24 * mag + (1.01 * r + 2.0 ** -24) * np.abs(d) + TINY[self.o]

    def check(self, D=None):
        got = (self.dD if D is None else D).get().double().numpy()
        want, tol = self.reference()
        assert (self.ws[self.size:] == 255).all(), "written past the workspace"
        assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)
        # by the norm: independent roundings of M terms, and the output's
        norm = np.linalg.norm(want)
        assert np.linalg.norm(got - want) <= (1.5 * HALF_STEP[self.o] + 2.0 ** -24 * (8 + self.M ** 0.5)) * norm + 1e-30


WG = [(1, 1, 1), (5, 3, 7), (64, 32, 128), (65, 33, 129), (130, 16, 40), (200, 128, 256), (257, 130, 70),
      (700, 200, 100), (2000, 8, 96), (1000, 20, 1000), (129, 300, 520), (4097, 9, 33)]


@pytest.mark.parametrize("how", ["vec", "vec_wide", "odd"])
@pytest.mark.parametrize("i,o", [(BF16, F32), (F16, F16), (BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("M,N,K", WG)
def test_wgrad(M, N, K, i, o, how):
    w = Wgrad(M, N, K, i, o, add=(M + N) % 2 == 1, how=how)
    w.call().check()


@pytest.mark.parametrize("i", [BF16, F16])
@pytest.mark.parametrize("M,N,K", [(64, 32, 64), (333, 70, 200), (1500, 16, 500), (1024, 300, 300)])
def test_wgrad_integers_are_exact(M, N, K, i):
    w = Wgrad(M, N, K, i, F32, add=True, ints=True).call()
    assert np.array_equal(w.dD.get().double().numpy(), w.reference()[0])


@pytest.mark.parametrize("M,N,K", [(300, 200, 64), (3000, 16, 256)])
def test_wgrad_in_place_adds_up(M, N, K):
    w = Wgrad(M, N, K, BF16, F32, add=True, ints=True)
    w.call(w.dC)
    w.call(w.dC)
    want = w.reference()[0] + w.G.double().numpy().T @ w.V
    assert np.array_equal(w.dC.get().double().numpy(), want)


@pytest.mark.parametrize("o", [F32, F16, BF16])
def test_wgrad_no_tokens(o):
    w = Wgrad(0, 5, 40, BF16, o, add=True).call()
    assert torch.equal(w.dD.get(), w.C)
    w = Wgrad(0, 5, 40, BF16, o).call()
    assert not w.dD.get().any()


def test_wgrad_nan_stays_in_its_column_and_row():
    w = Wgrad(200, 40, 96, BF16, F32)
    w.S[100, 1] = 255                      # a block that stands for NaN: columns 32 to 63
    w.dS.view.copy_(torch.from_numpy(w.S))
    w.G[7, 3] = float("inf")
    w.dG.view.copy_(w.G)
    got = w.call().dD.get().numpy()
    bad = np.zeros((40, 96), bool)
    bad[:, 32:64] = True
    bad[3] = True
    assert np.array_equal(~np.isfinite(got), bad)


def test_wgrad_same_bits_and_streams():
    w, v = Wgrad(3000, 16, 300), Wgrad(2500, 20, 200, seed=1)
    a, b = w.call().dD.get(), v.call().dD.get()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        w.call(s=s1.cuda_stream)
        v.call(s=s2.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(w.dD.get(), a) and torch.equal(v.dD.get(), b)


def test_wgrad_captured():
    w = Wgrad(3000, 16, 300, add=True)
    eager = w.call().dD.get()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.call()
    for i in range(3):
        w.dD.view.zero_()
        graph.replay()
        assert torch.equal(w.dD.get(), eager)
    w.dG.view.mul_(2)  # a replay follows its operands
    w.dC.view.mul_(2)
    graph.replay()
    assert torch.equal(w.dD.get(), 2 * eager)


def test_wgrad_long_offsets():
    """Q and G past 4 GiB, in bytes and in elements."""
    M, N, K, ldq, ldg = 80, 8, 64, 1 << 26, 1 << 25
    rng = np.random.default_rng(0)
    X = rng.integers(-3, 4, size=(M, K)).astype(np.float64)
    G = rng.integers(-3, 4, size=(M, N)).astype(np.float64)
    Q, S = ck.pack(X)
    dQ = torch.zeros((M - 1) * ldq + K, dtype=torch.int8, device="cuda")
    dG = torch.zeros((M - 1) * ldg + N, dtype=torch.bfloat16, device="cuda")
    for m in range(M):
        dQ[m * ldq:m * ldq + K] = torch.from_numpy(Q[m])
        dG[m * ldg:m * ldg + N] = torch.from_numpy(G[m]).bfloat16()
    dS = torch.from_numpy(S).cuda()
    D = torch.empty(N, K, device="cuda")
    ws = torch.empty(lg.gemm_checkpoint_wgrad_workspace(M, N, K) + 1, dtype=torch.uint8, device="cuda")
    ok(lg.gemm_checkpoint_wgrad(M, N, K, dG.data_ptr(), ldg, dQ.data_ptr(), ldq, dS.data_ptr(), S.shape[1], 0, K,
                                D.data_ptr(), K, BF16, F32, ws.data_ptr(), ws.numel(), stream()))
    assert np.array_equal(D.cpu().double().numpy(), G.T @ X)


# Tiles of 256 x 256, whole and in parts, their edges ragged; tiles of 128 in many parts, the
# last of them with less than 64 tokens; thin ones of several stretches.
WG_LARGE = [(520, 4100, 4090), (8200, 1530, 1540), (3203, 515, 520), (6410, 70, 300), (9000, 33, 130)]


@pytest.mark.parametrize("i,o,add", [(BF16, F32, True), (F16, F16, True), (BF16, BF16, False)])
@pytest.mark.parametrize("M,N,K", WG_LARGE)
def test_wgrad_large(M, N, K, i, o, add):
    w = Wgrad(M, N, K, i, o, add=add).call()
    w.check()
    if add:  # and in place, to the same bits
        first = w.dD.get()
        w.call(w.dC)
        assert torch.equal(w.dC.get(), first)


@pytest.mark.parametrize("M", [200, 1351])
@pytest.mark.parametrize("how", ["vec", "odd"])
def test_wgrad_nan_and_inf_in_tiles(M, how):
    """Also in the rows that the last step of a tile takes once more."""
    w = Wgrad(M, 200, 192, BF16, F32, how=how)
    w.S[M - 20, 1] = w.S[M - 60, 4] = 255  # columns 32 to 63 and 128 to 159
    w.dS.view.copy_(torch.from_numpy(w.S))
    w.G[M - 64, 3], w.G[M - 1, 150], w.G[5, 60] = float("inf"), float("nan"), float("-inf")
    w.dG.view.copy_(w.G)
    got = w.call().dD.get().numpy()
    bad = np.zeros((200, 192), bool)
    bad[:, 32:64] = bad[:, 128:160] = True
    bad[[3, 150, 60]] = True
    assert np.array_equal(~np.isfinite(got), bad)


@pytest.mark.parametrize("N", [16, 100])
@pytest.mark.parametrize("wide", [0, 16])
def test_wgrad_long_lines(N, wide):
    """Rows of G, Q and S past 4 GiB, at the longest lines of 32-bit offsets and past them."""
    M, K, ldg, ldq, lds = 140, 96, 1 << 24, (1 << 25) + wide, 1 << 25
    w = Wgrad(M, N, K, BF16, F32, ints=True)

    def spread(m, ld, dtype):
        buf = torch.empty((M - 1) * ld + m.shape[1], dtype=dtype, device="cuda")
        torch.as_strided(buf, tuple(m.shape), (ld, 1)).copy_(m if torch.is_tensor(m) else torch.from_numpy(m))
        return buf

    G, Q = spread(w.G, ldg, torch.bfloat16), spread(w.Q, ldq, torch.int8)
    S = spread(w.S, lds, torch.uint8)
    ok(lg.gemm_checkpoint_wgrad(M, N, K, G.data_ptr(), ldg, Q.data_ptr(), ldq, S.data_ptr(), lds, 0, w.dD.ld,
                                w.dD.ptr, w.dD.ld, BF16, F32, w.ws.data_ptr() if w.size else 0, w.size, stream()))
    assert np.array_equal(w.dD.get().double().numpy(), w.reference()[0])


def test_wgrad_tiles_captured():
    w = Wgrad(1500, 200, 300, add=True)
    assert w.size > 0
    eager = w.call().dD.get()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.call()
    for _ in range(3):
        w.dD.view.zero_()
        graph.replay()
        assert torch.equal(w.dD.get(), eager)
        w.call()


@pytest.mark.parametrize("a", [lg.GEMM_ACT_GELU, lg.GEMM_ACT_SILU])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_act_grad_tails(dtype, a):
    """The slope keeps its relative precision where it goes to 0, at every value of the
    format from -2^8 to 2^8, on G = 1 (fp16: 1024, whose subnormal values are rounded to 2^-25).

    With p = Phi(x), f = |x| phi(x) (SiLU: s, |x| s (1 - s)), for x < 0: (2^-20 + x^2 2^-24) (p + f)
    (SiLU: 2^-20 + |x| 2^-23).  An exponential's argument h is rounded, and its constant, to
    1.5 2^-24 h; the exponential and the reciprocal add 2^-23 each, the polynomial 4e-7, five
    more operations 2^-24 each.  What is below 2^-126 of an exponential may be 0: 2^-122 of GELU
    (|x| < 14 there), 2^-118 of SiLU (|x| < 88).  For x >= 0 1e-6, absolutely."""
    k = np.arange(-20, 9)  # S - 127
    Q = np.tile(np.arange(-127, 129).clip(max=127).astype(np.int8), (len(k), 1))
    S = np.tile((k + 127).astype(np.uint8)[:, None], (1, 8))
    V = ck.values(Q, S)
    g = 1024.0 if dtype == F16 else 1.0
    M, K = Q.shape
    dQ, dS = Lines(M, K, torch.int8, fill=torch.from_numpy(Q)), Lines(M, 8, torch.uint8, fill=torch.from_numpy(S))
    dG, dD = Lines(M, K, TORCH[dtype], fill=torch.full((M, K), g)), Lines(M, K, TORCH[dtype])
    ok(lg.gemm_checkpoint_act_grad(M, K, dQ.ptr, K, dS.ptr, 8, dG.ptr, K, a, dD.ptr, K, dtype, stream()))
    got = dD.get().double().numpy()
    n = np.abs(V)
    if a == lg.GEMM_ACT_GELU:
        p = 0.5 * np.vectorize(math.erfc)(n / math.sqrt(2.0))
        f = n * np.exp(-n * n / 2) / math.sqrt(2 * math.pi)
        rel, low = 2.0 ** -20 + V * V * 2.0 ** -24, 2.0 ** -122
    else:
        p = np.exp(-n) / (1 + np.exp(-n))
        f = n * p * (1 - p)
        rel, low = 2.0 ** -20 + n * 2.0 ** -23, 2.0 ** -118
    want = g * np.where(V < 0, p - f, 1 - p + f)  # both forms of the slope, without cancellation
    r = HALF_STEP[dtype]
    slope = g * (np.where(V < 0, rel * (p + f), 1e-6) + low)
    tol = r * np.abs(want) + (1 + r) * slope + TINY[dtype]
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)
    if dtype != F16:  # down to x = -12 the negative side is nothing but this slope
        far = (V <= -6) & (V >= -12)
        assert far.sum() > 100
        assert (np.abs(got - want)[far] <= (r + 1.1e-5) * np.abs(want[far])).all()


@pytest.mark.parametrize("how", ["vec", "odd"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_relu_grad_selects(dtype, how):
    """ReLU's gradient takes G or 0: an Inf or a NaN of G where X^ <= 0 is left out."""
    inf, nan = float("inf"), float("nan")
    Q = np.tile(np.array([1, -1, 0, 64, -64, 127, -127, 5], np.int8), (4, 5))
    S = np.full((4, 2), 127, np.uint8)
    S[2, 0], S[3] = 255, 0
    V = ck.values(Q, S)
    G = torch.tensor([inf, -inf, nan, 2.0, inf, nan, nan, -inf, 0.0, -3.0]).repeat(4, 4).to(TORCH[dtype])
    ldx, ldq, lds, sx, sq = layout(40, dtype, how)
    dQ, dS = Lines(4, 40, torch.int8, ldq, sq, torch.from_numpy(Q)), Lines(4, 2, torch.uint8, lds, sq, torch.from_numpy(S))
    dG, dD = Lines(4, 40, TORCH[dtype], ldx, sx, G), Lines(4, 40, TORCH[dtype], ldx, sx)
    ok(lg.gemm_checkpoint_act_grad(4, 40, dQ.ptr, ldq, dS.ptr, lds, dG.ptr, ldx, lg.GEMM_ACT_RELU, dD.ptr, ldx,
                                   dtype, stream()))
    want = np.where(np.isnan(V), np.nan, np.where(V > 0, G.double().numpy(), 0.0))
    assert np.array_equal(dD.get().double().numpy(), want, equal_nan=True)


def overflowing(M, N, K, tokens, how):
    """fp16 call of integers in which the first block of each of `tokens` lies past 65504, in
    values of both signs; (call, D by the definition)."""
    w = Wgrad(M, N, K, F16, F32, how=how, ints=True)
    for i, m in enumerate(tokens):
        w.S[m, 0] = 127 + 17
        w.Q[m, :32] = np.tile([64, -64, 100, -127], 8)[:min(K, 32)]
        w.G[m] = torch.tensor([3.0, -2.0, 0.0, 1.0]).repeat(N // 4 + 1)[i:i + N].half()
    w.dS.view.copy_(torch.from_numpy(w.S))
    w.dQ.view.copy_(torch.from_numpy(w.Q))
    w.dG.view.copy_(w.G)
    V = ck.values(w.Q, w.S)
    V = np.where(np.abs(V) > 65519, np.copysign(np.inf, V), V)
    G = w.G.double().numpy()
    hit = list(tokens)
    rest = np.setdiff1d(np.arange(M), hit)
    want = G[rest].T @ V[rest]
    with np.errstate(invalid="ignore"):
        for m in hit:
            want = want + G[m][:, None] * V[m][None, :]
    return w, want


@pytest.mark.parametrize("how", ["vec", "odd"])
@pytest.mark.parametrize("M,N,K,back", [
    (200, 100, 192, [20]), (200, 200, 192, [1]), (200, 200, 192, [64, 190]), (1351, 200, 200, [50]),
    (8200, 1530, 1540, [20]),  # parts of 256 x 256
    (200, 100, 192, [20, 30])])
def test_wgrad_overflowing_values_in_tiles(M, N, K, back, how):
    """Values past fp16's range are Inf, with their sign, wherever their token lies: also in the
    rows that the last step of a tile takes once more (the last 64 of a ragged M)."""
    w, want = overflowing(M, N, K, [M - b for b in back], how)
    assert np.isinf(want[:, :32]).any() and np.isfinite(want[:, 32:]).all()
    assert np.array_equal(w.call().dD.get().double().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("how", ["vec", "odd"])
@pytest.mark.parametrize("M,N,K,back", [
    (201, 16, 192, [1]), (201, 60, 192, [1]), (1037, 20, 300, [1]), (1037, 60, 300, [1, 13]), (201, 32, 192, [9, 40]),
    (9000, 33, 130, [1])])
def test_wgrad_overflowing_values_of_few_outputs(M, N, K, back, how):
    """The same for few outputs, whose last step of 16 tokens repeats the last one."""
    w, want = overflowing(M, N, K, [M - b for b in back], how)
    assert np.isinf(want[:, :32]).any() and np.isfinite(want[:, 32:]).all()
    assert np.array_equal(w.call().dD.get().double().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("how", ["vec", "odd"])
@pytest.mark.parametrize("M,N,K", [(200, 16, 64), (200, 100, 192)])
def test_wgrad_smallest_values(M, N, K, how):
    """X^ far below bf16's smallest normal value: the products with a large G are exact."""
    w = Wgrad(M, N, K, BF16, F32, how=how, ints=True)
    w.S[:] = np.random.default_rng(0).integers(0, 3, size=w.S.shape)
    w.dS.view.copy_(torch.from_numpy(w.S))
    w.G = (w.G.float() * 2.0 ** 100).bfloat16()
    w.dG.view.copy_(w.G)
    want = w.G.double().numpy().T @ ck.values(w.Q, w.S)
    assert np.array_equal(w.call().dD.get().double().numpy(), want)


@pytest.mark.parametrize("M,N,K", [(3000, 16, 256), (1500, 200, 300)])
@pytest.mark.parametrize("shift", [1, 100, 255])
def test_wgrad_workspace_at_any_address(M, N, K, shift):
    w = Wgrad(M, N, K)
    assert w.size > 0
    clean = w.call().dD.get()
    ws = torch.full((w.size + 256,), 255, dtype=torch.uint8, device="cuda")
    ok(lg.gemm_checkpoint_wgrad(M, N, K, w.dG.ptr, w.dG.ld, w.dQ.ptr, w.dQ.ld, w.dS.ptr, w.dS.ld, 0, K, w.dD.ptr,
                                w.dD.ld, w.i, w.o, ws.data_ptr() + shift, w.size, stream()))
    assert torch.equal(w.dD.get(), clean)
    assert (ws[:shift] == 255).all() and (ws[shift + w.size:] == 255).all()


@pytest.mark.parametrize("N,K", [((1 << 27) + 130, 5), (3, (1 << 27) + 170)])
def test_wgrad_more_than_one_launch(N, K):
    """More rows or columns of D than one launch takes: integers, checked on the device."""
    M = 3
    g = torch.Generator(device="cuda").manual_seed(0)
    G = torch.randint(-3, 4, (M, N), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    X = torch.randint(-3, 4, (M, K), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    Q, S = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, (K + 31) // 32, dtype=torch.uint8, device="cuda")
    ok(lg.gemm_checkpoint_pack(M, K, X.data_ptr(), K, BF16, Q.data_ptr(), K, S.data_ptr(), S.shape[1], stream()))
    D = torch.full((N * K + 64,), 77.0, device="cuda")
    size = lg.gemm_checkpoint_wgrad_workspace(M, N, K)
    ws = torch.empty(size + 1, dtype=torch.uint8, device="cuda")
    ok(lg.gemm_checkpoint_wgrad(M, N, K, G.data_ptr(), N, Q.data_ptr(), K, S.data_ptr(), S.shape[1], 0, K, D.data_ptr(), K,
                                BF16, F32, ws.data_ptr(), size, stream()))
    assert (D[N * K:] == 77).all()
    got = D[:N * K].view(N, K)
    for n0 in range(0, N, 1 << 24):
        for k0 in range(0, K, 1 << 24):
            a, b = G[:, n0:n0 + (1 << 24)].float(), X[:, k0:k0 + (1 << 24)].float()
            want = sum(a[m][:, None] * b[m][None, :] for m in range(M))
            assert torch.equal(got[n0:n0 + (1 << 24), k0:k0 + (1 << 24)], want)


def test_longest_row():
    """A row of 2^31 - 1 values, packed and back."""
    K = 2 ** 31 - 1
    X = (torch.arange(K, dtype=torch.int32, device="cuda") % 61 - 30).bfloat16()
    Q, S = torch.empty(K, dtype=torch.int8, device="cuda"), torch.empty((K + 31) // 32, dtype=torch.uint8, device="cuda")
    D = torch.full((K + 9,), 77.0, dtype=torch.bfloat16, device="cuda")
    ok(lg.gemm_checkpoint_pack(1, K, X.data_ptr(), K, BF16, Q.data_ptr(), K, S.data_ptr(), S.numel(), stream()))
    ok(lg.gemm_checkpoint_unpack(1, K, Q.data_ptr(), K, S.data_ptr(), S.numel(), D.data_ptr(), K, BF16, stream()))
    assert torch.equal(D[:K], X) and (D[K:] == 77).all()  # whole numbers below 64 are exact


@pytest.mark.parametrize("i,o,add", [(BF16, F32, True), (F16, F16, True), (BF16, BF16, False), (F16, F32, False)])
def test_wgrad_whole_large_tiles(i, o, add):
    """Tiles of 256 x 256 that take all of the tokens, a ragged number of them, and ragged edges."""
    w = Wgrad(292, 2973, 2973, i, o, add=add)
    assert w.size == 0
    w.call().check()


def test_wgrad_overflowing_values_in_whole_large_tiles():
    w, want = overflowing(292, 2973, 2973, [252, 291], "vec")
    assert np.isinf(want[:, :32]).any() and np.isfinite(want[:, 32:]).all()
    assert np.array_equal(w.call().dD.get().double().numpy(), want, equal_nan=True)

"""GPU parity of the low-rank adapters with their definition in 64 bits.

Tolerance, with e = 2^-24, r half a step of the input's 16-bit type (fp16 2^-11, bf16 2^-8)
and R half a step of the output's: the first product's fp32 sums of K terms (in up to 8
parts and 4 waves) are off by at most (K + 12) e sum|x a|; h is held in two parts for a
16-bit D and three for an fp32 one, which leaves r^2 |h| resp. r^3 |h|, and for fp16 what
is below 2^-34 (2^-38) of the token's largest |h|; the second sums 3 rank terms,
(3 rank + 4) e sum|h b|; the scale's multiplication adds e.  C is added in fp32 (e of the
result), and the result rounded once: R |d|.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_mixed_precision_tiled_amd as lg
from test_checkpoint_gpu import HALF_STEP, TINY, TORCH, Lines, ok, stream

pytestmark = pytest.mark.gpu

F32, F16, BF16 = lg.GEMM_F32, lg.GEMM_F16, lg.GEMM_BF16


class Lora:
    """One seeded call.  how: "vec" (16-byte lines), "odd" (unaligned everything)."""

    def __init__(self, T, K, N, rank, adapters, i=BF16, o=BF16, how="vec", ids="random", ranks=False,
                 scales=True, c=True, ints=False, seed=0):
        self.__dict__.update(T=T, K=K, N=N, rank=rank, adapters=adapters, i=i, o=o)
        g = torch.Generator().manual_seed(seed + T + 31 * K + 7 * N + rank)
        t = TORCH[i]
        if ints:
            pick = lambda n, m: torch.randint(-2, 3, (n, m), generator=g).to(t)  # noqa: E731
            self.X, self.A, self.B = pick(T, K), pick(adapters * rank, K), pick(adapters * N, rank)
            self.scales = torch.randint(1, 3, (adapters,), generator=g).float() if scales else None
            self.C = torch.randint(-9, 10, (T, N), generator=g).to(TORCH[o]) if c else None
        else:
            self.X = torch.randn(T, K, generator=g).to(t)
            self.A = (torch.randn(adapters * rank, K, generator=g) / K ** 0.5).to(t)
            self.B = (torch.randn(adapters * N, rank, generator=g) / rank ** 0.5).to(t)
            self.scales = torch.rand(adapters, generator=g) + 0.5 if scales else None
            self.C = torch.randn(T, N, generator=g).to(TORCH[o]) if c else None
        if ids == "random":  # any adapter, and none for some
            self.ids = torch.randint(-1, adapters, (T,), generator=g)
        elif ids == "runs":  # packed prompts
            cuts = torch.sort(torch.randint(0, max(T, 1), (7,), generator=g)).values
            self.ids = (torch.searchsorted(cuts, torch.arange(T), right=True) * 5 + 3) % (adapters + 1) - 1
        else:
            self.ids = torch.tensor(ids)
        self.ids = self.ids.to(torch.int32)
        self.ranks = torch.randint(-1, rank + 2, (adapters,), generator=g).int() if ranks else None
        up = lambda n, m: (n + m - 1) // m * m  # noqa: E731
        odd = how == "odd"
        line = lambda n, per: n + 3 if odd else up(n, per)  # noqa: E731
        sh = 1 if odd else 0
        self.dX = Lines(T, K, t, line(K, 8), sh, self.X)
        self.dA = Lines(adapters * rank, K, t, line(K, 8), sh, self.A)
        self.dB = Lines(adapters * N, rank, t, line(rank, 8), sh, self.B)
        for d in (self.dX, self.dA, self.dB):  # what lies between the rows must not matter
            pad = d.buf[d.shift:d.shift + d.rows * d.ld].view(d.rows, d.ld)[:, d.cols:]
            pad.fill_(float("nan"))
        self.dC = Lines(T, N, TORCH[o], line(N, 8), sh, self.C) if c else None
        self.dD = Lines(T, N, TORCH[o], line(N, 8), sh)
        self.dids = self.ids.cuda()
        self.dranks = None if self.ranks is None else self.ranks.cuda()
        self.dscales = None if self.scales is None else self.scales.cuda()
        ptr = lambda x: 0 if x is None else x.data_ptr()  # noqa: E731
        self.lora = lg.GemmLora(K, N, adapters, rank, self.dA.ptr, self.dA.ld, self.dB.ptr, self.dB.ld,
                                ptr(self.dranks), ptr(self.dscales))
        self.size = lg.gemm_lora_workspace(T, self.lora)
        assert self.size >= 0
        self.ws = torch.full((self.size + 64,), 255, dtype=torch.uint8, device="cuda")

    def call(self, D=None, s=None):
        D = self.dD if D is None else D
        C = self.dC
        ok(lg.gemm_lora_run(self.T, self.lora, self.dX.ptr, self.dX.ld, self.dids.data_ptr(),
                            0 if C is None else C.ptr, D.ld, D.ptr, D.ld, self.i, self.o, self.ws.data_ptr(),
                            self.size, stream() if s is None else s))
        return self

    def reference(self):
        """(D, bound of its error) in 64 bits."""
        T, K, N, rank = self.T, self.K, self.N, self.rank
        e, r, R = 2.0 ** -24, HALF_STEP[self.i], HALF_STEP[self.o]
        parts, low = (3, 2.0 ** -38) if self.o == F32 else (2, 2.0 ** -34)
        X, A, B = (v.double().numpy() for v in (self.X, self.A, self.B))
        A, B = A.reshape(self.adapters, rank, K), B.reshape(self.adapters, N, rank)
        D = self.C.double().numpy().copy() if self.C is not None else np.zeros((T, N))
        tol = np.zeros((T, N))
        for t in range(T):
            a = int(self.ids[t])
            if a < 0 or a >= self.adapters:
                continue
            k = rank if self.ranks is None else min(max(int(self.ranks[a]), 0), rank)
            if k == 0:
                continue
            s = 1.0 if self.scales is None else float(self.scales[a])
            h = A[a, :k] @ X[t]
            dh = (K + 12) * e * (np.abs(A[a, :k]) @ np.abs(X[t]))
            dh = dh + r ** parts * (np.abs(h) + dh)
            if self.i == F16:
                dh = dh + low * np.abs(h).max()
            Bk = np.abs(B[a, :, :k])
            D[t] += s * (B[a, :, :k] @ h)
            tol[t] = abs(s) * (Bk @ dh + (3 * rank + 6) * e * (Bk @ np.abs(h)))
        return D, 1.01 * tol + (1.01 * R + e) * np.abs(D) + TINY[self.o]

    def check(self, D=None):
        got = (self.dD if D is None else D).get().double().numpy()
        want, tol = self.reference()
        assert (self.ws[self.size:] == 255).all(), "written past the workspace"
        assert (np.abs(got - want) <= tol).all(), np.nanmax(np.abs(got - want) / tol)
        if self.o == F32:  # by the norm: roundings of independent signs
            assert np.linalg.norm(got - want) <= 2.0 ** -24 * (8 + self.K ** 0.5) * np.linalg.norm(want) + 1e-30
        return got


SHAPES = [  # T, K, N, rank, adapters
    (1, 64, 64, 8, 3), (1, 4096, 200, 16, 5), (2, 1, 1, 1, 1), (7, 100, 33, 5, 4), (16, 256, 64, 16, 16),
    (17, 520, 100, 12, 9), (33, 128, 300, 33, 6), (64, 1000, 70, 64, 40), (100, 96, 65, 7, 3), (5, 300, 80, 65, 2),
    (20, 200, 48, 200, 3), (31, 130, 40, 256, 2), (300, 160, 72, 16, 7), (1000, 72, 40, 24, 5)]


@pytest.mark.parametrize("how", ["vec", "odd"])
@pytest.mark.parametrize("i,o", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32), (F16, BF16)])
@pytest.mark.parametrize("T,K,N,rank,adapters", SHAPES)
def test_shapes(T, K, N, rank, adapters, i, o, how):
    Lora(T, K, N, rank, adapters, i, o, how, c=(T + N) % 3 != 0, ranks=T % 2 == 0, scales=K % 3 != 0).call().check()


# Past what one launch takes (more than 256 blocks of columns, a rank past 32 or a long A),
# and around it; prompts with long rows, large ranks and every token its own adapter.
LONGER = [
    (1, 2048, 256, 16, 2), (3, 2600, 520, 20, 2), (2, 8192, 40, 32, 2), (2, 8200, 40, 32, 2), (2, 16384, 40, 9, 2),
    (2, 16392, 40, 9, 2), (256, 40, 256, 4, 300), (129, 40, 257, 4, 3), (40, 1100, 2000, 12, 9), (70, 700, 1100, 30, 70),
    (5, 1200, 300, 128, 4), (290, 2100, 300, 100, 5), (500, 1500, 130, 256, 3), (300, 4100, 70, 33, 280),
    (321, 1024, 520, 64, 3)]


@pytest.mark.parametrize("how", ["vec", "odd"])
@pytest.mark.parametrize("i,o", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("T,K,N,rank,adapters", LONGER)
def test_longer_shapes(T, K, N, rank, adapters, i, o, how):
    Lora(T, K, N, rank, adapters, i, o, how, ranks=T % 2 == 0, seed=1).call().check()


@pytest.mark.parametrize("T,N", [(16, 1100), (80, 1100), (300, 1100)])
def test_bad_values_in_place_and_captured(T, N):
    """The three ways of the kernels: one launch, two, and prompts."""
    w = Lora(T, 128, N, 16, 4, ids=[t % 5 - 1 for t in range(T)])
    clean = w.call().dD.get()
    w.check()
    w.A[2 * 16 + 3, 7] = float("nan")
    w.X[1, 5] = float("inf")
    w.dA.view.copy_(w.A)
    w.dX.view.copy_(w.X)
    first = w.call().dD.get()
    for t in range(T):
        if t % 5 == 3:
            assert first[t].isnan().all()
        elif t == 1:
            assert not first[t].isfinite().any()
        else:
            assert torch.equal(first[t], clean[t])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.call(w.dC)
    for _ in range(3):
        w.dC.view.copy_(w.C)
        graph.replay()
        assert torch.equal(w.dC.get().view(torch.int16), first.view(torch.int16))
        w.call()


@pytest.mark.parametrize("i", [BF16, F16])
@pytest.mark.parametrize("T", [40, 257, 1100])
def test_packed_prompts(T, i):
    Lora(T, 264, 136, 16, 4, i, i, ids="runs").call().check()


@pytest.mark.parametrize("i", [BF16, F16])
@pytest.mark.parametrize("T,rank", [(3, 4), (33, 16), (300, 40)])
def test_integers_are_exact(T, rank, i):
    w = Lora(T, 96, 72, rank, 5, i, F32, ints=True).call()
    assert np.array_equal(w.dD.get().double().numpy(), w.reference()[0])


@pytest.mark.parametrize("T", [5, 40, 300])
def test_in_place(T):
    w = Lora(T, 128, 100, 8, 3).call()
    first = w.dD.get()
    w.call(w.dC)
    assert torch.equal(w.dC.get(), first)


def test_no_adapter_keeps_c():
    """Ids outside [0, adapters), of any value: D is C's very bits, NaN among them."""
    ids = [-1, 3, 2 ** 31 - 1, -2 ** 31, 0, 7, -5, 2] * 5
    w = Lora(40, 64, 72, 8, 3, ids=ids)
    w.C[1, 5] = float("nan")
    w.dC.view.copy_(w.C)
    got = w.call().dD.get()
    none = [t for t in range(40) if not 0 <= ids[t] < 3]
    assert torch.equal(got[none].view(torch.int16), w.C[none].view(torch.int16))
    w.call(w.dC)
    assert torch.equal(w.dC.get().view(torch.int16), got.view(torch.int16))


def test_every_token_alike_and_all_different():
    Lora(48, 136, 80, 16, 48, ids=[5] * 48).call().check()
    Lora(48, 136, 80, 16, 48, ids=list(range(48))).call().check()
    Lora(48, 136, 80, 16, 48, ids=[0, 1] * 24).call().check()
    Lora(1, 136, 80, 16, 1, ids=[-1]).call().check()


@pytest.mark.parametrize("i", [BF16, F16])
@pytest.mark.parametrize("T", [16, 300])
def test_bad_values_stay_with_their_tokens(T, i):
    """NaN in an adapter's weights, Inf in a token: other tokens do not see them."""
    w = Lora(T, 128, 96, 16, 4, i, i, ids=[t % 4 for t in range(T)])
    clean = w.call().dD.get()
    w.A[2 * 16 + 3, 7] = float("nan")
    w.B[1 * 96 + 11, 4] = float("inf")
    w.X[0, 5] = float("inf")
    for d, v in ((w.dA, w.A), (w.dB, w.B), (w.dX, w.X)):
        d.view.copy_(v)
    got = w.call().dD.get()
    for t in range(T):
        if t % 4 == 2:
            assert got[t].isnan().all()
        elif t == 0:
            assert not got[t].isfinite().any()
        elif t % 4 == 1:
            assert not got[t, 11].isfinite()
            keep = [n for n in range(96) if n != 11]
            assert torch.equal(got[t, keep], clean[t, keep])
        else:
            assert torch.equal(got[t], clean[t])


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -30, 1.0, 2.0 ** 30, 2.0 ** 80])
def test_fp16_inner_values_of_any_size(size):
    """h far outside fp16's range; the scale brings the result back."""
    w = Lora(20, 64, 40, 16, 3, F16, F32, c=False)
    # h = x A^T carries 2^14 at most from the operands; the rest of its size through fp32
    # partial sums is not reachable, so take it from X and A at their ends
    f = min(max(size, 2.0 ** -18), 2.0 ** 14)
    w.X, w.A = (w.X.float() * f ** 0.5).half(), (w.A.float() * f ** 0.5).half()
    w.scales = w.scales / size
    w.dX.view.copy_(w.X)
    w.dA.view.copy_(w.A)
    w.dscales.copy_(w.scales)
    w.call().check()


def test_fp16_inner_values_past_65504():
    w = Lora(20, 512, 40, 16, 3, F16, F32, c=False)
    w.X, w.A = torch.full_like(w.X, 200.0), torch.full_like(w.A, 30.0)  # h past 3e6
    w.A[::2] = 2.0 ** -14
    w.dX.view.copy_(w.X)
    w.dA.view.copy_(w.A)
    w.call().check()


def test_inf_rank_zero_and_scale_zero():
    w = Lora(12, 64, 40, 8, 3, ids=[0, 1, 2] * 4)
    w.dranks = torch.tensor([0, 8, 3], dtype=torch.int32, device="cuda")
    w.ranks = w.dranks.cpu()
    w.lora.ranks = w.dranks.data_ptr()
    w.scales[1] = 0.0
    w.dscales.copy_(w.scales)
    got = w.call().check()
    assert np.array_equal(got[0::3], w.C[0::3].double().numpy())
    assert np.array_equal(got[1::3], w.C[1::3].double().numpy())


def test_two_streams_and_same_bits():
    a, b = Lora(64, 512, 300, 16, 20), Lora(300, 256, 200, 8, 5, ids="runs", seed=3)
    ra, rb = a.call().dD.get(), b.call().dD.get()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.call(s=s1.cuda_stream)
        b.call(s=s2.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(a.dD.get(), ra) and torch.equal(b.dD.get(), rb)


def test_captured_follows_the_ids():
    w = Lora(40, 256, 136, 16, 6)
    w.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.call()
    for i in range(3):
        w.ids = torch.randint(-1, 6, (40,), generator=torch.Generator().manual_seed(i)).int()
        w.dids.copy_(w.ids)
        w.dD.view.zero_()
        graph.replay()
        got = w.check()
        w.call()  # eager work between the replays
        assert np.array_equal(w.dD.get().double().numpy(), got)


def test_long_offsets():
    """Lines so long that rows of X, A, B, C and D lie past 4 GiB."""
    T, K, N, rank, adapters, ld = 140, 32, 40, 3, 50, 1 << 24
    w = Lora(T, K, N, rank, adapters, BF16, F32, ids=[t % 51 - 1 for t in range(T)])

    def spread(m):
        buf = torch.empty((m.shape[0] - 1) * ld + m.shape[1], dtype=m.dtype, device="cuda")
        torch.as_strided(buf, m.shape, (ld, 1)).copy_(m)
        return buf

    X, A, C = spread(w.X), spread(w.A), spread(w.C)
    D = torch.empty_like(C)
    lora = lg.GemmLora(K, N, adapters, rank, A.data_ptr(), ld, w.dB.ptr, w.dB.ld, 0, w.dscales.data_ptr())
    ok(lg.gemm_lora_run(T, lora, X.data_ptr(), ld, w.dids.data_ptr(), C.data_ptr(), ld, D.data_ptr(), ld, BF16, F32,
                        w.ws.data_ptr(), w.size, stream()))
    w.dD.view.copy_(torch.as_strided(D, (T, N), (ld, 1)))
    w.check()


@pytest.mark.parametrize("o", [F32, BF16])
def test_long_offsets_of_prompts(o):
    """The same past 256 tokens, at the longest lines: a tile's own rows reach 2 GiB."""
    T, K, N, rank, adapters, ld = 300, 64, 72, 16, 10, 1 << 24
    w = Lora(T, K, N, rank, adapters, BF16, o, ids="runs")

    def spread(m):
        buf = torch.empty((m.shape[0] - 1) * ld + m.shape[1], dtype=m.dtype, device="cuda")
        torch.as_strided(buf, tuple(m.shape), (ld, 1)).copy_(m)
        return buf

    X, A, C = spread(w.X), spread(w.A), spread(w.C)
    D = torch.empty_like(C)
    lora = lg.GemmLora(K, N, adapters, rank, A.data_ptr(), ld, w.dB.ptr, w.dB.ld, 0, w.dscales.data_ptr())
    ok(lg.gemm_lora_run(T, lora, X.data_ptr(), ld, w.dids.data_ptr(), C.data_ptr(), ld, D.data_ptr(), ld, BF16, o,
                        w.ws.data_ptr(), w.size, stream()))
    w.dD.view.copy_(torch.as_strided(D, (T, N), (ld, 1)))
    w.check()


@pytest.mark.parametrize("o", [F32, BF16])
@pytest.mark.parametrize("T", [20, 300])
def test_bf16_inner_values_next_to_the_largest(T, o):
    """h between bf16's largest finite value and fp32's; the scale brings the result back."""
    w = Lora(T, 64, 40, 16, 3, BF16, o, c=False)
    w.X[:, :], w.A[:, :] = 0.0, 0.0
    w.X[:, :2] = 2.0 ** 64
    w.A[::2, 0], w.A[::2, 1] = 2.0 ** 63 * (2 - 2.0 ** -7), 2.0 ** 55 * 1.5  # 2^127 (2 - 2^-7 + 1.5 2^-8)
    w.A[1::4] = -w.A[::4]
    w.B = (w.B.float() * 2.0 ** -5).bfloat16()
    w.scales = w.scales * 2.0 ** -100
    for d, v in ((w.dX, w.X), (w.dA, w.A), (w.dB, w.B)):
        d.view.copy_(v)
    w.dscales.copy_(w.scales)
    h = float(w.A[0].double() @ w.X[0].double())
    assert torch.tensor(h).isfinite() and torch.tensor(h).bfloat16().isinf()
    w.call().check()


@pytest.mark.parametrize("o", [F32, F16, BF16])
@pytest.mark.parametrize("T", [20, 300])
def test_fp16_inner_values_beside_a_much_larger_one(T, o):
    """A rank whose h is far below the token's largest keeps its documented share: columns of D
    that use it alone are right but for 2^-38 of that largest value."""
    w = Lora(T, 64, 40, 16, 3, F16, o, c=False, ids=[t % 3 for t in range(T)])
    if o == F16:
        w.scales = w.scales * 2.0 ** -8  # D of the largest within its range
        w.dscales.copy_(w.scales)
    w.X[:, :], w.A[:, :], w.B[:, :] = 0.0, 0.0, 0.0
    w.X[:, 0], w.X[:, 1] = 2.0 ** 10, (1 + torch.arange(T) / 512).half()
    w.A.view(3, 16, 64)[:, 0, 0] = 2.0 ** 10                # h0 = 2^20
    for r in range(1, 16):                                  # h_r from 2^4 down to 2^-10
        w.A.view(3, 16, 64)[:, r, 1] = 2.0 ** (5 - r) * (1 + r / 16)
    for n in range(40):                                     # column n uses one rank
        w.B.view(3, 40, 16)[:, n, n % 16] = 1.0 + n / 64
    for d, v in ((w.dX, w.X), (w.dA, w.A), (w.dB, w.B)):
        d.view.copy_(v)
    got = w.call().dD.get().double().numpy()
    h = w.A.double().view(3, 16, 64)[0].numpy() @ w.X.double().numpy().T       # the three adapters are alike
    b = w.B.double().view(3, 40, 16)[0].numpy()
    for t in range(T):
        s = float(w.scales[t % 3])
        want = s * (b @ h[:, t])
        # h's parts, a rounding of h and of the two products, and the output's
        parts = (3 if o == F32 else 2) * 11
        tol = np.abs(b) @ np.abs(h[:, t]) * s * (2.0 ** -parts + 4 * 2.0 ** -24) + \
            s * np.abs(b).sum(1) * 2.0 ** -38 * np.abs(h[:, t]).max()
        tol = 1.01 * tol + HALF_STEP[o] * np.abs(want) + TINY[o]
        assert (np.abs(got[t] - want) <= tol).all(), np.max(np.abs(got[t] - want) / tol)


@pytest.mark.parametrize("how", ["vec", "odd"])
@pytest.mark.parametrize("i,o", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("T", [16, 80, 300])
def test_infinite_weights_give_infinities(T, i, o, how):
    """An Inf in B meets h as one number: D is Inf with the sign of h B, NaN only where h is 0 or
    two of them cancel.  (For 300 tokens h comes in parts, some of which are 0.)"""
    N = 1100
    w = Lora(T, 64, N, 40 if T == 300 else 16, 4, i, o, how, ids=[t % 5 - 1 for t in range(T)], ints=True)
    clean = w.call().dD.get()
    r = w.rank
    w.B[1 * N + 11, 4] = float("inf")
    w.B[1 * N + 1099, r - 1] = float("-inf")
    w.B[2 * N + 7, 0], w.B[2 * N + 7, 1] = float("inf"), float("inf")
    w.X[3] = 0.0  # a token of adapter 2 with h = 0
    w.dB.view.copy_(w.B)
    w.dX.view.copy_(w.X)
    got = w.call().dD.get()
    X, A, B = w.X.double(), w.A.double().view(4, r, 64), w.B.double().view(4, N, r)
    for t in range(T):
        a = t % 5 - 1
        if a not in (1, 2):
            assert torch.equal(got[t], clean[t])
            continue
        bad = [11, 1099] if a == 1 else [7]
        keep = [n for n in range(N) if n not in bad]
        if t != 3:
            assert torch.equal(got[t, keep], clean[t, keep])
        h = A[a] @ X[t]
        want = (B[a][bad] * h).sum(1)  # Inf, -Inf or NaN
        assert not want.isfinite().any()
        assert np.array_equal(got[t, bad].double().numpy(), want.numpy(), equal_nan=True)
    w.call(w.dC)  # and in place
    assert np.array_equal(w.dC.get().double().numpy(), got.double().numpy(), equal_nan=True)


@pytest.mark.parametrize("o", [F32, F16, BF16])
@pytest.mark.parametrize("T", [20, 300])
@pytest.mark.parametrize("size", ["large", "small", "mixed"])
def test_fp16_inner_values_far_from_one(T, o, size):
    """h at the ends of what fp16 operands reach (2^43 of a long row, 2^-42 of subnormal ones),
    tokens of very different size in one tile, and tokens whose h is 0."""
    K = 4096
    w = Lora(T, K, 40, 16, 3, F16, o, c=False)
    x = {"large": [60000.0], "small": [2.0 ** -20], "mixed": [60000.0, 2.0 ** -20, 1.0, 0.0]}[size]
    w.X = (w.X.float().clamp(-1, 1) * torch.tensor(x).repeat(T)[:T, None]).half()
    w.A = (w.A.float() * K ** 0.5).clamp(-1, 1) * {"large": 60000.0, "small": 2.0 ** -20, "mixed": 16.0}[size]
    w.A = w.A.half()
    if o != F32:  # results within the output's range
        w.scales = w.scales * {"large": 2.0 ** -36, "small": 2.0 ** 36, "mixed": 2.0 ** -18}[size]
        w.dscales.copy_(w.scales)
    w.dX.view.copy_(w.X)
    w.dA.view.copy_(w.A)
    w.call().check()


@pytest.mark.parametrize("T", [20, 300])
def test_bf16_smallest_inner_values(T):
    """Parts of h below bf16's smallest normal value still count."""
    w = Lora(T, 64, 40, 16, 3, BF16, F32, c=False)
    w.X, w.A = (w.X.float() * 2.0 ** -56).bfloat16(), (w.A.float() * 2.0 ** -56).bfloat16()
    w.B = (w.B.float() * 2.0 ** 20).bfloat16()
    w.scales = w.scales * 2.0 ** 90
    for d, v in ((w.dX, w.X), (w.dA, w.A), (w.dB, w.B)):
        d.view.copy_(v)
    w.dscales.copy_(w.scales)
    w.call().check()


@pytest.mark.parametrize("how", ["vec", "odd"])
def test_most_tokens(how):
    """2^20 tokens, the most there can be: integers, checked on the device."""
    T, K, N, rank, adapters = 1 << 20, 40, 24, 8, 7
    pad = 3 if how == "odd" else 0
    g = torch.Generator(device="cuda").manual_seed(0)
    pick = lambda n, m: torch.randint(-2, 3, (n, m + pad), generator=g, device="cuda").bfloat16()  # noqa: E731
    X, A, B, C = pick(T, K), pick(adapters * rank, K), pick(adapters * N, rank), pick(T, N)
    ids = (torch.arange(T, device="cuda") // 999 % (adapters + 1) - 1).int()
    D = torch.full((T + 1, N + pad), 77.0, device="cuda").bfloat16()
    lora = lg.GemmLora(K, N, adapters, rank, A.data_ptr(), K + pad, B.data_ptr(), rank + pad)
    ws = torch.empty(lg.gemm_lora_workspace(T, lora), dtype=torch.uint8, device="cuda")
    ok(lg.gemm_lora_run(T, lora, X.data_ptr(), K + pad, ids.data_ptr(), C.data_ptr(), N + pad, D.data_ptr(), N + pad,
                        BF16, BF16, ws.data_ptr(), ws.numel(), stream()))
    want = C[:, :N].float()
    for a in range(adapters):
        h = X[:, :K].float() @ A.float()[a * rank:(a + 1) * rank, :K].T
        want += torch.where((ids == a)[:, None], h @ B.float()[a * N:(a + 1) * N, :rank].T, 0.0)
    assert torch.equal(D[:T, :N], want.bfloat16()) and (D[T] == 77).all() and (D[:, N:] == 77).all()


@pytest.mark.parametrize("T", [1, 20, 300])
def test_widest(T):
    """K and N of 2^19, the largest."""
    K = N = 1 << 19
    g = torch.Generator(device="cuda").manual_seed(T)
    pick = lambda n, m, lo, hi: torch.randint(lo, hi, (n, m), generator=g, device="cuda").bfloat16()  # noqa: E731
    X, A, B = pick(T, K, 0, 2), pick(2 * 5, K, -1, 2), torch.zeros(2 * N, 8, device="cuda").bfloat16()
    B[:, :5] = pick(2 * N, 5, -1, 2)
    ids = (torch.arange(T, device="cuda") // 40 % 2).int()
    D = torch.full((T, N), 77.0, device="cuda")
    lora = lg.GemmLora(K, N, 2, 5, A.data_ptr(), K, B.data_ptr(), 8)
    ws = torch.empty(lg.gemm_lora_workspace(T, lora), dtype=torch.uint8, device="cuda")
    ok(lg.gemm_lora_run(T, lora, X.data_ptr(), K, ids.data_ptr(), 0, N, D.data_ptr(), N, BF16, F32, ws.data_ptr(),
                        ws.numel(), stream()))
    for a in (0, 1):
        rows = torch.nonzero(ids == a).flatten()
        h = X[rows].double() @ A[5 * a:5 * a + 5].double().T
        assert torch.equal(D[rows].double(), h @ B[a * N:(a + 1) * N, :5].double().T)  # sums below 2^24: exact


@pytest.mark.parametrize("T,N", [(16, 100), (80, 1100), (300, 136)])
@pytest.mark.parametrize("shift", [1, 100, 255])
def test_workspace_at_any_address(T, N, shift):
    w = Lora(T, 1100, N, 12, 3, F16, F32)
    clean = w.call().dD.get()
    ws = torch.full((w.size + 256,), 255, dtype=torch.uint8, device="cuda")
    ok(lg.gemm_lora_run(T, w.lora, w.dX.ptr, w.dX.ld, w.dids.data_ptr(), w.dC.ptr, w.dC.ld, w.dD.ptr, w.dD.ld, w.i,
                        w.o, ws.data_ptr() + shift, w.size, stream()))
    assert torch.equal(w.dD.get(), clean)
    assert (ws[:shift] == 255).all() and (ws[shift + w.size:] == 255).all()

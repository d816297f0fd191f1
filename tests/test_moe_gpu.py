"""GPU parity of the mixture-of-experts layer with its definition in 64 bits.

Tolerance, with e = 2^-24 and r half a step of the 16-bit type (fp16 2^-11, bf16
2^-8): the first product's fp32 sums of H terms are off by at most (H + 2) e
sum|x w|; the activation's slope is at most 1.13, and its own evaluation (the
exponential's argument of up to 30 is rounded, the function within 2 units)
2^-18 relative; h is held as two values of the type, the second of at most r |h|
and rounded once: r^2.  The second sums I terms in two parts (and adds up to
32 experts): (2 I + 40) e sum|h d|.  A weight's exponent is the difference of two
logits of size up to 10, its sum has E terms: (E + 40) e.  y is rounded once.  These
bounds add up absolutely and hold for every element.

They are far above the usual error, since roundings of independent signs do not
add up absolutely.  So the whole output is also compared by its 2-norm: the
rounding of y contributes at most r times the norm then, and 1.5 r leaves half as
much again for the rest.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import dense_mixed_precision_tiled_amd as lg
from gpu_util import log

pytestmark = pytest.mark.gpu

F16, BF16, I8 = lg.GEMM_F16, lg.GEMM_BF16, lg.GEMM_I8
TORCH = {F16: torch.float16, BF16: torch.bfloat16}
HALF_STEP = {F16: 2.0 ** -11, BF16: 2.0 ** -8}
SILU, GELU, RELU = lg.GEMM_ACT_SILU, lg.GEMM_ACT_GELU, lg.GEMM_ACT_RELU
SENTINEL = 12288.0  # exact in both types


def stream():
    return torch.cuda.current_stream().cuda_stream


def act64(x, act):
    if act == RELU:
        return np.maximum(x, 0)
    if act == GELU:
        return x * 0.5 * np.vectorize(math.erfc)(-x / math.sqrt(2.0))
    return x / (1 + np.exp(-x))


class Moe:
    """One seeded layer and call, on the CPU and on the device."""

    def __init__(self, T, H, I, E, topk, x=BF16, i8=False, act=SILU, renorm=False, pad=0, seed=0,
                 ints=False):
        g = torch.Generator().manual_seed(seed + T + 10 * H + 100 * I + 1000 * E)
        self.__dict__.update(T=T, H=H, I=I, E=E, topk=topk, x=x, i8=i8, act=act, renorm=renorm,
                             pad=pad)
        t = TORCH[x]
        if ints:  # sparse small integers: every sum and h is exact
            self.X = torch.randint(-1, 2, (T, H), generator=g).to(t)
            pick = lambda n, m: (torch.randint(-1, 2, (n, m), generator=g) *  # noqa: E731
                                 (torch.rand(n, m, generator=g) < 4.0 / m))
            self.W1, self.W2 = pick(E * 2 * I, H), pick(E * H, I)
        else:
            self.X = torch.randn(T, H, generator=g).to(t)
            self.W1 = torch.randn(E * 2 * I, H, generator=g)
            self.W2 = torch.randn(E * H, I, generator=g)
        self.s1 = self.s2 = None
        if i8:
            q = 1 if ints else 40
            self.W1 = (self.W1 * q).round().clamp(-128, 127).to(torch.int8)
            self.W2 = (self.W2 * q).round().clamp(-128, 127).to(torch.int8)
            self.s1 = torch.ones(E * 2 * I) if ints else \
                (torch.rand(E * 2 * I, generator=g) + 0.5) / (40 * H ** 0.5)
            self.s2 = torch.ones(E * H) if ints else \
                (torch.rand(E * H, generator=g) + 0.5) / (40 * I ** 0.5)
        elif ints:
            self.W1, self.W2 = self.W1.to(t), self.W2.to(t)
        else:
            self.W1, self.W2 = (self.W1 / H ** 0.5).to(t), (self.W2 / I ** 0.5).to(t)
        self.logits = torch.randn(T, E, generator=g) * 1.5

    def device(self):
        def lines(m, per):
            """Rows at the stride that pad asks for, the rest NaN (or -128)."""
            rows, cols = m.shape
            ld = cols + self.pad if self.pad else (cols + per - 1) // per * per
            fill = -128 if m.dtype == torch.int8 else float("nan")
            store = torch.full((rows, ld), fill, dtype=m.dtype)
            store[:, :cols] = m
            return store.cuda()

        per = 16 if self.i8 else 8
        self.dX, self.dW1, self.dW2 = lines(self.X, 8), lines(self.W1, per), lines(self.W2, per)
        self.dl = lines(self.logits, 1)
        self.ds1 = None if self.s1 is None else self.s1.cuda()
        self.ds2 = None if self.s2 is None else self.s2.cuda()
        self.dD = torch.full((self.T + 1, self.H + 4 + self.pad), SENTINEL, dtype=TORCH[self.x],
                             device="cuda")
        ptr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
        self.layer = lg.GemmMoe(self.H, self.I, self.E, self.topk, I8 if self.i8 else self.x,
                                ptr(self.dW1), self.dW1.shape[1], ptr(self.dW2), self.dW2.shape[1],
                                ptr(self.ds1), ptr(self.ds2), self.act, self.renorm)
        # a workspace of any content
        self.ws = torch.full((lg.gemm_moe_workspace(self.T, self.layer),), 255, dtype=torch.uint8,
                             device="cuda")
        return self

    def call(self, s=None):
        st = lg.gemm_moe_run(self.T, self.layer, self.dX.data_ptr(), self.dX.shape[1],
                             self.dl.data_ptr(), self.dl.shape[1], self.dD.data_ptr(),
                             self.dD.shape[1], self.x, self.ws.data_ptr(), self.ws.numel(),
                             stream() if s is None else s)
        assert st == 0, lg.gemm_status_string(st)

    def result(self):
        d = self.dD.cpu()
        assert (d[self.T:] == SENTINEL).all() and (d[:, self.H:] == SENTINEL).all(), \
            "written outside T x H"
        return d[:self.T, :self.H].double().numpy()

    def reference(self):
        """(y, bound of its error) in 64 bits."""
        T, H, I, E = self.T, self.H, self.I, self.E
        e24, r = 2.0 ** -24, HALF_STEP[self.x]
        X = self.X.double().numpy()
        W1, W2 = self.W1.double().numpy(), self.W2.double().numpy()
        if self.i8:
            W1 = W1 * self.s1.double().numpy()[:, None]
            W2 = W2 * self.s2.double().numpy()[:, None]
        W1, W2 = W1.reshape(E, 2 * I, H), W2.reshape(E, H, I)
        y, tol = np.zeros((T, H)), np.zeros((T, H))
        scale = 2 * e24 if self.i8 else 0.0  # a scale's multiplication, on each product
        for t in range(T):
            l = self.logits[t].double().numpy()
            if np.isnan(l).any() or np.isposinf(l).any():
                y[t] = np.nan
                continue
            if np.isneginf(l).all():
                continue
            p = np.exp(l - l.max())
            chosen = sorted(range(E), key=lambda j: (-l[j], j))[:self.topk]
            chosen = [j for j in chosen if l[j] > -np.inf]
            total = p[chosen].sum() if self.renorm else p.sum()
            for j in chosen:
                w = p[j] / total
                G, U = W1[j, :I], W1[j, I:]
                gate, up = G @ X[t], U @ X[t]
                ag, au = np.abs(G) @ np.abs(X[t]), np.abs(U) @ np.abs(X[t])
                a = act64(gate, self.act)
                h = a * up
                dh = 1.13 * np.abs(up) * ((H + 2) * e24 + scale) * ag + \
                    np.abs(a) * ((H + 2) * e24 + scale) * au + (2.0 ** -18 + r * r) * np.abs(h) + 2.0 ** -25
                if self.act == GELU:
                    dh += 2.2e-7 * np.maximum(1, np.abs(gate)) * np.abs(up)
                y[t] += w * (W2[j] @ h)
                D = np.abs(W2[j])
                tol[t] += w * (D @ dh + ((2 * I + 40) * e24 + (E + 40) * e24 + scale) * (D @ np.abs(h)))
            tol[t] = 1.01 * tol[t] + 1.01 * r * np.abs(y[t]) + 2.0 ** -25
        return y, tol

    def check(self, label=""):
        log("case: moe T%d H%d I%d E%d k%d x%d i8 %d pad %d %s" % (
            self.T, self.H, self.I, self.E, self.topk, self.x, self.i8, self.pad, label))
        self.device().call()
        got = self.result()
        ref, tol = self.reference()
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        got, ref = np.nan_to_num(got), np.nan_to_num(ref)
        err = np.abs(got - ref)
        worst = np.unravel_index(np.argmax(err - tol), err.shape)
        assert (err <= tol).all(), "at %s got %r ref %r tol %r" % (
            worst, got[worst], ref[worst], tol[worst])
        norm = np.linalg.norm(ref)
        if ref.size >= 64:
            assert np.linalg.norm(got - ref) <= 1.5 * HALF_STEP[self.x] * norm + 1e-6
        return got


TYPES = [(BF16, False), (F16, False), (BF16, True), (F16, True)]
# (T, H, I, E, topk): one token, batches at the row groups' edges, one expert,
# as many experts as pairs, more and fewer, odd and ragged widths
SIZES = [(1, 64, 32, 8, 2), (1, 1, 1, 1, 1), (1, 200, 100, 64, 8), (2, 256, 77, 16, 8),
         (3, 513, 130, 5, 5), (7, 100, 1000, 16, 4), (16, 512, 96, 32, 2), (17, 264, 40, 8, 3),
         (32, 128, 200, 100, 6), (33, 72, 24, 4, 1), (64, 320, 64, 16, 4), (64, 48, 520, 128, 8)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("x,i8", TYPES)
@pytest.mark.parametrize("pad", [0, 3])
def test_sizes_and_types(size, x, i8, pad):
    """pad 0: the vector loads; pad 3: element loads, padding NaN or -128."""
    Moe(*size, x=x, i8=i8, pad=pad).check()


@pytest.mark.parametrize("size", [(3, 4100, 72, 4, 2), (12, 4097, 100, 3, 1), (40, 4104, 136, 3, 2),
                                  (64, 4112, 40, 4, 1), (20, 2048, 300, 2, 1), (15, 2000, 64, 1, 1)])
@pytest.mark.parametrize("x,i8", TYPES)
@pytest.mark.parametrize("pad", [0, 3])
def test_wide_layers(size, x, i8, pad):
    """More columns than blocks of 8 for every CU, and just fewer."""
    Moe(*size, x=x, i8=i8, pad=pad).check()


@pytest.mark.parametrize("act", [SILU, GELU, RELU])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("x,i8", TYPES)
def test_activations_and_weights(act, renorm, x, i8):
    Moe(5, 136, 72, 12, 3, x=x, i8=i8, act=act, renorm=renorm, seed=7).check()


@pytest.mark.parametrize("T", [1, 16, 40, 64])
@pytest.mark.parametrize("x,i8", TYPES)
def test_exact_on_small_integers(T, x, i8):
    """One expert of weight 1, ReLU, integers whose sums every type holds: the
    result is the integer, so no element is left out, doubled or swapped."""
    m = Moe(T, 300, 150, 6, 1, x=x, i8=i8, act=RELU, renorm=True, ints=True)
    got = m.check("integers")
    W1, W2 = m.W1.double().numpy().reshape(6, 300, 300), m.W2.double().numpy().reshape(6, 300, 150)
    for t in range(T):
        e = int(np.argmax(m.logits[t].numpy()))
        gu = W1[e] @ m.X[t].double().numpy()
        want = W2[e] @ (np.maximum(gu[:150], 0) * gu[150:])
        assert np.abs(want).max() <= 256
        assert np.array_equal(got[t], want), t


@pytest.mark.parametrize("T,E,topk", [(1, 16, 4), (1, 300, 8), (6, 16, 4), (40, 24, 2)])
def test_ties_go_to_the_lower_expert(T, E, topk):
    m = Moe(T, 64, 48, E, topk)
    m.logits = (m.logits * 2).round().clamp(-1, 1)  # three values
    m.logits[m.logits == 0] = 0.0
    m.logits[0, ::2] *= -0.0 if T == 1 else 1.0     # -0 ties with 0
    m.check("ties")


@pytest.mark.parametrize("T,E,topk", [(7, 16, 4), (7, 40, 4), (1, 16, 4), (64, 8, 2)])
def test_masked_logits(T, E, topk):
    """Experts at -Inf are not chosen: fewer than topk, none at all; the weights
    of experts that no token may choose are NaN and stay unread.  NaN and +Inf
    give a NaN row, the lowest finite value does not mask."""
    m = Moe(T, 80, 40, E, topk, renorm=True)
    m.logits[:, E // 2:] = -float("inf")
    if not m.i8:
        m.W1.view(E, -1)[E // 2:] = float("nan")
        m.W2.view(E, -1)[E // 2:] = float("nan")
    m.logits[0, 1:] = -float("inf")              # one expert left
    if T > 1:
        m.logits[1] = -float("inf")              # none
        m.logits[2, 3] = float("nan")
        m.logits[3, 0] = float("inf")
        m.logits[4] = float("nan")
        m.logits[5, :3] = torch.finfo(torch.float32).min
    got = None
    m.device().call()
    got = m.result()
    ok = Moe(T, 80, 40, E, topk, renorm=True)    # finite weights for the reference
    ok.logits = m.logits
    ref, tol = ok.reference()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert (np.abs(np.nan_to_num(got) - np.nan_to_num(ref)) <= tol).all()
    if T > 1:
        assert (got[1] == 0).all() and np.isnan(got[2:5]).all()


@pytest.mark.parametrize("T", [2, 7, 40])
def test_a_token_that_is_nan_leaves_the_others_alone(T):
    """Tokens of one expert share matrix instructions, not values."""
    m = Moe(T, 256, 96, 4, 2, seed=8)
    ref, tol = m.reference()
    m.X[1, 5] = float("nan")
    m.device().call()
    got = m.result()
    assert np.isnan(got[1]).all()
    rest = [t for t in range(T) if t != 1]
    assert (np.abs(got[rest] - ref[rest]) <= tol[rest]).all()


def test_all_tokens_choose_the_same_expert():
    for T in (1, 16, 33, 64):
        for topk, E in ((1, 64), (2, 500)):
            m = Moe(T, 96, 56, E, topk)
            m.logits[:] = -3.0
            m.logits[:, 7] = 2.0
            m.logits[:, 3] = 1.0
            m.check("one expert")


def test_large_logits_keep_their_softmax():
    m = Moe(4, 64, 32, 8, 2)
    m.logits = m.logits * 1e4
    m.device().call()
    ref, tol = m.reference()
    # differences of logits of size 1e4 are rounded: 1e4 * 2^-24 in the exponent
    assert (np.abs(m.result() - ref) <= tol + 1e-3 * np.abs(ref)).all()


def test_weights_past_4_gib():
    """The last expert's weights start past 2^32 bytes."""
    H, I, E = 4096, 2048, 132
    W1 = torch.zeros(E * 2 * I, H, dtype=torch.bfloat16, device="cuda")
    W2 = torch.zeros(E * H, I, dtype=torch.bfloat16, device="cuda")
    assert (E - 1) * 2 * I * H * 2 > 2 ** 32 and W1.numel() * 2 > 2 ** 32
    m = Moe(2, 64, 32, 2, 1)  # the small layer only names the call's arguments
    g = torch.Generator(device="cuda").manual_seed(1)
    W1[-2 * I:] = torch.randn(2 * I, H, generator=g, device="cuda") / H ** 0.5
    W2[-H:] = torch.randn(H, I, generator=g, device="cuda") / I ** 0.5
    X = torch.randn(2, H, generator=g, device="cuda").bfloat16()
    logits = torch.zeros(2, E, device="cuda")
    logits[:, E - 1] = 5.0
    D = torch.empty(2, H, dtype=torch.bfloat16, device="cuda")
    layer = lg.GemmMoe(H, I, E, 1, BF16, W1.data_ptr(), H, W2.data_ptr(), I, renormalize=True)
    ws = torch.empty(lg.gemm_moe_workspace(2, layer), dtype=torch.uint8, device="cuda")
    st = lg.gemm_moe_run(2, layer, X.data_ptr(), H, logits.data_ptr(), E, D.data_ptr(), H, BF16,
                         ws.data_ptr(), ws.numel(), stream())
    assert st == 0
    x, w1, w2 = X.double().cpu(), W1[-2 * I:].double().cpu(), W2[-H:].double().cpu()
    g, u = x @ w1[:I].T, x @ w1[I:].T
    ref = (g * torch.sigmoid(g) * u) @ w2.T
    assert torch.linalg.norm(D.double().cpu() - ref) <= 3 * HALF_STEP[BF16] * torch.linalg.norm(ref)
    del m


def test_two_calls_on_two_streams():
    """Workspaces of their own: the calls may overlap."""
    a, b = Moe(9, 256, 128, 16, 4).device(), Moe(9, 256, 128, 16, 4, seed=50).device()
    a.call(), b.call()
    torch.cuda.synchronize()
    want = a.dD.clone(), b.dD.clone()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        a.dD.fill_(SENTINEL), b.dD.fill_(SENTINEL)
        torch.cuda.synchronize()
        a.call(s[0].cuda_stream), b.call(s[1].cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(a.dD, want[0]) and torch.equal(b.dD, want[1])


@pytest.mark.parametrize("T,E,topk", [(1, 64, 8), (20, 16, 2)])
def test_graphs_follow_the_logits(T, E, topk):
    """Two captured layers, replayed in turn on new tokens and logits with eager
    work between: every replay equals the eager result of its inputs."""
    layers = [Moe(T, 192, 96, E, topk, seed=s).device() for s in (0, 1)]
    graphs = []
    for m in layers:
        m.call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.call(stream())
        graphs.append(g)
    for step in range(3):
        for m, g in zip(layers, graphs):
            gen = torch.Generator(device="cuda").manual_seed(step)
            m.dX.copy_(torch.randn(m.dX.shape, generator=gen, device="cuda"))
            m.dl.copy_(torch.randn(m.dl.shape, generator=gen, device="cuda"))
            m.call()
            torch.cuda.synchronize()
            want = m.dD.clone()
            m.dD.fill_(SENTINEL)
            m.ws.fill_(17)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(m.dD, want)


@pytest.mark.parametrize("x,i8", TYPES)
def test_router_and_layer(x, i8):
    """As a program runs them: the router's product by gemm_run into fp32 logits,
    then the layer; with int8 weights, a scaled int8 product after it."""
    T, H, I, E, topk = 6, 256, 128, 16, 4
    m = Moe(T, H, I, E, topk, x=x, i8=i8, renorm=True).device()
    g = torch.Generator().manual_seed(3)
    router = (torch.randn(E, H, generator=g) / H ** 0.5).to(TORCH[x]).cuda()
    st = lg.gemm_run(T, E, H, m.dX.data_ptr(), H, lg.GEMM_ROW_MAJOR, router.data_ptr(), H,
                     lg.GEMM_COL_MAJOR, None, E, m.dl.data_ptr(), E, x, lg.GEMM_F32, lg.GEMM_F32, 0,
                     stream())
    assert st == 0
    m.call()
    m.logits = m.dl.cpu()
    assert torch.allclose(m.logits, m.X.float() @ router.cpu().float().T, rtol=1e-4, atol=1e-4)
    ref, tol = m.reference()
    got = m.result()
    assert (np.abs(got - ref) <= tol).all()
    if not i8:
        return
    # the next linear layer on y: quantised rows, scaled product
    W = torch.randint(-127, 128, (100, H), generator=g, dtype=torch.int8).cuda()
    sB = (torch.rand(100, generator=g) / 1000).cuda()
    Q = torch.empty(T, H, dtype=torch.int8, device="cuda")
    sA, out = torch.empty(T, device="cuda"), torch.empty(T, 100, device="cuda")
    assert lg.gemm_quantize_rows(T, H, m.dD.data_ptr(), m.dD.shape[1], x, Q.data_ptr(), H,
                                 sA.data_ptr(), stream()) == 0
    assert lg.gemm_run_scaled(T, 100, H, Q.data_ptr(), H, lg.GEMM_ROW_MAJOR, W.data_ptr(), H,
                              lg.GEMM_COL_MAJOR, sA.data_ptr(), sB.data_ptr(), None, 100,
                              out.data_ptr(), 100, I8, lg.GEMM_I32, lg.GEMM_F32, 0, None,
                              stream()) == 0
    y = got
    a = np.abs(y).max(1)
    q = np.rint(127 * y / a[:, None])
    P = q @ W.double().cpu().numpy().T * (a / 127)[:, None] * sB.double().cpu().numpy()
    assert (np.abs(out.double().cpu().numpy() - P) <= 8.1 * 2.0 ** -24 * np.abs(P)).all()


def rows_close(m, label):
    """Every token's row by its norm: y's rounding is at most r of it (2^-25 for an
    element that is subnormal in fp16), and half as much again is left for the rest."""
    log("case: moe T%d H%d I%d x%d i8 %d pad %d %s" % (m.T, m.H, m.I, m.x, m.i8, m.pad, label))
    m.device().call()
    got = m.result()
    with np.errstate(over="ignore"):  # exp of a large gate, whose silu is 0
        ref, _ = m.reference()
    assert np.isfinite(got).all(), label
    err, norm = np.linalg.norm(got - ref, axis=1), np.linalg.norm(ref, axis=1)
    bound = 1.5 * HALF_STEP[m.x] * norm + 2.0 ** -25 * m.H ** 0.5
    assert (err <= bound).all(), "%s: rows off by %s of their norm" % (label, (err / norm)[err > bound])


@pytest.mark.parametrize("T", [1, 2, 3, 7, 20, 50])
@pytest.mark.parametrize("H", [64, 2200])
@pytest.mark.parametrize("x,i8", TYPES)
def test_inner_values_of_any_size(T, H, x, i8):
    """h far below and above 1, y in the middle of its type's range: fp16 alone could
    not hold h and what rounding leaves of it.  Small and large tokens side by side."""
    for size, back in ((1e-1, 1e1), (1e-2, 1e3), (1e-3, 3e3), (300.0, 1e-3), (2000.0, 1e-4)):
        for pad in (0, 3):
            m = Moe(T, H, 333, 2, 1, x=x, i8=i8, renorm=True, pad=pad)
            m.X = (m.X * size).to(m.X.dtype)
            if i8:
                m.s2 = m.s2 * back
            else:
                m.W2 = (m.W2.float() * back).to(m.W2.dtype)
            rows_close(m, "x %g" % size)
    m = Moe(T, H, 333, 2, 1, x=x, i8=i8, renorm=True)
    m.X = (m.X * torch.logspace(-2, 2, T)[:, None]).to(m.X.dtype)
    # (y of the largest token's h, about 1e4, stays finite)
    rows_close(m, "tokens of 1e-2 to 1e2")


@pytest.mark.parametrize("T", [1, 3, 12, 50])
@pytest.mark.parametrize("H", [64, 2200])
@pytest.mark.parametrize("x,i8", TYPES)
def test_inner_values_that_grow_along_the_row(T, H, x, i8):
    """Rows of h that start with zeros or small values and grow, or shrink, over I."""
    I = 700
    for name, f in (("grow", torch.logspace(-4, 1, I)), ("shrink", torch.logspace(1, -4, I)),
                    ("late", torch.cat([torch.zeros(400), torch.full((I - 400,), 1e-2)]))):
        m = Moe(T, H, I, 2, 1, x=x, i8=i8, renorm=True)
        if i8:
            m.s1.view(2, 2, I)[:, 1] *= f
        else:
            m.W1.view(2, 2, I, H)[:, 1] *= f[:, None].to(m.W1.dtype)
        rows_close(m, name)


@pytest.mark.parametrize("T", [1, 2, 6, 40])
@pytest.mark.parametrize("x", [BF16, F16])
def test_inner_values_over_the_range_of_fp32(T, x):
    """int8 weights whose scales put h near 1e-24 or 1e22, and y near 1."""
    for up, down in ((1e-12, 1e24), (1e11, 1e-22)):
        m = Moe(T, 96, 300, 2, 1, x=x, i8=True, renorm=True)
        m.s1, m.s2 = m.s1 * up, m.s2 * down
        rows_close(m, "scales of %g" % up)


@pytest.mark.parametrize("T", [2, 7, 40])
@pytest.mark.parametrize("H", [64, 2200])
@pytest.mark.parametrize("x,i8", TYPES)
def test_an_infinite_token_leaves_the_others_alone(T, H, x, i8):
    """A token whose h is Inf or NaN shares the others' rows of the matrix units."""
    m = Moe(T, H, 333, 2, 1, x=x, i8=i8, seed=4)
    ref, tol = m.reference()
    m.X[0, 5] = float("inf")
    m.device().call()
    got = m.result()
    assert not np.isfinite(got[0]).any()
    assert (np.abs(got[1:] - ref[1:]) <= tol[1:]).all()


@pytest.mark.parametrize("size", [(4, 64, 1100, 32, 8), (3, 72, 1537, 64, 8), (1, 40, 4100, 8, 8),
                                  (2, 40, 600, 1024, 32)])
@pytest.mark.parametrize("x,i8", TYPES)
@pytest.mark.parametrize("pad", [0, 3])
def test_few_tokens_of_wide_experts(size, x, i8, pad):
    """Up to four tokens and a block of columns for each wave of the first kernel."""
    Moe(*size, x=x, i8=i8, pad=pad).check()


@pytest.mark.parametrize("T", [1, 5, 64])
@pytest.mark.parametrize("x,i8", TYPES)
def test_most_experts_and_ranks(T, x, i8):
    """1024 experts, top 32: the limits."""
    Moe(T, 32, 24, 1024, 32, x=x, i8=i8, renorm=T == 5).check()


@pytest.mark.parametrize("x", [BF16, F16])
def test_longest_lines(x):
    """Leading dimensions of 2^24 elements: X, D and the weights past 2 GiB, logits past 4."""
    T, H, I, E, ld = 64, 40, 24, 2, 2 ** 24
    m = Moe(T, H, I, E, 2, x=x)

    def lines(t):
        store = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype, device="cuda")
        store[:, :t.shape[1]] = t.cuda()
        return store

    log("case: moe lines of 2^24, x%d" % x)
    X, W1, W2, logits = lines(m.X), lines(m.W1), lines(m.W2), lines(m.logits)
    D = torch.full((T, ld), SENTINEL, dtype=TORCH[x], device="cuda")
    layer = lg.GemmMoe(H, I, E, 2, x, W1.data_ptr(), ld, W2.data_ptr(), ld)
    ws = torch.empty(lg.gemm_moe_workspace(T, layer), dtype=torch.uint8, device="cuda")
    st = lg.gemm_moe_run(T, layer, X.data_ptr(), ld, logits.data_ptr(), ld, D.data_ptr(), ld, x,
                         ws.data_ptr(), ws.numel(), stream())
    assert st == 0
    ref, tol = m.reference()
    assert (np.abs(D[:, :H].double().cpu().numpy() - ref) <= tol).all()
    assert (D[:, H:H + 64] == SENTINEL).all() and (D[:, ld - 64:] == SENTINEL).all()


@pytest.mark.parametrize("x", [BF16, F16])
def test_widest_inner_rows(x):
    """2048 pairs of 2^19 inner values: 4 GiB of them in the workspace."""
    T, H, I, E, topk = 64, 8, 2 ** 19, 32, 32
    t = TORCH[x]
    g = torch.Generator(device="cuda").manual_seed(12)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    X, logits = rand(T, H).to(t), rand(T, E)
    W1, W2 = (rand(E * 2 * I, H) / H ** 0.5).to(t), (rand(E * H, I) / I ** 0.5).to(t)
    D = torch.full((T + 1, H), SENTINEL, dtype=t, device="cuda")
    layer = lg.GemmMoe(H, I, E, topk, x, W1.data_ptr(), H, W2.data_ptr(), I)
    ws = torch.empty(lg.gemm_moe_workspace(T, layer), dtype=torch.uint8, device="cuda")
    log("case: moe widest inner rows, x%d, workspace %d" % (x, ws.numel()))
    st = lg.gemm_moe_run(T, layer, X.data_ptr(), H, logits.data_ptr(), E, D.data_ptr(), H, x,
                         ws.data_ptr(), ws.numel(), stream())
    assert st == 0
    w = torch.softmax(logits.double(), 1)
    ref = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        w1 = W1[e * 2 * I:(e + 1) * 2 * I].double()
        gate, up = X.double() @ w1[:I].t(), X.double() @ w1[I:].t()
        h = gate * torch.sigmoid(gate) * up
        ref += w[:, e:e + 1] * (h @ W2[e * H:(e + 1) * H].double().t())
    assert (D[T] == SENTINEL).all()
    # y's rounding, and as much again for sums of 2^19 terms of either sign
    err = torch.linalg.norm(D[:T].double() - ref, dim=1) / torch.linalg.norm(ref, dim=1)
    assert (err <= 2 * HALF_STEP[x]).all(), err.max().item()


@pytest.mark.parametrize("x,i8", TYPES)
@pytest.mark.parametrize("offset", [1, 100, 255])
def test_workspace_at_any_address(x, i8, offset):
    """The size that gemm_moe_workspace names is enough wherever the memory starts."""
    m = Moe(20, 96, 72, 8, 2, x=x, i8=i8).device()
    m.call()
    want = m.dD.clone()
    size = m.ws.numel()
    store = torch.full((offset + size + 64,), 99, dtype=torch.uint8, device="cuda")
    m.ws = store[offset:offset + size]
    m.dD.fill_(SENTINEL)
    m.call()
    assert torch.equal(m.dD, want)
    assert (store[:offset] == 99).all() and (store[offset + size:] == 99).all()


@pytest.mark.parametrize("T,H", [(1, 64), (3, 64), (10, 64), (40, 2200)])
@pytest.mark.parametrize("x,i8", [(F16, False), (F16, True)])
def test_graphs_follow_the_size_of_the_inner_values(T, H, x, i8):
    """fp16: a captured layer replayed on tokens of other sizes, up and down, with eager
    work between; every replay equals the eager result, which repeats itself."""
    m, other = (Moe(T, H, 333, 4, 2, x=x, i8=i8, seed=s).device() for s in (0, 1))
    m.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.call(stream())
    start = m.dX.clone()
    for size in (1.0, 2.0 ** -10, 2.0 ** 6, 2.0 ** -6):
        m.dX.copy_(start * size)
        m.dD.fill_(SENTINEL)
        m.ws.fill_(255)
        m.call()
        torch.cuda.synchronize()
        want = m.dD.clone()
        other.call()
        for fill in (0, 17):
            m.dD.fill_(SENTINEL)
            m.ws.fill_(fill)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(m.dD, want)

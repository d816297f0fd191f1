"""GPU parity of the router's balance loss, counts and gradient with their definitions in
64 bits.

Counts are compared exactly.  With e = 2^-24: an exponential's argument l - max (or
l - lse) of size a is rounded to a e, its evaluation adds at most 4 e relatively; a sum over
E experts adds (E + 2) e, so p is off by d = (2 a + E + 16) e relatively, with a the
spread of the token's logits (for the gradient also |lse| e from lse's rounding).  lse is
off by d + 4 e |lse|, from the logarithm and the addition of the maximum.  Sums over tokens
are fp32 over 32 of them (32 e of the sum) and fp64 beyond.  f is off by 3 e; the gradient's bracket adds a few products:
|g| p (balance E (|f| + sum f p) (2 d + 8 e) + 2 z (|lse| (d + 8 e) + d)), rounded once.
A p below 2^-126, fp32's smallest normal value, may be 0 (the exponential's result is not
kept as a subnormal), and products below that lose bits: twice 2^-126 of everything p is
multiplied with, and 2^-126 of g / n, z and lse's products on the way.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_mixed_precision_tiled_amd as lg
from test_checkpoint_gpu import HALF_STEP, TINY, TORCH, Lines, ok, stream

pytestmark = pytest.mark.gpu

F32, F16, BF16 = lg.GEMM_F32, lg.GEMM_F16, lg.GEMM_BF16
e24 = 2.0 ** -24


def reference(l, topk, mask, balance, z, g):
    """loss (3), counts, lse, dlogits and p in 64 bits, of logits without NaN or +Inf."""
    T, E = l.shape
    alive = (mask != 0) & (l > -np.inf).any(1)
    counts = np.zeros(E + 1, np.int64)
    counts[E] = n = int(alive.sum())
    p, lse = np.zeros((T, E)), np.where(mask != 0, -np.inf, 0.0)
    for t in np.flatnonzero(alive):
        order = sorted(range(E), key=lambda j: (-l[t, j], j))[:topk]
        for j in order:
            counts[j] += l[t, j] > -np.inf
        x = np.exp(l[t] - l[t].max())
        lse[t] = np.log(x.sum()) + l[t].max()
        p[t] = x / x.sum()
    if n == 0:
        return np.zeros(3), counts, lse, np.zeros((T, E)), p
    f = counts[:E] / (n * topk)
    b, zz = E * (f * p.sum(0)).sum() / n, (lse[alive] ** 2).sum() / n
    with np.errstate(invalid="ignore"):
        d = g / n * p * (balance * E * (f - (p @ f)[:, None]) + 2 * z * np.where(alive, lse, 0)[:, None])
    return np.array([balance * b + z * zz, b, zz]), counts, lse, d, p


class Balance:
    def __init__(self, T, E, topk, o=F32, mask=False, odd=False, balance=0.01, z=0.001, dloss=True, seed=0,
                 logits=None):
        self.__dict__.update(T=T, E=E, topk=topk, o=o, balance=balance, z=z)
        g = torch.Generator().manual_seed(seed + T + 17 * E + topk)
        self.l = torch.randn(T, E, generator=g) * 1.5 if logits is None else logits
        self.mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8) if mask else None
        self.g = 1.7 if dloss else 1.0
        up = (E + 3) // 4 * 4
        ld, sh = (E + 3, 1) if odd else (up, 0)
        self.dl = Lines(T, E, torch.float32, ld, sh, self.l)
        self.dD = Lines(T, E, TORCH[o], ld, sh)
        self.dmask = None if self.mask is None else self.mask.cuda()
        self.dloss = torch.tensor([1.7], device="cuda") if dloss else None
        self.loss, self.counts = Lines(1, 3, torch.float32), Lines(1, E + 1, torch.int32)
        self.lse = Lines(1, T, torch.float32)
        self.size = lg.gemm_moe_balance_workspace(T, E, topk)
        self.ws = torch.full((self.size + 64,), 255, dtype=torch.uint8, device="cuda")

    def call(self, s=None):
        s = stream() if s is None else s
        ptr = lambda x: 0 if x is None else x.data_ptr()  # noqa: E731
        ok(lg.gemm_moe_balance(self.T, self.E, self.topk, self.dl.ptr, self.dl.ld, ptr(self.dmask), self.balance,
                               self.z, self.loss.ptr, self.counts.ptr, self.lse.ptr, self.ws.data_ptr(), self.size, s))
        ok(lg.gemm_moe_balance_grad(self.T, self.E, self.topk, self.dl.ptr, self.dl.ld, ptr(self.dmask), self.balance,
                                    self.z, self.counts.ptr, self.lse.ptr, ptr(self.dloss), self.dD.ptr, self.dD.ld,
                                    self.o, s))
        return self

    def get(self):
        assert (self.ws[self.size:] == 255).all(), "written past the workspace"
        return (self.loss.get()[0], self.counts.get()[0], self.lse.get()[0], self.dD.get())

    def check(self):
        l = self.l.double().numpy()
        mask = np.ones(self.T) if self.mask is None else self.mask.numpy()
        b32, z32, g32 = (float(np.float32(v)) for v in (self.balance, self.z, self.g))
        loss, counts, lse, d, p = reference(l, self.topk, mask, b32, z32, g32)
        gl, gc, gs, gd = self.get()
        assert np.array_equal(gc.numpy(), counts)
        with np.errstate(invalid="ignore"):
            spread = np.where(np.isfinite(l), l.max(1, keepdims=True) - l, 0)
        flse = np.where(np.isfinite(lse), np.abs(lse), 0)
        rel = (2 * spread + self.E + 16) * e24
        dl = rel.max(1) + 4 * e24 * flse + e24
        same = np.isinf(lse)
        assert np.array_equal(gs.numpy()[same], lse[same].astype(np.float32))
        assert (np.abs(gs.double().numpy()[~same] - lse[~same]) <= dl[~same]).all()
        n = max(counts[-1], 1)
        f = counts[:-1] / (n * self.topk)
        db = self.E * (f * (p * rel).sum(0)).sum() / n + 34 * e24 * loss[1]
        dz = (2 * flse * dl + dl ** 2).sum() / n + 34 * e24 * loss[2]
        got = gl.double().numpy()
        bound = [abs(b32) * db + abs(z32) * dz + 2 * e24 * (abs(b32) * loss[1] + abs(z32) * loss[2]), db, dz]
        for v, want, b in zip(got, loss, bound):
            # (what lies past fp32's largest value is rounded to Inf: lse^2 of a row at its lowest)
            assert v == np.inf if want > 3.5e38 else abs(v - want) <= b
        dr = rel + (flse * e24 + dl)[:, None]
        fp = (p @ f)[:, None]
        tol = abs(g32) / n * p * (abs(b32) * self.E * (f + fp) * (2 * dr + (8 + self.E) * e24) +
                                  2 * abs(z32) * (flse[:, None] * (dr + 8 * e24) + dl[:, None]))
        r = HALF_STEP[self.o]
        pull = abs(b32) * self.E * (f + fp) + 2 * abs(z32) * flse[:, None]
        low = 2.0 ** -125 * abs(g32) / n * (pull + 1)
        tol = 1.01 * tol + 1.01 * r * np.abs(d) + TINY[self.o] + low
        err = np.abs(gd.double().numpy() - d)
        assert (err <= tol).all(), np.max(err / tol)
        return self


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("o", [F32, F16, BF16])
@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (1, 4, 2), (2, 5, 5), (7, 8, 2), (33, 9, 3), (64, 16, 4), (100, 17, 1),
                                      (65, 33, 8), (50, 64, 8), (31, 65, 6), (20, 130, 32), (9, 256, 8), (5, 257, 4),
                                      (6, 1000, 32), (3, 1024, 8)])
def test_shapes(T, E, topk, o, odd):
    Balance(T, E, topk, o, mask=T > 6, odd=odd, dloss=T % 2 == 0).call().check()


@pytest.mark.parametrize("T,E,topk", [(5000, 8, 2), (3001, 60, 4), (9000, 3, 1)])
def test_many_tokens(T, E, topk):
    Balance(T, E, topk, BF16, mask=True).call().check()


def test_more_tokens_than_threads():
    """Several tokens for each group of lanes, with 16 waves in a workgroup."""
    Balance(70000, 20, 2, F32, mask=True).call().check()


@pytest.mark.parametrize("balance,z", [(0.0, 0.0), (1.0, 0.0), (0.0, 1.0), (-2.0, 0.5)])
def test_weights(balance, z):
    Balance(50, 12, 3, balance=balance, z=z).call().check()


def test_ties_and_zeros():
    """Equal logits go to the lower index, -0 equals +0."""
    g = torch.Generator().manual_seed(0)
    l = torch.randint(-1, 2, (200, 24), generator=g).float()
    l[torch.rand(200, 24, generator=g) < 0.3] *= -1.0  # turns 0 into -0
    Balance(200, 24, 5, logits=l).call().check()
    Balance(30, 7, 3, logits=torch.zeros(30, 7)).call().check()


def test_masked_experts_and_empty_tokens():
    """Experts at -Inf are not chosen, also where fewer than topk are left; a token of -Inf
    alone, or of masked ones alone, does not count."""
    g = torch.Generator().manual_seed(1)
    l = torch.randn(60, 10, generator=g)
    l[torch.rand(60, 10, generator=g) < 0.6] = -float("inf")
    l[::7] = -float("inf")
    l[3, 1:] = -float("inf")
    l[4] = torch.finfo(torch.float32).min  # the type's lowest value is a number like others
    b = Balance(60, 10, 4, mask=True, logits=l).call().check()
    assert not b.get()[3][0].any()
    none = Balance(20, 10, 4, logits=torch.full((20, 10), -float("inf"))).call().check()
    loss, counts, _, d = none.get()
    assert not loss.any() and not counts.any() and not d.any()


def test_every_token_masked():
    b = Balance(20, 10, 4, mask=True)
    b.mask.zero_()
    b.dmask.zero_()
    b.dl.view.fill_(float("nan"))  # masked tokens are not read
    b.call()
    loss, counts, lse, d = b.get()
    assert not loss.any() and not counts.any() and not d.any() and not lse.any()


def test_no_tokens():
    b = Balance(0, 6, 2).call()
    loss, counts, _, _ = b.get()
    assert not loss.any() and not counts.any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_tokens(bad):
    """A NaN or +Inf makes the loss and the token's own gradients NaN, not the others'."""
    b = Balance(40, 12, 3)
    clean = b.call().get()
    b.l[17, 5] = bad
    b.dl.view.copy_(b.l)
    loss, counts, _, d = b.call().get()
    assert loss.isnan().all() and d[17].isnan().all()
    rest = [t for t in range(40) if t != 17]
    assert d[rest].isfinite().all()
    order = lambda row: sorted(range(12), key=lambda j: (-row[j] if row[j] == row[j] else float("inf"), j))  # noqa: E731
    want = np.zeros(12, int)
    for t in range(40):
        want[order(b.l[t].tolist())[:3]] += 1
    assert np.array_equal(counts[:12].numpy(), want) and int(counts[12]) == 40
    if np.array_equal(want, clean[1][:12].numpy()):
        assert torch.equal(d[rest], clean[3][rest])


def test_large_logits():
    """Rows of a large spread, and rows far from zero."""
    g = torch.Generator().manual_seed(2)
    l = torch.randn(64, 16, generator=g) * 50
    l[::3] += 1e4
    l[1::3] -= 3e3
    Balance(64, 16, 4, logits=l).call().check()


def test_gradient_is_the_differences_of_the_loss():
    """The loss of the kernel itself, a step up and down along each logit (small enough that
    no choice changes): the fp32 loss is off by 2^-22 of about 1, and the step's cube by
    h^2 / 6 times a third derivative of at most about 4."""
    l = torch.tensor([[0.9, -0.4, 1.8, 0.1], [2.0, 0.6, -1.0, -0.2], [0.3, 1.4, 0.7, -0.9]])
    h = 2.0 ** -6
    for bal, z in ((1.0, 0.0), (0.0, 1.0), (0.5, 0.25)):
        make = lambda m: Balance(3, 4, 2, balance=bal, z=z, dloss=False, logits=m).call()  # noqa: E731
        grad = make(l).get()[3].double()
        for t in range(3):
            for j in range(4):
                up, down = l.clone(), l.clone()
                up[t, j] += h
                down[t, j] -= h
                num = (float(make(up).get()[0][0]) - float(make(down).get()[0][0])) / (2 * h)
                assert abs(num - float(grad[t, j])) <= 2.0 ** -21 * 4 / h + 4 * h * h / 6


def test_two_streams_and_same_bits():
    a, b = Balance(3000, 64, 8), Balance(5000, 12, 2, BF16, mask=True)
    ra, rb = a.call().get(), b.call().get()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.call(s1.cuda_stream)
        b.call(s2.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.get(), ra))
    assert all(torch.equal(x, y) for x, y in zip(b.get(), rb))


def test_captured_follows_the_logits():
    b = Balance(500, 24, 4, mask=True)
    b.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.call()
    for i in range(3):
        b.l = torch.randn(500, 24, generator=torch.Generator().manual_seed(i))
        b.dl.view.copy_(b.l)
        b.dD.view.zero_()
        graph.replay()
        replayed = b.check().get()
        b.call()
        assert all(torch.equal(x, y) for x, y in zip(b.get(), replayed))


def gradient(l, topk, balance, z, g):
    """The gradient by the definition in 64 bits, and |terms| of its bracket."""
    T, E = l.shape
    x = np.exp(l - l.max(1, keepdims=True))
    p = x / x.sum(1, keepdims=True)
    lse = np.log(x.sum(1)) + l.max(1)
    counts = np.zeros(E)
    for t in range(T):
        for j in sorted(range(E), key=lambda j: (-l[t, j], j))[:topk]:
            counts[j] += 1
    f = counts / (T * topk)
    fp = (p @ f)[:, None]
    pull = abs(balance) * E * (f + fp) + 2 * abs(z) * np.abs(lse)[:, None]
    return g / T * p * (balance * E * (f - fp) + 2 * z * lse[:, None]), abs(g) / T * p * pull


@pytest.mark.parametrize("far", [0.0, -1e4, 1e6, -1e6, 1e9, -1e9, 1e30, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("T,E,topk,odd", [(40, 64, 8, False), (33, 5, 2, True), (20, 300, 4, False)])
def test_probabilities_of_rows_far_from_zero(T, E, topk, odd, far):
    """Adding a constant to a row changes no p: rows of equal logits and of a few steps of fp32
    around a constant, whose log-sum-exp cannot hold log E beside it.  An exponential's
    argument a is rounded to a 2^-24, its evaluation and the sum over E experts add at most
    (E + 16) 2^-24, and the bracket's terms as much again."""
    g = torch.Generator().manual_seed(E)
    l = torch.full((T, E), far)
    step = max(abs(far) * 2.0 ** -22, 0.5)  # whole steps of fp32 there; each is exact
    if abs(far) < 1e7:  # (past that a step is more than all of the softmax's range)
        l[::2] += torch.randint(-3, 4, (l[::2].shape), generator=g) * step
    b = Balance(T, E, topk, odd=odd, balance=1.0, z=0.0, logits=l).call()
    d = b.get()[3].double().numpy()
    want, size = gradient(l.double().numpy(), topk, 1.0, 0.0, float(np.float32(1.7)))
    spread = (l.double().max(1, keepdim=True).values - l.double()).numpy()
    tol = size * (2 * spread.max(1, keepdims=True) + 2 * E + 40) * e24 + 2.0 ** -125
    assert (np.abs(d - want) <= tol).all(), np.max(np.abs(d - want) / tol)
    # each row's gradient adds up to 0 (all of the experts' pulls cancel)
    assert (np.abs(d.sum(1)) <= E * e24 * size.sum(1) + tol.sum(1)).all()


@pytest.mark.parametrize("z", [0.0, 1e-40, 0.5])
def test_loss_of_rows_at_the_lowest_value(z):
    """lse^2 of a row held at the type's lowest value does not fit fp32: loss[2] is Inf there,
    and the weight decides whether loss[0] is."""
    g = torch.Generator().manual_seed(3)
    l = torch.randn(60, 10, generator=g)
    l[4] = l[59] = torch.finfo(torch.float32).min
    b = Balance(60, 10, 4, balance=0.5, z=z, logits=l).call()
    loss = b.get()[0].double().numpy()
    want = reference(l.double().numpy(), 4, np.ones(60), 0.5, float(np.float32(z)), 1.7)[0]
    assert want[2] > 3.5e38 and loss[2] == np.inf
    assert abs(loss[1] - want[1]) <= 1e-5 * want[1]
    assert loss[0] == np.inf if want[0] > 3.5e38 else abs(loss[0] - want[0]) <= 1e-5 * want[0]


def test_loss_of_large_squares():
    """Squares that fit fp64 alone, and a mean that fits fp32."""
    l = torch.zeros(4000, 4)
    l[0] = -3e19  # 9e38 / 4000
    loss = Balance(4000, 4, 2, balance=0.0, z=1.0, logits=l).call().get()[0].double().numpy()
    want = 9e38 / 4000  # (the others' log(4)^2 is nothing beside it)
    assert abs(loss[2] - want) <= 1e-6 * want and abs(loss[0] - want) <= 1e-6 * want


@pytest.mark.parametrize("o", [F32, BF16])
@pytest.mark.parametrize("balance,z", [(1.0, 1.0), (3e38, 0.0), (0.0, 3e38), (1e37, 1e37)])
def test_gradients_whose_factors_leave_the_range(balance, z, o):
    """Results that fit fp32, of products on the way that do not: a row at the type's lowest
    value with a full z weight, and weights near fp32's largest on small p."""
    g = torch.Generator().manual_seed(4)
    T, E, topk = 6000, 64, 4
    l = torch.randn(T, E, generator=g)
    if z == 1.0:
        l[5] = l[77] = torch.finfo(torch.float32).min
    b = Balance(T, E, topk, o, balance=balance, z=z, logits=l, dloss=False).call()
    d = b.get()[3].double().numpy()
    want, size = gradient(l.double().numpy(), topk, float(np.float32(balance)), float(np.float32(z)), 1.0)
    assert np.abs(want).max() < 3.3e38
    spread = (l.double().max(1, keepdim=True).values - l.double()).numpy()
    lse = np.abs(np.log(np.exp(l.double().numpy() - l.double().numpy().max(1, keepdims=True)).sum(1)) + l.double().numpy().max(1))
    # (lse itself is off by (2 spread + E + 20) 2^-24, and by half a step of its own)
    dlse = (2 * spread.max(1) + E + 20 + 4 * lse) * e24
    tol = size * (2 * spread.max(1, keepdims=True) + 2 * E + 40) * e24 + (2 * z / T * dlse)[:, None] + 2.0 ** -125
    tol = tol + HALF_STEP[o] * np.abs(want)
    assert (np.abs(d - want) <= tol).all(), np.max(np.abs(d - want) / tol)


def test_many_tokens_for_each_thread():
    """More than 32 tokens for each group of lanes, whose sums go on in fp64; compared with torch
    in 64 bits on the device, to the bounds above (E = 3: p within 40 e, sums over tokens 34 e)."""
    T, E, topk = 20000003, 3, 1
    g = torch.Generator(device="cuda").manual_seed(0)
    l = torch.randn(T, E, generator=g, device="cuda")
    mask = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8)
    loss, counts, lse = torch.empty(3, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda"), \
        torch.empty(T, device="cuda")
    D = torch.empty(T, E, device="cuda")
    ws = torch.empty(lg.gemm_moe_balance_workspace(T, E, topk), dtype=torch.uint8, device="cuda")
    ok(lg.gemm_moe_balance(T, E, topk, l.data_ptr(), E, mask.data_ptr(), 1.0, 0.5, loss.data_ptr(), counts.data_ptr(),
                           lse.data_ptr(), ws.data_ptr(), ws.numel(), stream()))
    ok(lg.gemm_moe_balance_grad(T, E, topk, l.data_ptr(), E, mask.data_ptr(), 1.0, 0.5, counts.data_ptr(), lse.data_ptr(),
                                0, D.data_ptr(), E, F32, stream()))
    d = l.double()
    live = mask != 0
    n = int(live.sum())
    c = torch.bincount(l[live].argmax(1), minlength=E)  # no ties among normal values of one row, or few
    same = int(((l == l.max(1, keepdim=True).values).sum(1) > 1)[live].sum())
    got = counts.long()
    assert int(got[E]) == n and int((got[:E] - c).abs().sum()) <= 2 * same and int(got[:E].sum()) == n
    p = torch.softmax(d, 1) * live[:, None]
    f = got[:E].double() / n
    want_lse = torch.logsumexp(d, 1) * live
    b, z = float(E * (f * p.sum(0)).sum() / n), float((want_lse ** 2).sum() / n)
    assert abs(float(loss[1]) - b) <= 80 * e24 * b and abs(float(loss[2]) - z) <= 200 * e24 * z
    assert abs(float(loss[0]) - (b + 0.5 * z)) <= 200 * e24 * (b + 0.5 * z)
    assert float((lse.double() - want_lse).abs().max()) <= 60 * e24 * 8
    fp = (p * f).sum(1, keepdim=True)
    assert bool((fp >= 0).all())
    pull = E * (f - fp) + want_lse[:, None]
    size = p * (E * (f + fp) + want_lse.abs()[:, None] + 1)
    assert bool(((D.double() * n - p * pull).abs() <= 200 * e24 * size + 1e-30).all())


@pytest.mark.parametrize("shift", [1, 100, 255])
def test_workspace_at_any_address(shift):
    b = Balance(3000, 40, 4)
    clean = b.call().get()
    ws = torch.full((b.size + 256,), 255, dtype=torch.uint8, device="cuda")
    ok(lg.gemm_moe_balance(b.T, b.E, b.topk, b.dl.ptr, b.dl.ld, 0, b.balance, b.z, b.loss.ptr, b.counts.ptr, b.lse.ptr,
                           ws.data_ptr() + shift, b.size, stream()))
    assert all(torch.equal(x, y) for x, y in zip(b.get(), clean))
    assert (ws[:shift] == 255).all() and (ws[shift + b.size:] == 255).all()

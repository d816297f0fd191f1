"""The operators as programs use them, one after the other on one stream: a training step of
a layer of experts' router and of an activated linear layer from 8-bit checkpoints, and a
served quantised projection with adapters, eager and as a captured graph.

Every stage is compared with its definition in 64 bits on the values that the stages
before it produced, by the 2-norm: an output's rounding contributes at most half a step r
relatively; 1.5 r leaves half as much for the sums in fp32 (2^-24 sqrt(terms), below
2^-16 of the norm here, where an fp32 result is compared)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import checkpoint_util as ck
import dense_mixed_precision_tiled_amd as lg
from test_balance_gpu import reference as balance_reference
from test_checkpoint_gpu import HALF_STEP, ok, slope64, stream

pytestmark = pytest.mark.gpu

F32, F16, BF16 = lg.GEMM_F32, lg.GEMM_F16, lg.GEMM_BF16
R, C = lg.GEMM_ROW_MAJOR, lg.GEMM_COL_MAJOR


def near(got, want, dtype):
    want = np.asarray(want)
    got = got.double().cpu().numpy()
    r = 2.0 ** -16 if dtype == F32 else 1.5 * HALF_STEP[dtype]
    assert np.linalg.norm(got - want) <= r * np.linalg.norm(want)


def f64(t):
    return t.double().cpu().numpy()


def empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Step:
    """Forward and backward of: logits = X Wr^T (router, balance loss), Z = X W^T + b,
    Y = gelu(Z); X and Z are kept in 8 bits."""

    def __init__(self, M=300, K=136, N=96, E=12, topk=3):
        self.__dict__.update(M=M, K=K, N=N, E=E, topk=topk)
        g = torch.Generator().manual_seed(7)
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.X = rand(M, K).bfloat16().cuda()
        self.Wr, self.W = (rand(E, K) / K ** 0.5).bfloat16().cuda(), (rand(N, K) / K ** 0.5).bfloat16().cuda()
        self.b, self.dY = (0.1 * rand(N)).cuda(), rand(M, N).bfloat16().cuda()
        self.dWr0, self.dW0 = rand(E, K).cuda(), rand(N, K).cuda()  # gradients so far
        self.logits, self.Z = empty(M, E), empty(M, N, dtype=torch.bfloat16)
        self.kb, self.nb = (K + 31) // 32, (N + 31) // 32
        ldq = (K + 15) // 16 * 16
        self.QX, self.SX = empty(M, ldq, dtype=torch.int8), empty(M, self.kb, dtype=torch.uint8)
        self.QZ, self.SZ = empty(M, N, dtype=torch.int8), empty(M, self.nb, dtype=torch.uint8)
        self.loss, self.counts, self.lse = empty(3), empty(E + 1, dtype=torch.int32), empty(M)
        self.dlogits, self.dZ = empty(M, E, dtype=torch.bfloat16), empty(M, N, dtype=torch.bfloat16)
        self.dWr, self.dW = self.dWr0.clone(), self.dW0.clone()
        self.epi = lg.GemmEpilogue(bias=self.b.data_ptr())
        sizes = (lg.gemm_moe_balance_workspace(M, E, topk), lg.gemm_checkpoint_wgrad_workspace(M, E, K),
                 lg.gemm_checkpoint_wgrad_workspace(M, N, K))
        self.ws = empty(max(sizes) + 1, dtype=torch.uint8)  # one after the other: one workspace

    def run(self):
        s, M, K, N, E = stream(), self.M, self.K, self.N, self.E
        p = lambda t: t.data_ptr()  # noqa: E731
        ws, size = p(self.ws), self.ws.numel()
        ok(lg.gemm_checkpoint_pack(M, K, p(self.X), K, BF16, p(self.QX), self.QX.shape[1], p(self.SX), self.kb, s))
        ok(lg.gemm_run(M, E, K, p(self.X), K, R, p(self.Wr), K, C, 0, E, p(self.logits), E, BF16, F32, F32, 0, s))
        ok(lg.gemm_moe_balance(M, E, self.topk, p(self.logits), E, 0, 0.5, 0.01, p(self.loss), p(self.counts),
                               p(self.lse), ws, size, s))
        ok(lg.gemm_run_ex(M, N, K, p(self.X), K, R, p(self.W), K, C, 0, N, p(self.Z), N, BF16, F32, BF16, 0, self.epi, s))
        ok(lg.gemm_checkpoint_pack(M, N, p(self.Z), N, BF16, p(self.QZ), N, p(self.SZ), self.nb, s))
        # backward
        ok(lg.gemm_checkpoint_act_grad(M, N, p(self.QZ), N, p(self.SZ), self.nb, p(self.dY), N, lg.GEMM_ACT_GELU,
                                       p(self.dZ), N, BF16, s))
        ok(lg.gemm_checkpoint_wgrad(M, N, K, p(self.dZ), N, p(self.QX), self.QX.shape[1], p(self.SX), self.kb,
                                    p(self.dW), K, p(self.dW), K, BF16, F32, ws, size, s))
        ok(lg.gemm_moe_balance_grad(M, E, self.topk, p(self.logits), E, 0, 0.5, 0.01, p(self.counts), p(self.lse), 0,
                                    p(self.dlogits), E, BF16, s))
        ok(lg.gemm_checkpoint_wgrad(M, E, K, p(self.dlogits), E, p(self.QX), self.QX.shape[1], p(self.SX), self.kb,
                                    p(self.dWr), K, p(self.dWr), K, BF16, F32, ws, size, s))

    def check(self):
        X, K, N = f64(self.X), self.K, self.N
        Q, S = ck.pack(X)
        assert np.array_equal(self.QX[:, :K].cpu().numpy(), Q) and np.array_equal(self.SX.cpu().numpy(), S)
        V = ck.values(Q, S)
        near(self.logits, X @ f64(self.Wr).T, F32)
        loss, counts, lse, d, _ = balance_reference(f64(self.logits), self.topk, np.ones(self.M), 0.5,
                                                    float(np.float32(0.01)), 1.0)
        assert np.array_equal(self.counts.cpu().numpy(), counts)
        near(self.loss, loss, F32)
        near(self.lse, lse, F32)
        near(self.dlogits, d, BF16)
        near(self.dWr, f64(self.dlogits).T @ V + f64(self.dWr0), F32)
        near(self.Z, X @ f64(self.W).T + f64(self.b), BF16)
        Q, S = ck.pack(f64(self.Z))
        assert np.array_equal(self.QZ.cpu().numpy(), Q) and np.array_equal(self.SZ.cpu().numpy(), S)
        near(self.dZ, f64(self.dY) * slope64(ck.values(Q, S), lg.GEMM_ACT_GELU), BF16)
        near(self.dW, f64(self.dZ).T @ V + f64(self.dW0), F32)


def test_training_step():
    s = Step()
    s.run()
    s.check()


def test_training_step_captured():
    """The step as a graph, replayed on new activations.  (M is above 16: no product of it
    splits K, which would take the library's own workspace.)"""
    s = Step()
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for i in range(3):
        s.X.copy_(torch.randn(s.M, s.K, generator=torch.Generator().manual_seed(i)).bfloat16())
        s.dW.copy_(s.dW0)
        s.dWr.copy_(s.dWr0)
        graph.replay()
        s.check()
        got = s.dW.clone()
        s.dW.copy_(s.dW0)  # eager work between the replays
        s.dWr.copy_(s.dWr0)
        s.run()
        assert torch.equal(s.dW, got)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_served_projection_with_adapters(M):
    """Quantiser, int8 product and adapters in place on its output."""
    K, N, rank, adapters = 256, 200, 16, 5
    g = torch.Generator().manual_seed(M)
    X = torch.randn(M, K, generator=g).bfloat16().cuda()
    W = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    sW = ((torch.rand(N, generator=g) + 0.5) / (64 * K ** 0.5)).cuda()
    A = (torch.randn(adapters * rank, K, generator=g) / K ** 0.5).bfloat16().cuda()
    B = torch.randn(adapters * N, rank, generator=g).bfloat16().cuda()
    ids = torch.randint(-1, adapters, (M,), generator=g).int().cuda()
    Q, sX, Y = empty(M, K, dtype=torch.int8), empty(M), empty(M, N, dtype=torch.bfloat16)
    lora = lg.GemmLora(K, N, adapters, rank, A.data_ptr(), K, B.data_ptr(), rank)
    ws = empty(lg.gemm_lora_workspace(M, lora), dtype=torch.uint8)
    p = lambda t: t.data_ptr()  # noqa: E731

    def serve():
        s = stream()
        ok(lg.gemm_quantize_rows(M, K, p(X), K, BF16, p(Q), K, p(sX), s))
        ok(lg.gemm_run_scaled(M, N, K, p(Q), K, R, p(W), K, C, p(sX), p(sW), 0, N, p(Y), N, lg.GEMM_I8, lg.GEMM_I32,
                              BF16, 0, None, s))
        base = Y.clone()
        ok(lg.gemm_lora_run(M, lora, p(X), K, p(ids), p(Y), N, p(Y), N, BF16, BF16, p(ws), ws.numel(), s))
        return base

    base = serve()
    near(base, (f64(Q) @ f64(W).T) * f64(sX)[:, None] * f64(sW), BF16)
    want = f64(base)
    for t, a in enumerate(ids.tolist()):
        if a >= 0:
            h = f64(A)[a * rank:(a + 1) * rank] @ f64(X)[t]
            want[t] += f64(B)[a * N:(a + 1) * N] @ h
    near(Y, want, BF16)

"""Argument checks of gemm_lora_run on the host: every documented refusal and the
workspace's size (no GPU needed)."""
import pytest

import dense_mixed_precision_tiled_amd as lg

F32, F16, BF16, I8 = lg.GEMM_F32, lg.GEMM_F16, lg.GEMM_BF16, lg.GEMM_I8
# fake, distinct, aligned addresses far apart: the checks never dereference
X0, I0, A0, B0, R0, S0, C0, D0, WS = (0x100000000 * n for n in range(1, 10))


def lora(K=64, N=48, adapters=6, rank=8, A=A0, lda=None, B=B0, ldb=None, ranks=R0, scales=S0):
    return lg.GemmLora(K, N, adapters, rank, A, K if lda is None else lda, B,
                       rank if ldb is None else ldb, ranks, scales)


def check(T=5, m=None, X=X0, ldx=64, ids=I0, C=C0, ldc=48, D=D0, ldd=48, i=BF16, o=BF16, ws=WS,
          size=1 << 30, **kw):
    return lg.gemm_validate_lora(T, lora(**kw) if m is None else m, X, ldx, ids, C, ldc, D, ldd, i,
                                 o, ws, size)


def test_accepts():
    for i in (F16, BF16):
        for o in (F32, F16, BF16):
            assert check(i=i, o=o) == 0
    assert check(C=None, ldc=0) == 0 and check(C=D0) == 0
    assert check(ranks=0, scales=0) == 0 and check(lda=65, ldb=9, ldx=70, ldc=49, ldd=50) == 0
    assert check(T=0, X=None, ids=None, C=None, D=None, ws=None, size=0) == 0
    assert check(rank=256, ldb=256) == 0 and check(adapters=2 ** 20) == 0
    assert check(T=1, ldx=2 ** 24) == 0


def test_refuses():
    assert check(T=-1) == -1 and check(K=0) == -1 and check(N=0) == -1
    assert check(adapters=0) == -1 and check(rank=0) == -1
    assert check(K=2 ** 19 + 1, ldx=2 ** 20) == -1 and check(N=2 ** 19 + 1, ldd=2 ** 20, ldc=2 ** 20) == -1
    assert check(T=2 ** 20 + 1) == -4 and check(adapters=2 ** 20 + 1) == -4 and check(rank=257) == -4
    assert check(i=F32) == -4 and check(i=I8) == -4 and check(o=lg.GEMM_I32) == -4
    assert check(ldx=63) == -2 and check(lda=63) == -2 and check(ldb=7) == -2
    assert check(ldc=47) == -2 and check(ldd=47) == -2 and check(ldx=2 ** 24 + 1) == -2
    for name in ("X", "ids", "D", "ws", "A", "B"):
        assert check(**{name: None}) == -3, name
    assert lg.gemm_validate_lora(1, None, X0, 64, I0, C0, 48, D0, 48, BF16, BF16, WS, 1 << 20) == -3
    for name in ("X", "ids", "A", "B", "ranks", "scales"):
        assert check(**{name: D0 + 16}) == -6, name
        assert check(**{name: WS + 16}) == -6, name
    assert check(C=WS) == -6 and check(C=D0 + 2) == -6 and check(C=D0, ldc=49) == -6
    assert check(ws=D0 + 100) == -6


@pytest.mark.parametrize("T,K,rank", [(1, 64, 1), (16, 4096, 16), (17, 5000, 12), (4096, 4096, 64)])
def test_workspace(T, K, rank):
    m = lora(K=K, rank=rank, ranks=0, scales=0)
    n = lg.gemm_lora_workspace(T, m)
    assert n >= T * rank * 4
    args = dict(T=T, m=m, ldx=K)
    assert check(size=n, **args) == 0 and check(size=n - 1, **args) == -9
    assert lg.gemm_lora_workspace(0, m) >= 0
    assert lg.gemm_lora_workspace(-1, m) == -1 and lg.gemm_lora_workspace(2 ** 20 + 1, m) == -4
    assert lg.gemm_lora_workspace(1, None) == -3

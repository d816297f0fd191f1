"""Argument checks of the checkpoint calls on the host: every documented refusal and the
workspace's size; the format's own definition on known values (no GPU needed)."""
import numpy as np
import pytest

import checkpoint_util as ck
import dense_mixed_precision_tiled_amd as lg

F32, F16, BF16, I8 = lg.GEMM_F32, lg.GEMM_F16, lg.GEMM_BF16, lg.GEMM_I8
# fake, distinct, aligned addresses far apart: the checks never dereference
X0, Q0, S0, D0, G0, C0, WS = (0x100000000 * n for n in range(1, 8))


def pack(M=5, K=70, X=X0, ldx=70, i=BF16, Q=Q0, ldq=70, S=S0, lds=3):
    return lg.gemm_validate_checkpoint_pack(M, K, X, ldx, i, Q, ldq, S, lds)


def unpack(M=5, K=70, Q=Q0, ldq=70, S=S0, lds=3, D=D0, ldd=70, o=BF16):
    return lg.gemm_validate_checkpoint_unpack(M, K, Q, ldq, S, lds, D, ldd, o)


def act(M=5, K=70, Q=Q0, ldq=70, S=S0, lds=3, G=G0, ldg=70, a=lg.GEMM_ACT_GELU, D=D0, ldd=70,
        o=BF16):
    return lg.gemm_validate_checkpoint_act_grad(M, K, Q, ldq, S, lds, G, ldg, a, D, ldd, o)


def wgrad(M=5, N=9, K=70, G=G0, ldg=9, Q=Q0, ldq=70, S=S0, lds=3, C=None, ldc=70, D=D0, ldd=70,
          i=BF16, o=F32, ws=WS, size=1 << 40):
    return lg.gemm_validate_checkpoint_wgrad(M, N, K, G, ldg, Q, ldq, S, lds, C, ldc, D, ldd, i, o,
                                             ws, size)


@pytest.mark.parametrize("check", [pack, unpack, act, wgrad])
def test_common(check):
    assert check() == 0
    assert check(M=-1) == -1 and check(K=-1) == -1 and check(M=2 ** 31) == -1
    assert check(K=2 ** 31) == -1
    assert check(ldq=69) == -2 and check(lds=2) == -2 and check(ldq=2 ** 40 + 1) == -2
    assert check(Q=None) == -3 and check(S=None) == -3
    assert check(K=0, ldq=0) == -2 and check(lds=0) == -2


def test_pack():
    for i in (F32, F16, BF16):
        assert pack(i=i) == 0
    assert pack(i=I8) == -4 and pack(i=lg.GEMM_FP8_E4M3) == -4
    assert pack(ldx=69) == -2 and pack(X=None) == -3
    assert pack(M=0, X=None, Q=None, S=None) == 0
    assert pack(K=0, X=None, Q=None, S=None) == 0
    assert pack(Q=X0 + 8) == -6 and pack(S=X0 + 8) == -6 and pack(S=Q0 + 8) == -6


def test_unpack_and_act_grad():
    for o in (F32, F16, BF16):
        assert unpack(o=o) == 0 and act(o=o) == 0
    assert unpack(o=I8) == -4 and act(o=lg.GEMM_I32) == -4
    for a in (lg.GEMM_ACT_RELU, lg.GEMM_ACT_GELU, lg.GEMM_ACT_SILU):
        assert act(a=a) == 0
    assert act(a=lg.GEMM_ACT_NONE) == -4 and act(a=4) == -4
    assert unpack(ldd=69) == -2 and act(ldd=69) == -2 and act(ldg=69) == -2
    assert unpack(D=None) == -3 and act(D=None) == -3 and act(G=None) == -3
    assert unpack(M=0, Q=None, S=None, D=None) == 0 and act(M=0, Q=None, S=None, D=None, G=None) == 0
    assert unpack(D=Q0) == -6 and unpack(D=S0) == -6 and act(D=S0) == -6
    assert act(D=G0) == 0 and act(D=G0, ldd=72) == -6 and act(D=G0 + 2) == -6


def test_wgrad():
    for i in (F16, BF16):
        for o in (F32, F16, BF16):
            assert wgrad(i=i, o=o) == 0
    assert wgrad(i=F32) == -4 and wgrad(o=lg.GEMM_I32) == -4
    assert wgrad(N=-1) == -1 and wgrad(N=2 ** 31) == -1
    assert wgrad(ldg=8) == -2 and wgrad(ldd=69) == -2 and wgrad(C=C0, ldc=69) == -2
    assert wgrad(ldc=0) == 0                       # no C: its line is not looked at
    assert wgrad(G=None) == -3 and wgrad(D=None) == -3
    assert wgrad(M=0, G=None, Q=None, S=None) == 0  # D = C, or 0
    assert wgrad(M=0, D=None) == -3
    assert wgrad(N=0, D=None, G=None) == 0 and wgrad(K=0, D=None, G=None) == 0
    for name in ("G", "Q", "S"):
        assert wgrad(**{name: D0 + 16}) == -6, name
    assert wgrad(C=D0) == 0 and wgrad(C=D0, ldc=71) == -6 and wgrad(C=D0 + 4) == -6


@pytest.mark.parametrize("M,N,K", [(8192, 16, 4096), (100000, 8, 64), (4096, 128, 128)])
def test_wgrad_workspace(M, N, K):
    need = lg.gemm_checkpoint_wgrad_workspace(M, N, K)
    assert need > 0
    args = dict(M=M, N=N, K=K, ldg=N, ldq=K, lds=K // 32, ldc=K, ldd=K)
    assert wgrad(size=need, **args) == 0 and wgrad(size=need - 1, **args) == -9
    assert wgrad(ws=None, **args) == -3
    for name in ("G", "Q", "S", "D"):
        assert wgrad(**args, **{name: WS + 16}) == -6, name
    assert wgrad(C=WS, **args) == -6


def test_wgrad_without_workspace():
    assert lg.gemm_checkpoint_wgrad_workspace(4096, 4096, 4096) == 0
    assert lg.gemm_checkpoint_wgrad_workspace(0, 16, 16) == 0
    assert lg.gemm_checkpoint_wgrad_workspace(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1) == 0
    assert lg.gemm_checkpoint_wgrad_workspace(-1, 1, 1) == -1
    assert wgrad(ws=None, size=0, M=0) == 0


def test_format():
    # 1.0 opens a block at S = 127, 64 units; the largest values below 2 are held at 127
    Q, S = ck.pack(np.array([[1.0, -0.5, 1 / 128, 3 / 128, 1.99, 127.5 / 64, 0.0]]))
    assert S.tolist() == [[127]]
    assert Q.tolist() == [[64, -32, 0, 2, 127, 127, 0]]
    assert ck.values(Q, S)[0, :4].tolist() == [1.0, -0.5, 0.0, 2 / 64]
    # every value is within half a step, or a whole one where it was held
    x = np.random.default_rng(0).normal(size=(50, 333)) * np.exp(3 * np.random.default_rng(1).normal(size=(50, 1)))
    Q, S = ck.pack(x)
    step = np.repeat(np.ldexp(1.0, S.astype(int) - 133), 32, axis=1)[:, :333]
    err = np.abs(ck.values(Q, S) - x) / step
    assert (err[np.abs(Q) < 127] <= 0.5).all() and (err < 1).all()
    Q, S = ck.pack(np.array([[0.0] * 32 + [np.inf] + [1.0] * 31 + [5e-324]]))
    assert S.tolist() == [[0, 255, 0]] and not Q.any()
    assert np.isnan(ck.values(Q, S)[0, 32:64]).all()

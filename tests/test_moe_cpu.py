"""Argument checks of gemm_moe_run on the host: every documented refusal and
the workspace's size (no GPU needed)."""
import pytest

import dense_mixed_precision_tiled_amd as lg

F16, BF16, I8 = lg.GEMM_F16, lg.GEMM_BF16, lg.GEMM_I8
# fake, distinct, aligned addresses far apart: the checks never dereference
X0, L0, W1, W2, S1, S2, D0, WS = (0x100000000 * n for n in range(1, 9))


def layer(H=64, I=32, E=8, topk=2, w=BF16, ld1=None, ld2=None, W1=W1, W2=W2, s1=0, s2=0,
          act=lg.GEMM_ACT_SILU, renorm=False):
    return lg.GemmMoe(H, I, E, topk, w, W1, H if ld1 is None else ld1, W2,
                      I if ld2 is None else ld2, s1, s2, act, renorm)


def check(T=3, m=None, X=X0, ldx=64, l=L0, ldl=8, D=D0, ldd=64, i=BF16, ws=WS, size=1 << 20, **kw):
    return lg.gemm_validate_moe(T, layer(**kw) if m is None else m, X, ldx, l, ldl, D, ldd, i, ws,
                                size)


def test_accepts():
    assert check() == 0
    assert check(i=F16, w=F16) == 0
    assert check(w=I8, s1=S1, s2=S2) == 0 and check(w=I8, s1=S1, s2=S2, i=F16) == 0
    for act in (lg.GEMM_ACT_SILU, lg.GEMM_ACT_GELU, lg.GEMM_ACT_RELU):
        assert check(act=act, renorm=True) == 0
    assert check(T=64) == 0 and check(ldx=100, ldl=9, ldd=65, ld1=65, ld2=33) == 0
    assert check(T=0, X=None, l=None, D=None, ws=None, size=0) == 0
    assert check(E=1024, topk=32, ldl=1024) == 0


def test_refuses():
    assert check(T=-1) == -1 and check(H=0) == -1 and check(I=0) == -1
    assert check(E=0) == -1 and check(topk=0) == -1 and check(topk=9) == -1
    assert check(H=2 ** 19 + 1) == -1 and check(I=2 ** 19 + 1) == -1
    assert check(T=65) == -4 and check(E=1025, ldl=1025) == -4
    assert check(E=64, topk=33, ldl=64) == -4
    assert check(i=lg.GEMM_F32) == -4 and check(i=F16) == -4      # bf16 weights
    assert check(w=lg.GEMM_FP8_E4M3) == -4 and check(act=lg.GEMM_ACT_NONE) == -4
    assert check(ldx=63) == -2 and check(ldl=7) == -2 and check(ldd=63) == -2
    assert check(ld1=63) == -2 and check(ld2=31) == -2
    assert check(ldx=2 ** 24 + 1) == -2 and check(ld1=2 ** 24) == 0
    for name in ("X", "l", "D", "ws"):
        assert check(**{name: None}) == -3, name
    assert check(W1=0) == -3 and check(W2=0) == -3
    assert check(w=I8, s1=S1) == -3 and check(w=I8, s2=S2) == -3
    assert lg.gemm_validate_moe(1, None, X0, 64, L0, 8, D0, 64, BF16, WS, 1 << 20) == -3
    for name in ("X", "l", "W1", "W2"):
        assert check(**{name: D0 + 16}) == -6, name
        assert check(**{name: WS + 16}) == -6, name
    assert check(w=I8, s1=D0, s2=S2) == -6 and check(w=I8, s1=S1, s2=WS) == -6
    assert check(ws=D0 + 100) == -6


@pytest.mark.parametrize("T,E,topk,I", [(1, 8, 2, 100), (64, 64, 8, 1000), (3, 1000, 32, 7)])
def test_workspace(T, E, topk, I):
    m = layer(E=E, topk=topk, I=I)
    n = lg.gemm_moe_workspace(T, m)
    pairs = T * topk
    # the pairs' inner rows (two values of 16 bits each), and less than 16 bytes for each slot and token beside them
    assert 4 * pairs * I <= n <= 4 * pairs * (I + 7) + 4 * (2 + T) * min(E, pairs) + 4 * pairs + 600
    args = dict(T=T, m=m, ldl=E)
    assert check(size=n, **args) == 0 and check(size=n - 1, **args) == -9
    assert lg.gemm_moe_workspace(0, m) >= 0
    assert lg.gemm_moe_workspace(65, m) == -4 and lg.gemm_moe_workspace(-1, m) == -1
    assert lg.gemm_moe_workspace(1, None) == -3

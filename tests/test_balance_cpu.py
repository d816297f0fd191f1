"""Argument checks of the router's balance on the host: every documented refusal and the
workspace's size (no GPU needed)."""
import pytest

import dense_mixed_precision_tiled_amd as lg

F32, F16, BF16 = lg.GEMM_F32, lg.GEMM_F16, lg.GEMM_BF16
# fake, distinct, aligned addresses far apart: the checks never dereference
L0, M0, O0, N0, S0, D0, G0, WS = (0x100000000 * n for n in range(1, 9))


def forward(T=50, E=8, k=2, l=L0, ldl=8, mask=M0, b=0.01, z=0.001, loss=O0, counts=N0, lse=S0,
            ws=WS, size=1 << 24):
    return lg.gemm_validate_moe_balance(T, E, k, l, ldl, mask, b, z, loss, counts, lse, ws, size)


def grad(T=50, E=8, k=2, l=L0, ldl=8, mask=M0, b=0.01, z=0.001, counts=N0, lse=S0, dloss=G0, D=D0,
         ldd=8, o=F32):
    return lg.gemm_validate_moe_balance_grad(T, E, k, l, ldl, mask, b, z, counts, lse, dloss, D,
                                             ldd, o)


@pytest.mark.parametrize("check", [forward, grad])
def test_common(check):
    assert check() == 0 and check(mask=None) == 0 and check(b=0.0, z=0.0) == 0
    assert check(E=1024, k=32, ldl=1024, **({"ldd": 1024} if check is grad else {})) == 0
    assert check(T=-1) == -1 and check(T=2 ** 31) == -1 and check(E=0) == -1 and check(k=0) == -1
    assert check(k=9) == -1
    assert check(E=1025, ldl=1025) == -4 and check(E=64, k=33, ldl=64) == -4
    for bad in (float("nan"), float("inf"), -float("inf")):
        assert check(b=bad) == -4 and check(z=bad) == -4
    assert check(ldl=7) == -2 and check(ldl=2 ** 40 + 1) == -2
    for name in ("l", "counts", "lse"):
        assert check(**{name: None}) == -3, name


def test_forward():
    for name in ("loss", "ws"):
        assert forward(**{name: None}) == -3, name
    assert forward(T=0, l=None, lse=None) == 0 and forward(T=0, loss=None) == -3
    outs = {"loss": O0, "counts": N0, "lse": S0, "ws": WS}
    for name, at in outs.items():
        for other in ("l", "mask", "loss", "counts", "lse", "ws"):
            if other != name:
                assert forward(**{other: at}) == -6, (name, other)


def test_grad():
    assert grad(dloss=None) == 0
    for o in (F32, F16, BF16):
        assert grad(o=o) == 0
    assert grad(o=lg.GEMM_I8) == -4 and grad(ldd=7) == -2 and grad(D=None) == -3
    assert grad(T=0, l=None, counts=None, lse=None, D=None) == 0
    for name in ("l", "mask", "counts", "lse", "dloss"):
        assert grad(**{name: D0}) == -6, name


@pytest.mark.parametrize("T,E,k", [(0, 1, 1), (1, 8, 2), (1 << 20, 64, 8), (2 ** 31 - 1, 1024, 32)])
def test_workspace(T, E, k):
    n = lg.gemm_moe_balance_workspace(T, E, k)
    assert 0 < n <= 1 << 22
    args = dict(T=T, E=E, k=k, ldl=E, mask=None)
    # (addresses far enough apart for the longest rows)
    assert forward(size=n, l=1 << 50, lse=1 << 51, **args) == 0
    assert forward(size=n - 1, l=1 << 50, lse=1 << 51, **args) == -9
    assert lg.gemm_moe_balance_workspace(-1, E, k) == -1
    assert lg.gemm_moe_balance_workspace(T, 1025, k) == -4

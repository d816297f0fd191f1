"""Argument checks of gemm_quantize_rows and gemm_run_scaled on the host: every
documented refusal, before any HIP call (no GPU needed)."""
import pytest

import dense_mixed_precision_tiled_amd as lg

R, C = lg.GEMM_ROW_MAJOR, lg.GEMM_COL_MAJOR
# fake, distinct, 16-byte aligned addresses: the checks never dereference
A0, B0, C0, D0, SA, SB = (0x10000000 * n for n in range(1, 7))


def scaled(M=8, N=6, K=32, A=A0, lda=None, la=R, B=B0, ldb=None, lb=C, sa=SA, sb=SB, c=None,
           ldc=None, D=D0, ldd=None, i=lg.GEMM_I8, a=lg.GEMM_I32, o=lg.GEMM_BF16, epi=None):
    ld_row = epi is None or epi.layoutD == R
    lda = max(1, K if la == R else M) if lda is None else lda
    ldb = max(1, N if lb == R else K) if ldb is None else ldb
    ldd = max(1, N if ld_row else M) if ldd is None else ldd
    return lg.gemm_validate_scaled(M, N, K, A, lda, la, B, ldb, lb, sa, sb, c,
                                   max(1, N) if ldc is None else ldc, D, ldd, i, a, o, epi)


@pytest.mark.parametrize("out", [lg.GEMM_F32, lg.GEMM_F16, lg.GEMM_BF16])
def test_scaled_accepts(out):
    for la, lb in ((R, C), (R, R), (C, C), (C, R)):
        assert scaled(la=la, lb=lb, o=out) == 0
    assert scaled(sa=None, sb=None, o=out) == 0
    assert scaled(c=C0, o=out) == 0
    assert scaled(c=D0, o=out) == 0                       # in place
    assert scaled(M=0, A=None, B=None, D=None, o=out) == 0
    assert scaled(K=0, A=None, B=None, o=out) == 0
    assert scaled(K=2 ** 17 - 1, o=out) == 0
    epi = lg.GemmEpilogue(0.5, 0.0, 0x70000000, lg.GEMM_ACT_GELU, R, C)
    assert scaled(epi=epi, o=out) == 0


def test_scaled_refuses():
    assert scaled(M=-1) == -1 and scaled(N=2 ** 31) == -1
    assert scaled(lda=31) == -2 and scaled(ldb=31) == -2 and scaled(ldd=5) == -2
    assert scaled(c=C0, ldc=5) == -2
    assert scaled(A=None) == -3 and scaled(B=None) == -3 and scaled(D=None) == -3
    assert scaled(i=lg.GEMM_F16) == -4 and scaled(i=lg.GEMM_FP8_E4M3) == -4
    assert scaled(a=lg.GEMM_F32) == -4 and scaled(o=lg.GEMM_I32) == -4
    assert scaled(K=2 ** 17) == -4                       # the int32 sum could wrap
    assert scaled(epi=lg.GemmEpilogue(activation=9)) == -4
    assert scaled(la=2) == -5 and scaled(lb=-1) == -5
    assert scaled(D=A0 + 16) == -6 and scaled(D=B0) == -6
    assert scaled(c=D0 + 4) == -6
    assert scaled(sa=D0 + 8) == -6 and scaled(sb=D0 + 8) == -6
    assert scaled(sa=D0 - 28) == -6                      # the last of M scales inside D
    assert scaled(sa=D0 - 32) == 0
    assert scaled(epi=lg.GemmEpilogue(bias=D0)) == -6


def quant(M=4, K=40, X=A0, ldx=40, i=lg.GEMM_F16, Q=B0, ldq=48, s=SA):
    return lg.gemm_validate_quantize_rows(M, K, X, ldx, i, Q, ldq, s)


def test_silu_is_for_the_experts_layer_only():
    epi = lg.GemmEpilogue(activation=lg.GEMM_ACT_SILU)
    assert scaled(epi=epi) == -4
    assert lg.gemm_validate_ex(8, 6, 32, A0, 32, R, B0, 32, C, None, 6, D0, 6, lg.GEMM_F16,
                               lg.GEMM_F32, lg.GEMM_F32, epi) == -4


def test_quantize_accepts():
    for t in (lg.GEMM_F16, lg.GEMM_BF16, lg.GEMM_F32):
        assert quant(i=t) == 0
    assert quant(M=0, X=None, Q=None, s=None) == 0
    assert quant(K=0, X=None, Q=None) == 0


def test_quantize_refuses():
    assert quant(M=-1) == -1 and quant(K=-1) == -1 and quant(K=2 ** 31) == -1
    assert quant(ldx=39) == -2 and quant(ldq=39) == -2 and quant(K=0, ldx=0) == -2
    assert quant(X=None) == -3 and quant(Q=None) == -3 and quant(s=None) == -3
    assert quant(K=0, s=None) == -3
    assert quant(i=lg.GEMM_I8) == -4 and quant(i=lg.GEMM_FP8_E5M2) == -4
    assert quant(Q=A0 + 16) == -6 and quant(s=A0) == -6 and quant(s=B0 + 8) == -6

"""Host-side refusals of the single-token calls (no GPU): every bad argument is answered before
anything is launched. The addresses are stand-ins that are never dereferenced."""
import ctypes

import pytest

from w4a4_post_quantized_zigzag_amd import binding as bd

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)
BY4 = ctypes.c_void_p(0x10004)
NULL = None


@pytest.fixture(scope="module")
def L():
    return bd.lib()


def gemv(L, *, X=FAKE, dt=bd.W4A4_F16, M=2, K=256, ldx=256, wt=FAKE, s=FAKE, group=64, N=48, Y=FAKE,
         ldy=48, epi=0, res=NULL, ldr=0):
    return L.w4a4_gemv_w4g(X, dt, M, K, ldx, wt, s, group, N, Y, ldy, epi, res, ldr, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(group=16), bd.W4A4_ERR_UNSUPPORTED),
    (dict(group=0), bd.W4A4_ERR_UNSUPPORTED),
    (dict(group=512), bd.W4A4_ERR_UNSUPPORTED),
    (dict(group=96), bd.W4A4_ERR_UNSUPPORTED),
    (dict(K=224, ldx=224), bd.W4A4_ERR_SHAPE),          # not a multiple of the group
    (dict(K=0), bd.W4A4_ERR_ARG),
    (dict(K=-64), bd.W4A4_ERR_ARG),
    (dict(N=0), bd.W4A4_ERR_ARG),
    (dict(M=-1), bd.W4A4_ERR_ARG),
    (dict(M=(1 << 21) + 1), bd.W4A4_ERR_UNSUPPORTED),
    (dict(K=(1 << 23) + 64, ldx=(1 << 23) + 64), bd.W4A4_ERR_UNSUPPORTED),
    (dict(dt=3), bd.W4A4_ERR_ARG),
    (dict(ldx=255), bd.W4A4_ERR_SHAPE),
    (dict(ldy=47), bd.W4A4_ERR_SHAPE),
    (dict(X=NULL), bd.W4A4_ERR_ARG),
    (dict(Y=NULL), bd.W4A4_ERR_ARG),
    (dict(wt=NULL), bd.W4A4_ERR_ARG),
    (dict(s=NULL), bd.W4A4_ERR_ARG),
    (dict(wt=BY4), bd.W4A4_ERR_ALIGN),
    (dict(s=ODD), bd.W4A4_ERR_ALIGN),
    (dict(X=ODD), bd.W4A4_ERR_ALIGN),
    (dict(X=ctypes.c_void_p(0x10002), dt=bd.W4A4_F32), bd.W4A4_ERR_ALIGN),
    (dict(Y=ODD), bd.W4A4_ERR_ALIGN),
    (dict(epi=3), bd.W4A4_ERR_ARG),
    (dict(epi=bd.EPI_RESIDUAL, ldr=48), bd.W4A4_ERR_ARG),
    (dict(epi=bd.EPI_RESIDUAL, res=FAKE, ldr=47), bd.W4A4_ERR_SHAPE),
    (dict(epi=bd.EPI_RESIDUAL, res=ODD, ldr=48), bd.W4A4_ERR_ALIGN),
])
def test_gemv_w4g_rejects(L, kw, code):
    assert gemv(L, **kw) == code
    assert L.w4a4_last_error() != b""


def test_gemv_w4g_empty_batch(L):
    assert gemv(L, M=0, X=NULL, Y=NULL) == bd.W4A4_OK
    assert gemv(L, M=0, dt=bd.W4A4_BF16) == bd.W4A4_OK


@pytest.mark.parametrize("kw,code", [
    (dict(group=48), bd.W4A4_ERR_UNSUPPORTED),
    (dict(K=320, ldw=320, group=128), bd.W4A4_ERR_SHAPE),
    (dict(N=0), bd.W4A4_ERR_ARG),
    (dict(dt=9), bd.W4A4_ERR_ARG),
    (dict(ldw=128), bd.W4A4_ERR_SHAPE),
    (dict(W=NULL), bd.W4A4_ERR_ARG),
    (dict(wt=NULL), bd.W4A4_ERR_ARG),
    (dict(wt=BY4), bd.W4A4_ERR_ALIGN),
    (dict(s=ODD), bd.W4A4_ERR_ALIGN),
])
def test_pack_w4g_rejects(L, kw, code):
    a = dict(W=FAKE, dt=bd.W4A4_F16, N=32, K=256, ldw=256, group=64, wt=FAKE, s=FAKE) | kw
    assert L.w4a4_pack_weights_w4g(a["W"], a["dt"], a["N"], a["K"], a["ldw"], a["group"], a["wt"], a["s"],
                                   NULL) == code
    assert L.w4a4_last_error() != b""


def test_codes_to_w4g_rejects_and_sizes(L):
    assert L.w4a4_codes_to_w4g(FAKE, 16, 48, FAKE, NULL) == bd.W4A4_ERR_SHAPE
    assert L.w4a4_codes_to_w4g(NULL, 16, 64, FAKE, NULL) == bd.W4A4_ERR_ARG
    assert L.w4a4_codes_to_w4g(FAKE, 16, 64, BY4, NULL) == bd.W4A4_ERR_ALIGN
    assert L.w4a4_codes_to_w4g(FAKE, 0, 64, FAKE, NULL) == bd.W4A4_ERR_ARG
    assert L.w4a4_w4g_operand_bytes(17, 160) == 2 * 2 * 1024
    assert L.w4a4_w4g_operand_bytes(1 << 14, 1 << 14) == 1 << 27
    assert L.w4a4_w4g_operand_bytes(0, 64) == 0


def test_other_calls_still_refuse_bf16(L):
    """bf16 is known to the single-token calls only."""
    assert L.w4a4_rotate_quant_act(FAKE, bd.W4A4_BF16, 16, 256, 256, 64, FAKE, FAKE, FAKE, 8, 0, FAKE,
                                   FAKE, NULL, NULL, 0, NULL) == bd.W4A4_ERR_ARG
    assert L.w4a4_pack_weights(FAKE, bd.W4A4_BF16, 16, 256, 256, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                               1 << 30, NULL) == bd.W4A4_ERR_ARG


def test_binding_refuses_before_the_library():
    import torch
    wt = torch.zeros(1024, dtype=torch.uint8)
    s = torch.ones((1, 16), dtype=torch.float16)
    X = torch.zeros((2, 128), dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        bd.gemv_w4g(X, wt, s)
    with pytest.raises(ValueError, match="wt"):
        bd.gemv_w4g(X, wt[:512], s)
    with pytest.raises(ValueError, match="Y must"):
        bd.gemv_w4g(X, wt, s, Y=torch.zeros((2, 16)))
    with pytest.raises(ValueError, match="residual must"):
        bd.gemv_w4g(X, wt, s, epilogue=bd.EPI_RESIDUAL, residual=torch.zeros((2, 17), dtype=torch.float16))
    with pytest.raises(ValueError, match="groups"):
        bd.gemv_w4g(X[:, :100], wt, torch.ones((3, 16), dtype=torch.float16))
    with pytest.raises(TypeError):
        bd.gemv_w4g(X.double(), wt, s)

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
    (dict(K=1 << 20, ldx=1 << 20, N=1 << 20, ldy=1 << 20), bd.W4A4_ERR_UNSUPPORTED),  # N K above 2^34
    (dict(ldx=(1 << 24) + 8), bd.W4A4_ERR_UNSUPPORTED),
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


# ---- norm, rotation, append --------------------------------------------------------------------

def rope(L, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dt=bd.W4A4_F16, M=4, H=8, KV=2, D=64, ldq=512, ldk=128, ldv=128, qw=FAKE,
             kw=FAKE, eps=1e-6, f=FAKE, rot=64, inter=0, pos=FAKE, qo=FAKE, ldqo=512, ko=NULL, ldko=0,
             kc=FAKE, vc=FAKE, P=10, page=16, stride=2 * 16 * 64, slots=FAKE) | kw
    return L.w4a4_qk_norm_rope(*[a[n] for n in (
        "q", "k", "v", "dt", "M", "H", "KV", "D", "ldq", "ldk", "ldv", "qw", "kw", "eps", "f", "rot",
        "inter", "pos", "qo", "ldqo", "ko", "ldko", "kc", "vc", "P", "page", "stride", "slots")], NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=bd.W4A4_F32), bd.W4A4_ERR_ARG),
    (dict(M=-1), bd.W4A4_ERR_ARG),
    (dict(M=(1 << 25) + 1), bd.W4A4_ERR_UNSUPPORTED),
    (dict(H=0), bd.W4A4_ERR_ARG),
    (dict(KV=0), bd.W4A4_ERR_ARG),
    (dict(D=0), bd.W4A4_ERR_ARG),
    (dict(H=5000), bd.W4A4_ERR_UNSUPPORTED),
    (dict(D=72, rot=0), bd.W4A4_ERR_UNSUPPORTED),
    (dict(D=528, rot=0), bd.W4A4_ERR_UNSUPPORTED),
    (dict(rot=80), bd.W4A4_ERR_SHAPE),
    (dict(rot=8), bd.W4A4_ERR_SHAPE),
    (dict(rot=-16), bd.W4A4_ERR_SHAPE),
    (dict(eps=-1.0), bd.W4A4_ERR_ARG),
    (dict(eps=float("nan")), bd.W4A4_ERR_ARG),
    (dict(ldq=511), bd.W4A4_ERR_SHAPE),
    (dict(ldk=127), bd.W4A4_ERR_SHAPE),
    (dict(ldv=127), bd.W4A4_ERR_SHAPE),
    (dict(ldqo=511), bd.W4A4_ERR_SHAPE),
    (dict(ko=FAKE, ldko=127), bd.W4A4_ERR_SHAPE),
    (dict(q=NULL), bd.W4A4_ERR_ARG),
    (dict(k=NULL), bd.W4A4_ERR_ARG),
    (dict(v=NULL), bd.W4A4_ERR_ARG),
    (dict(qo=NULL), bd.W4A4_ERR_ARG),
    (dict(kc=NULL), bd.W4A4_ERR_ARG),
    (dict(vc=NULL), bd.W4A4_ERR_ARG),
    (dict(kc=NULL, vc=NULL), bd.W4A4_ERR_ARG),           # keys would go nowhere
    (dict(slots=NULL), bd.W4A4_ERR_ARG),
    (dict(pos=NULL), bd.W4A4_ERR_ARG),
    (dict(f=NULL), bd.W4A4_ERR_ARG),
    (dict(P=0), bd.W4A4_ERR_ARG),
    (dict(page=8), bd.W4A4_ERR_UNSUPPORTED),
    (dict(page=48, stride=1 << 16), bd.W4A4_ERR_UNSUPPORTED),
    (dict(page=8192, stride=1 << 30), bd.W4A4_ERR_UNSUPPORTED),
    (dict(stride=2 * 16 * 64 - 8), bd.W4A4_ERR_SHAPE),
    (dict(stride=2 * 16 * 64 + 4), bd.W4A4_ERR_ALIGN),
    (dict(kc=BY4), bd.W4A4_ERR_ALIGN),
    (dict(vc=BY4), bd.W4A4_ERR_ALIGN),
    (dict(q=ODD), bd.W4A4_ERR_ALIGN),
    (dict(f=BY4), bd.W4A4_ERR_ALIGN),
    (dict(pos=BY4), bd.W4A4_ERR_ALIGN),
    (dict(slots=BY4), bd.W4A4_ERR_ALIGN),
    (dict(qw=ODD), bd.W4A4_ERR_ALIGN),
])
def test_qk_norm_rope_rejects(L, kw, code):
    assert rope(L, **kw) == code
    assert L.w4a4_last_error() != b""


def test_qk_norm_rope_empty(L):
    assert rope(L, M=0) == bd.W4A4_OK
    assert rope(L, M=0, kc=NULL, vc=NULL, v=NULL, slots=NULL, q=NULL, k=NULL, qo=NULL) == bd.W4A4_OK


# ---- attention over the cache ------------------------------------------------------------------

def attn(L, **kw):
    a = dict(q=FAKE, dt=bd.W4A4_BF16, B=2, H=8, KV=2, D=64, ldq=512, kc=FAKE, vc=FAKE, P=10, page=16,
             stride=2 * 16 * 64, table=FAKE, width=4, ldt=4, lens=FAKE, max_len=64, scale=0.125, window=0,
             sinks=0, out=FAKE, ldo=512, ws=NULL, wsb=0) | kw
    return L.w4a4_paged_attn_decode(*[a[n] for n in (
        "q", "dt", "B", "H", "KV", "D", "ldq", "kc", "vc", "P", "page", "stride", "table", "width", "ldt",
        "lens", "max_len", "scale", "window", "sinks", "out", "ldo", "ws", "wsb")], NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=bd.W4A4_F32), bd.W4A4_ERR_ARG),
    (dict(B=-1), bd.W4A4_ERR_ARG),
    (dict(B=1 << 16), bd.W4A4_ERR_UNSUPPORTED),
    (dict(B=60000, H=256, ldq=1 << 14, ldo=1 << 14), bd.W4A4_ERR_UNSUPPORTED),  # B heads above 2^23
    (dict(H=0), bd.W4A4_ERR_ARG),
    (dict(H=9, ldq=576, ldo=576), bd.W4A4_ERR_SHAPE),      # heads not a multiple of kv_heads
    (dict(D=80, ldq=640, ldo=640), bd.W4A4_ERR_UNSUPPORTED),
    (dict(D=32), bd.W4A4_ERR_UNSUPPORTED),
    (dict(D=512, ldq=4096, ldo=4096), bd.W4A4_ERR_UNSUPPORTED),
    (dict(ldq=511), bd.W4A4_ERR_SHAPE),
    (dict(ldo=511), bd.W4A4_ERR_SHAPE),
    (dict(q=NULL), bd.W4A4_ERR_ARG),
    (dict(out=NULL), bd.W4A4_ERR_ARG),
    (dict(kc=NULL), bd.W4A4_ERR_ARG),
    (dict(vc=NULL), bd.W4A4_ERR_ARG),
    (dict(table=NULL), bd.W4A4_ERR_ARG),
    (dict(lens=NULL), bd.W4A4_ERR_ARG),
    (dict(P=0), bd.W4A4_ERR_ARG),
    (dict(P=1 << 30, page=4096, stride=1 << 20), bd.W4A4_ERR_UNSUPPORTED),
    (dict(page=24), bd.W4A4_ERR_UNSUPPORTED),
    (dict(page=1), bd.W4A4_ERR_UNSUPPORTED),
    (dict(stride=100), bd.W4A4_ERR_SHAPE),
    (dict(stride=2 * 16 * 64 + 2), bd.W4A4_ERR_ALIGN),
    (dict(kc=BY4), bd.W4A4_ERR_ALIGN),
    (dict(width=0, ldt=0), bd.W4A4_ERR_ARG),
    (dict(ldt=3), bd.W4A4_ERR_SHAPE),
    (dict(width=(1 << 26) + 1, ldt=(1 << 26) + 1), bd.W4A4_ERR_UNSUPPORTED),
    (dict(table=ctypes.c_void_p(0x10002)), bd.W4A4_ERR_ALIGN),
    (dict(lens=ctypes.c_void_p(0x10002)), bd.W4A4_ERR_ALIGN),
    (dict(max_len=-1), bd.W4A4_ERR_ARG),
    (dict(window=-1), bd.W4A4_ERR_ARG),
    (dict(sinks=-1), bd.W4A4_ERR_ARG),
    (dict(scale=float("inf")), bd.W4A4_ERR_ARG),
    (dict(max_len=100000), bd.W4A4_ERR_WORKSPACE),
    (dict(max_len=100000, ws=BY4, wsb=1 << 30), bd.W4A4_ERR_ALIGN),
])
def test_paged_attn_rejects(L, kw, code):
    assert attn(L, **kw) == code
    assert L.w4a4_last_error() != b""


def test_paged_attn_empty_and_workspace(L):
    assert attn(L, B=0, q=NULL, out=NULL, table=NULL, lens=NULL) == bd.W4A4_OK
    assert L.w4a4_paged_attn_workspace_bytes(2, 8, 2, 64, 32, 0, 0) == 0          # nothing to split
    assert attn(L, B=0, q=NULL, out=NULL, table=NULL, lens=NULL, max_len=1 << 30) == bd.W4A4_OK
    big = L.w4a4_paged_attn_workspace_bytes(2, 8, 2, 64, 100000, 0, 0)
    assert big > 0
    # a window bounds what there is to split
    assert L.w4a4_paged_attn_workspace_bytes(2, 8, 2, 64, 100000, 40, 4) < big
    assert L.w4a4_paged_attn_workspace_bytes(2, 9, 2, 64, 100000, 0, 0) == 0


def test_binding_checks_shapes():
    import torch
    q = torch.zeros((2, 4, 64), dtype=torch.float16)
    kc = torch.zeros((3, 2, 16, 64), dtype=torch.float16)
    table, lens = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    call = bd.paged_attn_decode
    with pytest.raises(ValueError, match="GPU"):
        call(q, kc, kc.clone(), table, lens)
    with pytest.raises(ValueError, match="cache"):
        call(q, kc.bfloat16(), kc, table, lens)
    with pytest.raises(ValueError, match="alike"):
        call(q, kc, kc[:2], table, lens)
    with pytest.raises(ValueError, match="dense"):
        t = torch.zeros((3, 16, 2, 64), dtype=torch.float16).transpose(1, 2)
        call(q, t, t, table, lens)
    with pytest.raises(ValueError, match="table"):
        call(q, kc, kc, table.long(), lens)
    with pytest.raises(ValueError, match="lens"):
        call(q, kc, kc, table, lens.long())
    with pytest.raises(ValueError, match="adjacent"):
        call(q[:, ::2], kc, kc, table, lens)
    with pytest.raises(TypeError):
        call(q.float(), kc.float(), kc.float(), table, lens)
    k = torch.zeros((2, 2, 64), dtype=torch.float16)
    w, f, pos = torch.ones(64), torch.ones(32, dtype=torch.float64), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        bd.qk_norm_rope(q, k, w, w, f, pos)
    with pytest.raises(ValueError, match="inv_freq"):
        bd.qk_norm_rope(q, k, w, w, f.float(), pos)
    with pytest.raises(ValueError, match="positions"):
        bd.qk_norm_rope(q, k, w, w, f, pos.int())
    with pytest.raises(ValueError, match="q_weight"):
        bd.qk_norm_rope(q, k, w.half(), w, f, pos)
    with pytest.raises(ValueError, match="slots"):
        bd.qk_norm_rope_append(q, k, k, w, w, f, pos, kc, kc.clone(), pos.int())
    with pytest.raises(ValueError, match="required"):
        bd.qk_norm_rope_append(q, k, None, w, w, f, pos, kc, kc, pos)


@pytest.mark.parametrize("B,H,KV,D,max_len", [(32, 32, 8, 128, 8191), (64, 16, 16, 64, 8000), (1, 8, 1, 256, 20000),
                                              (2, 8, 8, 128, 131071), (4, 4, 2, 96, 65), (3, 40, 2, 192, 5000)])
def test_paged_attn_plans_a_window_that_hides_nothing_as_none(L, B, H, KV, D, max_len):
    """The lengths differ as much as without a window, so the work is split the same way (the workspace is a
    measure of it)."""
    size = lambda window, sinks: L.w4a4_paged_attn_workspace_bytes(B, H, KV, D, max_len, window, sinks)  # noqa: E731
    most = (1 << 31) - 1
    for window, sinks in ((max_len, 0), (max_len - 3, 3), (max_len - 40, 100), (1, max_len), (most, 0), (1, most), (most, most)):
        assert size(window, sinks) == size(0, 0) == size(0, sinks), (window, sinks)

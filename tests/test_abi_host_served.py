"""Host-side refusals of the calls around a quantized cache, a shared prefix and low-rank adapters (no GPU): every bad
argument is answered before anything is launched. The addresses are stand-ins that are never dereferenced."""
import ctypes

import pytest

from w4a4_post_quantized_zigzag_amd import binding as bd

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)
BY2 = ctypes.c_void_p(0x10002)
BY4 = ctypes.c_void_p(0x10004)
BY8 = ctypes.c_void_p(0x10008)
NULL = None
A, S, U, AL, W = (bd.W4A4_ERR_ARG, bd.W4A4_ERR_SHAPE, bd.W4A4_ERR_UNSUPPORTED, bd.W4A4_ERR_ALIGN, bd.W4A4_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def L():
    return bd.lib()


# a cache of 10 pages of 16 tokens, 2 heads of 64, in int8
CACHE = dict(fmt=bd.KV_INT8, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, P=10, page=16, stride=2 * 16 * 64, ss=2 * 16)
CACHE_NAMES = ("fmt", "kc", "vc", "ks", "vs", "P", "page", "stride", "ss")
BAD_CACHE = [
    (dict(fmt=0), A),
    (dict(fmt=3), A),
    (dict(kc=NULL), A),
    (dict(vc=NULL), A),
    (dict(ks=NULL), A),
    (dict(vs=NULL), A),
    (dict(kc=BY8), AL),
    (dict(vc=BY8), AL),
    (dict(ks=BY8), AL),
    (dict(vs=BY8), AL),
    (dict(P=0), A),
    (dict(P=1 << 30, stride=1 << 20, ss=1 << 10), U),
    (dict(P=1 << 30, stride=2048, ss=1 << 20), U),
    (dict(page=8), U),
    (dict(page=24), U),
    (dict(page=8192, stride=1 << 30, ss=1 << 20), U),
    (dict(stride=2 * 16 * 64 - 16), S),
    (dict(stride=2 * 16 * 64 + 8), AL),
    (dict(ss=31), S),
    (dict(ss=34), AL),
    (dict(fmt=bd.KV_FP4, ss=63), S),            # two groups of 32 channels
    (dict(fmt=bd.KV_FP4, ss=72), AL),
    (dict(fmt=bd.KV_FP4, stride=2 * 16 * 32 - 16, ss=64), S),
]


def rope(L, **kw):
    a = CACHE | dict(q=FAKE, k=FAKE, v=FAKE, dt=bd.W4A4_F16, M=4, H=8, KV=2, D=64, ldq=512, ldk=128, ldv=128, qw=FAKE,
                     kw=FAKE, eps=1e-6, f=FAKE, rot=64, inter=0, pos=FAKE, qo=FAKE, ldqo=512, ko=NULL, ldko=0,
                     slots=FAKE) | kw
    return L.w4a4_qk_norm_rope_quant(*[a[n] for n in (
        "q", "k", "v", "dt", "M", "H", "KV", "D", "ldq", "ldk", "ldv", "qw", "kw", "eps", "f", "rot", "inter", "pos",
        "qo", "ldqo", "ko", "ldko", *CACHE_NAMES, "slots")], NULL)


@pytest.mark.parametrize("kw,code", BAD_CACHE + [
    (dict(dt=bd.W4A4_F32), A),
    (dict(M=-1), A),
    (dict(M=(1 << 25) + 1), U),
    (dict(D=80, rot=0), U),
    (dict(D=32, rot=0), U),
    (dict(D=512, rot=0, ldq=4096, ldqo=4096, ldk=1024, ldv=1024), U),
    (dict(rot=80), S),
    (dict(eps=float("nan")), A),
    (dict(ldq=511), S),
    (dict(ldk=127), S),
    (dict(ldv=127), S),
    (dict(ldqo=511), S),
    (dict(ko=FAKE, ldko=127), S),
    (dict(q=NULL), A),
    (dict(k=NULL), A),
    (dict(v=NULL), A),
    (dict(qo=NULL), A),
    (dict(slots=NULL), A),
    (dict(pos=NULL), A),
    (dict(f=NULL), A),
    (dict(v=ODD), AL),
    (dict(slots=BY4), AL),
    (dict(qw=ODD), AL),
])
def test_norm_rope_rejects(L, kw, code):
    assert rope(L, **kw) == code
    assert L.w4a4_last_error() != b""


def append(L, **kw):
    a = CACHE | dict(k=FAKE, v=FAKE, dt=bd.W4A4_BF16, M=4, KV=2, D=64, ldk=128, ldv=128, slots=FAKE) | kw
    return L.w4a4_kv_append_quant(*[a[n] for n in ("k", "v", "dt", "M", "KV", "D", "ldk", "ldv", *CACHE_NAMES, "slots")],
                                  NULL)


def read(L, **kw):
    a = CACHE | dict(k=FAKE, v=FAKE, dt=bd.W4A4_BF16, M=4, KV=2, D=64, ldk=128, ldv=128, slots=FAKE) | kw
    return L.w4a4_kv_read_quant(*[a[n] for n in (*CACHE_NAMES, "slots", "M", "KV", "D", "dt", "k", "ldk", "v", "ldv")],
                                NULL)


ROWS = BAD_CACHE + [
    (dict(dt=bd.W4A4_F32), A),
    (dict(M=-1), A),
    (dict(M=(1 << 25) + 1), U),
    (dict(KV=0), A),
    (dict(KV=5000), U),
    (dict(D=0), A),
    (dict(D=48), U),
    (dict(ldk=127), S),
    (dict(ldv=127), S),
    (dict(k=ODD), AL),
    (dict(v=ODD), AL),
    (dict(slots=NULL), A),
    (dict(slots=BY4), AL),
]


@pytest.mark.parametrize("kw,code", ROWS + [(dict(k=NULL), A), (dict(v=NULL), A)])
def test_append_rejects(L, kw, code):
    assert append(L, **kw) == code
    assert L.w4a4_last_error() != b""


@pytest.mark.parametrize("kw,code", ROWS + [(dict(k=NULL, v=NULL), A)])
def test_read_rejects(L, kw, code):
    assert read(L, **kw) == code
    assert L.w4a4_last_error() != b""


def test_rows_empty(L):
    assert rope(L, M=0) == bd.W4A4_OK
    assert append(L, M=0, k=NULL, v=NULL, slots=NULL) == bd.W4A4_OK
    assert read(L, M=0, k=NULL, v=NULL, slots=NULL) == bd.W4A4_OK
    for D in (64, 96, 128, 192, 256):
        for fmt, row, groups in ((bd.KV_INT8, D, 1), (bd.KV_FP4, D // 2, D // 32)):
            kw = dict(M=0, D=D, fmt=fmt, ldk=2 * D, ldv=2 * D, stride=2 * 16 * row, ss=2 * 16 * groups)
            assert append(L, **kw) == bd.W4A4_OK and read(L, **kw) == bd.W4A4_OK


def attn(L, **kw):
    a = CACHE | dict(q=FAKE, dt=bd.W4A4_BF16, B=2, H=8, KV=2, D=64, ldq=512, table=FAKE, width=4, ldt=4, lens=FAKE,
                     max_len=64, scale=0.125, window=0, sinks=0, out=FAKE, ldo=512, ws=NULL, wsb=0) | kw
    return L.w4a4_paged_attn_decode_quant(*[a[n] for n in (
        "q", "dt", "B", "H", "KV", "D", "ldq", *CACHE_NAMES, "table", "width", "ldt", "lens", "max_len", "scale",
        "window", "sinks", "out", "ldo", "ws", "wsb")], NULL)


def shared(L, **kw):
    a = CACHE | dict(q=FAKE, dt=bd.W4A4_BF16, B=2, H=8, KV=2, D=64, ldq=512, pt=FAKE, pw=3, pl=FAKE, max_prefix=48,
                     table=FAKE, width=4, ldt=4, lens=FAKE, max_len=64, scale=0.125, out=FAKE, ldo=512, ws=FAKE,
                     wsb=1 << 30) | kw
    return L.w4a4_paged_attn_shared(*[a[n] for n in (
        "q", "dt", "B", "H", "KV", "D", "ldq", *CACHE_NAMES, "pt", "pw", "pl", "max_prefix", "table", "width", "ldt",
        "lens", "max_len", "scale", "out", "ldo", "ws", "wsb")], NULL)


ATTN = [
    (dict(dt=bd.W4A4_F32), A),
    (dict(B=-1), A),
    (dict(B=1 << 16), U),
    (dict(B=60000, H=256, ldq=1 << 14, ldo=1 << 14), U),
    (dict(H=0), A),
    (dict(H=9, ldq=576, ldo=576), S),
    (dict(D=80, ldq=640, ldo=640), U),
    (dict(ldq=511), S),
    (dict(ldo=511), S),
    (dict(q=NULL), A),
    (dict(out=NULL), A),
    (dict(table=NULL), A),
    (dict(lens=NULL), A),
    (dict(width=0, ldt=0), A),
    (dict(ldt=3), S),
    (dict(width=(1 << 26) + 1, ldt=(1 << 26) + 1), U),
    (dict(table=BY2), AL),
    (dict(lens=BY2), AL),
    (dict(max_len=-1), A),
    (dict(scale=float("inf")), A),
]


@pytest.mark.parametrize("kw,code", BAD_CACHE + ATTN + [
    (dict(window=-1), A),
    (dict(sinks=-1), A),
    (dict(max_len=100000), W),
    (dict(max_len=100000, ws=BY4, wsb=1 << 30), AL),
])
def test_attn_rejects(L, kw, code):
    assert attn(L, **kw) == code
    assert L.w4a4_last_error() != b""


@pytest.mark.parametrize("kw,code", [(k, c) for k, c in BAD_CACHE if k.get("fmt") != 0] + ATTN + [
    (dict(pt=NULL), A),
    (dict(pl=NULL), A),
    (dict(pt=BY2), AL),
    (dict(pl=BY2), AL),
    (dict(pw=-1), A),
    (dict(max_prefix=-1), A),
    (dict(pw=(1 << 26) + 1), U),
    (dict(ws=NULL), W),
    (dict(wsb=100), W),
    (dict(ws=BY4), AL),
    (dict(fmt=bd.KV_16BIT, ks=NULL, vs=NULL, ss=0, stride=2 * 16 * 64 + 4), AL),
    (dict(fmt=bd.KV_16BIT, ks=NULL, vs=NULL, ss=0, stride=2 * 16 * 64 - 8), S),
])
def test_shared_rejects(L, kw, code):
    assert shared(L, **kw) == code
    assert L.w4a4_last_error() != b""


def test_attn_empty_and_workspaces(L):
    none = dict(B=0, q=NULL, out=NULL, table=NULL, lens=NULL, ws=NULL, wsb=0)
    assert attn(L, **none) == bd.W4A4_OK
    assert shared(L, **none, pt=NULL, pl=NULL) == bd.W4A4_OK
    assert shared(L, **none, pt=NULL, pl=NULL, pw=0, fmt=bd.KV_16BIT, ks=NULL, vs=NULL, ss=0) == bd.W4A4_OK
    f, g = L.w4a4_paged_attn_quant_workspace_bytes, L.w4a4_paged_attn_shared_workspace_bytes
    assert f(2, 8, 2, 64, 32, 0, 0) == 0 and f(2, 8, 2, 64, 100000, 0, 0) > 0
    assert f(2, 9, 2, 64, 100000, 0, 0) == 0 and f(-1, 8, 2, 64, 100, 0, 0) == 0 and f(2, 8, 2, 64, -1, 0, 0) == 0
    assert g(2, 8, 2, 64, 0, 0) > 0                      # the parts are always joined
    assert g(2, 8, 2, 64, -1, 0) == 0 and g(0, 8, 2, 64, 100, 100) == 0
    for B in (1, 7, 64, 4096):                            # never more parts than the join weighs
        for H, KV in ((8, 1), (32, 8), (4, 4)):
            for n in (1, 1000, 1 << 20, 1 << 30):
                assert g(B, H, KV, 64, n, n) <= 256 * B * H * (64 * 4 + 8) + 512


def adapter(L, **kw):
    a = dict(X=FAKE, dt=bd.W4A4_F16, M=4, K=64, ldx=64, A=FAKE, sa=16 * 64, B=FAKE, sb=48 * 16, n=3, R=16, ids=FAKE,
             scale=FAKE, N=48, Y=FAKE, ldy=48, epi=0, res=NULL, ldr=0, out=FAKE, ldo=48, ws=FAKE, wsb=1 << 20) | kw
    return L.w4a4_adapter_add(*[a[n] for n in (
        "X", "dt", "M", "K", "ldx", "A", "sa", "B", "sb", "n", "R", "ids", "scale", "N", "Y", "ldy", "epi", "res", "ldr",
        "out", "ldo", "ws", "wsb")], NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=bd.W4A4_F32), A),
    (dict(M=-1), A),
    (dict(K=0), A),
    (dict(N=0), A),
    (dict(n=0), A),
    (dict(R=0), A),
    (dict(K=60), S),
    (dict(R=12), S),
    (dict(R=264, sa=264 * 64, sb=48 * 264), U),
    (dict(M=(1 << 25) + 1), U),
    (dict(K=(1 << 23) + 8, ldx=1 << 24, sa=1 << 40), U),
    (dict(N=(1 << 24) + 1, ldy=1 << 25, ldo=1 << 25, sb=1 << 40), U),
    (dict(n=1 << 30, sa=1 << 20), U),
    (dict(ldx=63), S),
    (dict(ldy=47), S),
    (dict(ldo=47), S),
    (dict(sa=16 * 64 - 1), S),
    (dict(sb=48 * 16 - 1), S),
    (dict(X=NULL), A),
    (dict(A=NULL), A),
    (dict(B=NULL), A),
    (dict(ids=NULL), A),
    (dict(Y=NULL), A),
    (dict(out=NULL), A),
    (dict(X=ODD), AL),
    (dict(A=ODD), AL),
    (dict(B=ODD), AL),
    (dict(Y=ODD), AL),
    (dict(out=ODD), AL),
    (dict(ids=BY2), AL),
    (dict(scale=BY2), AL),
    (dict(epi=3), A),
    (dict(epi=bd.EPI_RESIDUAL, ldr=48), A),
    (dict(epi=bd.EPI_RESIDUAL, res=FAKE, ldr=47), S),
    (dict(epi=bd.EPI_RESIDUAL, res=ODD, ldr=48), AL),
    (dict(ws=NULL), W),
    (dict(wsb=64), W),
    (dict(ws=BY4), AL),
])
def test_adapter_rejects(L, kw, code):
    assert adapter(L, **kw) == code
    assert L.w4a4_last_error() != b""


def test_adapter_empty_and_workspace(L):
    assert adapter(L, M=0, X=NULL, Y=NULL, out=NULL, ids=NULL, ws=NULL, wsb=0) == bd.W4A4_OK
    f = L.w4a4_adapter_workspace_bytes
    assert f(1, 64, 16) == 256 and f(0, 64, 16) == 0 and f(1, 0, 16) == 0
    assert f(1, 1 << 20, 16) <= 16 * 16 * 4 and f(1 << 20, 4096, 64) >= (1 << 20) * 64 * 4


# ---- the binding, on CPU tensors: shapes and types are refused before the device is looked at ---------------------

def test_binding_caches():
    import torch
    for kind in ("int8", "fp4"):
        for D in (64, 96, 128, 192, 256):
            c = bd.quant_pages(3, 2, 16, D, kind, device="cpu")
            assert isinstance(c, tuple) and len(c) == 4
            x = torch.zeros((5, 2, D), dtype=torch.float16)
            slots = torch.zeros(5, dtype=torch.int64)
            with pytest.raises(ValueError, match="GPU"):
                bd.kv_append_quant(x, x, c, slots)
            with pytest.raises(ValueError, match="GPU"):
                bd.kv_append_quant(x, x, tuple(c), slots)
            with pytest.raises(ValueError, match="GPU"):
                bd.kv_read_quant(c, slots, torch.bfloat16)
            with pytest.raises(ValueError, match="scales must"):
                bd.kv_append_quant(x, x, c._replace(k_scale=c.k_scale[:, :1]), slots)
            with pytest.raises(ValueError, match="laid out alike"):
                bd.kv_append_quant(x, x, c._replace(v=c.v[:2]), slots)
            with pytest.raises(ValueError, match="another number of heads"):
                bd.kv_append_quant(x[:, :1], x[:, :1], c, slots)
            with pytest.raises(ValueError, match="slots"):
                bd.kv_append_quant(x, x, c, slots[:4])
            with pytest.raises(ValueError, match="do not hold"):
                bd.kv_append_quant(x[..., :32].contiguous(), x[..., :32].contiguous(), c, slots)
            with pytest.raises(ValueError, match="dense"):
                bd.kv_append_quant(x, x, c._replace(k=c.k.transpose(0, 2)[:3].transpose(0, 2),
                                                    v=c.v.transpose(0, 2)[:3].transpose(0, 2)), slots)
            with pytest.raises(TypeError):
                bd.kv_append_quant(x.float(), x.float(), c, slots)
            with pytest.raises(TypeError, match="tuple"):
                bd.kv_append_quant(x, x, list(c), slots)
            with pytest.raises(ValueError, match="k_scale"):
                bd.kv_append_quant(x, x, (c.k, c.v), slots)
    with pytest.raises(ValueError, match="int8 or fp4"):
        bd.quant_pages(1, 1, 16, 64, "int4", device="cpu")


def test_binding_attention():
    import torch
    q = torch.zeros((2, 4, 64), dtype=torch.float16)
    c = bd.quant_pages(3, 2, 16, 64, "int8", device="cpu")
    table, lens = torch.zeros((2, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    pt, pl = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for cache in (c, (q.new_zeros((3, 2, 16, 64)),) * 2):
        with pytest.raises(ValueError, match="GPU"):
            bd.paged_attn_shared(q, cache, pt, pl, table, lens)
    with pytest.raises(ValueError, match="GPU"):
        bd.paged_attn_decode_quant(q, c, table, lens)
    with pytest.raises(ValueError, match="table"):
        bd.paged_attn_decode_quant(q, c, table[:1], lens)
    with pytest.raises(ValueError, match="lens"):
        bd.paged_attn_decode_quant(q, c, table, lens.long())
    with pytest.raises(ValueError, match="prefix_len"):
        bd.paged_attn_shared(q, c, pt, lens, table, lens)
    with pytest.raises(ValueError, match="prefix_table"):
        bd.paged_attn_shared(q, c, table, pl, table, lens)
    with pytest.raises(ValueError, match="two tensors"):
        bd.paged_attn_shared(q, (q.new_zeros((3, 2, 16, 64)).bfloat16(),) * 2, pt, pl, table, lens)
    with pytest.raises(ValueError, match="out must"):
        bd.paged_attn_decode_quant(q, c, table, lens, out=q[:1])


def test_binding_adapters():
    import torch
    h = torch.float16
    X, Y = torch.zeros((3, 64), dtype=h), torch.zeros((3, 40), dtype=h)
    A, B = torch.zeros((2, 8, 64), dtype=h), torch.zeros((2, 40, 8), dtype=h)
    ids = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        bd.adapter_add(Y, X, A, B, ids)
    for kw in (dict(A=A[:1]), dict(B=B[:, :, :4]), dict(A=A.bfloat16()), dict(ids=ids.long()), dict(ids=ids[:2]),
               dict(Y=Y[:2]), dict(Y=Y.float()), dict(scale=torch.ones(3)), dict(out=Y[:, :39]), dict(residual=Y.T),
               dict(A=A.transpose(1, 2).contiguous().transpose(1, 2))):
        a = dict(Y=Y, X=X, A=A, B=B, ids=ids) | kw
        with pytest.raises(ValueError):
            bd.adapter_add(**a)
    with pytest.raises(TypeError):
        bd.adapter_add(Y.float(), X.float(), A.float(), B.float(), ids)

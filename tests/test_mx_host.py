"""Argument checks of the microscaled-storage entry points; they run on the
host before any CUDA call, so the pointers below are never dereferenced."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
INVALID, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from layer_streamed_qlora_b200 import _lib, build
    build.build()
    return _lib


def test_scale_stride(L):
    assert [L.soup_mx4_scale_stride(i) for i in (32, 512, 544, 4096)] == [16, 16, 32, 128]


def test_scale_stride_is_the_librarys(L):
    f = L.lib().soup_mx4_scale_stride
    assert all(L.soup_mx4_scale_stride(i) == f(i) for i in (-32, 0, 1, 31, 32, 512, 513, 544, 4096, 14336, 1 << 29))


def test_quantise_refusals(L):
    f = L.lib().soup_mx4_quantize

    def call(W=P(0x1000), typ=0, out=4, inp=64, ldw=64, codes=P(0x2000), scales=P(0x3000), values=None):
        return f(W, typ, out, inp, ldw, codes, scales, values, None, None)

    assert call(W=None) == INVALID and call(codes=None) == INVALID and call(scales=None) == INVALID
    assert call(typ=2) == INVALID
    assert call(inp=48, ldw=48) == SHAPE and call(out=0) == SHAPE and call(inp=0) == SHAPE and call(ldw=32) == SHAPE
    assert call(out=1 << 29, inp=1 << 20, ldw=1 << 20) == SHAPE
    assert call(W=P(0x1004)) == ALIGN and call(ldw=66) == ALIGN and call(values=P(0x4008)) == ALIGN
    assert call(typ=1, ldw=68) == ALIGN


def test_dequant_refusals(L):
    f = L.lib().soup_mx4_dequant
    assert f(None, P(16), 4, 64, P(16), None) == INVALID
    assert f(P(16), P(16), 4, 40, P(16), None) == SHAPE
    assert f(P(16), P(16), 4, 64, P(24), None) == ALIGN


def _weight(L, **kw):
    d = dict(kind=L.SOUP_WEIGHT_MXFP4, out_features=64, in_features=96, codes=0x1000, scales=0x2000) | kw
    return L.SoupWeight(d["kind"], d["out_features"], d["in_features"], d["codes"], None, None, d["scales"])


@pytest.mark.parametrize("fn", ["soup_linear_fwd", "soup_linear_bwd"])
def test_linear_refusals(L, fn):
    f = getattr(L.lib(), fn)

    def call(W=None, a=P(0x1000), lda=96, T=4, c=P(0x2000), ldc=96, ws=None, nws=0):
        return f(ctypes.byref(W or _weight(L)), a, lda, T, c, ldc, ws, nws, None)

    assert f(None, P(16), 96, 4, P(16), 96, None, 0, None) == INVALID
    assert call(T=0, a=None, c=None) == 0
    assert call(T=-1) == SHAPE and call(T=1 << 31) == SHAPE
    assert call(a=None) == INVALID and call(c=None) == INVALID
    assert call(lda=56) == SHAPE and call(ldc=56) == SHAPE
    assert call(lda=100) == ALIGN and call(a=P(0x1008)) == ALIGN and call(ldc=100) == ALIGN
    assert call(ws=P(0x1010), nws=1 << 20) == ALIGN and call(ws=None, nws=1 << 20) == ALIGN
    assert call(W=_weight(L, kind=3)) == INVALID and call(W=_weight(L, scales=None)) == INVALID
    assert call(W=_weight(L, in_features=80)) == SHAPE and call(W=_weight(L, out_features=56)) == SHAPE
    assert call(W=_weight(L, codes=0x1008)) == ALIGN and call(W=_weight(L, scales=0x2008)) == ALIGN


def test_linear_wrapper_refuses_host_tensors_and_shapes(L):
    W = _weight(L)
    x, y = torch.zeros(4, 96, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not on the current CUDA device"):
        L.soup_linear_fwd(W, x, y)
    with pytest.raises(ValueError, match="must be"):
        L.soup_linear_fwd(W, x, y[:3])
    with pytest.raises(ValueError, match="must be"):
        L.soup_linear_bwd(W, x, y)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        L.soup_mx4_quantize(x.half(), None, None)


def test_weight_refuses_short_or_wrong_buffers(L):
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)
    codes, scales = u8((64, 48)), u8((64, 16))
    assert L.weight_mxfp4(codes, scales, 64, 96).scales == scales.data_ptr()
    for c, s in ((codes[:63], scales), (codes, u8((64, 3))), (codes.int(), scales), (codes, scales.float()),
                 (u8((64, 96))[:, :48], scales)):
        with pytest.raises(ValueError, match="weight_mxfp4"):
            L.weight_mxfp4(c, s, 64, 96)


def test_layer_blob_holds_the_scales(L):
    cfg = L.LayerCfg(256, 2, 1, 128, 640, 16, 32.0, 1e-5, 5e5, 0, 0)
    w = L.soup_layer_blob_views(cfg, L.SOUP_WEIGHT_MXFP4, 0)
    assert w.down.in_features == 640 and w.down.scales - w.down.codes == 256 * 320
    assert w.norm1 - w.down.scales == 256 * 32  # 20 scale bytes a row, padded to 32
    full = L.LayerCfg(4096, 32, 8, 128, 14336, 16, 32.0, 1e-5, 5e5, 0, 0)
    mx, nf = (L.soup_layer_blob_bytes(full, k) for k in (L.SOUP_WEIGHT_MXFP4, L.SOUP_WEIGHT_NF4))
    n = 6144 * 4096 + 4096 * 4096 + 28672 * 4096 + 4096 * 14336
    assert mx == n // 2 + n // 32 + 2 * 8192 and nf - mx == n // 32


def _tensor(L, k, n=100, **kw):
    base = 0x100000 * (k + 1)
    d = {name: base + 0x10000 * i for i, name in
         enumerate(("theta", "theta_bf16", "grad", "m", "v", "m_scale", "v_scale"))} | kw
    return L.AdamWTensor(n, *(d[x] for x in ("theta", "theta_bf16", "grad", "m", "v", "m_scale", "v_scale")))


def test_group_refusals(L):
    lib = L.lib()
    h = L.AdamWGroupHandle()

    def init(ts, bits=8, grad=0, tables=P(0x10), nbytes=1 << 20):
        arr = (L.AdamWTensor * max(1, len(ts)))(*ts)
        return lib.soup_adamw_group_init(arr, len(ts), bits, grad, tables, nbytes, ctypes.byref(h), None)

    one = _tensor(L, 0)
    assert init([]) == SHAPE and init([one], bits=16) == INVALID and init([one], grad=3) == INVALID
    assert init([_tensor(L, 0, n=-1)]) == SHAPE
    assert init([_tensor(L, 0, theta=None)]) == INVALID and init([_tensor(L, 0, v_scale=None)]) == INVALID
    assert init([_tensor(L, 0, m=0x130004)]) == ALIGN
    assert init([one, one]) == INVALID and b"overlap" in lib.soup_last_error()
    # the second tensor's gradient starts inside the first one's
    assert init([one, _tensor(L, 1, grad=0x120000 + 0x100)]) == INVALID
    assert init([one], nbytes=8) == INVALID and init([one], tables=None) == INVALID and init([one], tables=P(8)) == ALIGN

    step = lib.soup_adamw_group_step
    h.tables, h.n_chunks, h.state_bits, h.grad_type = 0x10, 1, 8, 0
    ok = dict(lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, gs=1.0, t=1)

    def call(**kw):
        return step(ctypes.byref(h), *(ok | kw).values(), 0, 0, None, None)

    assert call(t=0) == INVALID and call(b1=1.0) == INVALID and call(b2=-0.1) == INVALID
    assert call(eps=0.0) == INVALID and call(lr=-1.0) == INVALID and call(wd=-1.0) == INVALID
    h.tables = None
    assert call() == INVALID

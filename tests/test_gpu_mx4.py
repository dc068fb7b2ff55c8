"""GPU parity of the MXFP4 storage: quantisation and dequantisation bit for bit
against the oracle, the frozen products against 64-bit sums, and LoRA linear,
decoder layer and streamed model over an MXFP4 base bit for bit against the
same over a bf16 base that holds the stored values."""
import numpy as np
import pytest
import torch

import soup_synth as ss
from oracle import mx
from oracle.lora import lora_bwd, lora_fwd
from tests.gpu_util import assert_close, dev_bf16, dev_f32, host

pytestmark = pytest.mark.gpu
L = None


@pytest.fixture(scope="module", autouse=True)
def _lib():
    global L
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_streamed_qlora_b200 import _lib as lib
    lib.lib()
    L = lib
    yield
    assert lib.device_error() == 0


def quantize(W, values=False, nonfinite=None):
    out_f, in_f = W.shape
    codes = torch.full((out_f, in_f // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((out_f, mx.scale_stride(in_f)), 0xEE, dtype=torch.uint8, device="cuda")
    Wb = torch.empty((out_f, in_f), dtype=torch.bfloat16, device="cuda") if values else None
    L.soup_mx4_quantize(W, codes, scales, Wb, nonfinite)
    return codes, scales, Wb


def special_weights():
    """Ties, saturation, zeros of both signs, extreme and non-finite blocks."""
    W = np.zeros((9, 160), np.float32)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99, 0.0, -0.0], np.float32)
    W[0, :36] = np.concatenate([ties, np.nextafter(ties, np.float32(9)), -np.nextafter(ties, np.float32(-9))])
    W[0, 31] = 4.0
    W[1, :32] = 2.0 ** -149 * np.arange(32)
    W[2, :32] = 2.0 ** -126 * np.linspace(0.5, 4, 32)
    W[3, :32] = np.float32(3.4028235e38)
    W[4, 5] = np.nan
    W[5, 40] = -np.inf
    W[6, :] = np.linspace(-3, 3, 160)
    W[7, 64:96] = -0.0
    W[8, ::7] = 2.0 ** -130
    return W


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (257, 544), (64, 4096)])
def test_quantise_bit_exact(shape, dtype):
    W = dev_f32(ss.normal_f32(3, f"mx.{shape}", shape, std=0.02)).to(dtype)
    codes, scales, Wb = quantize(W, values=True)
    oc, os_ = mx.mx4_quantize(W.float().cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), oc)
    assert np.array_equal(scales.cpu().numpy(), os_)
    assert np.array_equal(Wb.double().cpu().numpy(), mx.mx4_dequant(oc, os_))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantise_special_values_and_strided_rows(dtype):
    S = special_weights()
    W = torch.full((9, 192), float("nan"), dtype=dtype, device="cuda")
    W[:, :160] = torch.from_numpy(S).cuda()
    W = W[:, :160]                    # row stride 192: what lies between rows is not read
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales, Wb = quantize(W, True, flag)
    oc, os_ = mx.mx4_quantize(W.float().cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), oc) and np.array_equal(scales.cpu().numpy(), os_)
    assert np.array_equal(Wb.double().cpu().numpy(), mx.mx4_dequant(oc, os_), equal_nan=True)
    assert flag.item() == 1
    flag.zero_()
    quantize(W[6:8], nonfinite=flag)
    assert flag.item() == 0


def test_dequantise_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()            # [256, 256]: every byte
    scales = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 16).contiguous().cuda()
    Wb = torch.empty((256, 512), dtype=torch.bfloat16, device="cuda")
    L.soup_mx4_dequant(codes, scales, 256, 512, Wb)
    want = mx.mx4_dequant(codes.cpu().numpy(), scales.cpu().numpy())
    big = np.abs(want) >= 2.0 ** 128  # beyond bf16
    want[big] = np.sign(want[big]) * np.inf
    assert np.array_equal(Wb.double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_buffers_aligned_to_16_bytes_only(dtype):
    """W, codes, scales and the stored values 16 but not 32 bytes into their storage, rows too: the aligned bits."""
    out_f, in_f, e = 37, 544, 16 // dtype.itemsize
    whole = torch.randn((out_f, in_f + e), device="cuda").to(dtype)
    W = whole[:, e:]                  # row stride 16 bytes beyond a multiple of 32
    assert W.data_ptr() % 32 == 16
    ss_ = mx.scale_stride(in_f)
    flat = lambda n, t, skip: torch.full((n + 64,), 7, dtype=t, device="cuda")[skip:skip + n]
    codes, scales = flat(out_f * in_f // 2, torch.uint8, 16), flat(out_f * ss_, torch.uint8, 16)
    Wb, Wd = flat(out_f * in_f, torch.bfloat16, 8), flat(out_f * in_f, torch.bfloat16, 8)
    L.soup_mx4_quantize(W, codes, scales, Wb)
    L.soup_mx4_dequant(codes, scales, out_f, in_f, Wd)
    c0, s0, W0 = quantize(W.contiguous(), values=True)
    assert torch.equal(codes.view_as(c0), c0) and torch.equal(scales.view_as(s0), s0)
    assert torch.equal(Wb.view_as(W0), W0) and torch.equal(Wd, Wb)
    x = torch.randn((40, in_f), device="cuda").to(torch.bfloat16)
    for T in (3, 40):
        y = torch.empty((T, out_f // 16 * 16), dtype=torch.bfloat16, device="cuda")
        L.soup_linear_fwd(L.weight_mxfp4(codes, scales, out_f // 16 * 16, in_f), x[:T], y)
        check_product(y, x[:T], W0[:out_f // 16 * 16].T, "y")


def test_offsets_beyond_32_bits():
    """More than 2^32 weights: the last rows quantise, dequantise and multiply as they do on their own."""
    out_f, in_f, n = 131_200, 32_768, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    W = torch.empty((out_f, in_f), dtype=torch.bfloat16, device="cuda")
    for r in range(0, out_f, 8200):
        W[r:r + 8200] = torch.randn((8200, in_f), generator=g, device="cuda") * 0.02
    codes, scales, _ = quantize(W)
    c0, s0, last = quantize(W[-n:].contiguous(), values=True)
    assert torch.equal(codes[-n:], c0) and torch.equal(scales[-n:], s0)
    L.soup_mx4_dequant(codes, scales, out_f, in_f, W)
    assert torch.equal(W[-n:], last)
    del W
    w = L.weight_mxfp4(codes, scales, out_f, in_f)
    for T in (1, 40, 1100):
        ws = torch.empty(L.soup_linear_workspace(w, T), dtype=torch.uint8, device="cuda")
        x = torch.randn((T, in_f), generator=g, device="cuda").to(torch.bfloat16)
        y = torch.empty((T, out_f), dtype=torch.bfloat16, device="cuda")
        L.soup_linear_fwd(w, x, y, workspace=ws)
        check_product(y[:, -n:], x, last.T, f"y, T={T}")
        dy = torch.zeros((T, out_f), dtype=torch.bfloat16, device="cuda")
        dy[:, -n:] = torch.randn((T, n), generator=g, device="cuda")
        dx = torch.empty((T, in_f), dtype=torch.bfloat16, device="cuda")
        L.soup_linear_bwd(w, dy, dx, workspace=ws)
        check_product(dx, dy[:, -n:], last, f"dx, T={T}")


def mx_weight(out_f, in_f, seed=5, std=0.02):
    W = torch.from_numpy(ss.normal_f32(seed, f"w{out_f}x{in_f}", (out_f, in_f), std=std)).cuda()
    codes, scales, Wb = quantize(W, values=True)
    # what pads a row of scales is read by nothing
    scales[:, in_f // 32:] = 0xFF
    return L.weight_mxfp4(codes, scales, out_f, in_f), Wb, (codes, scales)


def check_product(got, a, B, name):
    """|got - a B| <= half a bf16 step of the result + K fp32 steps (2^-23) of the sum of magnitudes: each of
    the K additions is off by at most one step of a partial sum, which that sum bounds."""
    a, B = a.double(), B.double()
    want = a @ B
    bound = 2.0 ** -8 * want.abs() + a.shape[1] * 2.0 ** -23 * (a.abs() @ B.abs()) + 2.0 ** -133
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), name
    over = ((got.double() - want).abs() / bound)[fine].max().item() if fine.any() else 0.0
    assert over <= 1, f"{name}: {over} of the bound"


@pytest.mark.parametrize("T,out_f,in_f", [(1, 16, 32), (1, 4096, 4096), (2, 272, 96), (5, 1040, 4128), (8, 48, 2048),
                                          (16, 512, 1056), (17, 2048, 512), (33, 80, 160), (64, 768, 3104),
                                          (100, 4096, 544), (128, 144, 64), (129, 528, 8224), (300, 2048, 11008),
                                          (515, 272, 2016), (1024, 6144, 4096), (1025, 272, 2016), (1100, 2064, 8224),
                                          (2049, 528, 544)])
@pytest.mark.parametrize("workspace", [False, True])
def test_products_against_64_bits(T, out_f, in_f, workspace):
    W, Wb, keep = mx_weight(out_f, in_f)
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda n: torch.randn((T, n), generator=g, device="cuda").to(torch.bfloat16)
    ws = None
    if workspace:  # contents need no initialisation
        ws = torch.full((L.soup_linear_workspace(W, T),), 0x5A, dtype=torch.uint8, device="cuda")
    # strided rows; what lies between them stays
    x, dy = rand(in_f + 24), rand(out_f + 8)
    y = torch.full((T, out_f + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full((T, in_f + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        L.soup_linear_fwd(W, x[:, :in_f], y[:, :out_f], workspace=ws)
        L.soup_linear_bwd(W, dy[:, :out_f], dx[:, :in_f], workspace=ws)
        check_product(y[:, :out_f], x[:, :in_f], Wb.T, "y")
        check_product(dx[:, :in_f], dy[:, :out_f], Wb, "dx")
    assert (y[:, out_f:] == 7).all() and (dx[:, in_f:] == 7).all()
    y1 = y.clone()
    L.soup_linear_fwd(W, x[:, :in_f], y[:, :out_f], workspace=ws)
    assert torch.equal(y, y1)  # the same bits on every run


@pytest.mark.parametrize("kind", ["nf4", "bf16"])
@pytest.mark.parametrize("T", [1, 200, 600])
def test_products_of_the_other_storages(kind, T):
    out_f, in_f = 528, 2048
    W32 = torch.from_numpy(ss.normal_f32(7, "other", (out_f, in_f), std=0.02)).cuda()
    if kind == "nf4":
        codes = torch.empty((out_f, in_f // 2), dtype=torch.uint8, device="cuda")
        absmax = torch.empty((out_f, in_f // 64), dtype=torch.float32, device="cuda")
        L.soup_nf4_quantize(W32, codes, absmax, torch.zeros(1, dtype=torch.int32, device="cuda"))
        Wb = torch.empty((out_f, in_f), dtype=torch.bfloat16, device="cuda")
        L.soup_nf4_dequant(codes, absmax, out_f, in_f, Wb)
        W = L.weight_nf4(codes, absmax, out_f, in_f)
    else:
        Wb = W32.to(torch.bfloat16)
        W = L.weight_bf16(Wb)
    x, dy = (torch.randn((T, n), device="cuda").to(torch.bfloat16) for n in (in_f, out_f))
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    ws = torch.empty(L.soup_linear_workspace(W, T), dtype=torch.uint8, device="cuda")
    L.soup_linear_fwd(W, x, y, workspace=ws)
    L.soup_linear_bwd(W, dy, dx, workspace=ws)
    check_product(y, x, Wb.T, "y")
    check_product(dx, dy, Wb, "dx")


@pytest.mark.parametrize("T", [3, 12, 40, 1100])
@pytest.mark.parametrize("byte", [1, 129, 200, 253])
def test_products_with_extreme_scales(T, byte):
    """Block scales far from 1: subnormal stored values, and scales above 2 (a second factor in the decode)."""
    out_f, in_f = 48, 160
    W, Wb, (codes, scales) = mx_weight(out_f, in_f)
    scales[:, :5] = byte
    scales[::3, 1] = 120
    L.soup_mx4_dequant(codes, scales, out_f, in_f, Wb)
    for a, B, f, n in ((in_f, Wb.T, L.soup_linear_fwd, out_f), (out_f, Wb, L.soup_linear_bwd, in_f)):
        # inputs that bring the products of the extreme scale back to about 1
        x = (torch.randn((T, a), device="cuda") * 2.0 ** max(-100, min(100, 127 - byte))).to(torch.bfloat16)
        y = torch.empty((T, n), dtype=torch.bfloat16, device="cuda")
        f(W, x, y)
        check_product(y, x, B, f"T={T} scale byte {byte}")


def test_products_with_no_tokens_and_non_finite_inputs():
    W, Wb, keep = mx_weight(64, 128)
    e = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    L.soup_linear_fwd(W, e, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    x = torch.randn((3, 128), device="cuda").to(torch.bfloat16)
    x[1, 5] = float("nan")
    keep[1][7, 1] = 255  # one block of row 7 is NaN
    y = torch.empty((3, 64), dtype=torch.bfloat16, device="cuda")
    L.soup_linear_fwd(W, x, y)
    nan = torch.isnan(y)
    assert nan[1].all() and nan[:, 7].all()
    nan[1], nan[:, 7] = False, False
    assert not nan.any()


@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
def test_products_with_less_workspace(kind):
    """Any size of workspace is allowed; what lies behind it stays."""
    W, Wb, keep = mx_weight(2064, 8224)
    if kind == "bf16":
        Wb = Wb[:, :8192].contiguous()  # a weight holds pointers, not tensors
        W = L.weight_bf16(Wb)
    in_f = Wb.shape[1]
    x = torch.randn((1100, in_f), device="cuda").to(torch.bfloat16)
    full = L.soup_linear_workspace(W, 1100)
    assert full > 4 << 20
    for n in (1, 3000, 600_000, 1 << 20, full // 2 + 17, full):
        buf = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        y = torch.empty((1100, 2064), dtype=torch.bfloat16, device="cuda")
        L.soup_linear_fwd(W, x, y, workspace=buf[:n])
        check_product(y, x, Wb.T, f"{n} bytes")
        assert (buf[n:] == 0x5A).all()


@pytest.mark.parametrize("T", [1, 13, 77, 1027])
def test_products_leave_the_rows_behind_the_tokens(T):
    """Rows beyond T are neither read (NaN there) nor written."""
    W, Wb, keep = mx_weight(272, 96)
    x = torch.full((T + 300, 96), float("nan"), dtype=torch.bfloat16, device="cuda")
    dy = torch.full((T + 300, 272), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[:T], dy[:T] = torch.randn((T, 96), device="cuda"), torch.randn((T, 272), device="cuda")
    y, dx = torch.full_like(dy, 7.0), torch.full_like(x, 7.0)
    L.soup_linear_fwd(W, x[:T], y[:T])
    L.soup_linear_bwd(W, dy[:T], dx[:T])
    check_product(y[:T], x[:T], Wb.T, "y")
    check_product(dx[:T], dy[:T], Wb, "dx")
    assert (y[T:] == 7).all() and (dx[T:] == 7).all()


@pytest.mark.parametrize("T,in_f", [(1, 4096), (40, 4096), (300, 4096), (1100, 8192)])
def test_products_captured_replayed_and_concurrent(T, in_f):
    """Replays of one graph give the first run's bits, and two calls with a workspace each may overlap (1100 x 8192
    cuts its tiles along K and so uses the workspace)."""
    W, Wb, keep = mx_weight(2048, in_f)
    xs = [torch.randn((T, in_f), device="cuda").to(torch.bfloat16) for _ in range(2)]
    ys = [torch.empty((T, 2048), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    wss = [torch.empty(L.soup_linear_workspace(W, T), dtype=torch.uint8, device="cuda") for _ in range(2)]
    for x, y, ws in zip(xs, ys, wss):
        L.soup_linear_fwd(W, x, y, workspace=ws)
    torch.cuda.synchronize()
    want = [y.clone() for y in ys]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.soup_linear_fwd(W, xs[0], ys[0], workspace=wss[0])
    for _ in range(3):
        ys[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[0], want[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for y in ys:
        y.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, x, y, ws in zip(streams, xs, ys, wss):
            L.soup_linear_fwd(W, x, y, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for y, w in zip(ys, want))


@pytest.mark.parametrize("T", [1, 50])
def test_a_chain_of_launches_sees_what_came_before(T):
    """Each launch may start while the one before it ends: a chain in which every call reads what the last one
    wrote, and one overwrites what the last one read, gives the bits of the calls made one by one; eagerly, and
    captured with a fork and a join."""
    n = 1024
    W0 = torch.randn((n, n), device="cuda") * 0.03
    new = lambda: dict(codes=torch.zeros((n, n // 2), dtype=torch.uint8, device="cuda"),
                       scales=torch.zeros((n, n // 32), dtype=torch.uint8, device="cuda"),
                       Wb=torch.zeros((n, n), dtype=torch.bfloat16, device="cuda"),
                       x=torch.ones((T, n), dtype=torch.bfloat16, device="cuda"),
                       y=torch.zeros((T, n), dtype=torch.bfloat16, device="cuda"),
                       z=torch.zeros((T, n), dtype=torch.bfloat16, device="cuda"))

    def chain(b, between):
        w = L.weight_mxfp4(b["codes"], b["scales"], n, n)
        side = torch.cuda.Stream()
        L.soup_mx4_quantize(W0, b["codes"], b["scales"])
        for _ in range(4):
            between()
            L.soup_linear_fwd(w, b["x"], b["y"])
            between()
            side.wait_stream(torch.cuda.current_stream())
            L.soup_linear_bwd(w, b["y"], b["z"], stream=side)       # reads y
            L.soup_mx4_dequant(b["codes"], b["scales"], n, n, b["Wb"])
            torch.cuda.current_stream().wait_stream(side)
            between()
            L.soup_linear_fwd(w, b["z"], b["x"])                    # overwrites the first product's input
            between()
            L.soup_mx4_quantize(b["Wb"], b["codes"], b["scales"])   # overwrites the weight just read
            between()
            L.soup_mx4_dequant(b["codes"], b["scales"], n, n, b["Wb"])

    want = new()
    chain(want, torch.cuda.synchronize)
    torch.cuda.synchronize()
    got = new()
    torch.cuda.synchronize()
    chain(got, lambda: None)
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    assert torch.isfinite(got["x"]).all() and got["x"].any()
    cap = new()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain(cap, lambda: None)
    for _ in range(3):
        cap["x"].fill_(1)
        for k in ("codes", "scales", "Wb"):
            cap[k].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(cap[k], want[k]) for k in want)


@pytest.mark.parametrize("T,in_f", [(64, 512), (1, 512), (300, 544)])
def test_lora_linear_over_mxfp4(T, in_f):
    out_f, r, s = 512, 8, 2.0
    W, Wb, keep = mx_weight(out_f, in_f)
    vals = lambda name, shape, std=1.0: ss.to_bf16_values(ss.normal_f32(9, name, shape, std=std))
    x, dy = vals("x", (T, in_f)), vals("dy", (T, out_f))
    A, B = vals("A", (r, in_f), 0.02), vals("B", (out_f, r), 0.02)
    xd, Ad, Bd, dyd = (dev_bf16(a) for a in (x, A, B, dy))
    y = torch.empty((T, out_f), dtype=torch.bfloat16, device="cuda")
    u = torch.zeros((r, (T + 7) // 8 * 8), dtype=torch.bfloat16, device="cuda")
    L.soup_lora_linear_fwd(W, Ad, Bd, r, s, xd, T, y, u)
    dx = torch.empty((T, in_f), dtype=torch.bfloat16, device="cuda")
    dA, dB = torch.empty((r, in_f), device="cuda"), torch.empty((out_f, r), device="cuda")
    ws = torch.empty(L.soup_lora_linear_bwd_workspace(T, r, out_f), dtype=torch.uint8, device="cuda")
    L.soup_lora_linear_bwd(W, Ad, Bd, r, s, xd, u, dyd, T, dx, dA, dB, ws)
    Wd = host(Wb)
    ry, ru = lora_fwd(x, Wd, A, B, s)
    rdx, rdA, rdB = lora_bwd(x, Wd, A, B, s, dy)
    for got, want, name in ((y, ry, "y"), (dx, rdx, "dx"), (dA, rdA, "dA"), (dB, rdB, "dB")):
        assert_close(host(got), want, name)


SMALL = ss.LayerShape(hidden=512, n_q_heads=4, n_kv_heads=2, head_dim=128, intermediate=1024, rank=16, alpha=32.0,
                      eps=1e-5, theta=5e5, vocab=512, n_layers=1)
ODD_KV = ss.LayerShape(hidden=256, n_q_heads=3, n_kv_heads=1, head_dim=128, intermediate=640, rank=16, alpha=32.0,
                       eps=1e-5, theta=5e5, vocab=512, n_layers=1)


@pytest.mark.parametrize("shape,B,S", [(SMALL, 2, 64), (SMALL, 3, 200), (ODD_KV, 1, 77)])
def test_layer_over_mxfp4_equals_bf16_layer_of_the_stored_values(shape, B, S):
    """Forward, saved activations' backward and recompute backward: the fused decode gives the bf16 operand."""
    from tests.layer_fixture import DevLayer
    dl = DevLayer(L, shape, seed=2, kind="bf16")
    keep, packed, plain = [], [], []
    for name in ("qkv", "o", "gate_up", "down"):
        W = dev_f32(dl.W_oracle[name])
        codes, scales, Wb = quantize(W, values=True)
        keep += [codes, scales, Wb]
        packed.append(L.weight_mxfp4(codes, scales, *W.shape))
        plain.append(L.weight_bf16(Wb))
    norms = (dl.norm1.data_ptr(), dl.norm2.data_ptr())
    T, H = B * S, shape.hidden
    h = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    dh = torch.randn((T, H), device="cuda")
    ws = torch.empty(L.soup_decoder_layer_workspace(dl.cfg, B, S), dtype=torch.uint8, device="cuda")
    got = []
    for w in (packed, plain):
        W = L.LayerWeights(*w, *norms)
        out, dhi = torch.empty_like(h), torch.empty_like(dh)
        L.soup_decoder_layer_fwd(W, dl.lora, dl.cfg, h, B, S, out, True, ws)
        L.soup_decoder_layer_bwd(W, dl.lora, dl.cfg, h, dh, B, S, dhi, dl.grads, True, ws)
        torch.cuda.synchronize()
        got.append([out, dhi] + [g.clone() for g in dl.grads_t.values()])
    for a, b in zip(*got):
        assert torch.equal(a, b)


class StoredValues:
    """Weights whose projections are the MXFP4 values of another source's."""

    def __init__(self, source):
        self.source = source

    def __getattr__(self, name):
        return getattr(self.source, name)

    def layer(self, l):
        w = dict(self.source.layer(l))
        for k in ("qkv", "o", "gate_up", "down"):
            w[k] = quantize(w[k].contiguous(), values=True)[2].float()
        return w


@pytest.mark.parametrize("source", ["ram", "disk"])
def test_streamed_model_over_mxfp4(source, tmp_path):
    """A streamed SFT step over an MXFP4 base (RAM and disk tiers) equals the step over the stored values in
    bf16, bit for bit; its optimiser step with 8-bit states moves the factors."""
    import dataclasses
    from layer_streamed_qlora_b200 import model as M
    from tests.model_fixture import NumpyWeights
    cfg = M.ModelConfig(hidden=512, n_q_heads=4, n_kv_heads=2, head_dim=128, intermediate=1024, rank=16, alpha=32.0,
                        vocab=512, n_layers=3, kind="mxfp4")
    w = NumpyWeights(cfg, 0)
    ids = torch.from_numpy(ss.uniform_ids(1, "ids", (2, 64), cfg.vocab).astype(np.int32))
    got = []
    for kind, weights in (("mxfp4", w), ("bf16", StoredValues(w))):
        extra = dict(stream_source=source, shard_dir=str(tmp_path)) if source == "disk" and kind == "mxfp4" else {}
        m = M.StreamedLoRAModel(dataclasses.replace(cfg, kind=kind), 2, 64, n_buffers=2, weights=weights,
                                head_chunk=48, adamw=M.AdamW(state_bits=8, seed=4), **extra)
        try:
            m.set_ids(ids)
            loss = float(m.sft_step().item())
            grads = m.grad_flat.clone()
            before = m.master_flat.clone()
            m.optimizer_step()
            torch.cuda.synchronize()
            assert m.adam_m.dtype == torch.uint8 and not m.grad_flat.any() and m.nonfinite.item() == 0
            moved = m.master_flat != before
            assert moved[grads != 0].float().mean() > 0.99 and not moved[grads == 0].any()
            assert torch.equal(m.lora_flat, m.master_flat.to(torch.bfloat16))
            got.append((loss, grads, m.master_flat.clone(), m.adam_v.clone()))
        finally:
            m.close()
    assert got[0][0] == got[1][0] and all(torch.equal(a, b) for a, b in zip(got[0][1:], got[1][1:]))


def test_streamed_model_refuses_non_finite_weights_and_state_bits():
    from layer_streamed_qlora_b200 import model as M
    from tests.model_fixture import NumpyWeights
    cfg = M.ModelConfig(hidden=512, n_q_heads=4, n_kv_heads=2, head_dim=128, intermediate=1024, rank=16, alpha=32.0,
                        vocab=512, n_layers=1, kind="mxfp4")
    w = NumpyWeights(cfg, 0)
    with pytest.raises(ValueError, match="state_bits"):
        M.StreamedLoRAModel(cfg, 2, 64, weights=w, adamw=M.AdamW(state_bits=16))
    w.f32[0]["up"][3, 4] = np.nan
    with pytest.raises(ValueError, match="non-finite"):
        M.StreamedLoRAModel(cfg, 2, 64, weights=w, head_chunk=48)

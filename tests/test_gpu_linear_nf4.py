"""Frozen products over NF4 and bf16 weights, exact: sizes that end inside a
tile of the one-CTA and the CTA-pair kernels in both directions (rows of W that
are no multiple of 64, columns that no tile width divides)."""
import pytest
import torch

from tests.exact_products import integers, product

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


def weight(kind, out_f, in_f, g):
    """A weight of -s, 0 and s with s = 1 or 2 per block of 64 (codes 0, 7 and 15 of NF4), and its values."""
    W = integers((out_f, in_f), g, 1).float().view(out_f, -1, 64)
    W[..., 0] = 1.0
    W = (W * torch.randint(1, 3, (out_f, in_f // 64, 1), generator=g, device="cuda")).view(out_f, in_f)
    if kind == "bf16":
        return L.weight_bf16(W.to(torch.bfloat16)), W
    codes = torch.empty((out_f, in_f // 2), dtype=torch.uint8, device="cuda")
    absmax = torch.empty((out_f, in_f // 64), dtype=torch.float32, device="cuda")
    L.soup_nf4_quantize(W, codes, absmax, torch.zeros(1, dtype=torch.int32, device="cuda"))
    Wb = torch.empty((out_f, in_f), dtype=torch.bfloat16, device="cuda")
    L.soup_nf4_dequant(codes, absmax, out_f, in_f, Wb)
    assert torch.equal(Wb.float(), W)
    return L.weight_nf4(codes, absmax, out_f, in_f), W


@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("out_f", [16, 80, 528, 1040])
@pytest.mark.parametrize("in_f", [64, 128, 192, 256, 320, 448, 1088, 2048])
@pytest.mark.parametrize("kind", ["nf4", "bf16"])
def test_products(kind, in_f, out_f, T):
    g = torch.Generator(device="cuda").manual_seed(in_f + out_f + T)
    W, values = weight(kind, out_f, in_f, g)
    x, dy = integers((T, in_f), g), integers((T, out_f + 8), g)[:, :out_f]
    y = torch.full((T, out_f + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full((T, in_f + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    L.soup_linear_fwd(W, x, y[:, :out_f])
    L.soup_linear_bwd(W, dy, dx[:, :in_f])
    assert torch.equal(y[:, :out_f], product(x, values.T))
    assert torch.equal(dx[:, :in_f], product(dy, values))
    assert (y[:, out_f:] == 7).all() and (dx[:, in_f:] == 7).all()


@pytest.mark.parametrize("out_f,in_f", [(80, 192), (528, 320), (272, 1088), (64, 64)])
def test_lora_linear_gradient_of_such_sizes(out_f, in_f):
    """The same transposed products with the adapter's K block behind them (an adapter of zeros)."""
    T, r = 40, 8
    g = torch.Generator(device="cuda").manual_seed(out_f)
    W, values = weight("nf4", out_f, in_f, g)
    x, dy = integers((T, in_f), g), integers((T, out_f), g)
    A, B = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((r, in_f), (out_f, r)))
    y, dx, u = torch.empty_like(dy), torch.empty_like(x), torch.zeros((r, T), dtype=torch.bfloat16, device="cuda")
    dA, dB = torch.empty((r, in_f), device="cuda"), torch.empty((out_f, r), device="cuda")
    ws = torch.empty(L.soup_lora_linear_bwd_workspace(T, r, out_f), dtype=torch.uint8, device="cuda")
    L.soup_lora_linear_fwd(W, A, B, r, 2.0, x, T, y, u)
    L.soup_lora_linear_bwd(W, A, B, r, 2.0, x, u, dy, T, dx, dA, dB, ws)
    assert torch.equal(y, product(x, values.T)) and torch.equal(dx, product(dy, values))
    assert not dA.any() and not dB.any()

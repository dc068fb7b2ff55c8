"""Frozen products over MXFP4 weights with exact sums, bit for bit: every kernel
and both sides of the rules that choose between them, K from one block to
32,768, few tokens through projections of many rows, strided rows, and offsets
beyond 32 bits."""
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


def values_of(codes, scales, in_f):
    """fp32 values by the format's definition: (-1)^S 2^(max(E, 1) - 1) (E > 0 + M / 2) 2^(s - 127)."""
    n = torch.stack((codes & 15, codes >> 4), dim=-1).view(codes.shape[0], in_f).int()
    E, M = (n >> 1) & 3, n & 1
    v = torch.exp2((E.clamp_min(1) - 1).float()) * ((E > 0).float() + 0.5 * M)
    s = torch.exp2(scales[:, :in_f // 32].float() - 127.0).repeat_interleave(32, 1)
    return torch.where(n >= 8, -v, v) * s


def weight(out_f, in_f, g):
    """Random codes of every kind with block scales 1 and 2, and the values (multiples of 1/2 up to 12)."""
    codes = torch.randint(0, 256, (out_f, in_f // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(127, 129, (out_f, L.soup_mx4_scale_stride(in_f)), generator=g, device="cuda",
                           dtype=torch.uint8)
    scales[:, in_f // 32:] = 0xFF  # what pads a row of scales is read by nothing
    return L.weight_mxfp4(codes, scales, out_f, in_f), values_of(codes, scales, in_f), codes, scales


def run(f, W, x, n, pad, ws=None):
    """f's product [T, n] into rows of n + pad elements, what lies between them untouched."""
    y = torch.full((x.shape[0], n + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    f(W, x, y[:, :n], workspace=ws)
    assert (y[:, n:] == 7).all()
    return y[:, :n]


def both(T, out_f, in_f, workspace=True):
    g = torch.Generator(device="cuda").manual_seed(T + out_f + in_f)
    W, values, *_ = weight(out_f, in_f, g)
    ws = None
    if workspace:
        ws = torch.full((L.soup_linear_workspace(W, T),), 0x5A, dtype=torch.uint8, device="cuda")
    x, dy = integers((T, in_f + 16), g)[:, :in_f], integers((T, out_f + 8), g)[:, :out_f]
    assert torch.equal(run(L.soup_linear_fwd, W, x, out_f, 40, ws), product(x, values.T))
    assert torch.equal(run(L.soup_linear_bwd, W, dy, in_f, 8, ws), product(dy, values))


@pytest.mark.parametrize("T", [8, 9, 13, 16, 17])
@pytest.mark.parametrize("rows", ["16 per SM", "one tile more", 4096, 6144, 28672])
def test_few_tokens_on_both_sides_of_the_row_limit(T, rows):
    """9 to 16 tokens take another kernel where the rows are more than 16 for each SM; K ends inside a k-block."""
    limit = 16 * torch.cuda.get_device_properties(0).multi_processor_count
    out_f = {"16 per SM": limit, "one tile more": limit + 16}.get(rows, rows)
    both(T, out_f, 4128 if out_f < 28672 else 544)


@pytest.mark.parametrize("T", [1, 5, 12, 16, 33, 100, 256, 257, 1024, 1025, 2100])
@pytest.mark.parametrize("out_f,in_f", [(16, 32), (144, 96), (272, 2016), (2064, 1056), (5136, 544)])
@pytest.mark.parametrize("workspace", [False, True])
def test_products(T, out_f, in_f, workspace):
    both(T, out_f, in_f, workspace)


@pytest.mark.parametrize("T", [1, 8, 12, 16, 40, 300, 1024, 1100])
@pytest.mark.parametrize("out_f,in_f", [(144, 32768), (2400, 32768), (32784, 160)])
def test_long_sums(T, out_f, in_f):
    """K of 32,768 in the forward (512 k-blocks) and of 32,784 in the backward."""
    both(T, out_f, in_f)


@pytest.mark.parametrize("T", [9, 13, 16])
@pytest.mark.parametrize("byte", [1, 129, 200, 240])
def test_extreme_scales_of_few_tokens_through_many_rows(T, byte):
    """One block in three has a scale far from 1, and is met by zeros or, in the last token, by the power of two that
    brings it back: the decode's second factor and bf16's subnormals, exact."""
    out_f, in_f = 4096, 192
    g = torch.Generator(device="cuda").manual_seed(byte)
    W, values, codes, scales = weight(out_f, in_f, g)
    scales[:, 2], scales[:, 5] = byte, byte
    values = values_of(codes, scales, in_f)
    x = integers((T, in_f), g)
    x[:, 64:96] = 0
    x[:, 160:] = 0
    x[-1] = 0
    x[-1, 64:96] = 2.0 ** (127 - byte) if byte < 250 else 0
    want = x.double() @ values.double().T
    got = run(L.soup_linear_fwd, W, x, out_f, 8)
    assert torch.equal(got, want.float().to(torch.bfloat16))


def test_offsets_beyond_32_bits():
    """More than 2^32 weights: the last rows multiply as they do on their own, in both directions."""
    out_f, in_f, n = 131_200, 32_768, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    codes = torch.empty((out_f, in_f // 2), dtype=torch.uint8, device="cuda")
    for r in range(0, out_f, 8200):
        codes[r:r + 8200] = torch.randint(0, 256, (8200, in_f // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(127, 129, (out_f, in_f // 32), generator=g, device="cuda", dtype=torch.uint8)
    W, last = L.weight_mxfp4(codes, scales, out_f, in_f), values_of(codes[-n:], scales[-n:], in_f)
    for T in (1, 16, 40, 1100):
        ws = torch.empty(L.soup_linear_workspace(W, T), dtype=torch.uint8, device="cuda")
        x = integers((T, in_f), g)
        y = run(L.soup_linear_fwd, W, x, out_f, 8, ws)
        assert torch.equal(y[:, -n:], product(x, last.T)), T
        dy = torch.zeros((T, out_f), dtype=torch.bfloat16, device="cuda")
        dy[:, -n:] = integers((T, n), g)
        dx = run(L.soup_linear_bwd, W, dy, in_f, 8, ws)
        assert torch.equal(dx, product(dy[:, -n:], last)), T

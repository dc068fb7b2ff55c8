"""A subnormal second moment next to a small eps: what the step may take for
zero depends on the bias correction that multiplies its root."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("g,beta2,eps", [(4e-16, 1 - 2.0 ** -24, 2e-12), (3e-18, 0.999, 3e-17), (3e-18, 0.999, 1e-10),
                                         (1e-16, 1 - 2.0 ** -20, 1.01e-12), (2e-17, 0.999, 1.1e-12), (1e-3, 0.999, 1e-8)])
def test_first_step_with_small_gradients(bits, g, beta2, eps):
    """theta = -lr g / (sqrt(v) / sqrt(1 - beta2) + eps) from a zero state, v = (1 - beta2) g^2 as fp32 holds it.
    The errors: v's rounding where it is subnormal (half of 2^-149) and, by half of each relative one in the root,
    two roundings of v; 2^-21 of the update for quotient, root, sum and products and 4 of 2^-24 for the constants
    and the bias-corrected m; half a step of theta."""
    from layer_streamed_qlora_b200 import _lib as L
    f = lambda x: float(np.float32(x))
    n, lr = 64, 1e-3
    t = dict(theta=torch.zeros(n, device="cuda"), grad=torch.full((n,), g, device="cuda"))
    for k in ("m", "v"):
        if bits == 32:
            t[k] = torch.zeros(n, device="cuda")
        else:
            t[k] = torch.zeros(n, dtype=torch.uint8, device="cuda")
            t[k + "_scale"] = torch.zeros(n // 32, dtype=torch.uint8, device="cuda")
    L.AdamWGroup([t], bits).step(lr, 0.9, beta2, eps, 0.0, 1.0, 1)
    b2 = f(beta2)
    root = np.sqrt((1 - b2) * f(g) ** 2)
    c = 1 / np.sqrt(1 - b2)
    want = -f(lr) * f(g) / (root * c + f(eps))
    droot = c * (2.0 ** -150 / (2 * root) + 2.0 ** -24 * root)  # of the bias-corrected root
    bound = abs(want) * (droot / (root * c + f(eps)) + 2.0 ** -21 + 4 * 2.0 ** -24) + 2.0 ** -24 * abs(want)
    got = t["theta"].double().cpu().numpy()
    assert (np.abs(got - want) <= bound).all(), (got[0], want, np.abs(got - want).max() / bound)


@pytest.mark.parametrize("eps", [1e-8, 1e-30])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
def test_32_bit_update_is_within_its_bound(eps, grad):
    """From theta = 0, theta is the documented update of the new m and v, which the step also returns, to 2^-21."""
    from layer_streamed_qlora_b200 import _lib as L
    n, t = 1 << 18, 9
    rng = np.random.default_rng(0)
    new = lambda std: torch.from_numpy((rng.standard_normal(n) * std).astype(np.float32)).cuda()
    d = dict(theta=torch.zeros(n, device="cuda"), grad=new(1e-3).to(grad), m=new(1e-3), v=new(1e-3).square())
    L.AdamWGroup([d], 32).step(3e-3, 0.9, 0.999, eps, 0.05, 1.0, t)
    f = lambda x: float(np.float32(x))
    m, v, got = (d[k].double().cpu().numpy() for k in ("m", "v", "theta"))
    step, c = f(f(3e-3) / (1 - f(0.9) ** t)), f(1 / np.sqrt(1 - f(0.999) ** t))
    want = -step * m / (np.sqrt(v) * c + f(eps))
    assert (np.abs(got - want) <= 2.0 ** -21 * np.abs(want)).all()

"""The AdamW step over a group of tensors against the oracle: 32-bit states
against 64-bit arithmetic, 8-bit states code for code against the same fp32
operations on the CPU, and over many steps against fp32 states."""
import numpy as np
import pytest
import torch

from oracle import mx
from oracle.nf4 import round_to_bf16

pytestmark = pytest.mark.gpu
L = None
HP = dict(lr=3e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.05, grad_scale=0.25)
TABLE = {"m": mx.E4M3, "v": mx.E5M2}
SIZES = [1, 31, 32, 33, 2047, 2048, 2049, 0, 5000, 16, 100_003]


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


def make(n, bits, grad, rng, bf16=True):
    spread = np.exp2(rng.uniform(-10, 4, n))
    t = {"theta": rng.standard_normal(n) * 0.02, "grad": rng.standard_normal(n) * 1e-3 * spread}
    t["grad"][rng.random(n) < 0.05] = 0.0
    t = {k: torch.from_numpy(v.astype(np.float32)).cuda() for k, v in t.items()}
    t["grad"] = t["grad"].to(grad)
    if bf16:
        t["theta_bf16"] = t["theta"].to(torch.bfloat16)
    m, r = rng.standard_normal(n) * 1e-4 * spread, np.abs(rng.standard_normal(n)) * 3e-4 * spread
    if bits == 32:
        t["m"], t["v"] = (torch.from_numpy(a.astype(np.float32)).cuda() for a in (m, r * r))
    else:
        for k, a in (("m", m), ("v", r * r)):
            c, s = mx.state_encode_nearest(a, TABLE[k])
            t[k], t[k + "_scale"] = torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()
    return t


def snapshot(t):
    return {k: (v.float() if v.dtype == torch.bfloat16 else v).cpu().numpy().copy() for k, v in t.items()}


def moments32(t0, t, hp):
    """The step's new theta, m and v in fp32, operation by operation."""
    f = np.float32
    b1, b2, lr, eps, wd, gs = (f(hp[k]) for k in ("beta1", "beta2", "lr", "eps", "weight_decay", "grad_scale"))
    g = t0["grad"].astype(np.float32) * gs
    if t0["m"].dtype == np.uint8:
        m, v = (mx.state_decode(t0[k], t0[k + "_scale"], TABLE[k]).astype(np.float32) for k in ("m", "v"))
    else:
        m, v = t0["m"], t0["v"]
    m = m * b1 + g * f(1.0 - float(b1))
    v = v * b2 + (g * g) * f(1.0 - float(b2))
    denom = np.sqrt(v) * f(1.0 / np.sqrt(1.0 - float(b2) ** t)) + eps
    p = t0["theta"] * f(1.0 - float(lr) * float(wd)) - f(float(lr) / (1.0 - float(b1) ** t)) * (m / denom)
    return p, m, v


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("zero", [False, True])
def test_32_bit_states(grad, zero):
    rng = np.random.default_rng(0)
    ts = [make(n, 32, grad, rng, bf16=i % 3 != 1) for i, n in enumerate(SIZES)]
    before = [snapshot(t) for t in ts]
    L.AdamWGroup(ts, 32).step(**HP, t=9, zero_grad=zero)
    torch.cuda.synchronize()
    for t0, t in zip(before, ts):
        hp = {k: float(np.float32(v)) for k, v in HP.items()}
        g = t0["grad"].astype(np.float64) * hp["grad_scale"]
        m = hp["beta1"] * t0["m"].astype(np.float64) + (1 - hp["beta1"]) * g
        v = hp["beta2"] * t0["v"].astype(np.float64) + (1 - hp["beta2"]) * g * g
        up = hp["lr"] / (1 - hp["beta1"] ** 9) * m / (np.sqrt(v / (1 - hp["beta2"] ** 9)) + hp["eps"])
        th = t0["theta"] * (1 - hp["lr"] * hp["weight_decay"]) - up
        now = snapshot(t)
        # three fp32 roundings of terms no larger than the magnitudes below (and three of the constants)
        sm = np.abs(t0["m"]) + np.abs(g)
        assert (np.abs(now["m"] - m) <= 6 * 2.0 ** -24 * sm).all()
        assert (np.abs(now["v"] - v) <= 6 * 2.0 ** -24 * v + 1e-45).all()
        # theta: decay and subtraction (and the decay's constant); the update: m's error over the denominator
        # and sixteen fp32 half steps for its quotient, root, sum, products and the constants' roundings
        derr = hp["lr"] / (1 - hp["beta1"] ** 9) * 6 * 2.0 ** -24 * sm / (np.sqrt(v / (1 - hp["beta2"] ** 9)) + hp["eps"])
        assert (np.abs(now["theta"] - th) <= 4 * 2.0 ** -24 * np.abs(t0["theta"]) + 16 * 2.0 ** -24 * np.abs(up) + derr).all()
        if "theta_bf16" in now:
            np.testing.assert_array_equal(now["theta_bf16"], round_to_bf16(now["theta"]))
        np.testing.assert_array_equal(now["grad"], 0 * t0["grad"] if zero else t0["grad"])


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("zero", [False, True])
def test_8_bit_states_code_for_code(grad, zero):
    """Every operation up to the codes is one correctly rounded fp32 operation, so the codes are equal.  theta
    is not: its update's quotient, root, sum and products are off by up to eight fp32 steps of 2^-23 (2^-20), the
    decayed parameter by one rounding, the difference by another of a result below their sum."""
    rng = np.random.default_rng(1)
    ts = [make(n, 8, grad, rng, bf16=i % 3 != 1) for i, n in enumerate(SIZES)]
    before = [snapshot(t) for t in ts]
    L.AdamWGroup(ts, 8).step(**HP, t=70_001, seed=99, zero_grad=zero)
    torch.cuda.synchronize()
    for k, (t0, t) in enumerate(zip(before, ts)):
        n = t0["theta"].size
        p, m, v = moments32(t0, 70_001, HP)
        now = snapshot(t)
        up = np.abs(p - t0["theta"] * np.float32(1.0 - HP["lr"] * HP["weight_decay"]))
        assert (np.abs(now["theta"].astype(np.float64) - p) <= 2.0 ** -20 * up + 2.0 ** -22 * np.abs(t0["theta"])).all()
        if "theta_bf16" in now:
            np.testing.assert_array_equal(now["theta_bf16"], round_to_bf16(now["theta"]))
        rnd = mx.random16(n, k, 99, 70_001)
        for name, x in (("m", m), ("v", v)):
            c, s = mx.state_encode_stochastic(x.astype(np.float64), rnd, TABLE[name], keep_nonzero=name == "v")
            np.testing.assert_array_equal(now[name + "_scale"], s)
            np.testing.assert_array_equal(now[name], c)
        np.testing.assert_array_equal(now["grad"], 0 * t0["grad"] if zero else t0["grad"])


def test_first_step_from_zero_states_and_zero_gradients():
    n = 4096
    z = lambda *a: torch.zeros(*a, dtype=torch.uint8, device="cuda")
    t = dict(theta=torch.randn(n, device="cuda"), grad=torch.randn(n, device="cuda"), m=z(n), v=z(n),
             m_scale=z(n // 32), v_scale=z(n // 32))
    t["grad"][:1024] = 0.0
    th = t["theta"].clone()
    L.AdamWGroup([t], 8).step(1e-3, 0.9, 0.999, 1e-8, 0.0, 1.0, 1)
    # bias-corrected first step: theta - lr sign(g) (eps and a few roundings aside), nothing where g = 0
    want = th - 1e-3 * torch.sign(t["grad"])
    assert torch.allclose(t["theta"], want, rtol=0, atol=1e-6)
    assert torch.equal(t["theta"][:1024], th[:1024])
    assert not t["m"][:1024].any() and not t["v_scale"][:32].any()


def test_non_finite_gradients_stay_in_their_element():
    n = 256
    rng = np.random.default_rng(2)
    for bits in (8, 32):
        t = make(n, bits, torch.float32, rng)
        t["grad"][5], t["grad"][100] = float("nan"), float("inf")
        ref = {k: v.clone() for k, v in t.items()}
        ref["grad"][5], ref["grad"][100] = 0.0, 0.0
        flag, flag0 = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
        L.AdamWGroup([t], bits).step(**HP, t=3, seed=1, nonfinite=flag)
        L.AdamWGroup([ref], bits).step(**HP, t=3, seed=1, nonfinite=flag0)
        assert flag.item() == 1 and flag0.item() == 0
        others = [i for i in range(n) if i // 32 not in (0, 3)]
        for k in ("theta", "m", "v"):
            assert torch.equal(t[k][others], ref[k][others])
        if bits == 8:
            assert (t["m"][[5, 100]] & 0x7F == 0x7F).all() and (t["v"][[5, 100]] == 0x7F).all()
            assert (t["v"] == 0x7F).sum() == 2


@pytest.mark.parametrize("bits", [8, 32])
def test_same_bits_on_every_run_stream_and_replay(bits):
    def fresh():
        return [make(n, bits, torch.float32, np.random.default_rng(3)) for n in (777, 4096, 9)]

    runs = []
    for how in ("plain", "plain", "stream", "graph"):
        ts = fresh()
        g = L.AdamWGroup(ts, bits)
        if how == "stream":
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            g.step(**HP, t=5, seed=7, stream=s)
            s.synchronize()
        elif how == "graph":
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                g.step(**HP, t=5, seed=7)
            graph.replay()
        else:
            g.step(**HP, t=5, seed=7)
        torch.cuda.synchronize()
        runs.append(ts)
    for ts in runs[1:]:
        for a, b in zip(runs[0], ts):
            assert all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)


def test_8_bit_moments_follow_the_gradients():
    """From m = 0 and a second moment 100 times too large, 3000 steps of constant gradient g: fp32 states reach
    m = g and decay to v = g^2 (1 + 99 e^-3) = 5.93 g^2; rounding to nearest would leave m near 0.65 g and v at
    100 g^2.  The stored mean is unbiased.  Its noise: a step adds to an element a variance below the distance it
    moves times a code step, so over the decay by a factor 17 of v, in parts of v, below ln(17) / 4 (steps of at
    most 1/4), and for m less: a relative deviation below 0.9, of the mean over 4096 elements 0.014; 5 of them."""
    n = 4096
    z = lambda *a: torch.zeros(*a, dtype=torch.uint8, device="cuda")
    c, s = mx.state_encode_nearest(np.full(n, 1e-4), mx.E5M2)
    t = dict(theta=torch.zeros(n, device="cuda"), grad=torch.full((n,), 1e-3, device="cuda"), m=z(n),
             v=torch.from_numpy(c).cuda(), m_scale=z(n // 32), v_scale=torch.from_numpy(s).cuda())
    v0 = float(mx.state_decode(c[:1], s[:1], mx.E5M2)[0])
    g = L.AdamWGroup([t], 8)
    for step in range(1, 3001):
        g.step(0.0, 0.9, 0.999, 1e-8, 0.0, 1.0, step, seed=5)
    m, v = (mx.state_decode(t[k].cpu().numpy(), t[k + "_scale"].cpu().numpy(), TABLE[k]) for k in ("m", "v"))
    want = 1e-6 + (v0 - 1e-6) * 0.999 ** 3000
    assert abs(v.mean() / want - 1) < 0.07
    assert abs(m.mean() / 1e-3 - 1) < 0.07


@pytest.mark.parametrize("bits", [8, 32])
def test_tensors_aligned_to_16_bytes_only(bits):
    """Views 16 but not 32 bytes into their storage give the bits of aligned tensors, and their neighbours stay."""
    rng = np.random.default_rng(6)
    n = 4100
    a = make(n, bits, torch.float32, rng)
    b, whole = {}, {}
    for k, v in a.items():
        skip = 16 // v.element_size() if "scale" not in k else 3
        whole[k] = torch.full((n + 64,), 7, dtype=v.dtype, device="cuda")
        b[k] = whole[k][skip:skip + v.numel()]
        b[k].copy_(v)
    for t in (a, b):
        L.AdamWGroup([t], bits).step(**HP, t=5, seed=2, zero_grad=True)
    for k, v in a.items():
        skip = 16 // v.element_size() if "scale" not in k else 3
        assert torch.equal(b[k].view(torch.uint8), v.view(torch.uint8)), k
        assert (whole[k][:skip] == 7).all() and (whole[k][skip + v.numel():] == 7).all()


def test_an_eps_near_zero_divides_by_the_root():
    """eps below 1e-12 takes the IEEE path: a gradient of 1e-21 (its square subnormal in the second moment) still
    moves theta by about the learning rate."""
    n = 64
    t = {k: torch.zeros(n, device="cuda") for k in ("theta", "m", "v")}
    t["grad"] = torch.full((n,), 1e-21, device="cuda")
    L.AdamWGroup([t], 32).step(1e-3, 0.0, 0.0, 1e-30, 0.0, 1.0, 1)
    # v = 1e-42 is subnormal, with steps of 1.4e-45: its root is off by 1e-3 of itself
    assert torch.allclose(t["theta"], torch.full((n,), -1e-3, device="cuda"), rtol=2e-3)


def test_group_wrapper_refusals():
    t = make(64, 8, torch.float32, np.random.default_rng(4))
    with pytest.raises(ValueError, match="no tensors"):
        L.AdamWGroup([], 8)
    with pytest.raises(ValueError, match="m is torch.uint8"):
        L.AdamWGroup([t], 32)
    with pytest.raises(ValueError, match="contiguous"):
        L.AdamWGroup([dict(t, grad=t["grad"][:32])], 8)
    with pytest.raises(ValueError, match="not on the current"):
        L.AdamWGroup([dict(t, theta=t["theta"].cpu())], 8)
    with pytest.raises(L.SoupError, match="overlap"):
        L.AdamWGroup([t, t], 8)
    with pytest.raises(L.SoupError, match="null pointer"):
        L.AdamWGroup([{k: v for k, v in t.items() if k != "v_scale"}], 8)


def test_group_made_and_stepped_on_a_side_stream():
    rng = np.random.default_rng(8)
    a = make(5000, 8, torch.bfloat16, rng)
    b = {k: v.clone() for k, v in a.items()}
    L.AdamWGroup([a], 8).step(**HP, t=3, seed=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = L.AdamWGroup([b], 8, stream=s)
    g.step(**HP, t=3, seed=1, stream=s)
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k


@pytest.mark.parametrize("bits", [8, 32])
def test_elements_beyond_32_bits(bits):
    """The last elements of a tensor of more than 2^31 step as they do in a tensor of their own (8-bit codes are
    rounded by other random bits: within one)."""
    n, tail = 2 ** 31 + 5000, 4096 + 904  # the tail starts on a block of 32
    state = torch.uint8 if bits == 8 else torch.float32
    big = {"theta": torch.zeros(n, device="cuda"), "grad": torch.zeros(n, dtype=torch.bfloat16, device="cuda"),
           "m": torch.zeros(n, dtype=state, device="cuda"), "v": torch.zeros(n, dtype=state, device="cuda")}
    if bits == 8:
        big |= {k: torch.zeros((n + 31) // 32, dtype=torch.uint8, device="cuda") for k in ("m_scale", "v_scale")}
    small = make(tail, bits, torch.bfloat16, np.random.default_rng(11), bf16=False)
    for k, v in big.items():
        v[-small[k].numel():] = small[k]
    for t in (big, small):
        L.AdamWGroup([t], bits).step(**HP, t=7, seed=3)
    for k, v in big.items():
        a, b = v[-small[k].numel():], small[k]
        if bits == 8 and k in ("m", "v"):
            assert (a.int() - b.int()).abs().max() <= 1, k
        else:
            assert torch.equal(a, b), k
    assert not big["theta"][:2 ** 31 - 8].any()

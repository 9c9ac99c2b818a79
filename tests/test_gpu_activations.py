"""The activations and their gradients over the whole range of a sum, where the sigmoid is below the smallest normal fp32
number and the activation is not: against 64 bits.

All are z s(v) with the sigmoid s, v = z for silu and v = 2 sqrt(2/pi) (z + 0.044715 z^3) for gelu's tanh form, written as such
here too: 1 + tanh(v/2) has no digits left in 64 bits where it is below 1e-16.  Bounds, of the magnitudes of the terms: 2^-19
for the functions (ops_ref), and for the tanh form, whose v comes out of four fp32 operations on terms of one sign, 4 |v|
2^-24 more, which is what an error of v does to e^v."""
import math

import pytest
import torch

from tests import ops_ref as R

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def eff():
    import expert_ffn_serving_amd as e
    e.lib()
    return e


def sums():
    """Every 1/8 from -110 to 30, every 1/128 in [-14, 14] (where gelu_tanh's tail is), and far out; exact in bf16 or not
    used (a bf16 step at 100 is 1/2)."""
    z = torch.cat([torch.arange(-880, 240) / 8, torch.arange(-1792, 1792) / 128, torch.tensor([-1e30, -3e4, -300., 300., 3e4, 1e30])])
    return z[z.to(BF).float() == z].unique()


def argument(z, act):
    """v and dv/dz in 64 bits."""
    z = z.double()
    if act != R.GELU_TANH:
        return z, torch.ones_like(z)
    c = 2 * math.sqrt(2 / math.pi)
    return c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)


def relative(v, act):
    return R.FUNC + (v.abs() * 2.0 ** -22 if act == R.GELU_TANH else 0.0)


def product_of(z, act):
    """x, w whose sums are z (SwiGLU: gates z, ups 1)."""
    x, w = torch.zeros(len(z), 8, dtype=BF), torch.zeros(16 if act == R.SWIGLU else 8, 8, dtype=BF)
    x[:, 0], x[:, 1] = z.to(BF), 1.0
    w[:8, 0] = 1.0
    if act == R.SWIGLU:
        w[8:, 1] = 1.0
    return x, w


@pytest.mark.parametrize("rows", [7, None])        # the few-row kernel, and the tiles
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("act", [R.SILU, R.GELU_TANH, R.SWIGLU])
def test_activations(eff, act, out, rows):
    z = sums()
    x, w = product_of(z, act)
    y = torch.full((len(z), 8), 7.0, dtype=out, device="cuda")
    step = rows or len(z)
    for i in range(0, len(z), step):
        eff.matmul(x[i:i + step].cuda(), w.cuda(), y[i:i + step], act=act)
    v, _ = argument(z, act)
    ref = z.double() / (1 + torch.exp(-v))
    R.assert_within(y, ref[:, None].expand(-1, 8), (relative(v, act) * ref.abs())[:, None].expand(-1, 8), "activation %d" % act)


@pytest.mark.parametrize("act", [R.SILU, R.GELU_TANH, R.SWIGLU])
def test_gradients(eff, act):
    """w is the identity, so dx is dz rounded to bf16 (one product each, exact)."""
    z = sums()
    n = 8
    nw = 16 if act == R.SWIGLU else 8
    pre = z.to(BF)[:, None].repeat(1, nw)
    dy = torch.full((len(z), n), 2.0, dtype=F32)
    if act == R.SWIGLU:
        pre[:, n:] = 3.0
    dx = torch.full((len(z), nw), 7.0, dtype=BF, device="cuda")
    eff.matmul_backward(dy.cuda(), torch.zeros(len(z), nw, dtype=BF, device="cuda"), torch.eye(nw, dtype=BF, device="cuda"), dx=dx, act=act,
                        pre=pre.cuda())
    v, dv = argument(z, act)
    s = 1 / (1 + torch.exp(-v))
    # for v > 0 the kernel's 1 - s is off by 2^-24 of 1, not of itself
    slope, size = s + z.double() * s * (1 - s) * dv, s + z.double().abs() * dv * torch.where(v > 0, 1.0, s * (1 - s))
    ref, err = 2 * slope, 2 * relative(v, act) * size
    if act == R.SWIGLU:                        # d gate: dy up silu'; d up: dy silu
        half = lambda a, b: torch.cat([a[:, None].expand(-1, n), b[:, None].expand(-1, n)], 1)  # noqa: E731
        up = 2 * z.double() * s
        ref, err = half(3 * ref, up), half(3 * err, relative(v, act) * up.abs())
    else:
        ref, err = ref[:, None].expand(-1, nw), err[:, None].expand(-1, nw)
    R.assert_within(dx, ref, err, "gradient %d" % act)

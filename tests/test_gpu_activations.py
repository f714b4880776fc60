"""The activations of the linear layers and their slopes where they are small: relative to their own value, not
to that of z, against 64 bits.  The values of z are bf16 numbers and reach the epilogue exactly (a product
with a column of ones)."""
import math

import pytest
import torch

import self_attention_gb300 as sa
import _block_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_attention_gb300.build import build
    sa.load_library(build())


def _bf16_between(lo, hi):
    """Every bf16 number from lo to hi (0 < lo < hi)."""
    a, b = (torch.tensor(v).bfloat16().view(torch.int16).item() for v in (lo, hi))
    return torch.arange(a, b + 1, dtype=torch.int16).view(torch.bfloat16).cuda()


def _rows(z, M):
    x = torch.zeros(M, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = z.repeat(M // len(z) + 1)[:M]
    return x


def _value64(z, name):
    z = z.double()
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":     # (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)), without the cancellation
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z)


# down to where the values leave 2^-119
RANGES = {"gelu": (2.0 ** -9, 12.5), "gelu_tanh": (2.0 ** -9, 9.7), "silu": (2.0 ** -9, 84.0)}


@pytest.mark.parametrize("name", RANGES)
@pytest.mark.parametrize("M", [1, 40, 6000])
def test_values_left_of_zero(name, M):
    """y is the bf16 number next to a value that is off by at most 2^-12 of itself: half a bf16 step of the
    result, taken at the larger of the two binades where the error crosses into the next, and 2^-12."""
    zs = -_bf16_between(*RANGES[name])
    if M == 1:
        zs = zs[::37]
    w = torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")
    w[0] = 1
    for z in ([v.view(1) for v in zs] if M == 1 else [zs]):
        x = _rows(z, max(M, len(z)))
        y = sa.linear_forward(x, w, activation=name)
        want = _value64(x[:, :1], name).expand(-1, 16)
        off = 2.0 ** -12 * want.abs()
        half = torch.exp2(torch.floor(torch.log2(want.abs() + off)) - 8)
        assert float(want.abs().min()) >= 2.0 ** -119
        ref.check(f"{name}", y, want, off + half)
    assert sa.attn_get_device_status() == 0


def test_slope_of_gelu_left_of_zero():
    """dbias of one row is its dz, unrounded.  The slope is phi(a) (m - a) for z = -a, with the ratio
    m = erfc(a / sqrt 2) / (2 phi(a)) <= 1 / a: the approximation's 2^-12 enters as m / (a - m) <= 1 / (a^2 - 1);
    the exponent a^2 / 2 log2(e) <= 113 is rounded three times (2^-24 each, 113 ln 2 2^-22.4 = 2^-16.1), beside half
    a dozen more fp32 roundings and two MUFU results of 2^-22: 2^-15."""
    a = _bf16_between(2.0, 12.5)
    z = (-a).view(1, -1)[:, :len(a) // 8 * 8].contiguous()
    n = z.shape[1]
    x, w = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, n, dtype=torch.bfloat16, device="cuda")
    _, _, db = sa.linear_backward(x, w, torch.ones(1, n, dtype=torch.bfloat16, device="cuda"), z, "gelu")
    z = z.double()[0]
    # erfc and the normal density both in 64 bits: their difference loses at most a factor a^2
    want = 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    ref.check("slope", db, want, want.abs() * (2.0 ** -12 / (z * z - 1) + 2.0 ** -15))

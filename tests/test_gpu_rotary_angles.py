"""The angles of the rotary positions: off by at most 2^-25 of half a turn, at fractions of a turn chosen where rounding
in two steps would pass that."""
import math

import pytest
import torch

import self_attention_gb300 as sa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_attention_gb300.build import build
    sa.load_library(build())


# Fractions of a turn in 2^-64 next to a quarter and three quarters, where the cosine is the angle's distance from there: the
# 24 bits of an fp32 fraction end 128 units of 2^32 apart, so that 64 of them and some more lie past the middle.
LOW = [0, 1, 1 << 31, (1 << 32) - 1]
NEAR = [(s * ((1 << 30) + n) << 32) + low for s in (1, -1) for n in (0, 1, 63, 64, 65, 127, 128, 191, 192) for low in LOW]
NEAR += [-x for x in NEAR]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("call", ["forward", "backward", "append"])
def test_angles_next_to_quarters_of_a_turn(interleaved, call):
    turns = [x - (1 << 64) if x >> 63 else x for x in (x % (1 << 64) for x in NEAR)]
    for i in range(0, len(turns), 32):
        part = (turns[i:i + 32] + [0] * 32)[:32]
        x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
        (x[..., 0::2] if interleaved else x[..., :32]).fill_(1)
        t = torch.tensor(part, dtype=torch.int64, device="cuda")
        at = torch.ones(1, 1, dtype=torch.int32, device="cuda")
        if call == "append":
            y = torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16, device="cuda")
            sa.cache_append(x, x, y, torch.zeros_like(y), torch.zeros(1, dtype=torch.int32, device="cuda"), t, at, interleaved)
            y = y[0, 0, 0]
        else:
            y = (sa.rotary_forward if call == "forward" else sa.rotary_backward)(x, t, at, interleaved)[0, 0, 0]
        y = y.double().cpu()
        cos, sin = (y[0::2], y[1::2]) if interleaved else (y[:32], y[32:])
        for j, turn in enumerate(part):
            sign = 1 if turn > 0 else -1                 # of the quarter that it is next to
            # cos(pi u) = -sin(pi (|u| - 1/2)), u = 2 turn / 2^64: the distance is exact
            off = (abs(turn) - (1 << 62)) / 2.0 ** 63
            want = -math.sin(math.pi * off) if turn else 1.0
            # the angle's bound, the cosine's 2 steps of 2^-23 and the rounding to bf16, half a step
            tol = math.pi * 2.0 ** -25 + (2.0 ** -22 + 2.0 ** -8) * abs(cos[j].item())
            assert abs(cos[j].item() - want) <= tol, (turn, cos[j].item(), want)
            if turn:
                assert sin[j].item() == sign * (-1 if call == "backward" else 1)

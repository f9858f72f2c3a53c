"""Angles of far positions, against the product of the position and the
frequency as they are, with no rounding on the way."""
import math
from fractions import Fraction

import pytest
import torch

import adaptive_vector_quantized_b200 as avq

pytestmark = pytest.mark.gpu

# pi to 60 digits: the product with 2^31 and frequencies of 53 bits keeps 40
PI = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("base", [1e4, 5e5])
def test_angles_of_far_positions(base, dtype):
    pos = [1, 1000, 1000003, 2 ** 24 + 1, 2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1, -1, -777777, -2 ** 31]
    d, pairs = 128, 64
    freqs, _ = avq.avq_rotary_freqs(d, base=base)
    X = torch.zeros(1, 1, len(pos), d, dtype=dtype, device="cuda")
    X[..., :pairs] = 1.0  # (1, 0) turns to (cos, sin)
    Y, _ = avq.avq_rotary(X, freqs=freqs.cuda(), positions=torch.tensor(pos, dtype=torch.int32).cuda())
    Y = Y[0, 0].cpu().double()
    for i, p in enumerate(pos):
        for j, f in enumerate(freqs.tolist()):
            turns = Fraction(f) * p / (2 * PI)
            angle = 2 * math.pi * float(turns - round(turns))
            # the fraction of a turn in 24 bits; the frequency in turns (a product with a rounded constant)
            # times the position; sine, cosine and what rounds in fp32; for bf16 the fast forms (2^-21.19 and
            # their argument's rounding) and one rounding of the result
            off = 2 * math.pi * (2.0 ** -26 + abs(p) * f / (2 * math.pi) * 2.0 ** -52) + 4 * 2.0 ** -24
            if dtype == torch.bfloat16:
                off += 2.0 ** -21.19 + math.pi * 2.0 ** -24
            for got, want in ((Y[i, j], math.cos(angle)), (Y[i, pairs + j], math.sin(angle))):
                tol = off + (2.0 ** -8 * abs(want) if dtype == torch.bfloat16 else 0.0)
                assert abs(got.item() - want) <= tol, (p, f, got.item(), want)

"""GPU test of the angles at far positions, against decimal arithmetic: a pair (1, 0) turned by position * frequency.
The frequency is off by at most 2^-63 of a turn for each position (64 bits, and the last places of a long double's
power), the phase is cut after 2^-32 and rounded by up to 2^-28: 2^-27 of a turn for positions below 2^32, and 4 u
for the series and the products."""
import decimal
import math

import numpy as np
import pytest
import torch

from dlrm_sparse_embedding_amd import emb as E

pytestmark = pytest.mark.gpu
PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628621")


def angles(pos, rot, base):
    """position * base^(-2i / rot) modulo 2 pi, in 60 digits."""
    with decimal.localcontext() as c:
        c.prec = 60
        f = [(-(decimal.Decimal(2 * i) / rot) * decimal.Decimal(base).ln()).exp() for i in range(rot // 2)]
        return np.array([[float((p * x) % (2 * PI)) for x in f] for p in pos])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot", [(64, 64), (7, 6)])          # 16-byte units, element by element
def test_far_positions(layout, dim, rot):
    pos = [0, 1, 4095, (1 << 20) + 1, (1 << 24) - 1, 999999937, (1 << 31) - 1, (1 << 32) - 3, -5, -(1 << 31), -(1 << 32) + 1]
    x = torch.zeros((len(pos), 1, dim), device="cuda")
    a = slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)
    b = slice(rot // 2, rot) if layout == "half" else slice(1, rot, 2)
    x[..., a] = 1.0
    y = torch.empty_like(x)
    r = E.Rotary(rot, layout=layout, base=10000.0)
    E.emb_rotary_apply(r.handle, torch.tensor(pos).cuda(), x, y)
    ang = angles(pos, rot, 10000)
    y = y.double().cpu().numpy()[:, 0]
    tol = 2 * math.pi * 2.0 ** -27 + 4 * 2.0 ** -24
    assert np.abs(y[:, a] - np.cos(ang)).max() <= tol and np.abs(y[:, b] - np.sin(ang)).max() <= tol

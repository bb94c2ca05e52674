"""The gradients of a pool's factors (qlora_multi_bwd) where their operands are
extreme: infinities, and the largest fp32 values."""
import numpy as np
import pytest
import torch

from bit_nf4_quantized_07_b200 import api
from tests.test_gpu_multi import U2, Case

pytestmark = pytest.mark.gpu
INF = float("inf")


def _exact_g(c):
    """Factors B with one element per column, so that G_t = dY_t B is an element of dY times one of B: 16 bits, exact."""
    for a in range(c.count):
        c.B[a] = 0
        for j in range(c.r):
            c.B[a, (7 * j + a) % c.rows, j] = 1 + (j % 64) / 128
    c.pool = api.AdapterPool(c.A, c.B, c.s, c.rank)
    G = torch.zeros(c.n, c.r, dtype=torch.float32, device="cuda")
    for a, at, k, _ in c.groups():
        G[at, :k] = (c.dY[at].double() @ c.B[a, :, :k].double()).float()
    return G


def _signed(got, want):
    """The infinities and NaN of `want`, and finite where it is."""
    inf = torch.isinf(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[inf].double(), want[inf].double())
    assert torch.isfinite(got[torch.isfinite(want)]).all()


@pytest.mark.parametrize("shape,n,r", [((256, 512), 60, 16), ((192, 320), 200, 40), ((128, 256), 5, 64), ((256, 128), 90, 128)])
@pytest.mark.parametrize("short", [False, True])
def test_infinities_in_x_and_dy_keep_their_sign(shape, n, r, short):
    """short: G and U of few bits (powers of two and zeros among them), whose lower parts would be zero."""
    c = Case(*shape, n, 3, r, "random", seed=23)
    c.ids[0], c.ids[1], c.ids[2] = 0, 1, 2
    if short:
        c.dY[:, ::3], c.dY[:, 1::5] = 0.5, 0
        _exact_g(c)
        c.U = torch.full((n, r), 0.5, device="cuda")
        c.U[:, 1::4], c.U[:, 2::4] = -2.0 ** -90, 0
    else:
        _, c.U = c.fwd()
    clean = c.bwd(U=c.U)
    c.X[1, 11], c.X[1, 12], c.dY[2, 3], c.dY[2, 5] = INF, -INF, -INF, INF
    _, dA, dB = c.bwd(U=c.U)
    assert torch.equal(dA[0], clean[1][0]) and torch.equal(dB[0], clean[2][0])
    for a, at, k, s in c.groups():
        y, x, u = c.dY[at].double(), c.X[at].double(), c.U[at].double()
        G = (y[:, :, None] * c.B[a].double()).sum(1)  # term by term, as the formula has it
        _signed(dA[a], s * (G[:, :, None] * x[:, None]).sum(0))
        _signed(dB[a], s * (y[:, :, None] * u[:, None]).sum(0))


def test_the_largest_g_and_u_stay_finite():
    """Values above the largest bf16, whose rounding to bf16 would be infinite."""
    c = Case(128, 256, 6, 2, 8, "random", seed=24)
    top = float(np.finfo(np.float32).max)
    c.U = torch.full((6, 8), top, device="cuda")
    c.dY.fill_(2.0 ** -20)
    c.s.fill_(1.0)
    _, _, dB = c.bwd(U=c.U)
    for a, at, _, _ in c.groups():
        want = len(at) * top * 2.0 ** -20
        assert torch.isfinite(dB[a]).all() and ((dB[a].double() - want).abs() <= 8 * U2 * want).all()

"""The gradients of a pool's factors (qlora_multi_bwd) where their operands are
extreme: what fp32 values of G and U give beside bf16 ones, and infinities.

Tolerances: u = 2^-24, half a step of fp32.  G and U take part as the fp32
values they are, in three bf16 parts whose products with bf16 are exact; the
tensor cores' running sums may truncate, so a sum over n tokens may be off by
n 2u of the sum of its terms' magnitudes.  Of a sum of terms with random signs
at most a few hundred of those roundings add up alike: in norm an error of
1e-6 (17 u) is allowed.  Two parts would leave up to 2^-17 of a term: 2.5e-6 in norm."""
import numpy as np
import pytest
import torch

from bit_nf4_quantized_07_b200 import api
from tests.test_gpu_multi import U2, Case, _near

pytestmark = pytest.mark.gpu
INF = float("inf")


def _given(c, G):
    """dA and dB in float64 of given G and U (fp32 values), their bounds without any error of G or U themselves."""
    dA, dB = torch.zeros(c.A.shape).double().cuda(), torch.zeros(c.B.shape).double().cuda()
    tA, tB = torch.zeros_like(dA), torch.zeros_like(dB)
    for a, at, k, s in c.groups():
        y, x, u, g = c.dY[at].double(), c.X[at].double(), c.U[at, :k].double(), G[at, :k].double()
        e = abs(s) * (len(at) + 4) * U2
        dA[a, :k], dB[a, :, :k] = s * (g.T @ x), s * (y.T @ u)
        tA[a, :k], tB[a, :, :k] = e * (g.abs().T @ x.abs()), e * (y.abs().T @ u.abs())
    return (dA, 1.01 * tA), (dB, 1.01 * tB)


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


@pytest.mark.parametrize("rows,cols,n,count,r,kind,vary", [
    (256, 512, 9, 7, 16, "random", False),      # one token or two of an adapter: nothing hides a missing part
    (192, 320, 3, 1, 8, "one", False), (256, 320, 40, 30, 24, "random", True), (512, 256, 33, 12, 64, "random", True),
    (320, 512, 70, 40, 128, "random", False), (256, 512, 1500, 2, 16, "random", False)])
def test_all_bits_of_g_and_u_take_part(rows, cols, n, count, r, kind, vary):
    c = Case(rows, cols, n, count, r, kind, vary, seed=21)
    g = torch.Generator("cuda").manual_seed(n)
    c.U = torch.randn(n, r, generator=g, device="cuda")  # any fp32 values: not rounded to fewer bits
    G = _exact_g(c)
    _, dA, dB = c.bwd(U=c.U)
    for name, x, (ref, tol) in zip(("dA", "dB"), (dA, dB), _given(c, G)):
        _near(name, x, ref, tol)
        assert ((x.double() - ref).norm() / ref.norm()).item() < 1e-6, name


@pytest.mark.parametrize("n,count,r", [(3000, 2, 16), (700, 3, 40), (5000, 1, 64)])
def test_long_sums_in_norm(n, count, r):
    c = Case(256, 512, n, count, r, "random", seed=22)
    _, c.U = c.fwd()
    _, dA, dB = c.bwd(U=c.U)
    ref = c.backward_ref(U=c.U)
    for name, x, (want, _) in zip(("dA", "dB"), (dA, dB), ref[1:]):
        # dA's G is a sum of 256 products of its own, off by 256 2u / sqrt(256) of its norm where the truncations add up
        assert ((x.double() - want).norm() / want.norm()).item() < (1e-6 if name == "dB" else 1e-6 + 16 * U2), name


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

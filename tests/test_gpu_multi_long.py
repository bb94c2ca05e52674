"""Batches whose tensors pass 2^31 elements: their first, last and middle tokens' rows, and the gradients over all of
them, against float64 (bounds as in test_gpu_multi.py, evaluated on the rows that are looked at)."""
import pytest
import torch

from bit_nf4_quantized_07_b200 import api
from tests.test_gpu_multi import H, U2, _near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,n", [(128, 8192, 270001), (8192, 64, 270001), (64, 8192, 270001), (128, 64, 1 << 20)])
def test_long_batch(rows, cols, n):
    g = torch.Generator("cuda").manual_seed(rows)
    count, r = 3, 8
    t = lambda shape, std: torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)  # noqa: E731
    w = api.quantize_weight(torch.randn(rows, cols, generator=g, device="cuda") * 0.02)
    W = api.nf4_dequant(w).double()
    X, dY, A, B = t((n, cols), 1.0), t((n, rows), 1.0), t((count, r, cols), 0.05), t((count, rows, r), 0.05)
    s = torch.tensor([0.5, -2.0, 1.0], device="cuda")
    ids = torch.randint(-1, count, (n,), generator=g, device="cuda").int()
    pool = api.AdapterPool(A, B, s)
    Y, U = api.qlora_multi_fwd(w, pool, X, ids, want_u=True)
    dX, dA, dB = api.qlora_multi_bwd(w, pool, X, ids, dY, U=U)
    look = torch.cat([torch.arange(200), torch.arange(n // 2, n // 2 + 100), torch.arange(n - 300, n)]).cuda()
    Ad, Bd = A.double(), B.double()

    def side(x, f, W, other, K):
        """x W^T + s (x f^T) other of the tokens in `look`, its bound, and x f^T with its own."""
        x = x[look].double()
        y, base = x @ W.T, x.abs() @ W.abs().T
        tol, low, ltol = (K + r) * U2 * base, torch.zeros(len(look), r).double().cuda(), torch.zeros(len(look), r).double().cuda()
        for a in range(count):
            at = ids[look] == a
            u, ue = x[at] @ f[a].T, K * U2 * (x[at].abs() @ f[a].abs().T)
            low[at], ltol[at], k = u, ue, abs(s[a].item())
            y[at] += s[a].item() * (u @ other[a])
            tol[at] += k * ((H * (1 + H) + (K + r) * U2) * (u.abs() @ other[a].abs()) + (1 + H) * (ue @ other[a].abs()))
        return y, H * y.abs() + 1.01 * tol, low, ltol
    Yr, Yt, Ur, Ut = side(X, Ad, W, Bd.transpose(1, 2), cols)
    _near("Y", Y[look], Yr, Yt)
    _near("U", U[look], Ur, Ut)
    dXr, dXt, _, _ = side(dY, Bd.transpose(1, 2), W.T, Ad, rows)
    _near("dX", dX[look], dXr, dXt)
    # the gradients in norm: sums of n terms of random signs in fp32 pieces (and G's own rounding, rows 2u of it)
    for a in range(count):
        refA, refB = torch.zeros_like(Ad[a]), torch.zeros_like(Bd[a])
        for part in (ids == a).nonzero()[:, 0].split(1 << 15):
            x, y = X[part].double(), dY[part].double()
            refA += s[a].item() * ((y @ Bd[a]).T @ x)
            refB += s[a].item() * (y.T @ U[part].double())
        assert ((dA[a].double() - refA).norm() / refA.norm()).item() < 2e-6 + rows ** 0.5 * U2
        assert ((dB[a].double() - refB).norm() / refB.norm()).item() < 2e-6

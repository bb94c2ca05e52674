"""Batches whose tensors pass 2^31 elements: their first, last and middle tokens' rows, and the gradients over all of
them, against float64 (bounds as in test_gpu_multi.py, evaluated on the rows that are looked at)."""
import pytest
import torch

from bit_nf4_quantized_07_b200 import api
from tests.test_gpu_multi import H, U2, _near

pytestmark = pytest.mark.gpu


def _side(x, W, f, other, s, ids):
    """x W^T + s (x f_a^T) other_a, a = ids, of tokens x, its bound, and x f_a^T with its own; f, other: per adapter, cut
    to its rank."""
    x, K, r = x.double(), x.shape[1], max(len(k) for k in f.values())
    y, base = x @ W.T, x.abs() @ W.abs().T
    tol, low, ltol = (K + r) * U2 * base, torch.zeros(len(x), r).double().cuda(), torch.zeros(len(x), r).double().cuda()
    for a in f:
        at, k, fa, oa = ids == a, abs(s[a].item()), f[a].double(), other[a].double()
        u, ue = x[at] @ fa.T, K * U2 * (x[at].abs() @ fa.abs().T)
        low[at, :len(fa)], ltol[at, :len(fa)] = u, ue
        y[at] += s[a].item() * (u @ oa)
        tol[at] += k * ((H * (1 + H) + (K + r) * U2) * (u.abs() @ oa.abs()) + (1 + H) * (ue @ oa.abs()))
    return y, H * y.abs() + 1.01 * tol, low, ltol


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
    Ad, Bd, every = A.double(), B.double(), range(count)
    up, down = {a: Ad[a] for a in every}, {a: Bd[a].T for a in every}
    Yr, Yt, Ur, Ut = _side(X[look], W, up, down, s, ids[look])
    _near("Y", Y[look], Yr, Yt)
    _near("U", U[look], Ur, Ut)
    dXr, dXt, _, _ = _side(dY[look], W.T, down, up, s, ids[look])
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


@pytest.mark.parametrize("rows,cols", [(128, 17408), (17408, 128), (64, 17408), (17408, 64)])
@pytest.mark.parametrize("n", [5, 30, 70])
def test_pool_of_more_than_2_31_elements(rows, cols, n):
    """Adapters from both ends of a pool whose A or B passes 2^31 elements, and the gradients of the others."""
    g = torch.Generator("cuda").manual_seed(n)
    count, r = 1024, 128
    t = lambda shape, std: torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)  # noqa: E731
    w = api.quantize_weight(torch.randn(rows, cols, generator=g, device="cuda") * 0.02)
    X, dY, A, B = t((n, cols), 1.0), t((n, rows), 1.0), t((count, r, cols), 0.05), t((count, rows, r), 0.05)
    s, rank = torch.randn(count, generator=g, device="cuda"), torch.randint(1, r + 1, (count,), generator=g, device="cuda").int()
    own = torch.tensor([0, 3, 700, 1000, 1021, 1023], device="cuda")
    pick = torch.randint(0, len(own), (n,), generator=g, device="cuda")
    pick[:5] = torch.arange(1, 6)
    ids = own[pick].int()
    W = api.nf4_dequant(w).double()
    pool = api.AdapterPool(A, B, s, rank)
    Y, U = api.qlora_multi_fwd(w, pool, X, ids, want_u=True)
    dX, dA, dB = api.qlora_multi_bwd(w, pool, X, ids, dY, U=U)
    up = {a: A[a, :rank[a]] for a in own.tolist()}
    down = {a: B[a, :, :rank[a]].T for a in own.tolist()}
    Yr, Yt, Ur, Ut = _side(X, W, up, down, s, ids)
    if n <= 32:  # the weight stream's rounding of the book and its unrounded weights, see test_gpu_multi_variants.py
        Yt += 7 * (H + H / 2) * W.norm(dim=1)
    k = Ur.shape[1]
    _near("U", U[:, :k], Ur, Ut)
    assert not U[:, k:].any()
    _near("Y", Y, Yr, Yt)
    dXr, dXt, Gr, Gt = _side(dY, W.T, down, up, s, ids)
    _near("dX", dX, dXr, dXt)
    for a in own.tolist():
        at, q, sa = ids == a, int(rank[a]), s[a].item()
        x, y, u, e = X[at].double(), dY[at].double(), U[at, :q].double(), (int(at.sum()) + 4) * U2
        _near("dA", dA[a, :q], sa * (Gr[at, :q].T @ x), 1.01 * abs(sa) * ((Gt[at, :q] + e * Gr[at, :q].abs()).T @ x.abs()))
        _near("dB", dB[a, :, :q], sa * (y.T @ u), 1.01 * abs(sa) * e * (y.abs().T @ u.abs()))
        assert not dA[a, q:].any() and not dB[a, :, q:].any()
    others = torch.ones(count, dtype=torch.bool, device="cuda")
    others[own] = False
    others = others.nonzero()[:, 0]
    assert not dA[others[::37]].any() and not dB[others[::37]].any() and not dA[others[-1]].any()


@pytest.mark.parametrize("n", [6, 30, 100])
@pytest.mark.parametrize("shape", [(192, 320), (256, 512)])
def test_ranks_outside_the_pools_are_the_nearer_end(shape, n):
    g = torch.Generator("cuda").manual_seed(n)
    t = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    w = api.quantize_weight(torch.randn(*shape, generator=g, device="cuda") * 0.02)
    X, dY, A, B, s = t(n, shape[1]), t(n, shape[0]), t(5, 24, shape[1]), t(5, shape[0], 24), torch.randn(5, device="cuda")
    ids = (torch.arange(n, device="cuda") % 5).int()
    out = []
    for rank in ([-1, 25, 1 << 30, -1 << 31, 11], [0, 24, 24, 0, 11]):
        pool = api.AdapterPool(A, B, s, torch.tensor(rank, dtype=torch.int32, device="cuda"))
        Y, U = api.qlora_multi_fwd(w, pool, X, ids, want_u=True)
        out.append((Y, U) + api.qlora_multi_bwd(w, pool, X, ids, dY, U=U))
    assert all(torch.equal(a, b) for a, b in zip(*out))

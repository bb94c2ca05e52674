"""The linear with a pool of adapters on every variant that its launchers choose
among: the weight stream over one epoch and several, and the tcgen05 GEMM with
one or two weight sub-tiles, one or two token sub-tiles, and K split over up to
four CTAs, forward and transposed.  The sizes are chosen for the variants, which
test_sizes_take_the_variants_they_are_for looks up in the launches themselves.

Tolerances, element by element, are those of test_gpu_multi.py without its
allowance for the codebook at n <= 32.  Only the weight stream needs one.  It
does not round W' to bf16 (2^-8 of a weight at most) but the book (2^-9): the
values of X are independent standard normal and know nothing of the weights'
roundings d, so what these add to Y is normal with a standard deviation of
|d| <= (2^-8 + 2^-9) |W'_row|, and 7 of those are allowed (3e-12 of all).

In norm: a bf16 rounding is off by at most half a step, evenly distributed over
it, so by 2^-7 / sqrt(12) of the value or less in the mean.  Y = P + T, P = X W'^T
and T the adapter term, rounds once, bf16(s U) once in T, and the stream leaves
the rounding of W' out of P and rounds the book (6.3e-4 in norm).  The means are
taken over thousands of values; 5 % are allowed on top."""
import json
import math

import pytest
import torch

from bit_nf4_quantized_07_b200 import api
from tests.test_gpu_multi import H, U2, Case, _ids, _near

pytestmark = pytest.mark.gpu
A2 = 2.0 ** -14 / 12  # mean square of a bf16 rounding
BOOK2 = 6.3e-4 ** 2
INF = float("inf")


class Big(Case):
    """A Case with its values drawn on the device."""

    def __init__(self, rows, cols, n, count, r, kind, vary=False, weight="int8", seed=0):
        import numpy as np
        g = np.random.Generator(np.random.PCG64([rows, cols, n, count, r, seed]))
        gen = torch.Generator("cuda").manual_seed(rows + 3 * cols + 7 * n + seed)
        t = lambda shape, std: (torch.randn(shape, generator=gen, device="cuda") * std).bfloat16()  # noqa: E731
        self.w = api.quantize_weight(torch.randn(rows, cols, generator=gen, device="cuda") * 0.02,
                                     double_quant=weight != "plain", dq_format="e4m3" if weight == "e4m3" else "int8")
        self.W = api.nf4_dequant(self.w)
        self.X, self.dY = t((n, cols), 1.0), t((n, rows), 1.0)
        self.A, self.B = t((count, r, cols), 0.05), t((count, rows, r), 0.05)
        self.s = torch.from_numpy(g.uniform(-2, 2, count).astype(np.float32)).cuda()
        rank = np.concatenate([[0, r, 1], g.integers(0, r + 1, count)])[:count] if vary else None
        self.rank = None if rank is None else torch.from_numpy(rank.astype(np.int32)).cuda()
        self.ranks = [r] * count if rank is None else rank.tolist()
        self.ids = torch.from_numpy(_ids(kind, n, count, g).astype(np.int32)).cuda()
        self.rows, self.cols, self.n, self.count, self.r = rows, cols, n, count, r
        self.pool = api.AdapterPool(self.A, self.B, self.s, self.rank)


def _check_forward(c, stream):
    Y, U = c.fwd()
    Yr, Yt, Ur, Ut = c.forward_ref()
    _near("U", U, Ur, Ut)
    W, X = c.W.double(), c.X.double()
    P = X @ W.T
    if c.n <= 32:
        Yt -= 1.01 * 2 * H * (X.abs() @ W.abs().T)
    if stream:
        Yt += 7 * (H + H / 2) * W.norm(dim=1)
    _near("Y", Y, Yr, Yt)
    err2 = (Y.double() - Yr).square().sum().item()
    want2 = A2 * (Yr.square().sum() + (Yr - P).square().sum()).item() + stream * (A2 + BOOK2) * P.square().sum().item()
    assert err2 <= 1.05 ** 2 * want2, (math.sqrt(err2) / Yr.norm().item(), math.sqrt(want2) / Yr.norm().item())


def _check_backward(c):
    _, U = c.fwd()
    got = c.bwd(U=U)
    for name, x, (ref, tol) in zip(("dX", "dA", "dB"), got, c.backward_ref(U=U)):
        _near(name, x, ref, tol)
        if name == "dX":
            P = c.dY.double() @ c.W.double()
            want2 = A2 * (ref.square().sum() + (ref - P).square().sum()).item()
            assert (x.double() - ref).square().sum().item() <= 1.05 ** 2 * want2
        elif ref.norm() > 0:  # G's own sum of `rows` terms, then the sum over the tokens: roundings of random signs
            assert ((x.double() - ref).norm() / ref.norm()).item() < 1e-6 + math.sqrt(c.rows) * U2 * (name == "dA"), name


# rows, cols, n, adapters, r, ids, ranks, weight
STREAM = [(4096, 4096, 1, 40, 16, "random", False, "int8"), (4096, 4096, 8, 40, 16, "holes", True, "e4m3"),
          (2048, 1024, 3, 3, 128, "random", True, "plain"), (1024, 11008, 8, 9, 24, "random", False, "int8"),
          (28672, 4096, 8, 12, 16, "random", True, "int8"), (28672, 8192, 1, 4, 16, "random", False, "int8"),
          (28672, 8192, 8, 8, 64, "holes", True, "int8"), (8192, 28672, 1, 3, 128, "random", False, "e4m3"),
          (8192, 28672, 8, 8, 16, "random", True, "plain"),                     # several epochs
          (1024, 11008, 12, 20, 64, "random", True, "int8"), (1024, 11008, 24, 40, 64, "random", False, "int8"),
          (16384, 1024, 24, 40, 64, "random", True, "int8"),                    # many pairs of a tile and an adapter
          (4096, 4096, 24, 40, 128, "holes", True, "plain"), (4096, 4096, 16, 2, 40, "random", False, "e4m3"),
          # rows that the GEMM's tiles do not divide
          (4160, 4096, 9, 9, 16, "random", False, "int8"), (1088, 2048, 24, 40, 24, "holes", True, "e4m3"),
          (4160, 4096, 32, 32, 64, "random", False, "int8"), (64, 4096, 25, 40, 128, "random", True, "plain"),
          (11072, 4096, 30, 3, 16, "holes", True, "int8"), (192, 512, 32, 32, 8, "random", False, "int8")]
# product rows (outputs), its depth, n, adapters, r, ids, ranks, weight: weight sub-tiles, token sub-tiles, K split
GEMM = {(1024, 2048, 100, 9, 16, "random", True, "int8"): (1, 1, 4), (4096, 8192, 16, 9, 16, "random", True, "int8"): (1, 1, 4),
        (4096, 11008, 12, 6, 32, "holes", False, "e4m3"): (1, 1, 4), (1024, 4096, 32, 32, 16, "random", False, "plain"): (1, 1, 4),
        (4096, 4096, 333, 5, 8, "blocks", False, "int8"): (1, 1, 2), (5120, 1024, 100, 40, 40, "random", True, "int8"): (1, 1, 3),
        (8192, 512, 700, 24, 24, "blocks", True, "int8"): (1, 2, 1), (8192, 4096, 300, 5, 64, "holes", True, "e4m3"): (1, 2, 2),
        (5120, 4096, 333, 100, 8, "random", False, "plain"): (1, 2, 3), (4096, 8192, 333, 7, 128, "blocks", True, "int8"): (1, 2, 4),
        (8192, 1024, 900, 300, 16, "random", True, "int8"): (2, 1, 1), (11008, 4096, 500, 3, 128, "blocks", False, "e4m3"): (2, 1, 1),
        (14336, 4096, 16, 16, 64, "random", True, "int8"): (2, 1, 2), (11008, 4096, 203, 24, 32, "blocks", True, "int8"): (2, 1, 3),
        (11008, 4096, 2048, 8, 16, "runs", False, "int8"): None}  # what it takes differs between the directions


def _id(g):
    return "-".join(map(str, g))


@pytest.mark.parametrize("g", STREAM, ids=_id)
def test_weight_stream(g):
    _check_forward(Big(*g), True)


@pytest.mark.parametrize("g", list(GEMM), ids=_id)
def test_gemm_forward(g):
    _check_forward(Big(*g), False)


@pytest.mark.parametrize("g", list(GEMM), ids=_id)
def test_gemm_backward(g):
    _check_backward(Big(g[1], g[0], *g[2:]))


def _launches(tmp_path, call):
    """(name, grid) of the kernels that a call launches."""
    call()
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        call()
        torch.cuda.synchronize()
    path = str(tmp_path / "trace.json")
    prof.export_chrome_trace(path)
    with open(path) as f:
        got = [(e["name"], e["args"]["grid"]) for e in json.load(f)["traceEvents"] if e.get("cat") == "kernel"]
    if not got:
        pytest.skip("the profiler records no kernels here")
    return got


def test_sizes_take_the_variants_they_are_for(tmp_path):
    wrong = []
    for g in STREAM:
        names = [k for k, _ in _launches(tmp_path, Big(*g).fwd)]
        if not any(f"nf4_decode_fwd_kernel<{-(-g[2] // 8)}, true>" in k for k in names):
            wrong.append((g, names))
    for g, want in GEMM.items():
        if want is None:
            continue
        for trans in (False, True):
            c = Big(*(g[1::-1] if trans else g[:2]), *g[2:])
            found = _launches(tmp_path, c.bwd if trans else c.fwd)
            name = f"nf4_tc_gemm_kernel<{str(trans).lower()}, {want[0]}, {want[1]}, true>"
            if not any(name in k and grid[2] == want[2] for k, grid in found):
                wrong.append((g, trans, want, found))
    assert not wrong, wrong


NONFINITE = [(4096, 4096, 8, 16), (1024, 11008, 24, 64), (1088, 2048, 32, 16),                   # the stream (forward)
             (1088, 2048, 100, 24),                                                             # the register-level GEMM
             (1024, 2048, 100, 16), (4096, 4096, 333, 24), (8192, 512, 700, 24), (5120, 4096, 333, 16),
             (8192, 1024, 900, 40), (11008, 4096, 203, 32)]


@pytest.mark.parametrize("g", NONFINITE, ids=_id)
@pytest.mark.parametrize("trans", [False, True])
def test_factors_that_are_not_finite(g, trans):
    """An infinity or NaN in a factor reaches the outputs that it is a term of, in their own tokens, with its sign; every
    other output keeps its bits.  Values past a rank take no part."""
    M, K, n, r = g
    c = Big(*((K, M) if trans else (M, K)), n, 4, r, "random", seed=3)
    c.rank = torch.tensor([r - 3, r, r - 5, r], dtype=torch.int32, device="cuda")
    c.ids[:4] = torch.arange(4, dtype=torch.int32, device="cuda")
    c.ranks, c.pool = c.rank.tolist(), api.AdapterPool(c.A, c.B, c.s, c.rank)
    _, U = c.fwd()
    run = (lambda: c.bwd(U=U)[0]) if trans else (lambda: c.fwd()[0])
    clean = run()
    factor = c.A.transpose(1, 2) if trans else c.B  # [count][M][r] either way
    factor[0, :, r - 3:], factor[2, :, r - 5:] = float("nan"), INF
    assert torch.equal(run(), clean)
    at = [(1, M - 1, 0, INF), (1, 130, r - 1, -INF), (3, M // 2 + 5, 2, -INF), (3, 7, 1, float("nan")),
          (3, M - 1, r // 2, -INF)]  # adapter, output, column, value
    for a, m, j, x in at:
        factor[a, m, j] = x
    got = run()
    low = torch.zeros(n, r, dtype=torch.float64, device="cuda")  # U, or G = dY B
    for a, tok, k, s in c.groups():
        low[tok, :k] = s * (c.dY[tok].double() @ c.B[a, :, :k].double() if trans else U[tok, :k].double())
    spoiled = torch.zeros_like(clean, dtype=torch.bool)
    for a, m, j, x in at:
        tok = (c.ids == a).nonzero()[:, 0]
        spoiled[tok, m] = True
        want = x * low[tok, j].sign()
        assert torch.equal(torch.isnan(got[tok, m]), torch.isnan(want))
        assert math.isnan(x) or torch.equal(got[tok, m].double(), want)
    assert torch.equal(got[~spoiled], clean[~spoiled])


@pytest.mark.parametrize("g", NONFINITE, ids=_id)
@pytest.mark.parametrize("trans", [False, True])
def test_an_infinite_factor_times_an_infinite_product(g, trans):
    """U = X A^T is infinite where A is, and so is its product with an infinity of B: with the sign of the two, not NaN
    (and dX from G = dY B and A the same way)."""
    M, K, n, r = g
    c = Big(*((K, M) if trans else (M, K)), n, 3, r, "random", seed=4)
    c.ids[:3] = torch.arange(3, dtype=torch.int32, device="cuda")
    _, U = c.fwd()
    down, up = (c.B.transpose(1, 2), c.A.transpose(1, 2)) if trans else (c.A, c.B)  # [count][r][K], [count][M][r]
    x = c.dY if trans else c.X
    tok = (c.ids == 1).nonzero()[:, 0]
    x[tok, 9] = x[tok, 9].abs() + 1  # not zero, one sign
    down[1, 2, 9] = -INF
    up[1, 5, 2], up[1, M - 1, 2], up[1, 6, 2] = INF, -INF, 0
    got = (c.bwd(U=U)[0] if trans else c.fwd()[0])[tok].double()
    low = -INF * c.s[1].item()
    want = low * up[1, :, 2].double().sign()
    assert torch.equal(torch.isnan(got), torch.isnan(want).expand_as(got))
    there = ~torch.isnan(want)
    assert torch.equal(got[:, there], want[there].expand(len(tok), -1))

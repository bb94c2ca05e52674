"""GPU parity of the linear with a pool of adapters (qlora_multi_fwd,
qlora_multi_bwd) against the formulas in float64, element by element.

Tolerances.  u = 2^-24 is half a step of fp32; the tensor cores' running sums
may truncate, so a sum of k products is allowed k 2u of the sum of their
magnitudes |.|; a bf16 rounding is off by at most 2^-8 of its value.
  U   K 2u |X||A|
  Y   2^-8 |Y*|, the operand bf16(s U): 2^-8 |sU||B|, U's own error times |sB|,
      and (K + r) 2u (|X||W'| + |sU||B|); for n <= 32 the codebook's entries
      enter as bf16 before the block constant: 2^-8 |X||W'| more (W' itself is
      bf16 of the product: another 2^-8).
  dX  as Y, of dY, W', G = dY B and A.
  dA  G as hi + lo: 2^-16 |G|, G's own error dout 2u |dY||B|, and the sum over
      the tokens: n 2u; three more roundings for scale and flushes.
  dB  the same of U and dY."""
import numpy as np
import pytest
import torch

from bit_nf4_quantized_07_b200 import api

pytestmark = pytest.mark.gpu
U2 = 2.0 ** -23
H = 2.0 ** -8


def _ids(kind, n, count, g):
    if kind == "random":
        return g.integers(0, count, n)
    if kind == "runs":
        return np.sort(g.integers(0, count, n))[::-1].copy()
    if kind == "holes":  # ids outside the pool: no adapter
        a = g.integers(-1, count + 1, n)
        return np.where(a == count, 2 ** 31 - 1, np.where(a < 0, -2 ** 31, a))
    if kind == "none":
        return np.full(n, -1)
    if kind == "one":
        return np.full(n, count - 1)
    if kind == "blocks":  # runs of uneven lengths in no order
        return np.repeat(g.integers(-1, count, n), g.integers(1, 40, n))[:n]
    raise ValueError(kind)


class Case:
    def __init__(self, rows, cols, n, count, r, kind, vary=False, weight="int8", seed=0):
        g = np.random.Generator(np.random.PCG64([rows, cols, n, count, r, seed]))
        t = lambda shape, std: torch.from_numpy((g.standard_normal(shape) * std).astype(np.float32)).cuda().bfloat16()  # noqa: E731
        W0 = torch.from_numpy((g.standard_normal((rows, cols)) * 0.02).astype(np.float32)).cuda()
        self.w = api.quantize_weight(W0, double_quant=weight != "plain", dq_format="e4m3" if weight == "e4m3" else "int8")
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

    def fwd(self, **k):
        return api.qlora_multi_fwd(self.w, self.pool, self.X, self.ids, want_u=True, **k)

    def bwd(self, **k):
        return api.qlora_multi_bwd(self.w, self.pool, self.X, self.ids, self.dY, **k)

    def groups(self):
        ids = self.ids.cpu().numpy()
        for a in range(self.count):
            yield a, torch.from_numpy(np.flatnonzero(ids == a)).cuda(), self.ranks[a], float(self.s[a])

    def forward_ref(self, A=None, B=None, X=None):
        """Y, U and their bounds in float64."""
        X, W = (self.X if X is None else X).double(), self.W.double()
        A, B = (self.A if A is None else A).double(), (self.B if B is None else B).double()
        K, r = self.cols, self.r
        Y, base = X @ W.T, X.abs() @ W.abs().T
        tol = K * U2 * base + (2 * H * base if self.n <= 32 else 0)
        Uf, Utol = torch.zeros(self.n, r).double().cuda(), torch.zeros(self.n, r).double().cuda()
        for a, at, k, s in self.groups():
            x, f, b = X[at], A[a, :k], B[a, :, :k]
            u, ue = x @ f.T, K * U2 * (x.abs() @ f.abs().T)
            Uf[at, :k], Utol[at, :k] = u, ue
            Y[at] += s * (u @ b.T)
            mag = abs(s) * (u.abs() @ b.abs().T)
            tol[at] += (H * (1 + H) + (K + r) * U2) * mag + K * U2 * 0 + abs(s) * (ue @ b.abs().T) * (1 + H) + r * U2 * base[at]
        return Y, H * Y.abs() + 1.01 * tol, Uf, Utol

    def backward_ref(self, A=None, B=None, X=None, U=None):
        X, W, dY = (self.X if X is None else X).double(), self.W.double(), self.dY.double()
        A, B = (self.A if A is None else A).double(), (self.B if B is None else B).double()
        K, r = self.rows, self.r
        dX, base = dY @ W, dY.abs() @ W.abs()
        tol = K * U2 * base
        dA, dB = torch.zeros(self.A.shape).double().cuda(), torch.zeros(self.B.shape).double().cuda()
        tA, tB = torch.zeros_like(dA), torch.zeros_like(dB)
        for a, at, k, s in self.groups():
            y, x, f, b = dY[at], X[at], A[a, :k], B[a, :, :k]
            G, ge = y @ b, K * U2 * (y.abs() @ b.abs())
            u, ue = (x @ f.T, self.cols * U2 * (x.abs() @ f.abs().T)) if U is None else (U[at, :k].double(), 0)
            dX[at] += s * (G @ f)
            mag = abs(s) * (G.abs() @ f.abs())
            tol[at] += (H * (1 + H) + (K + r) * U2) * mag + abs(s) * (ge @ f.abs()) * (1 + H) + r * U2 * base[at]
            dA[a, :k], dB[a, :, :k] = s * (G.T @ x), s * (y.T @ u)
            e = H * H + (len(at) + 4) * U2
            tA[a, :k] = abs(s) * ((ge + e * G.abs()).T @ x.abs())
            tB[a, :, :k] = abs(s) * (y.abs().T @ (ue + e * u.abs()))
        return (dX, H * dX.abs() + 1.01 * tol), (dA, 1.01 * tA), (dB, 1.01 * tB)


def _near(name, got, ref, tol):
    assert got.shape == ref.shape, name
    bad = ~((got.double() - ref).abs() <= tol)  # NaN is not within
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}: " \
                          f"{got[bad][0].item()} for {ref[bad][0].item()} +- {tol[bad][0].item()}"


SHAPES = [(128, 256), (192, 320), (640, 768), (64, 64), (512, 1024)]
TOKENS = [1, 2, 7, 9, 31, 32, 33, 63, 64, 65, 127, 200, 300, 777]
KINDS = ["random", "runs", "holes", "none", "one", "blocks"]
GRID = [(SHAPES[i % 5], n, KINDS[(i + j) % 6], [8, 16, 40, 64, 128][(i + 2 * j) % 5], [1, 3, 7, 40][(i + j) % 4],
         (i + j) % 2 == 1, ["int8", "plain", "e4m3"][(i + j) % 3])
        for i, n in enumerate(TOKENS) for j in range(3)]


def _name(g):
    (rows, cols), n, kind, r, count, vary, weight = g
    return f"{rows}x{cols}-n{n}-{kind}-r{r}-{count}{'-ranks' if vary else ''}-{weight}"


@pytest.mark.parametrize("g", GRID, ids=_name)
def test_forward(g):
    (rows, cols), n, kind, r, count, vary, weight = g
    c = Case(rows, cols, n, count, r, kind, vary, weight)
    Y, U = c.fwd()
    ws = torch.full((api.workspace_bytes(api.OP_MULTI_FWD, rows, cols, n, r),), 255, dtype=torch.uint8, device="cuda")
    Y2, _ = api.qlora_multi_fwd(c.w, c.pool, c.X, c.ids, ws=ws)  # no U, a workspace with leftovers
    Yr, Yt, Ur, Ut = c.forward_ref()
    _near("U", U, Ur, Ut)
    _near("Y", Y, Yr, Yt)
    assert torch.equal(Y, Y2)
    assert api.device_status(ws) == 0


@pytest.mark.parametrize("g", GRID, ids=_name)
def test_backward(g):
    (rows, cols), n, kind, r, count, vary, weight = g
    c = Case(rows, cols, n, count, r, kind, vary, weight)
    _, U = c.fwd()
    ws = torch.full((api.workspace_bytes(api.OP_MULTI_BWD, rows, cols, n, r),), 255, dtype=torch.uint8, device="cuda")
    out = [torch.full(s, float("nan"), dtype=d, device="cuda")  # every element has to be written
           for s, d in ((c.X.shape, torch.bfloat16), (c.A.shape, torch.float32), (c.B.shape, torch.float32))]
    got = c.bwd(U=U, dX=out[0], dA=out[1], dB=out[2], ws=ws)
    assert all(x is y for x, y in zip(got, out))
    for name, x, (ref, tol) in zip(("dX", "dA", "dB"), got, c.backward_ref(U=U)):
        _near(name, x, ref, tol)
    again = c.bwd()  # U recomputed
    for name, x, (ref, tol) in zip(("dX", "dA", "dB"), again, c.backward_ref()):
        _near(name + " without U", x, ref, tol)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert api.device_status(ws) == 0


@pytest.mark.parametrize("rows,cols,n", [(1024, 4096, 20), (1024, 4096, 48), (1024, 2048, 32), (1024, 11008, 12),
                                         (4096, 8192, 20), (4096, 8192, 16), (1024, 8192, 300)])
def test_forward_long_sums(rows, cols, n):
    c = Case(rows, cols, n, 9, 16, "random", True)
    Y, U = c.fwd()
    Yr, Yt, Ur, Ut = c.forward_ref()
    _near("U", U, Ur, Ut)
    _near("Y", Y, Yr, Yt)


def test_backward_many_tokens_of_one_adapter():
    """The sums over 5000 tokens keep fp32 accuracy in norm: far inside the bound, 2e-6 (an fp32 sum of n terms of
    random sign errs by about sqrt(n) u, the pair of bf16 values by 2^-17 / sqrt(3) of a term)."""
    c = Case(256, 512, 5000, 2, 16, "one")
    _, U = c.fwd()
    got = c.bwd(U=U)
    for name, x, (ref, tol) in zip(("dX", "dA", "dB"), got, c.backward_ref(U=U)):
        _near(name, x, ref, tol)
        if name != "dX":
            assert ((x.double() - ref).norm() / ref.norm()).item() < 5e-6


@pytest.mark.parametrize("n", [5, 32, 40, 64, 300])
@pytest.mark.parametrize("shape", [(192, 320), (256, 512)])
def test_what_is_not_finite_stays_with_its_own(n, shape):
    """Infinities and NaN in one adapter's factors, in one token, and past the ranks: the other tokens and adapters get
    the bits that they get without them, and the token or adapter itself is not finite."""
    rows, cols = shape
    clean = Case(rows, cols, n, 4, 16, "random", seed=3)
    clean.rank = torch.tensor([5, 16, 9, 16], dtype=torch.int32, device="cuda")
    clean.ids[1], clean.ids[2], clean.ids[3] = 1, 2, 3
    dirty = Case(rows, cols, n, 4, 16, "random", seed=3)
    dirty.rank, dirty.ids = clean.rank, clean.ids
    dirty.A[0, 5:], dirty.B[0, :, 5:], dirty.A[2, 9:] = float("nan"), float("inf"), float("-inf")  # past the ranks
    dirty.A[3, 2, 7], dirty.B[3, 5, 1], dirty.B[3, 6, 2] = float("inf"), float("nan"), float("-inf")
    dirty.X[2, 11], dirty.dY[2, 3] = float("nan"), float("inf")
    for c in (clean, dirty):
        c.pool = api.AdapterPool(c.A, c.B, c.s, c.rank)
    ids = clean.ids.cpu()
    hit = (ids == 3) | (torch.arange(n) == 2)
    keep = (~hit).nonzero()[:, 0].cuda()
    (Y0, U0), (Y1, U1) = clean.fwd(), dirty.fwd()
    assert torch.equal(Y0[keep], Y1[keep]) and torch.equal(U0[keep], U1[keep])
    assert torch.isnan(Y1[2]).all()
    assert not torch.isfinite(Y1[3, 5]) and not torch.isfinite(U1[3, 2])
    assert torch.isfinite(Y0).all()
    g0, g1 = clean.bwd(U=U0), dirty.bwd(U=U0)
    assert torch.equal(g0[0][keep], g1[0][keep])
    for a in (0, 1):
        assert torch.equal(g0[1][a], g1[1][a]) and torch.equal(g0[2][a], g1[2][a]), a
    assert not torch.isfinite(g1[0][3, 7]) and not torch.isfinite(g1[1][2, :9]).any()
    assert (g1[1][2, 9:] == 0).all() and (g1[2][2, :, 9:] == 0).all()


def test_infinite_factor_gives_its_own_tokens_the_signed_infinity():
    c = Case(256, 512, 100, 3, 16, "random", seed=5)
    c.B[1, 17, 4] = float("inf")
    Y, U = c.fwd()
    for t in (c.ids == 1).nonzero()[:, 0].tolist():
        assert Y[t, 17].item() == float("inf") * float(np.sign(U[t, 4].item() * c.s[1].item()))
    assert torch.isfinite(Y[c.ids != 1]).all()


@pytest.mark.parametrize("n", [5, 32, 40, 300])
@pytest.mark.parametrize("shape", [(192, 320), (256, 512)])
def test_rank_zero_adds_nothing_whatever_its_scale(n, shape):
    c = Case(*shape, n, 3, 16, "random", seed=9)
    c.ids[0] = 1
    c.s[1], c.rank = float("inf"), torch.tensor([7, 0, 16], dtype=torch.int32, device="cuda")
    c.pool = api.AdapterPool(c.A, c.B, c.s, c.rank)
    at = c.ids == 1
    Y, U = c.fwd()
    dX, dA, dB = c.bwd(U=U)
    c.ids = torch.where(at, -1, c.ids).int()  # the same without an adapter
    Y0, U0 = c.fwd()
    assert torch.equal(Y, Y0) and torch.equal(U, U0) and (U[at] == 0).all()
    assert torch.equal(dX, c.bwd(U=U0)[0]) and (dA[1] == 0).all() and (dB[1] == 0).all()


def test_gradients_agree_with_differences():
    """L = sum dY Y is linear in A, in B and in X each, so central differences of the float64 forward are its
    derivatives up to rounding; the kernels' gradients have to give the same along random directions."""
    c = Case(256, 320, 90, 3, 16, "holes", True, seed=8)
    _, U = c.fwd()
    dX, dA, dB = c.bwd(U=U)
    (_, tX), (_, tA), (_, tB) = c.backward_ref()
    loss = lambda **k: (c.dY.double() * c.forward_ref(**k)[0]).sum()  # noqa: E731
    gen = torch.Generator("cuda").manual_seed(1)
    for name, grad, tol in (("A", dA, tA), ("B", dB, tB), ("X", dX, tX)):
        x = getattr(c, name).double()
        for _ in range(3):
            d = torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)
            diff = (loss(**{name: x + 0.5 * d}) - loss(**{name: x - 0.5 * d})).item()
            got, allowed = (grad.double() * d).sum().item(), (tol * d.abs()).sum().item()
            assert abs(got - diff) <= allowed + 1e-9 * abs(diff), (name, got, diff, allowed)


@pytest.mark.parametrize("n", [17, 48, 200])
def test_same_bits_again_on_another_stream_and_from_a_graph(n):
    c = Case(256, 512, n, 5, 16, "random", True)
    Y, U = c.fwd()
    G = c.bwd(U=U)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Ys, Us = c.fwd()
        Gs = c.bwd(U=Us)
    torch.cuda.synchronize()
    assert torch.equal(Y, Ys) and torch.equal(U, Us) and all(torch.equal(a, b) for a, b in zip(G, Gs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Yg, Ug = c.fwd()
        Gg = c.bwd(U=Ug)
    # the tables and inputs may change between replays
    c.ids.copy_(c.ids.flip(0))
    c.A.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    Y2, U2_ = c.fwd()
    G2 = c.bwd(U=U2_)
    assert torch.equal(Yg, Y2) and torch.equal(Ug, U2_) and all(torch.equal(a, b) for a, b in zip(Gg, G2))
    assert not torch.equal(Y, Y2)


def test_two_calls_at_once_on_two_streams():
    cases = [Case(512, 1024, n, 6, 32, "random", seed=n) for n in (24, 300)]
    want = [c.fwd() + c.bwd() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(c.fwd() + c.bwd())
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i % 2]))


def test_rows_behind_the_batch_stay_as_they_were():
    c = Case(256, 512, 70, 3, 16, "random")
    for n in (1, 30, 33, 65):
        X, ids, dY = c.X[:n], c.ids[:n], c.dY[:n]
        Y, U, dX = (torch.full(s, 7.0, dtype=d, device="cuda") for s, d in
                    ((c.dY.shape, torch.bfloat16), ((70, 16), torch.float32), (c.X.shape, torch.bfloat16)))
        api.qlora_multi_fwd(c.w, c.pool, X, ids, Y=Y[:n], U_out=U[:n])
        api.qlora_multi_bwd(c.w, c.pool, X, ids, dY, U=U[:n], dX=dX[:n])
        for t in (Y, U, dX):
            assert (t[n:] == 7).all() and not (t[:n] == 7).all(), n


def test_views_into_larger_buffers():
    """Inputs and outputs that begin inside other allocations, 16 bytes from their start; what lies around stays."""
    c = Case(256, 512, 90, 3, 16, "random")
    Y0, U0 = c.fwd()
    G0 = c.bwd(U=U0)

    def inside(t, fill=7.0):
        skip = 16 // t.element_size()
        whole = torch.full((t.numel() + 2 * skip,), fill, dtype=t.dtype, device="cuda")
        view = whole[skip:-skip].view(t.shape)
        view.copy_(t)
        return whole, view, skip
    (_, X, _), (_, dY, _), (_, ids, _) = inside(c.X), inside(c.dY), inside(c.ids, 0)
    (_, A, _), (_, B, _) = inside(c.A), inside(c.B)
    pool = api.AdapterPool(A, B, c.s)
    outs = [inside(torch.zeros_like(t)) for t in (Y0, U0, *G0)]
    api.qlora_multi_fwd(c.w, pool, X, ids, Y=outs[0][1], U_out=outs[1][1])
    api.qlora_multi_bwd(c.w, pool, X, ids, dY, U=outs[1][1], dX=outs[2][1], dA=outs[3][1], dB=outs[4][1])
    for (whole, view, skip), ref in zip(outs, (Y0, U0, *G0)):
        assert torch.equal(view, ref)
        assert (whole[:skip] == 7).all() and (whole[-skip:] == 7).all()


def test_malformed_weights_are_refused():
    c = Case(256, 512, 5, 2, 8, "random")
    for bad in (dict(codes=c.w.codes[:-16]), dict(qabs=c.w.qabs[:-1]), dict(dq_scale=c.w.dq_scale[:-1])):
        w = api.NF4Weight(**dict(dict(codes=c.w.codes, rows=256, cols=512, qabs=c.w.qabs, dq_scale=c.w.dq_scale,
                                      dq_mean=c.w.dq_mean), **bad))
        with pytest.raises(ValueError, match="weight"):
            api.qlora_multi_fwd(w, c.pool, c.X, c.ids)


def test_one_adapter_agrees_with_the_single_adapter_call():
    """With one adapter for all tokens the two entry points compute the same thing: Y and dX within two bf16 roundings
    (and the rounding of U and G to bf16), through different kernels."""
    c = Case(256, 512, 100, 1, 16, "one")
    Y, _ = c.fwd()
    Y1, U1 = api.qlora_linear_fwd(c.w, c.X, c.A[0], c.B[0], float(c.s[0]))
    Yr, Yt, _, _ = c.forward_ref()
    _near("Y against the single call", Y, Y1.double(), 2 * Yt + H * Yr.abs())
    dX, dA, dB = c.bwd()
    dX1, dA1, dB1 = api.qlora_linear_bwd(c.w, c.X, c.A[0], c.B[0], float(c.s[0]), c.dY, U=U1)
    assert (dA[0] - dA1).norm() < H * dA1.norm() and (dB[0] - dB1).norm() < H * dB1.norm()


def test_adapters_train_together_and_serve():
    """As they are used: three adapters trained in one batch (forward, backward, the 8-bit AdamW step over all factors),
    the updated pool then serving single tokens.  The step's parameters agree with the 32-bit step's up to fp32
    rounding, since both start from zero states and the update uses states that have not been rounded to 8 bits yet:
    step one moves a parameter by at most lr (m / d S = lr g / (|g| + eps')), which the 32-bit kernel forms within
    10 units of 2^-24 and the 8-bit one within 16 (its root and quotient are the hardware's approximate ones); the decay
    is 1 here, and both round the difference p' once: 26 u lr + 2 u |p'|."""
    c = Case(256, 512, 150, 3, 16, "blocks", seed=2)
    masters = [c.A.float(), c.B.float()]
    other = [m.clone() for m in masters]
    grads = [torch.zeros_like(m) for m in masters]
    st = [api.adamw8_state(m) for m in masters]
    t8 = api.AdamW8Tensors([m.view(-1) for m in masters], [g.view(-1) for g in grads], *map(list, zip(*st)),
                           params_bf16=[c.A.view(-1), c.B.view(-1)])
    zeros = [[torch.zeros(m.numel(), device="cuda") for m in masters] for _ in range(2)]
    t32 = api.AdamWTensors([m.view(-1) for m in other], [g.view(-1) for g in grads], *zeros)
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    Y, U = c.fwd()
    api.qlora_multi_bwd(c.w, c.pool, c.X, c.ids, c.dY, U=U, dA=grads[0], dB=grads[1])
    before = (c.A.clone(), c.B.clone())
    api.adamw8_multi_step(t8, step, 1e-2)
    api.adamw_multi_step(t32, step, 1e-2)
    torch.cuda.synchronize()
    for a, b in zip(masters, other):
        _near("parameters", a, b.double(), 2.0 ** -24 * (26 * 1e-2 + 2 * b.double().abs()))
    assert torch.equal(c.A, masters[0].bfloat16()) and torch.equal(c.B, masters[1].bfloat16())
    assert not torch.equal(c.A, before[0]) and not torch.equal(c.B, before[1])
    X, ids = c.X[:9].contiguous(), torch.tensor([0, 1, 2, -1, 2, 1, 0, 0, 5], dtype=torch.int32, device="cuda")
    c.X, c.ids, c.n = X, ids, 9
    Y, U = c.fwd()
    Yr, Yt, Ur, Ut = c.forward_ref()
    _near("Y", Y, Yr, Yt)
    _near("U", U, Ur, Ut)


@pytest.mark.parametrize("rows,cols,n,r,vary", [(64, 64, 1500, 8, True), (128, 128, 900, 24, True), (256, 512, 1100, 128, False),
                                                (512, 1024, 290, 40, True)])
def test_largest_pool(rows, cols, n, r, vary):
    """Hundreds of adapters within one tile of tokens, chunks of several ranks, with and without a K split."""
    c = Case(rows, cols, n, 1024, r, "random", vary)
    Y, U = c.fwd()
    Yr, Yt, Ur, Ut = c.forward_ref()
    _near("Y", Y, Yr, Yt)
    for name, x, (ref, tol) in zip(("dX", "dA", "dB"), c.bwd(U=U), c.backward_ref(U=U)):
        _near(name, x, ref, tol)

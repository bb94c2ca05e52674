"""GPU parity of the list updates (qln_adamw_multi_step, qln_adamw8_multi_step)
against the formula in float64, one step from states of any size.

Tolerances, u = 2^-24 (fp32 rounding, half a step), the hyper-parameters being
the fp32 values themselves:
  m  two products and a sum:            3 u (|b1 m| + |(1-b1) g|)
  v  g^2, two products, a sum, all >= 0: 5 u v
  p  decay 3 u |p|, the final difference u |p'|, and the step S m / d with
     d = sqrt(v) i + eps: m's error / d, and S, i (u each), the root (2.5 u + u),
     its product, the sum, the quotient and the last product (u each): 10 u.
8-bit states are restored with one rounding (m) or two (v: the root's product,
then the square: 3 u on v) before the step, which adds u |b1 m| to m, 3 u to v
and 2 u to d.  That kernel takes the approximate root (2 u instead of u) and
quotient (4 u instead of u), so its step is within 16 u.  A code is the nearest
E4M3 value to y = x / b, b = max fp32(1/448): half a step is 2^-4 |y|, below 2^-6
the fixed 2^-10; the quotient, the constant and its product have a rounding
each (3 u); a root raised to the smallest code is off by less than 2^-9."""
import ctypes

import numpy as np
import pytest
import torch

from bit_nf4_quantized_07_b200 import api
from oracle import adamw

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F = lambda x: float(np.float32(x))  # noqa: E731
LR, B1, B2, EPS, WD = F(2e-3), F(0.9), F(0.995), F(1e-8), F(0.01)
SIZES = [1, 3, 255, 256, 257, 2047, 2048, 2049, 4096 + 8, 5000, 70000 + 7]
GUARD = 64  # elements behind every buffer that must stay as they were


class Buf:
    """A tensor of n elements with guard elements behind it."""

    def __init__(self, values, dtype=torch.float32):
        n = len(values)
        self.whole = torch.full((n + GUARD,), 3.0).to(dtype)
        self.whole[:n] = torch.as_tensor(values).to(dtype)
        self.whole = self.whole.cuda()
        self.t = self.whole[:n]

    def guard_intact(self):
        return bool((self.whole[len(self.t):].float() == 3.0).all())


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _lists(sizes, seed, bf16):
    g = _rng(seed)
    spread = lambda n: 10 ** g.uniform(-5, -1, n)  # noqa: E731
    d = dict(p=[], g=[], m=[], v=[], b=[])
    for n in sizes:
        s = spread(n)
        d["p"].append(Buf((g.standard_normal(n) * 0.02).astype(np.float32)))
        d["g"].append(Buf((g.standard_normal(n) * s).astype(np.float32)))
        d["m"].append(Buf((0.3 * g.standard_normal(n) * s).astype(np.float32)))
        d["v"].append(Buf(((g.standard_normal(n) * s) ** 2).astype(np.float32)))
        d["b"].append(Buf(np.zeros(n, np.float32), torch.bfloat16))
    if bf16 == "none":
        d["b"] = None
    elif bf16 == "some":
        d["b"] = [b if i % 2 else None for i, b in enumerate(d["b"])]
    return d


def _ts(bufs):
    return None if bufs is None else [b and b.t for b in bufs]


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _check_p(p, p0, g, m0, mref, vref, t, extra):
    """The parameter after the step, within the derived bound."""
    size, inv = LR / (1 - B1 ** t), 1 / np.sqrt(1 - B2 ** t)
    d = np.sqrt(vref) * inv + EPS
    pref = p0 * (1 - LR * WD) - size * mref / d
    mtol = (3 + (1 if extra else 0)) * U * (np.abs(B1 * m0) + np.abs((1 - B1) * g))
    tol = 3 * U * np.abs(p0) + U * np.abs(pref) + size * (mtol + (16 if extra else 10) * U * np.abs(mref)) / d
    bad = np.abs(p - pref) > 1.01 * tol
    assert not bad.any(), (np.flatnonzero(bad)[:4], p[bad][:4], pref[bad][:4])


@pytest.mark.parametrize("t", [0, 1, 2, 1000, 1000003])
@pytest.mark.parametrize("bf16", ["all", "none", "some"])
def test_list_matches_formula(t, bf16):
    d = _lists(SIZES, 100 + t % 97, bf16)
    before = {k: [_f64(b.t) for b in d[k]] for k in "pgmv"}
    tensors = api.AdamWTensors(_ts(d["p"]), _ts(d["g"]), _ts(d["m"]), _ts(d["v"]), _ts(d["b"]))
    step = torch.full((1,), t, dtype=torch.int64, device="cuda")
    launches = api.launch_count()
    api.adamw_multi_step(tensors, step, LR, (B1, B2), EPS, WD)
    assert api.launch_count() == launches + 1
    torch.cuda.synchronize()
    t = max(t, 1)
    for i, n in enumerate(SIZES):
        p0, g, m0, v0 = (before[k][i] for k in "pgmv")
        pr, mr, vr = adamw.adamw_step(p0, g, m0, v0, t, LR, B1, B2, EPS, WD)
        m, v, p = (_f64(d[k][i].t) for k in "mvp")
        assert (np.abs(m - mr) <= 3.03 * U * (np.abs(B1 * m0) + np.abs((1 - B1) * g))).all()
        assert (np.abs(v - vr) <= 5.05 * U * vr + 2e-45).all()
        _check_p(p, p0, g, m0, mr, vr, t, False)
        assert np.array_equal(_f64(d["g"][i].t), g)
        if d["b"] and d["b"][i]:
            assert torch.equal(d["b"][i].t, d["p"][i].t.to(torch.bfloat16))
    assert all(b.guard_intact() for k in d if d[k] for b in d[k] if b)


def test_many_tensors_take_several_launches():
    sizes = [8 + i % 23 for i in range(1100)]
    d = _lists(sizes, 3, "none")
    e = _lists(sizes, 3, "none")
    step = torch.full((1,), 7, dtype=torch.int64, device="cuda")
    launches = api.launch_count()
    api.adamw_multi_step(api.AdamWTensors(*(_ts(d[k]) for k in "pgmv")), step, LR, (B1, B2), EPS, WD)
    assert api.launch_count() == launches + 3
    one = api.AdamWTensors([e["p"][1099].t], [e["g"][1099].t], [e["m"][1099].t], [e["v"][1099].t])
    api.adamw_multi_step(one, step, LR, (B1, B2), EPS, WD)
    torch.cuda.synchronize()
    assert all(torch.equal(d[k][1099].t, e[k][1099].t) for k in "pmv")
    assert all(not torch.equal(d["p"][i].t, e["p"][i].t) for i in range(1099))


# ---- 8-bit states ---------------------------------------------------------------
def _blocks(x):
    """[ceil(n / 256)][256], zero-padded."""
    return np.pad(x, (0, -len(x) % 256)).reshape(-1, 256)


def _restore(code, scale):
    c = _blocks(_f64(code)).astype(np.float32)
    return (c * scale.cpu().numpy()[:, None]).reshape(-1)[: len(code)].astype(np.float64)


def _lists8(sizes, seed, bf16, fresh=False):
    d = _lists(sizes, seed, bf16)
    d["ms"], d["vs"] = [], []
    for i, n in enumerate(sizes):
        for k, ks in (("m", "ms"), ("v", "vs")):
            x = _blocks(_f64(d[k][i].t) if k == "m" else np.sqrt(_f64(d[k][i].t)))
            b = (np.abs(x).max(1) / 448).astype(np.float32)
            y = x / np.where(b > 0, b, 1)[:, None]
            if k == "v":
                y = np.where(x > 0, np.maximum(y, 2.0 ** -9), 0)
            if fresh:
                b, y = b * 0, y * 0
            d[k][i] = Buf(torch.from_numpy(y.reshape(-1)[:n].astype(np.float32)), torch.float8_e4m3fn)
            d[ks].append(Buf(b))
    return d


def _tensors8(d):
    return api.AdamW8Tensors(*(_ts(d[k]) for k in ("p", "g", "m", "ms", "v", "vs", "b")))


def _check_state(code, scale, ref, ref_tol, root):
    """Codes and scales of a state against the float64 values it stands for."""
    x, tol = _blocks(ref), _blocks(ref_tol)
    b = scale.cpu().numpy().astype(np.float64)
    bmax = np.abs(x).max(1)
    assert (np.abs(b - bmax / 448) <= (tol.max(1) + 3 * U * bmax) / 448 + 2e-45).all()
    y = x / np.where(b > 0, b, 1)[:, None]
    ytol = tol / np.where(b > 0, b, 1)[:, None] + 3 * U * np.abs(y)
    half = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10)
    if root:
        half = np.where((y > 0) & (y < 2.0 ** -9), 2.0 ** -9, half)
    got = _blocks(_f64(code))
    bad = np.abs(got - y) > 1.07 * ytol + half
    assert not bad.any(), (got[bad][:4], y[bad][:4])
    assert (got[x == 0] == 0).all()
    if root:
        assert ((got > 0) | (x == 0)).all()


@pytest.mark.parametrize("t", [1, 2, 1000])
@pytest.mark.parametrize("bf16", ["all", "some"])
@pytest.mark.parametrize("fresh", [False, True])
def test_8bit_list_matches_formula(t, bf16, fresh):
    d = _lists8(SIZES, 200 + t % 89, bf16, fresh)
    before = [(_f64(d["p"][i].t), _f64(d["g"][i].t), _restore(d["m"][i].t, d["ms"][i].t),
               _restore(d["v"][i].t, d["vs"][i].t)) for i in range(len(SIZES))]
    step = torch.full((1,), t, dtype=torch.int64, device="cuda")
    api.adamw8_multi_step(_tensors8(d), step, LR, (B1, B2), EPS, WD)
    torch.cuda.synchronize()
    for i, n in enumerate(SIZES):
        p0, g, m0, r0 = before[i]
        pr, mr, vr = adamw.adamw_step(p0, g, m0, r0 * r0, t, LR, B1, B2, EPS, WD)
        _check_p(_f64(d["p"][i].t), p0, g, m0, mr, vr, t, True)
        _check_state(d["m"][i].t, d["ms"][i].t, mr, 4 * U * (np.abs(B1 * m0) + np.abs((1 - B1) * g)), False)
        _check_state(d["v"][i].t, d["vs"][i].t, np.sqrt(vr), 5 * U * np.sqrt(vr), True)
        if d["b"] and d["b"][i]:
            assert torch.equal(d["b"][i].t, d["p"][i].t.to(torch.bfloat16))
    assert all(b.guard_intact() for k in d if d[k] for b in d[k] if b)


def test_8bit_states_are_the_bits_of_their_definition():
    """The states in fp32, every operation correctly rounded (numpy's are; a fused product is formed in float64, where
    the product of two fp32 values is exact), and their codes: the same bits, the rare ones beside the middle of two
    codes among them."""
    n = 1 << 20
    d = _lists8([n], 31, "none")
    g, f = _f64(d["g"][0].t).astype(np.float32), np.float32
    m0 = _restore(d["m"][0].t, d["ms"][0].t).astype(f)
    r0 = _restore(d["v"][0].t, d["vs"][0].t).astype(f)
    api.adamw8_multi_step(_tensors8(d), torch.full((1,), 77, dtype=torch.int64, device="cuda"), LR, (B1, B2), EPS, WD)
    b1, b2, c1, c2 = f(B1), f(B2), f(1) - f(B1), f(1) - f(B2)
    fma = lambda a, b, c: (a.astype(np.float64) * b + c).astype(f)  # noqa: E731
    m = fma(g, c1, b1 * m0)
    v = fma(g * g, c2, b2 * (r0 * r0))
    for x, code, scale, root in ((m, "m", "ms", False), (np.sqrt(v), "v", "vs", True)):
        x = _blocks(x)
        b = np.abs(x).max(1) * (f(1) / f(448))
        y = x / b[:, None]
        if root:
            y = np.where(x > 0, np.maximum(y, f(2.0 ** -9)), y)
        want = torch.from_numpy(y.reshape(-1)[:n]).to(torch.float8_e4m3fn)
        assert np.array_equal(d[scale][0].t.cpu().numpy(), b)
        assert torch.equal(d[code][0].t.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("top", [1e-30, 1e-36, 3e-38, 1e-41, 1e-44])
def test_8bit_states_of_tiny_gradients(top):
    """Blocks whose scale is subnormal or zero: m keeps the codes of its definition, or zeros."""
    n, f = 512, np.float32
    g = (np.linspace(-1, 1, n) * top).astype(f)
    d = {k: torch.zeros(n, device="cuda") for k in ("p", "g")}
    d["g"].copy_(torch.from_numpy(g))
    m, ms, v, vs = api.adamw8_state(d["p"])
    api.adamw8_multi_step(api.AdamW8Tensors([d["p"]], [d["g"]], [m], [ms], [v], [vs]),
                          torch.ones(1, dtype=torch.int64, device="cuda"), LR, (B1, B2), EPS, WD)
    x = _blocks(g * (f(1) - f(B1)))
    b = np.abs(x).max(1) * (f(1) / f(448))
    y = np.where(b[:, None] > 0, x / np.where(b > 0, b, f(1))[:, None], f(0))
    assert np.array_equal(ms.cpu().numpy(), b)
    assert torch.equal(m.cpu().float(), torch.from_numpy(y.reshape(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).float())
    assert torch.isfinite(v.float()).all() and torch.isfinite(d["p"]).all()


def test_8bit_zero_gradients_and_states_only_decay():
    n = 700
    p0 = torch.randn(n, device="cuda")
    p = p0.clone()
    m, ms, v, vs = api.adamw8_state(p)
    t = api.AdamW8Tensors([p], [torch.zeros(n, device="cuda")], [m], [ms], [v], [vs])
    api.adamw8_multi_step(t, torch.ones(1, dtype=torch.int64, device="cuda"), LR, (B1, B2), EPS, WD)
    assert torch.equal(p, p0 * (np.float32(1) - np.float32(LR) * np.float32(WD)))
    assert all(not x.float().any() for x in (m, ms, v, vs))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 1e30])
def test_8bit_a_bad_gradient_spoils_its_own_element_only(value):
    """1e30 squares to infinity: its root is not finite, its m is."""
    n, at = 1000, 300
    d, e = _lists8([n], 9, "none"), _lists8([n], 9, "none")
    d["g"][0].t[at] = value
    e["g"][0].t[at] = 0.0
    step = torch.full((1,), 5, dtype=torch.int64, device="cuda")
    for x in (d, e):
        api.adamw8_multi_step(_tensors8(x), step, LR, (B1, B2), EPS, WD)
    other = torch.arange(n, device="cuda") != at
    block = torch.arange(n, device="cuda") // 256 == at // 256
    for k in ("p", "v", "vs"):
        same = d[k][0].t.float() == e[k][0].t.float()
        assert bool(same[other].all() if k != "vs" else same.all()), k
    assert torch.isnan(d["v"][0].t.float()[at])
    if value != 1e30:  # a finite m sets its block's scale; what is infinite does not
        assert torch.isnan(d["p"][0].t[at]) and torch.isnan(d["m"][0].t.float()[at])
        assert torch.equal(d["m"][0].t.float()[other], e["m"][0].t.float()[other])
    else:
        assert torch.equal(d["m"][0].t.float()[~block], e["m"][0].t.float()[~block])


def test_8bit_follows_32bit_over_steps():
    """Twenty steps: a restored state is the stored one within a code's
    half-step, and the decayed sum of those errors bounds the difference of the
    first moments: sum of b1^k 2^-4 < 10 half-steps of the largest moment."""
    n = 3000
    g = _rng(5)
    p = [torch.from_numpy((g.standard_normal(n) * 0.02).astype(np.float32)).cuda() for _ in range(2)]
    p[1].copy_(p[0])
    grad = torch.zeros(n, device="cuda")
    m32, v32 = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    m, ms, v, vs = api.adamw8_state(p[1])
    t32 = api.AdamWTensors([p[0]], [grad], [m32], [v32])
    t8 = api.AdamW8Tensors([p[1]], [grad], [m], [ms], [v], [vs])
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    env = np.zeros(n)
    for k in range(20):
        step += 1
        grad.copy_(torch.from_numpy(g.standard_normal(n).astype(np.float32)))
        api.adamw_multi_step(t32, step, LR, (B1, B2), EPS, WD)
        api.adamw8_multi_step(t8, step, LR, (B1, B2), EPS, WD)
        full = _blocks(_f64(m32))
        top = np.abs(full).max(1, keepdims=True)
        half = np.maximum(2.0 ** -4 * np.abs(full), 2.0 ** -10 * top / 448).reshape(-1)[:n]
        env = (1 + 2.0 ** -4) * B1 * env + 1.01 * half  # the error of the state carried on, and this step's own
        assert (np.abs(_restore(m, ms) - _f64(m32)) <= env + 2.0 ** -4 * env).all()


def test_graph_replay_reads_the_device_step_and_other_streams_work():
    d, e = _lists8([5000, 257], 17, "all"), _lists8([5000, 257], 17, "all")
    td, te = _tensors8(d), _tensors8(e)
    step_d, step_e = (torch.zeros(1, dtype=torch.int64, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_d.add_(1)
        api.adamw8_multi_step(td, step_d, LR, (B1, B2), EPS, WD)
    del td  # a captured launch holds its own table
    for _ in range(3):
        graph.replay()
    with torch.cuda.stream(side):
        for _ in range(3):
            step_e.add_(1)
            api.adamw8_multi_step(te, step_e, LR, (B1, B2), EPS, WD)
    torch.cuda.synchronize()
    for k in ("p", "m", "ms", "v", "vs", "b"):
        assert all(torch.equal(x.t.float(), y.t.float()) for x, y in zip(d[k], e[k])), k


def test_misaligned_views_are_refused():
    x = [torch.zeros(300, device="cuda") for _ in range(4)]
    t = api.AdamWTensors([x[0][1:257]], [x[1][:256]], [x[2][:256]], [x[3][:256]])
    with pytest.raises(api.QLNError, match="ALIGN"):
        api.adamw_multi_step(t, torch.ones(1, dtype=torch.int64, device="cuda"), LR)


@pytest.mark.parametrize("eight", [False, True])
def test_managed_states_paged_in_and_out(eight):
    """States in unified memory, prefetched in and back to the host: the same
    bits as in device memory."""
    from cuda.bindings import runtime as cudart
    n = 20000 + 5
    d = (_lists8 if eight else _lists)([n], 23, "none")
    e = (_lists8 if eight else _lists)([n], 23, "none")
    names = ("m", "ms", "v", "vs") if eight else ("m", "v")
    ptrs, host = {}, {}
    try:
        for k in names:
            t = d[k][0].t
            raw = t.view(torch.uint8).cpu().numpy()
            err, ptr = cudart.cudaMallocManaged(len(raw), cudart.cudaMemAttachGlobal)
            assert err == cudart.cudaError_t.cudaSuccess
            ptrs[k] = int(ptr)
            host[k] = np.ctypeslib.as_array(ctypes.cast(int(ptr), ctypes.POINTER(ctypes.c_uint8)), shape=(len(raw),))
            host[k][:] = raw
        P = lambda b: b.t.data_ptr()  # noqa: E731
        if eight:
            arr = (api.CAdamW8Tensor * 1)(api.CAdamW8Tensor(P(d["p"][0]), P(d["g"][0]), ptrs["m"], ptrs["ms"], ptrs["v"],
                                                            ptrs["vs"], None, n))
        else:
            arr = (api.CAdamWTensor * 1)(api.CAdamWTensor(P(d["p"][0]), P(d["g"][0]), ptrs["m"], ptrs["v"], None, n))
        step = torch.full((1,), 4, dtype=torch.int64, device="cuda")
        cfg = api.CAdamWConfig(LR, B1, B2, EPS, WD)
        fn = api.lib().qln_adamw8_multi_step if eight else api.lib().qln_adamw_multi_step
        for _ in range(2):
            assert fn(arr, 1, ctypes.byref(cfg), ctypes.c_void_p(step.data_ptr()),
                      api.ADAMW_PAGE_IN | api.ADAMW_PAGE_OUT, api._stream()) == 0
            if eight:
                api.adamw8_multi_step(_tensors8(e), step, LR, (B1, B2), EPS, WD)
            else:
                api.adamw_multi_step(api.AdamWTensors(*(_ts(e[k]) for k in "pgmv")), step, LR, (B1, B2), EPS, WD)
        torch.cuda.synchronize()
        for k in names:
            assert np.array_equal(host[k], e[k][0].t.view(torch.uint8).cpu().numpy()), k
        assert torch.equal(d["p"][0].t, e["p"][0].t)
    finally:
        for p in ptrs.values():
            cudart.cudaFree(p)

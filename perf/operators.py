"""The measured cases of the operators for many adapters: their inputs, their
plain forms in elementary torch operations, and their values in 64 bits.

Operators (``own`` calls them through ``bit_nf4_quantized_07_b200.api``):

fwd     Y = X W'^T + s_a (X A_a^T) B_a^T, each row t of X with the adapter
        a = ids[t] of a pool, over one NF4 projection W (qlora_multi_fwd).
bwd     dX, and dA, dB of every adapter of the pool (qlora_multi_bwd).
adamw   one AdamW step over many tensors, 32-bit states (adamw_multi_step).
adamw8  the same with 8-bit states in blocks of 256 (adamw8_multi_step).
"""
import math

import numpy as np
import torch

own = False

# The NF4 book as the library holds it (fp32 bit patterns).
_BOOK = np.array([0xbf800000, 0xbf3239b1, 0xbf066b2e, 0xbeca329e, 0xbe91a24b, 0xbe3d353d, 0xbdba7869, 0x00000000,
                  0x3da2fb01, 0x3e24cadf, 0x3e7c04da, 0x3ead0336, 0x3ee1a4b5, 0x3f1007a9, 0x3f3913b0, 0x3f800000],
                 dtype=np.uint32).view(np.float32)

# AdamW hyper-parameters; the library takes them as fp32 values.
_LR, _B1, _B2, _EPS, _WD = (float(np.float32(x)) for x in (2e-4, 0.9, 0.999, 1e-8, 0.01))
_BLOCK = 256  # elements of one 8-bit state block


def listed():
    return [
        # Serving, single tokens: one request alone on an attention projection.
        dict(name="fwd 1 token", op="fwd", rows=4096, cols=4096, n=1, count=4, r=16, ids="each", vary=False, u=False),
        # Serving, single tokens: a full decode batch, every request with its own adapter.
        dict(name="fwd 32 requests", op="fwd", rows=4096, cols=4096, n=32, count=32, r=16, ids="each", vary=False, u=False),
        # Serving, single tokens on the MLP's down projection, adapters of several ranks.
        dict(name="fwd 12 down", op="fwd", rows=4096, cols=11008, n=12, count=6, r=64, ids="each", vary=True, u=False),
        # Serving, a mixed step: some prompt pieces, single tokens and rows of the base model between them.
        dict(name="fwd 203 mixed", op="fwd", rows=11008, cols=4096, n=203, count=24, r=32, ids="mixed", vary=True, u=False),
        # Training or prefill: eight packed sequences of different lengths; U kept for the backward pass.
        dict(name="fwd packed", op="fwd", rows=11008, cols=4096, n=2048, count=8, r=16, ids="packed", vary=False, u=True),
        # Training: a short ragged batch on an attention projection, small and odd ranks.
        dict(name="bwd ragged", op="bwd", rows=4096, cols=4096, n=333, count=5, r=8, ids="mixed", vary=True),
        # Training: four packed sequences on the MLP's up projection.
        dict(name="bwd packed", op="bwd", rows=11008, cols=4096, n=2048, count=4, r=16, ids="packed", vary=False),
        # Training: the largest projection, eight adapters of rank 64.
        dict(name="bwd large", op="bwd", rows=28672, cols=8192, n=4096, count=8, r=64, ids="packed", vary=False),
        # Optimizer: the factors of one layer; latency counts.
        dict(name="adamw layer", op="adamw", layers=1, dim=4096, hidden=11008, r=8, odd=False),
        # Optimizer: the factors of a whole model of 32 layers.
        dict(name="adamw model", op="adamw", layers=32, dim=4096, hidden=11008, r=16, odd=False),
        # Optimizer with 8-bit states: one layer with odd tensor sizes, and the whole model.
        dict(name="adamw8 layer", op="adamw8", layers=1, dim=4095, hidden=11007, r=7, odd=True),
        dict(name="adamw8 model", op="adamw8", layers=32, dim=4096, hidden=11008, r=16, odd=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "adamw", "adamw8"])
    if op in ("adamw", "adamw8"):
        odd = rng.random() < 0.5
        dim, hidden = rng.choice([(512, 1408), (1024, 2816), (2048, 5504), (4096, 11008)])
        return dict(op=op, layers=_log(rng, 1, 32), dim=dim - odd * rng.randrange(1, 9), hidden=hidden - odd * rng.randrange(1, 9),
                    r=rng.randrange(1, 17) if odd else rng.choice([4, 8, 12, 16]), odd=odd)
    rows = rng.choice([512, 1024, 2048, 4096, 5120, 8192, 11008])
    cols = rng.choice([512, 1024, 2048, 4096, 5120, 8192])
    n = _log(rng, 1, 4096) if op == "fwd" else _log(rng, 16, 4096)
    case = dict(op=op, rows=rows, cols=cols, n=n, count=_log(rng, 1, 48), r=8 * _log(rng, 1, 16),
                ids="each" if n <= 48 else rng.choice(["packed", "mixed"]), vary=rng.random() < 0.5)
    if op == "fwd":
        case["u"] = rng.random() < 0.3
    return case


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed(1000003 * seed + salt)


def _normal(seed, salt, shape, std, dtype=torch.float32):
    return (torch.randn(shape, generator=_gen(seed, salt), device="cuda") * std).to(dtype)


def _nf4(seed, rows, cols):
    """A Gaussian weight, quantized: codes, int8 codes of the block constants, their scales and mean."""
    book = torch.from_numpy(_BOOK).cuda()
    w = _normal(seed, 1, (rows * cols // 64, 64), 0.02)
    absmax = w.abs().amax(1)
    q = torch.bucketize((w / absmax[:, None]).view(-1), (book[1:] + book[:-1]) / 2, out_int32=True).to(torch.uint8)
    codes = (q[0::2] << 4) | q[1::2]
    mean = absmax.mean().view(1)
    d = torch.nn.functional.pad(absmax - mean, (0, -len(absmax) % 256)).view(-1, 256)
    scale = d.abs().amax(1) / 127
    qabs = torch.where(scale[:, None] > 0, d / scale[:, None], 0.0).round().clamp(-127, 127).to(torch.int8).view(-1)
    return dict(codes=codes, qabs=qabs[: len(absmax)].clone(), scale=scale, mean=mean, rows=rows, cols=cols)


def _ids(case, seed):
    """The adapter of every row. "each": the requests' own; "packed": sequences one after the other; "mixed": sequences,
    single rows and rows without an adapter (-1) in any order."""
    n, count = case["n"], case["count"]
    rng = np.random.default_rng([seed, 7])
    perm = rng.permutation(count)
    if case["ids"] == "each":
        ids = perm[np.arange(n) % count]
    elif case["ids"] == "packed":
        cuts = np.sort(rng.integers(0, n + 1, count - 1))
        ids = perm[np.searchsorted(cuts, np.arange(n), side="right")]
    else:
        runs = np.maximum(1, rng.geometric(1.0 / max(2, n // (2 * count)), n))
        who = np.where(rng.random(n) < 0.1, -1, perm[np.arange(n) % count])
        ids = np.repeat(who, runs)[:n]
    return torch.from_numpy(ids.astype(np.int32)).cuda()


def _sizes(case):
    """Elements of A and B of the seven projections of every layer."""
    d, h, r = case["dim"], case["hidden"], case["r"]
    one = [d * r] * 8 + [d * r, h * r] * 2 + [h * r, d * r]
    return one * case["layers"]


def _round(n):
    return -(-n // _BLOCK) * _BLOCK


def _e4m3(x, keep):
    """Blocks of 256 of fp32 `x` as E4M3 codes and scales; with `keep`, no positive value becomes zero."""
    x = x.view(-1, _BLOCK)
    scale = x.abs().amax(1) / 448
    q = torch.where(scale[:, None] > 0, x / scale[:, None], 0.0)
    if keep:
        q = torch.where(x > 0, q.clamp_min(2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn).view(-1), scale


def prepare(case, seed):
    if case["op"] in ("adamw", "adamw8"):
        # the tensors are views of one buffer, as an optimizer with flat storage keeps them; each begins a block of 256
        sizes = _sizes(case)
        at = np.concatenate([[0], np.cumsum([_round(k) for k in sizes])])
        total = int(at[-1])
        real = torch.zeros(total, dtype=torch.bool, device="cuda")
        for a, k in zip(at, sizes):
            real[a: a + k] = True
        mag = torch.exp(2.0 * _normal(seed, 5, total, 1.0)) * 1e-4  # gradients of different sizes within a block
        flat = dict(p=_normal(seed, 1, total, 0.02) * real, g=_normal(seed, 2, total, 1.0) * mag * real,
                    m=0.3 * _normal(seed, 3, total, 1.0) * mag * real, v=(_normal(seed, 4, total, 1.0) * mag).square() * real)
        flat["p16"] = flat["p"].bfloat16()
        if case["op"] == "adamw8":
            flat["m"], flat["ms"] = _e4m3(flat["m"], False)
            flat["v"], flat["vs"] = _e4m3(flat["v"].sqrt(), True)
        state = dict(case=case, flat=flat, step=torch.full((1,), 1000, dtype=torch.int64, device="cuda"))
        if own:
            from bit_nf4_quantized_07_b200 import api
            cut = {key: [t[a // (_BLOCK if key in ("ms", "vs") else 1):][: (-(-k // _BLOCK) if key in ("ms", "vs") else k)]
                         for a, k in zip(at.tolist(), sizes)] for key, t in flat.items()}
            if case["op"] == "adamw":
                state["tensors"] = api.AdamWTensors(cut["p"], cut["g"], cut["m"], cut["v"], cut["p16"])
            else:
                state["tensors"] = api.AdamW8Tensors(cut["p"], cut["g"], cut["m"], cut["ms"], cut["v"], cut["vs"], cut["p16"])
        return state
    rows, cols, n, count, r = (case[k] for k in ("rows", "cols", "n", "count", "r"))
    rng = np.random.default_rng([seed, 11])
    state = dict(case=case, w=_nf4(seed, rows, cols), X=_normal(seed, 2, (n, cols), 1.0, torch.bfloat16),
                 A=_normal(seed, 3, (count, r, cols), 0.02, torch.bfloat16),
                 B=_normal(seed, 4, (count, rows, r), 0.02, torch.bfloat16),
                 s=torch.from_numpy(rng.uniform(0.5, 2.0, count).astype(np.float32)).cuda(),
                 rank=torch.from_numpy(rng.integers(1, r + 1, count).astype(np.int32)).cuda() if case["vary"] else None,
                 ids=_ids(case, seed))
    if case["op"] == "bwd":
        state["dY"] = _normal(seed, 5, (n, rows), 1.0, torch.bfloat16)
        state["U"] = _down(state["X"], state["A"], state).clone()
    if own:
        from bit_nf4_quantized_07_b200 import api
        w = state["w"]
        state["W"] = api.NF4Weight(codes=w["codes"], rows=rows, cols=cols, qabs=w["qabs"], dq_scale=w["scale"], dq_mean=w["mean"])
        state["pool"] = api.AdapterPool(state["A"], state["B"], state["s"], state["rank"])
    return state


# --------------------------------------------------------------------------
# plain forms (fp32)
# --------------------------------------------------------------------------
def _weight(w):
    """doubleDequant: w' = bf16(fp32(ahat c)), ahat = fp32(mu + fp32(b rhat)), as fp32 [rows][cols]."""
    book = torch.from_numpy(_BOOK).cuda()
    ahat = w["mean"] + w["scale"].repeat_interleave(256)[: len(w["qabs"])] * w["qabs"].float()
    c = torch.stack((book[(w["codes"] >> 4).int()], book[(w["codes"] & 15).int()]), 1).view(-1, 64)
    return (ahat[:, None] * c).bfloat16().float().view(w["rows"], w["cols"])


def _used(state):
    """Rows x (adapter, column of its rank): which entries of a [n][count * r] product belong to the row's adapter."""
    count, r = state["case"]["count"], state["case"]["r"]
    col = torch.arange(count * r, device="cuda")
    used = (col // r)[None, :] == state["ids"][:, None]
    return used if state["rank"] is None else used & (col % r < state["rank"].repeat_interleave(r))[None, :]


def _down(x, f, state):
    """[n][r]: x times the transposed factor (A as stored, B with its last two axes exchanged) of the row's adapter."""
    count, r, k = f.shape
    n = x.shape[0]
    every = torch.where(_used(state), x.float() @ f.float().reshape(count * r, k).T, 0.0)
    return every.view(n, count, r).sum(1)


def _placed(u, state):
    """[n][count * r]: s u in the columns of the row's adapter, zero elsewhere."""
    count, r = state["case"]["count"], state["case"]["r"]
    return torch.where(_used(state), u.repeat(1, count) * state["s"].repeat_interleave(r), 0.0)


def _fwd(state):
    A, B, X = state["A"], state["B"], state["X"].float()
    u = _down(X, A, state)
    y = X @ _weight(state["w"]).T + _placed(u, state) @ B.float().transpose(1, 2).reshape(-1, B.shape[1])
    return (y.bfloat16(), u) if state["case"]["u"] else y.bfloat16()


def _bwd(state):
    A, B, X, dY = state["A"], state["B"], state["X"].float(), state["dY"].float()
    count, r = state["case"]["count"], state["case"]["r"]
    sg = _placed(_down(dY, B.transpose(1, 2), state), state)
    dX = dY @ _weight(state["w"]) + sg @ A.float().reshape(count * r, -1)
    dA = (sg.T @ X).view(count, r, -1)
    dB = (_placed(state["U"], state).T @ dY).view(count, r, -1).transpose(1, 2).contiguous()
    return dX.bfloat16(), dA, dB


def _update(f, m, v, step):
    """AdamW on flat fp32 tensors; p in place, the new m and v are returned (m and v are overwritten)."""
    t = step.double()
    size = (_LR / (1 - _B1 ** t)).float()
    inv = (1 - _B2 ** t).rsqrt().float()
    m.mul_(_B1).add_(f["g"], alpha=1 - _B1)
    v.mul_(_B2).addcmul_(f["g"], f["g"], value=1 - _B2)
    f["p"].mul_(1 - _LR * _WD).sub_(size * m / (v.sqrt() * inv + _EPS))
    f["p16"].copy_(f["p"])
    return m, v


def _plain(state):
    op, f = state["case"]["op"], state.get("flat")
    if op == "fwd":
        return _fwd(state)
    if op == "bwd":
        return _bwd(state)
    if op == "adamw":
        _update(f, f["m"], f["v"], state["step"])
        return f["p"], f["m"], f["v"], f["p16"]
    wide = lambda q, s: (q.float().view(-1, _BLOCK) * s[:, None]).view(-1)  # noqa: E731
    m, v = _update(f, wide(f["m"], f["ms"]), wide(f["v"], f["vs"]).square(), state["step"])
    (f["m"], f["ms"]), (f["v"], f["vs"]) = _e4m3(m, False), _e4m3(v.sqrt(), True)
    return f["p"], f["m"], f["ms"], f["v"], f["vs"], f["p16"]


def run(state):
    if not own:
        return _plain(state)
    from bit_nf4_quantized_07_b200 import api
    case, f = state["case"], state.get("flat")
    if case["op"] == "fwd":
        y, u = api.qlora_multi_fwd(state["W"], state["pool"], state["X"], state["ids"], want_u=case["u"])
        return (y, u) if case["u"] else y
    if case["op"] == "bwd":
        return api.qlora_multi_bwd(state["W"], state["pool"], state["X"], state["ids"], state["dY"], U=state["U"])
    if case["op"] == "adamw":
        api.adamw_multi_step(state["tensors"], state["step"], _LR, (_B1, _B2), _EPS, _WD)
        return f["p"], f["m"], f["v"], f["p16"]
    api.adamw8_multi_step(state["tensors"], state["step"], _LR, (_B1, _B2), _EPS, _WD)
    return f["p"], f["m"], f["ms"], f["v"], f["vs"], f["p16"]


# --------------------------------------------------------------------------
# work and the values in 64 bits
# --------------------------------------------------------------------------
def work(case):
    if case["op"] in ("adamw", "adamw8"):
        k = sum(_sizes(case))
        blocks = sum(_round(s) // _BLOCK for s in _sizes(case))
        # p, g read; p, bf16 copy written; the states read and written
        return dict(bytes=k * 14 + (k * 16 if case["op"] == "adamw" else k * 4 + blocks * 16), flops=k * 16)
    rows, cols, n, count, r = (case[k] for k in ("rows", "cols", "n", "count", "r"))
    weight = rows * cols * (1 / 2 + 1 / 64 + 4 / 16384)
    factors = min(count, n) * r * (rows + cols) * 2
    if case["op"] == "fwd":
        return dict(bytes=weight + factors + 2 * n * (rows + cols) + 4 * n + 4 * n * r * case["u"],
                    flops=2 * n * (rows * cols + r * (rows + cols)))
    return dict(bytes=weight + factors + 4 * n * (rows + cols) + 4 * n + 4 * n * r + 4 * count * r * (rows + cols),
                flops=2 * n * (rows * cols + 2 * r * (rows + cols)))


def exact(case, seed):
    global own
    kept, own = own, False
    s = prepare(case, seed)
    own = kept
    if case["op"] in ("adamw", "adamw8"):
        f, eight = s["flat"], case["op"] == "adamw8"
        p, g = f["p"].double(), f["g"].double()
        if eight:
            m = f["m"].double() * f["ms"].double().repeat_interleave(_BLOCK)
            v = (f["v"].double() * f["vs"].double().repeat_interleave(_BLOCK)) ** 2
        else:
            m, v = f["m"].double(), f["v"].double()
        t = int(s["step"].item())
        m = _B1 * m + (1 - _B1) * g
        v = _B2 * v + (1 - _B2) * g * g
        p = p - _LR * _WD * p - _LR * (m / (1 - _B1 ** t)) / ((v / (1 - _B2 ** t)) ** 0.5 + _EPS)
        if not eight:
            return p, m, v, p
        out = [p]
        for x, keep in ((m, False), (v ** 0.5, True)):
            b = x.view(-1, _BLOCK).abs().max(1).values / 448
            y = x / b.repeat_interleave(_BLOCK)
            y[x == 0] = 0
            if keep:
                y[(x > 0) & (y < 2.0 ** -9)] = 2.0 ** -9
            out += [y.float().to(torch.float8_e4m3fn), b]
        return (*out, p)
    w, ids = s["w"], s["ids"].long()
    book = torch.from_numpy(_BOOK.astype(np.float64)).cuda()
    b = w["scale"].double()[torch.arange(len(w["qabs"]), device="cuda") // 256]
    ahat = (w["mean"].double() + (b * w["qabs"].double()).float().double()).float().double()  # fp32 roundings are part of the definition
    both = torch.empty(len(w["codes"]), 2, dtype=torch.float64, device="cuda")
    both[:, 0], both[:, 1] = book[(w["codes"].int() // 16)], book[(w["codes"].int() % 16)]
    W = (both.view(-1, 64) * ahat[:, None]).float().bfloat16().double().view(case["rows"], case["cols"])
    X = s["X"].double()
    rank = [case["r"]] * case["count"] if s["rank"] is None else s["rank"].tolist()
    if case["op"] == "fwd":
        Y = X @ W.T
        U = torch.zeros(case["n"], case["r"], dtype=torch.float64, device="cuda")
        for a in range(case["count"]):
            at = (ids == a).nonzero()[:, 0]
            u = X[at] @ s["A"][a, : rank[a]].double().T
            U[at, : rank[a]] = u
            Y[at] += s["s"][a].double() * (u @ s["B"][a, :, : rank[a]].double().T)
        return (Y, U) if case["u"] else Y
    dY, U = s["dY"].double(), s["U"].double()
    dX = dY @ W
    dA = torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda")
    dB = torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda")
    for a in range(case["count"]):
        at, k = (ids == a).nonzero()[:, 0], rank[a]
        sc = s["s"][a].double()
        G = dY[at] @ s["B"][a, :, :k].double()
        dX[at] += sc * (G @ s["A"][a, :k].double())
        dA[a, :k] = sc * (G.T @ X[at])
        dB[a, :, :k] = sc * (dY[at].T @ U[at, :k])
    return dX, dA, dB

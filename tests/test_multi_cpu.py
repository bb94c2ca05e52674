"""Host-side checks of the calls with a pool of adapters: argument errors of the
C entry points (fake addresses, nothing is launched), workspace sizes, and the
binding's checks of shapes, types and devices."""
import ctypes

import pytest
import torch

from bit_nf4_quantized_07_b200 import api

P = ctypes.c_void_p
A16 = 0x10000


@pytest.fixture(scope="module")
def L():
    from bit_nf4_quantized_07_b200 import build
    build.build()
    return api.lib()


def _w(rows=128, cols=256, **bad):
    return api.CNF4Weight(**dict(dict(codes=A16, absmax=A16, qabs=None, dq_scale=None, dq_mean=None, rows=rows, cols=cols,
                                      dq_format=0), **bad))


GOOD = dict(A=A16, B=A16, scale=A16, rank=None, count=3, r=16)


def _call(L, op, w=None, pool=None, X=A16, n=40, ids=A16, Y=A16, U=None, dY=A16, dX=A16, dA=A16, dB=A16, ws=0x40000,
          wsb=1 << 34):
    w = w or _w()
    pool = api.CAdapterPool(**dict(GOOD, **(pool or {})))
    wp, pp = ctypes.byref(w), ctypes.byref(pool)
    if op == "fwd":
        return L.qlora_multi_fwd(wp, pp, P(X), n, P(ids), P(Y), P(U), P(ws), wsb, None)
    return L.qlora_multi_bwd(wp, pp, P(X), n, P(ids), P(dY), P(U), P(dX), P(dA), P(dB), P(ws), wsb, None)


@pytest.mark.parametrize("op", ["fwd", "bwd"])
def test_argument_errors(L, op):
    call = lambda **k: _call(L, op, **k)  # noqa: E731
    assert call(X=None) == 1 and call(ids=None) == 1 and call(ws=None) == 1
    for name in ("A", "B", "scale"):
        assert call(pool={name: None}) == 1, name
    assert call(w=_w(codes=None)) == 1
    assert call(n=0) == 2 and call(n=(1 << 24) + 1) == 2
    assert call(pool=dict(count=0)) == 2 and call(pool=dict(count=1025)) == 2
    for r in (0, 4, 12, 136):
        assert call(pool=dict(r=r)) == 2, r
    assert call(w=_w(rows=100)) == 2 and call(w=_w(cols=96)) == 2
    assert call(X=A16 + 8) == 3 and call(ids=A16 + 2) == 3 and call(ws=0x40010) == 3 and call(U=A16 + 4) == 3
    assert call(pool=dict(A=A16 + 8)) == 3 and call(pool=dict(B=A16 + 8)) == 3
    assert call(pool=dict(scale=A16 + 2)) == 3 and call(pool=dict(rank=A16 + 2)) == 3
    for name in (("Y",) if op == "fwd" else ("dY", "dX", "dA", "dB")):
        assert call(**{name: None}) == 1, name
        assert call(**{name: A16 + 8}) == 3, name
    need = api.workspace_bytes(api.OP_MULTI_FWD if op == "fwd" else api.OP_MULTI_BWD, 128, 256, 40, 16)
    assert need % 256 == 0 and need > 256
    assert call(wsb=need - 1) == 4


def test_null_structs(L):
    w, pool = _w(), api.CAdapterPool(**GOOD)
    assert L.qlora_multi_fwd(None, ctypes.byref(pool), P(A16), 4, P(A16), P(A16), None, P(0x40000), 1 << 30, None) == 1
    assert L.qlora_multi_fwd(ctypes.byref(w), None, P(A16), 4, P(A16), P(A16), None, P(0x40000), 1 << 30, None) == 1


def test_workspace_sizes():
    for op in (api.OP_MULTI_FWD, api.OP_MULTI_BWD):
        assert api.workspace_bytes(op, 128, 256, 0, 16) == 0
        assert api.workspace_bytes(op, 128, 256, (1 << 24) + 1, 16) == 0
        a, b = (api.workspace_bytes(op, 4096, 4096, n, 16) for n in (100, 5000))
        assert 0 < a < b


def _pool(count=3, r=16, dout=128, din=256, **bad):
    t = dict(A=torch.zeros(count, r, din, dtype=torch.bfloat16), B=torch.zeros(count, dout, r, dtype=torch.bfloat16),
             scale=torch.ones(count), rank=None)
    t.update(bad)
    return api.AdapterPool(**t)


def test_pool_is_checked():
    bf = torch.bfloat16
    for bad, msg in ((dict(A=torch.zeros(16, 256, dtype=bf)), "count"),
                     (dict(B=torch.zeros(2, 128, 16, dtype=bf)), "disagree"),
                     (dict(B=torch.zeros(3, 128, 8, dtype=bf)), "disagree"),
                     (dict(A=torch.zeros(3, 16, 256)), "A must be"),
                     (dict(B=torch.zeros(3, 16, 128, dtype=bf).transpose(1, 2)), "B must be contiguous"),
                     (dict(scale=torch.ones(2)), "scale holds 2"),
                     (dict(scale=torch.ones(3, dtype=torch.float64)), "scale must be"),
                     (dict(rank=torch.ones(3)), "rank must be"),
                     (dict(rank=torch.ones(4, dtype=torch.int32)), "rank holds 4")):
        with pytest.raises(ValueError, match=msg):
            _pool(**bad)


def test_pool_keeps_the_memory_it_was_made_of():
    A = torch.nn.Parameter(torch.zeros(3, 16, 256, dtype=torch.bfloat16))
    pool = _pool(A=A)
    A.data = torch.ones(3, 16, 256, dtype=torch.bfloat16)
    assert pool.c.A == pool.A.data_ptr() != A.data_ptr() and (pool.A == 0).all()
    with pytest.raises(AttributeError):
        pool.A = A


def test_calls_check_shapes_types_and_device():
    pool = _pool()
    w = api.NF4Weight(codes=torch.zeros(128 * 128, dtype=torch.uint8), rows=128, cols=256, absmax=torch.zeros(512))
    X, ids, dY = torch.zeros(5, 256, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int32), torch.zeros(5, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="adapters 128 x 256"):
        api.qlora_multi_fwd(api.NF4Weight(codes=w.codes, rows=256, cols=128, absmax=w.absmax), pool, X, ids)
    with pytest.raises(ValueError, match="X must be"):
        api.qlora_multi_fwd(w, pool, X.float(), ids)
    with pytest.raises(ValueError, match="ids must be"):
        api.qlora_multi_fwd(w, pool, X, ids.long())
    with pytest.raises(ValueError, match="ids must be"):
        api.qlora_multi_fwd(w, pool, X, ids[:4])
    with pytest.raises(ValueError, match="Y must be"):
        api.qlora_multi_fwd(w, pool, X, ids, Y=torch.zeros(5, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="U must be"):
        api.qlora_multi_bwd(w, pool, X, ids, dY, U=torch.zeros(5, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="dB must be"):
        api.qlora_multi_bwd(w, pool, X, ids, dY, dB=torch.zeros(3, 16, 128))
    with pytest.raises(ValueError, match="CUDA"):
        api.qlora_multi_fwd(w, pool, X, ids)

"""Host-side checks of the list updates: argument errors of the C entry points
(fake addresses, nothing is launched) and of the tensor lists of the binding."""
import ctypes

import pytest
import torch

from bit_nf4_quantized_07_b200 import api

P = ctypes.c_void_p
A16, A8, A4 = 0x10000, 0x10008, 0x10004


@pytest.fixture(scope="module")
def L():
    from bit_nf4_quantized_07_b200 import build
    build.build()
    return api.lib()


CFG = ctypes.byref(api.CAdamWConfig(1e-3, 0.9, 0.999, 1e-8, 0.0))
GOOD32 = dict(param=A16, grad=A16, m=A16, v=A16, param_bf16=None, n=64)
GOOD8 = dict(param=A16, grad=A16, m=A8, m_scale=A4, v=A8, v_scale=A4, param_bf16=None, n=64)


@pytest.mark.parametrize("fn,ctype,good", [("qln_adamw_multi_step", api.CAdamWTensor, GOOD32),
                                           ("qln_adamw8_multi_step", api.CAdamW8Tensor, GOOD8)])
def test_argument_errors(L, fn, ctype, good):
    def call(count=2, cfg=CFG, step=P(A16), **bad):  # the second tensor is checked too
        arr = (ctype * 2)(ctype(**good), ctype(**dict(good, **bad)))
        return getattr(L, fn)(arr, count, cfg, step, 0, None)
    assert getattr(L, fn)(None, 1, CFG, P(A16), 0, None) == 1
    assert call(cfg=None) == 1
    assert call(step=None) == 1
    for name in good:
        if name not in ("n", "param_bf16"):
            assert call(**{name: None}) == 1, name
            assert call(**{name: 0x10002}) == 3, name
    assert call(param=A8) == 3
    assert call(grad=A8) == 3
    assert call(param_bf16=A4) == 3
    assert call(count=0) == 2
    assert call(count=-1) == 2
    assert call(n=0) == 2
    assert call(n=(1 << 32) + 1) == 2
    assert getattr(L, fn)((ctype * 1)(ctype(**good)), (1 << 20) + 1, CFG, P(A16), 0, None) == 2


def _t(k=3, n=300, **bad):
    t = {name: [torch.zeros(n) for _ in range(k)] for name in ("params", "grads", "m", "v")}
    t.update(bad)
    return t


def _t8(k=3, n=300, **bad):
    t = dict(params=[torch.zeros(n) for _ in range(k)], grads=[torch.zeros(n) for _ in range(k)])
    st = [api.adamw8_state(p) for p in t["params"]]
    t.update({name: [s[i] for s in st] for i, name in enumerate(("m", "m_scale", "v", "v_scale"))})
    t.update(bad)
    return t


def test_lists_are_checked():
    shared = torch.zeros(300)
    for bad, msg in ((dict(params=[]), "empty"),
                     (dict(grads=[torch.zeros(300)]), "1 grad tensors for 3"),
                     (dict(m=[torch.zeros(300, dtype=torch.float64)] * 3), "m must be"),
                     (dict(v=[torch.zeros(299)] * 3), "v holds 299"),
                     (dict(params=[torch.zeros(0)] * 3), "is empty"),
                     (dict(m=[torch.zeros(600)[::2]] * 3), "must be contiguous"),
                     (dict(params_bf16=[torch.zeros(300)] * 3), "param_bf16 must be"),
                     (dict(params=[shared, shared, torch.zeros(300)]), "overlap"),
                     (dict(m=[shared, torch.zeros(300), torch.zeros(300)], v=[torch.zeros(300), shared, torch.zeros(300)]),
                      "overlap"),
                     (dict(m=[shared, torch.zeros(300), torch.zeros(300)], grads=[shared] * 3), "overlap")):
        with pytest.raises(ValueError, match=msg):
            api.AdamWTensors(**_t(**bad))
    api.AdamWTensors(**_t())
    api.AdamWTensors(**_t(grads=[shared] * 3))  # only read: may be shared
    api.AdamWTensors(**_t(params_bf16=[None, torch.zeros(300, dtype=torch.bfloat16), None]))


def test_a_small_buffer_inside_a_large_one_is_an_overlap():
    big = torch.zeros(1000)
    with pytest.raises(ValueError, match="overlap"):
        api.AdamWTensors([big, torch.zeros(8)], [torch.zeros(1000), big[400:408]],
                         [torch.zeros(1000), torch.zeros(8)], [torch.zeros(1000), torch.zeros(8)])


def test_8bit_lists_are_checked():
    for bad, msg in ((dict(m=[torch.zeros(300)] * 3), "m must be"),
                     (dict(m_scale=[torch.zeros(1)] * 3), "m_scale holds 1"),
                     (dict(v_scale=[torch.zeros(2, dtype=torch.float16)] * 3), "v_scale must be")):
        with pytest.raises(ValueError, match=msg):
            api.AdamW8Tensors(**_t8(**bad))
    t = api.AdamW8Tensors(**_t8(n=256))
    assert t.array[0].n == 256 and t.tensors["m_scale"][0].numel() == 1


def test_calls_refuse_other_lists_steps_and_devices():
    t = api.AdamWTensors(**_t())
    with pytest.raises(ValueError, match="AdamW8Tensors"):
        api.adamw8_multi_step(t, torch.ones(1, dtype=torch.int64), 1e-3)
    with pytest.raises(ValueError, match="int64"):
        api.adamw_multi_step(t, torch.ones(1), 1e-3)
    with pytest.raises(ValueError, match="CUDA"):
        api.adamw_multi_step(t, torch.ones(1, dtype=torch.int64), 1e-3)


def test_lists_keep_the_memory_they_were_made_of():
    d = _t()
    t = api.AdamWTensors(**d)
    at = d["params"][1].data_ptr()
    d["params"][1].data = torch.ones_like(d["params"][1])
    assert t.array[1].param == at == t.tensors["param"][1].data_ptr() != d["params"][1].data_ptr()

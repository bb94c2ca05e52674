"""The list updates with tables of every length, and captured: the bits are those of the same tensors updated one by
one (each tensor's update depends on itself only)."""
import pytest
import torch

from bit_nf4_quantized_07_b200 import api

pytestmark = pytest.mark.gpu
HYPER = (2e-3, (0.9, 0.995), 1e-8, 0.01)


def _tensors(sizes, eight, seed=1):
    """Per tensor: param, grad, the states, bf16 copy (every third has none)."""
    g = torch.Generator("cuda").manual_seed(seed)
    t = lambda n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
    out = []
    for i, n in enumerate(sizes):
        p, grad = t(n), t(n) * 0.1
        b = None if i % 3 == 0 else torch.zeros(n, dtype=torch.bfloat16, device="cuda")
        if eight:
            m, ms, v, vs = api.adamw8_state(p)
            m.copy_((t(n) * 20).to(torch.float8_e4m3fn))
            v.copy_((t(n).abs() * 20 + 1).to(torch.float8_e4m3fn))
            ms.fill_(0.003)
            vs.fill_(0.002)
            out.append([p, grad, m, ms, v, vs, b])
        else:
            out.append([p, grad, t(n) * 0.1, t(n).square() * 0.01, b])
    return out


def _list(tensors, eight):
    return (api.AdamW8Tensors if eight else api.AdamWTensors)(*map(list, zip(*tensors)))


def _same(a, b):
    bits = lambda x: x.view(torch.uint8)  # noqa: E731
    for i, (x, y) in enumerate(zip(a, b)):
        for k, (u, v) in enumerate(zip(x, y)):
            assert (u is None and v is None) or torch.equal(bits(u), bits(v)), (i, k)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("count,launches", [(1, 1), (48, 1), (49, 1), (480, 1), (481, 2), (1000, 3)])
def test_a_list_of_any_length_is_its_tensors_one_by_one(eight, count, launches):
    step = (api.adamw8_multi_step if eight else api.adamw_multi_step)
    sizes = [1 + (7919 * i) % 5003 for i in range(count)]
    a, b = _tensors(sizes, eight), _tensors(sizes, eight)
    before = api.launch_count()
    step(_list(a, eight), torch.full((1,), 3, dtype=torch.int64, device="cuda"), *HYPER)
    assert api.launch_count() == before + launches
    for t in b:
        step(_list([t], eight), torch.full((1,), 3, dtype=torch.int64, device="cuda"), *HYPER)
    _same(a, b)
    assert all(not torch.equal(x[0], y[0]) for x, y in zip(a, _tensors(sizes, eight)))


@pytest.mark.parametrize("eight", [False, True])
def test_captured_steps_of_a_long_list(eight):
    step = (api.adamw8_multi_step if eight else api.adamw_multi_step)
    sizes = [1 + (7919 * i) % 5003 for i in range(500)]
    a, b = _tensors(sizes, eight), _tensors(sizes, eight)
    at_a, at_b = (torch.zeros(1, dtype=torch.int64, device="cuda") for _ in range(2))
    graph, la, lb = torch.cuda.CUDAGraph(), _list(a, eight), _list(b, eight)
    with torch.cuda.graph(graph):
        at_a += 1
        step(la, at_a, *HYPER)
    for _ in range(3):
        graph.replay()
        at_b += 1
        step(lb, at_b, *HYPER)
    torch.cuda.synchronize()
    _same(a, b)


@pytest.mark.parametrize("eight", [False, True])
def test_a_tensor_of_more_than_2_31_elements(eight):
    """Its first and last elements and those around 2^31 get the bits that they get in tensors of their own."""
    step = (api.adamw8_multi_step if eight else api.adamw_multi_step)
    n, at = (1 << 31) + 777, torch.full((1,), 3, dtype=torch.int64, device="cuda")
    spans = [(0, 5120), ((1 << 31) - 2560, 2560), (1 << 31, 777)]  # whole blocks of 256 but for the last
    # all but the spans is zero: zero gradients and states of zero parameters leave zeros
    whole = [torch.zeros(n, device="cuda") for _ in range(2)]
    if eight:
        whole += [torch.zeros(-(-n // k), dtype=d, device="cuda") for _ in range(2)
                  for k, d in ((1, torch.float8_e4m3fn), (256, torch.float32))]
    else:
        whole += [torch.zeros(n, device="cuda") for _ in range(2)]
    small = _tensors([k for _, k in spans], eight)
    cut = lambda x, a, k: x[a // 256:a // 256 + -(-k // 256)] if len(x) < n else x[a:a + k]  # noqa: E731
    for (a, k), t in zip(spans, small):
        t[-1] = None
        for x, y in zip(whole, t):
            cut(x, a, k).copy_(y)
    step(_list([whole + [None]], eight), at, *HYPER)
    step(_list(small, eight), at, *HYPER)
    for (a, k), t in zip(spans, small):
        _same([[cut(x, a, k) for x in whole]], [t[:-1]])
    assert not any(x[10240:20480].float().any() for x in whole)

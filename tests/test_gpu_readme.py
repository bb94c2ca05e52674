"""The README's example runs as it stands, and every step takes its own gradients."""
import os
import re

import pytest
import torch

from bit_nf4_quantized_07_b200 import api

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_of_several_adapters():
    with open(os.path.join(ROOT, "README.md")) as f:
        code = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    assert len(code) == 1
    g = torch.Generator("cuda").manual_seed(1)
    t = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    W0, A, B, scale = t(256, 512) * 0.02, (t(3, 16, 512) * 0.05).bfloat16(), (t(3, 256, 16) * 0.05).bfloat16(), t(3)
    batches = [(t(n, 512).bfloat16(), torch.randint(-1, 3, (n,), generator=g, device="cuda").int()) for n in (40, 7, 90)]
    grad = lambda Y: (Y.float() * 0.01 - 0.003).bfloat16()  # noqa: E731
    ns = dict(W0=W0, A=A.clone(), B=B.clone(), scale=scale, batches=batches, loss_gradient=grad)
    exec(code[0], ns)
    # the same steps with a list of each step's own gradients
    w, pool = api.quantize_weight(W0), api.AdapterPool(A, B, scale)
    masters = [A.float(), B.float()]
    state = [api.adamw8_state(p) for p in masters]
    for k, (X, ids) in enumerate(batches):
        Y, U = api.qlora_multi_fwd(w, pool, X, ids, want_u=True)
        _, dA, dB = api.qlora_multi_bwd(w, pool, X, ids, grad(Y), U=U)
        own = api.AdamW8Tensors(masters, [dA, dB], *zip(*state), params_bf16=[A, B])
        api.adamw8_multi_step(own, torch.full((1,), k + 1, dtype=torch.int64, device="cuda"), lr=2e-4)
    for mine, theirs in ((ns["masters"], masters), ((ns["A"], ns["B"]), (A, B))):
        assert all(torch.equal(x, y) for x, y in zip(mine, theirs))

"""The norm with rotation at the largest number of tokens, 2^31 - 1: places in the
arrays are past 32 bits, and a position among the tokens is next to the end of them."""
import pytest
import torch

import ops_ref as R
from tensor_adamw_optimizer_amd import ops

pytestmark = pytest.mark.gpu
T = 2 ** 31 - 1


def test_forward_and_backward():
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    dev, bf = "cuda", torch.bfloat16
    # heads of one value, 1 or -1 but for the last tokens: y = x w / sqrt(x^2 + eps)
    gen = torch.Generator(device=dev).manual_seed(1)
    q = torch.ones(T, 1, 1, dtype=bf, device=dev)
    q[torch.randint(0, T, (1 << 20,), generator=gen, device=dev)] = -1
    ends = [slice(0, 5000), slice(T // 2, T // 2 + 5000), slice(T - 9000, T)]
    for e in ends:
        q[e] = torch.randn(q[e].shape, generator=gen, device=dev).to(bf)
    k, w = q[:, :, :1], torch.full((1,), 1.5, dtype=bf, device=dev)
    pos = torch.zeros((), dtype=torch.int64, device=dev).expand(T)
    how = dict(rotary_dim=0, eps=0.25)
    qy, ky = ops.qk_norm_rope_forward(q, k, w, w, pos, **how)
    assert torch.equal(qy, ky)
    for e in ends:
        R.within(qy[e], *R.qk(q[e], w, pos[e], bf, rotary=0, eps=0.25)[0], "y")
    rest = qy[5000:T // 2]
    assert torch.equal(rest.abs().amax(), rest.abs().amin()) and torch.equal(rest < 0, q[5000:T // 2] < 0)
    del qy, ky, rest
    dx, _, dw, dkw = ops.qk_norm_rope_backward(q, k, q, k, w, w, pos, **how)
    for e in ends:
        R.within(dx[e], *R.qk(q[e], w, pos[e], bf, rotary=0, eps=0.25, dy=q[e])[1], "dx")
    assert torch.equal(dw, dkw) and dw.isfinite().all()

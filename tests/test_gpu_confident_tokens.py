"""The gradient at the target of confident tokens: dz = dloss (p - 1) with 1 - p
from 1e-3 to 1e-5, at logits of 30 and 120, against float64.

p - 1 is formed from exp(z - lse) before it is rounded to bf16, so an error of z
- lse is absolute in 1 - p.  The logits of the backward are the forward's, bit
for bit, so that their own error cancels against lse's; what is left is lse as
fp32 holds it (one rounding, and one half of an ulp for the parts that it is
joined from) and the exponentials."""
import numpy as np
import pytest
import torch

from tests.step_util import U16, U32, Rand, dev, f64

pytestmark = pytest.mark.gpu

V = 601


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from top_routing_grouped_moe_gb300 import _binding
    return _binding


def _inputs(T, d, level, seed):
    """Logits near `level` for all ids and above it for the target.  Channel t
    is 1 in token t and 0 elsewhere, and 0 in W: dW[v, t] = dz[t, v]."""
    R = Rand(seed)
    free = d - T
    u = R.normal(free, dtype=torch.float64).abs() + 0.5  # every product of the level positive: the sums grow steadily
    w = R.normal(V, free, dtype=torch.float64)
    w -= (w @ u / (u @ u))[:, None] * u  # (the rows' own parts leave the level alone)
    target = torch.randperm(V, generator=R.g)[:T]
    q = 10.0 ** -(3.0 + 2.0 * torch.arange(T, dtype=torch.float64) / (T - 1))
    gap = torch.log((V - 1) / q)
    own = w[target]
    x = level * u / (u @ u) + gap[:, None] * own / (own * own).sum(1, keepdim=True)
    W = torch.cat([torch.zeros(V, T, dtype=torch.float64), u + w], 1)
    X = torch.cat([torch.eye(T, dtype=torch.float64), x], 1)
    return X.to(torch.bfloat16), W.to(torch.bfloat16), target.to(torch.int32)


@pytest.mark.parametrize("T", [40, 200])
@pytest.mark.parametrize("d", [576, 2048, 4096])
@pytest.mark.parametrize("level", [15.0, 105.0])
def test_gradient_at_the_target(B, T, d, level):
    x, W, t = _inputs(T, d, level, seed=T + d)
    z = f64(x) @ f64(W).T
    top = z.max(1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(1))
    at = t.numpy().astype(np.int64)
    rows = np.arange(T)
    others = z.copy()
    others[rows, at] = -np.inf
    rest = np.exp(others - lse[:, None]).sum(1)  # 1 - p, without the subtraction
    assert (rest < 3e-3).all() and (rest > 3e-6).all() and rest.min() < 3e-5 < 3e-4 < rest.max()

    x, W, t = dev(x), dev(W), dev(t)
    up = torch.ones(T, device="cuda")
    n = B.moe_cross_entropy_workspace(T, d, V)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    loss, got_lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dW = torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    B.moe_cross_entropy(x, W, t, T, d, V, 0.0, loss, got_lse, ws, n)
    B.moe_cross_entropy_bwd(x, W, t, got_lse, up, T, d, V, 0.0, 0, None, dW, ws, n)
    got = -f64(dW)[at, rows]
    # lse: half an ulp for its own rounding, as much again for its parts; s, p:
    # base-2 exponentials of about 2^-22 and their arguments.  The other ids'
    # share of 1 - p: differences of logits, each off by its 32 truncated sums
    # of 512 columns and the d / 512 roundings that add them.  Then dz and dW,
    # a rounding to bf16 each.
    e_lse = 2 * U32 * np.abs(lse) + 8 * U32
    e_z = 2 * U32 * (32 + d / 512) * 2 * np.abs(lse)
    bound = e_lse + rest * (e_z + 2 * U16 + U16**2)
    bad = np.abs(got - rest) > bound
    worst = int(np.argmax(np.abs(got - rest) / bound))
    assert not bad.any(), (f"{bad.sum()} of {T}; token {worst}: 1 - p = {rest[worst]:.3e}, got {got[worst]:.3e}, "
                           f"bound {bound[worst]:.1e}")
    assert B.moe_device_status() == 0

"""Main paths of the training-step operators that need more than a small shape:
the loss of many tokens over several 512-column parts of the width, and the
residual norm's backward over many more groups of rows than its ring holds."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as so
from tests import test_gpu_cross_entropy as ce
from tests import test_gpu_residual_norm as rn
from tests.step_util import U32, check, dev, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from top_routing_grouped_moe_gb300 import _binding
    return _binding


@pytest.mark.parametrize("T,V,d", [(300, 700, 576), (300, 701, 2048), (200, 300, 1088), (513, 257, 4096),
                                   (40, 701, 576), (128, 700, 1600), (129, 1000, 1600)])
def test_loss_over_several_parts_of_the_width(B, T, V, d):
    x, W, t, up = ce._inputs(T, V, d, seed=T + d)
    out = ce._run(B, x, W, t, up, 1e-3)
    ce._compare(out, x, W, t, up, 1e-3)
    loss, lse, z = so.cross_entropy(f64(x), f64(W), t.numpy().astype(np.int64), 1e-3)
    # a logit: at most 32 truncated additions of a part of 512 columns and the
    # parts' own, relative to the sum of magnitudes
    ez = (32 + d / 512 + 2) * 2 * U32 * (np.abs(f64(x)) @ np.abs(f64(W)).T).max(1)
    e_lse = ez + (np.abs(lse) + 1) * 8 * U32 + 4 * ce.EXP
    check("lse", out["lse"], lse, e_lse)
    check("loss", out["loss"], loss, np.where(t.numpy() >= 0, 2 * e_lse * (1 + 2e-3 * np.abs(lse)) +
                                              8 * U32 * np.abs(z).max(1), 0.0))
    assert B.moe_device_status() == 0


# every CTA of the 152-SM part's one to three per SM walks at least two rings of
# up to eight groups of rows
@pytest.mark.parametrize("T,d,f32", [(6000, 2048, False), (6000, 2048, True), (2600, 4096, False), (2600, 4096, True),
                                     (1300, 8192, False), (1300, 8192, True), (8000, 1280, False), (21000, 320, False),
                                     (21000, 320, True), (40001, 64, False)])
@pytest.mark.parametrize("kind", ["channel", "token"])
def test_norm_backward_over_many_rings(B, T, d, f32, kind):
    alpha = 0.75
    i = rn._inputs(T, d, kind, True, f32, seed=T + d)
    h = {k: f64(v) for k, v in i.items()}
    got = rn._forward(B, i, kind, f32, alpha, T, d)
    g = {k: dev(v) for k, v in i.items()}
    F = torch.float32
    e = lambda *s, dt=F: torch.full(s, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    out = dict(dr=e(T, d, dt=F if f32 else torch.bfloat16), d_o=e(T, d, dt=torch.bfloat16), dw_pre=e(d), dw_post=e(d),
               dgate=e(len(i["gate"])))
    n = B.moe_residual_norm_workspace(T, d)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    B.moe_residual_norm_bwd(g["dx"], g["dr_out"], g["o"], g["gate"], rn._kind(B, kind), g["w_post"], g["w_pre"],
                            got["r_out"], got["rstd_post"], got["rstd_pre"], T, d, f32, alpha, out["dr"], out["d_o"],
                            out["dgate"], out["dw_post"], out["dw_pre"], ws, n)
    r_out, ro, rp = f64(got["r_out"]), f64(got["rstd_post"])[:, None], f64(got["rstd_pre"])[:, None]
    ref = so.residual_norm_bwd(h["dx"], h["dr_out"], h["o"], h["gate"], kind, h["w_post"], h["w_pre"], r_out,
                               ro[:, 0], rp[:, 0], alpha)
    # magnitudes of the terms, as the roundings are relative to them
    xh, a = np.abs(r_out) * rp, np.abs(h["dx"] * h["w_pre"])
    Gm = np.abs(h["dr_out"]) + rp * (a + xh * (a * xh).mean(1, keepdims=True))
    oh, wpo = np.abs(h["o"]) * ro, np.abs(h["w_post"])
    gm = np.abs(h["gate"])[:, None] if kind == "token" else np.abs(h["gate"])
    dnm = alpha * gm * Gm
    am = dnm * wpo
    # a column: its CTA's rows in turn (at most T / 152 of them), up to 456 CTAs'
    # partials in 32 warps, the warps; and each term's own error
    COL = (T / 152 + 456 / 32 + 32) * U32 + 2 * rn.SUM
    check("dr", out["dr"], ref["dr"], rn.SUM * Gm)
    check("d_o", out["d_o"], ref["d_o"], 2 * rn.SUM * ro * (am + oh * (am * oh).mean(1, keepdims=True)))
    check("dw_pre", out["dw_pre"], ref["dw_pre"], COL * (np.abs(h["dx"]) * xh).sum(0))
    check("dw_post", out["dw_post"], ref["dw_post"], COL * (dnm * oh).sum(0))
    n_mag = alpha * (Gm * oh * wpo)
    check("dgate", out["dgate"], ref["dgate"], 2 * rn.SUM * n_mag.sum(1) if kind == "token" else COL * n_mag.sum(0))
    assert B.moe_device_status() == 0

"""The layer operators as a block uses them: residual sum and norm, the
projections (torch products), the gated recurrence, forward and backward
through the whole block against float64 autograd; and the same block decoding
token by token against its own prefill."""
import numpy as np
import pytest
import torch

from gpu_util import log, rel_l2

pytestmark = pytest.mark.gpu


def block64(x, r, w, b, Wp, Wo, h0):
    """The block in float64 autograd on the CPU: norm, one projection to x, f
    and g, the recurrence token by token, the output projection."""
    s = x + r
    c = s - s.mean(-1, keepdim=True)
    n = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * w + b
    xi, f, g = (n @ Wp).chunk(3, -1)
    h, ys = h0, []
    for t in range(x.shape[1]):
        a = torch.sigmoid(f[:, t])
        h = a * h + (1 - a) * xi[:, t]
        ys.append(h * torch.nn.functional.silu(g[:, t]))
    return torch.stack(ys, 1) @ Wo, s, h


def test_block_forward_backward_and_decode():
    """In float32 throughout: what differs from float64 is rounding, held to
    1e-4 relative over each tensor (products over 96 terms, 280 tokens of
    recurrence: each well under a thousand roundings of 6e-8)."""
    import state_space_sequence_exp_amd as m3
    gen = torch.Generator().manual_seed(9)
    B, T, W, D = 2, 280, 96, 72
    rn = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    v = dict(x=rn(B, T, W), r=rn(B, T, W), w=rn(W) * 0.2 + 1, b=rn(W) * 0.2, Wp=rn(W, 3 * D) * W ** -0.5,
             Wo=rn(D, W) * D ** -0.5, h0=rn(B, D))
    v = {k: t.float().double().requires_grad_() for k, t in v.items()}
    out, s64, h64 = block64(**v)
    dout, ds = rn(B, T, W).float().double(), rn(B, T, W).float().double()
    ref = dict(zip(v, torch.autograd.grad([out, s64], list(v.values()), [dout, ds])))

    t = {k: a.detach().float().cuda() for k, a in v.items()}
    y, s, mean, rstd = m3.layer_norm(t["x"], t["w"], t["b"], residual=t["r"])
    proj = y @ t["Wp"]
    xi, f, g = proj.chunk(3, -1)                      # slices, read in place
    yr, last, states = m3.gated_scan(xi, f, g, h0=t["h0"], want_states=True)
    o = yr @ t["Wo"]
    go, gs = dout.float().cuda(), ds.float().cuda()
    got = {"Wo": yr.flatten(0, 1).T @ go.flatten(0, 1)}
    dproj = torch.empty_like(proj)
    d = m3.gated_scan_backward(go @ t["Wo"].T, xi, f, g, states,
                               **dict(zip(("dx", "df", "dg"), dproj.chunk(3, -1))))
    got["h0"] = d["h0"]
    got["Wp"] = y.flatten(0, 1).T @ dproj.flatten(0, 1)
    n = m3.layer_norm_backward(dproj @ t["Wp"].T, s, t["w"], mean, rstd, dsum=gs)
    got.update(x=n["x"], r=n["x"], w=n["weight"], b=n["bias"])
    errs = {k: rel_l2(got[k].double().cpu().numpy(), ref[k].numpy()) for k in ref}
    errs["out"] = rel_l2(o.double().cpu().numpy(), out.detach().numpy())
    errs["h"] = rel_l2(last.double().cpu().numpy(), h64.detach().numpy())
    log("   " + "  ".join("%s %.1e" % e for e in errs.items()))
    assert max(errs.values()) <= 1e-4

    # the last tokens one by one from the state before them
    T0 = T - 6
    _, h, _ = m3.gated_scan(xi[:, :T0], f[:, :T0], g[:, :T0], h0=t["h0"]) if B == 1 else \
        m3.gated_scan(*(a[:, :T0].contiguous() for a in (xi, f, g)), h0=t["h0"])
    for k in range(T0, T):
        yn = m3.layer_norm(t["x"][:, k], t["w"], t["b"], residual=t["r"][:, k], want_stats=False)[0]
        y1, h = m3.gated_scan_step(h, *(yn @ t["Wp"]).chunk(3, -1))
        assert rel_l2((y1 @ t["Wo"]).double().cpu().numpy(), out[:, k].detach().numpy()) <= 1e-4
    assert rel_l2(h.double().cpu().numpy(), h64.detach().numpy()) <= 1e-4

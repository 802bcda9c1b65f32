"""The selective layer and the feed-forward block as a model runs them: norm,
input projection, short convolution, the projections to dt, B and C, the scan, the
output projection, then norm and the gated feed-forward products; a padded batch
of prompts against float64, its tokens one by one from pools of states, and the
block's training gradients."""
import numpy as np
import pytest
import torch

from gpu_util import log, rel_l2

pytestmark = pytest.mark.gpu
B, T, W, D, N, R, F = 3, 200, 48, 72, 16, 6, 100
SiLU = torch.nn.functional.silu


def weights(gen):
    rn = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    p = dict(n1=rn(W) * 0.1 + 1, b1=rn(W) * 0.1, Win=rn(W, 2 * D) * W ** -0.5, cw=rn(D, 4) * 0.5, cb=rn(D) * 0.1,
             Wx=rn(D, R + 2 * N) * D ** -0.5, Wdt=rn(R, D) * R ** -0.5, dtb=rn(D) - 2, A=-torch.exp(rn(D, N) * 0.5),
             skip=rn(D), Wout=rn(D, W) * D ** -0.5, n2=rn(W) * 0.1 + 1, b2=rn(W) * 0.1, wg=rn(F, W) * W ** -0.5,
             wu=rn(F, W) * W ** -0.5, Wd=rn(F, W) * F ** -0.5)
    return {k: v.float().double() for k, v in p.items()}


def norm64(x, w, b):
    c = x - x.mean(-1, keepdim=True)
    return c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * w + b


def layer64(x, p):
    """One sequence [T,W] in float64: the block's output, and the conv's and scan's states."""
    xi, z = (norm64(x, p["n1"], p["b1"]) @ p["Win"]).chunk(2, -1)
    pad = torch.cat([xi.new_zeros(3, D), xi])
    c = SiLU(sum(pad[k:k + len(x)] * p["cw"][:, k] for k in range(4)) + p["cb"])
    dt, Bt, Ct = (c @ p["Wx"]).split([R, N, N], -1)
    s = torch.nn.functional.softplus(dt @ p["Wdt"] + p["dtb"])
    h, ys = xi.new_zeros(D, N), []
    for t in range(len(x)):
        h = torch.exp(s[t, :, None] * p["A"]) * h + (s[t] * c[t])[:, None] * Bt[t]
        ys.append((h * Ct[t]).sum(-1) + p["skip"] * c[t])
    x = x + (torch.stack(ys) * SiLU(z)) @ p["Wout"]
    n = norm64(x, p["n2"], p["b2"])
    return x + (SiLU(n @ p["wg"].T) * (n @ p["wu"].T)) @ p["Wd"], pad[len(x):], h


def test_prompts_then_tokens():
    """In float32: what differs from float64 is rounding, held to 1e-4 relative over
    each tensor (products over 100 terms, 200 tokens of recurrence, two norms: each
    well under a thousand roundings of 6e-8)."""
    import state_space_sequence_exp_amd as m3
    gen = torch.Generator().manual_seed(3)
    p = weights(gen)
    g = {k: v.float().cuda() for k, v in p.items()}
    x = torch.randn(B, T + 5, W, generator=gen, dtype=torch.float64).float().double()
    n = [T, 77, 1]
    want = [layer64(x[b, :n[b] + 5], p) for b in range(B)]

    def mix(x, conv, scan):
        y, s, _, _ = m3.layer_norm(x, g["n1"], g["b1"])
        xi, z = (y @ g["Win"]).chunk(2, -1)                       # slices, read in place
        c = conv(xi)
        dt, Bt, Ct = (c @ g["Wx"]).split([R, N, N], -1)
        o = scan(c, dt @ g["Wdt"], Bt, Ct, z)
        y, s, _, _ = m3.layer_norm(o @ g["Wout"], g["n2"], g["b2"], residual=x)
        return s + m3.gated_ffn(y, g["wg"], g["wu"])[0] @ g["Wd"]

    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    kept = {}

    def conv(xi):
        c, kept["conv"] = m3.causal_conv(xi, g["cw"], g["cb"], silu=True, lengths=lengths)
        return c

    def scan(c, dt, Bt, Ct, z):
        y, kept["scan"] = m3.selective_scan(c, dt, g["A"], Bt, Ct, g["skip"], z, dt_bias=g["dtb"], lengths=lengths)
        return y

    xp = x[:, :T].float().cuda()
    for b in range(B):
        xp[b, n[b]:] = float("nan")                               # a norm of padding is NaN, and stays there
    out = mix(xp, conv, scan)
    errs = [rel_l2(out[b, :n[b]].double().cpu().numpy(), want[b][0][:n[b]].numpy()) for b in range(B)]

    # the states go into pools, in another order; a padded batch of four takes five tokens
    pools = torch.zeros(5, 3, D, device="cuda"), torch.zeros(5, D, N, device="cuda")
    slots = torch.tensor([4, 0, 2, -1], dtype=torch.int32, device="cuda")
    at = slots[:B].long()
    pools[0][at], pools[1][at] = kept["conv"], kept["scan"]
    conv1 = lambda xi: m3.causal_conv_step(pools[0], xi, g["cw"], g["cb"], silu=True, slots=slots)
    scan1 = lambda c, dt, Bt, Ct, z: m3.selective_scan_step(pools[1], c, dt, g["A"], Bt, Ct, g["skip"], z,
                                                            dt_bias=g["dtb"], slots=slots)
    for k in range(5):
        xt = torch.zeros(4, W, device="cuda")
        xt[:B] = torch.stack([x[b, n[b] + k] for b in range(B)]).float().cuda()
        o = mix(xt, conv1, scan1)
        errs += [rel_l2(o[b].double().cpu().numpy(), want[b][0][n[b] + k].numpy()) for b in range(B)]
    for pool, i in zip(pools, (1, 2)):
        errs += [rel_l2(pool[at[b]].double().cpu().numpy(), want[b][i].numpy()) for b in range(B)]
        assert not pool[[1, 3]].any()
    log("   worst %.1e" % max(errs))
    assert max(errs) <= 1e-4


def test_feed_forward_block_gradients():
    """Norm with the residual sum, the gated projections, the down projection, in
    float32 against float64 autograd through the whole block."""
    import state_space_sequence_exp_amd as m3
    gen = torch.Generator().manual_seed(4)
    p = weights(gen)
    rn = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64).float().double()
    v = {"x": rn(B, T, W), "r": rn(B, T, W), **{k: p[k] for k in ("n2", "b2", "wg", "wu", "Wd")}}
    leaf = {k: a.clone().requires_grad_() for k, a in v.items()}
    s = leaf["x"] + leaf["r"]
    n = norm64(s, leaf["n2"], leaf["b2"])
    out = s + (SiLU(n @ leaf["wg"].T) * (n @ leaf["wu"].T)) @ leaf["Wd"]
    dout = rn(B, T, W)
    ref = dict(zip(leaf, torch.autograd.grad(out, list(leaf.values()), dout)))

    t = {k: a.float().cuda() for k, a in v.items()}
    y, s, mean, rstd = m3.layer_norm(t["x"], t["n2"], t["b2"], residual=t["r"])
    h, gate, up = m3.gated_ffn(y, t["wg"], t["wu"], want_pre=True)
    go = dout.float().cuda()
    got = {"Wd": h.flatten(0, 1).T @ go.flatten(0, 1)}
    d = m3.gated_ffn_backward(go @ t["Wd"].T, y, t["wg"], t["wu"], gate, up)
    got.update(wg=d["w_gate"], wu=d["w_up"])
    dn = m3.layer_norm_backward(d["x"], s, t["n2"], mean, rstd, dsum=go)
    got.update(x=dn["x"], r=dn["x"], n2=dn["weight"], b2=dn["bias"])
    errs = {k: rel_l2(got[k].double().cpu().numpy(), ref[k].numpy()) for k in ref}
    errs["out"] = rel_l2((s + h @ t["Wd"]).double().cpu().numpy(), out.detach().numpy())
    log("   " + "  ".join("%s %.1e" % e for e in errs.items()))
    assert max(errs.values()) <= 1e-4

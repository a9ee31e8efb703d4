"""fp64 CPU oracle of the gated delta rule, its gated epilogue and the
residual norm.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``.

The delta rule runs one token after the other as its definition states it,
and its gradient is the reverse of those steps:
    P = a S;  u = v - P k;  S' = P + beta u k^T;  y = scale S' q
Shapes as in include/gdr.h: q, k [B, T, Hk, K], v [B, T, Hv, V], g, beta
[B, T, Hv], states [sequences, Hv, V, K].  ``starts`` packs sequences into
one row (B = 1).
"""
import torch

EPS = 1e-6


def _d(x):
    return None if x is None else x.detach().to("cpu", torch.float64)


def _norm(x):
    n = torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)
    return x / n, n


def _sequences(B, T, starts):
    if starts is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, lo, hi) for lo, hi in zip(starts[:-1], starts[1:])]


def _steps(q, k, v, a, beta, S):
    """One sequence's [T, H, .] tokens; yields the states before each step
    and the last."""
    y, states = torch.empty_like(v), [S]
    for t in range(q.shape[0]):
        P = a[t][:, None, None] * S
        u = v[t] - (P * k[t][:, None, :]).sum(-1)
        S = P + (beta[t][:, None] * u)[..., None] * k[t][:, None, :]
        y[t] = (S * q[t][:, None, :]).sum(-1)
        states.append(S)
    return y, states


def _reverse(q, k, v, a, beta, states, dy, dS):
    dq, dk, dv, da, db = (torch.empty_like(x) for x in (q, k, v, a, beta))
    for t in range(q.shape[0] - 1, -1, -1):
        P = a[t][:, None, None] * states[t]
        u = v[t] - (P * k[t][:, None, :]).sum(-1)
        dq[t] = (states[t + 1] * dy[t][..., None]).sum(-2)
        dS = dS + dy[t][..., None] * q[t][:, None, :]
        dSk = (dS * k[t][:, None, :]).sum(-1)
        db[t] = (dSk * u).sum(-1)
        du = beta[t][:, None] * dSk
        dk[t] = ((beta[t][:, None] * u)[..., None] * dS - du[..., None] * P).sum(-2)
        dv[t] = du
        dP = dS - du[..., None] * k[t][:, None, :]
        da[t] = (dP * states[t]).sum((-1, -2))
        dS = a[t][:, None, None] * dP
    return dq, dk, dv, da, db, dS


def rule(q, k, v, g, beta, s0=None, dy=None, dsT=None, *, starts=None, scale=None, norm_qk=False):
    """dict y, sT and, with dy, dq, dk, dv, dg, dbeta, ds0.  Tokens outside
    every sequence hold NaN."""
    q, k, v, g, beta, s0, dy, dsT = map(_d, (q, k, v, g, beta, s0, dy, dsT))
    B, T, Hk, K = q.shape
    Hv, V = v.shape[2:]
    group = Hv // Hk
    scale = K ** -0.5 if scale is None else scale
    one = torch.ones(())
    qn, nq = _norm(q) if norm_qk else (q, one)
    kn, nk = _norm(k) if norm_qk else (k, one)
    qs = (qn * scale).repeat_interleave(group, 2)
    ks = kn.repeat_interleave(group, 2)
    a = torch.exp(g)
    seqs = _sequences(B, T, starts)
    nan = float("nan")
    out = {"y": torch.full_like(v, nan), "sT": torch.zeros(len(seqs), Hv, V, K, dtype=torch.float64)}
    if dy is not None:
        out.update(dq=torch.full_like(qs, nan), dk=torch.full_like(ks, nan), dv=torch.full_like(v, nan),
                   dg=torch.full_like(g, nan), dbeta=torch.full_like(g, nan), ds0=torch.zeros_like(out["sT"]))
    for i, (b, lo, hi) in enumerate(seqs):
        S = torch.zeros(Hv, V, K, dtype=torch.float64) if s0 is None else s0[i]
        args = [x[b, lo:hi] for x in (qs, ks, v, a, beta)]
        out["y"][b, lo:hi], states = _steps(*args, S)
        out["sT"][i] = states[-1]
        if dy is None:
            continue
        dS = torch.zeros_like(S) if dsT is None else dsT[i]
        got = _reverse(*args, states, dy[b, lo:hi], dS)
        for n, x in zip(("dq", "dk", "dv", "dg", "dbeta"), got):
            out[n][b, lo:hi] = x * args[3] if n == "dg" else x
        out["ds0"][i] = got[5]
    if dy is not None:
        # the decay of a state that is forgotten (g <= -200) has no gradient
        out["dg"] = torch.where(g <= -200, torch.where(torch.isnan(out["dg"]), out["dg"], 0.0), out["dg"])
        dq = out["dq"].view(B, T, Hk, group, K).sum(3) * scale
        dk = out["dk"].view(B, T, Hk, group, K).sum(3)
        if norm_qk:
            dq = (dq - qn * (qn * dq).sum(-1, keepdim=True)) / nq
            dk = (dk - kn * (kn * dk).sum(-1, keepdim=True)) / nk
        out.update(dq=dq, dk=dk)
    return out


def epilogue(y, gate, w, dz=None, eps=1e-6):
    """dict z and, with dz, dy, dgate, dw."""
    y, gate, w, dz = map(_d, (y, gate, w, dz))
    N = y.shape[-1]
    r = 1 / torch.sqrt((y * y).sum(-1, keepdim=True) / N + eps)
    s = 1 / (1 + torch.exp(-gate))
    yn, act = y * r, gate * s
    out = {"z": yn * w * act}
    if dz is not None:
        out["dgate"] = dz * yn * w * (s + gate * s * (1 - s))
        dyn = dz * act
        dw = (dyn * yn).reshape(-1, *y.shape[-2:]).sum(0)
        out["dw"] = dw if w.shape[0] == y.shape[-2] else dw.sum(0, keepdim=True)
        dyn = dyn * w
        out["dy"] = r * dyn - yn * r * (dyn * yn).sum(-1, keepdim=True) / N
    return out


def residual_norm(x, y, w, scale=None, eps=1e-6):
    """dict x_out, h."""
    x, y, w, scale = map(_d, (x, y, w, scale))
    xo = x if y is None else x + (y if scale is None else scale * y)
    return {"x_out": xo, "h": xo / torch.sqrt((xo * xo).mean(-1, keepdim=True) + eps) * w}


def residual_norm_backward(dh, dx_out, x_out, w, y=None, scale=None, eps=1e-6):
    """dict dx, dw and, with a scale, dy, dscale."""
    dh, dx_out, xo, w, y, scale = map(_d, (dh, dx_out, x_out, w, y, scale))
    D = xo.shape[-1]
    r = 1 / torch.sqrt((xo * xo).sum(-1, keepdim=True) / D + eps)
    xn, dn = xo * r, dh * w
    dx = r * (dn - xn * (dn * xn).sum(-1, keepdim=True) / D)
    if dx_out is not None:
        dx = dx + dx_out
    out = {"dx": dx, "dw": (dh * xn).reshape(-1, D).sum(0)}
    if scale is not None:
        out.update(dy=scale * dx, dscale=(dx * y).reshape(-1, D).sum(0))
    return out

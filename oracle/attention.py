"""fp64 CPU oracle of softmax attention: the norm and rotation of queries and
keys, causal attention with its gradients, the paged cache and attention over
it.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``.

Shapes as in include/attention.h.  ``starts`` packs sequences into one row
(B = 1); rows outside every sequence are NaN in the results.  Beside each
result x that is a weighted sum, ``x_1`` is the sum of its terms' magnitudes
and ``x_2`` the root of the sum of their squares: what roundings of the
weights are relative to.
"""
import math

import torch


def _d(x):
    return None if x is None else x.detach().to("cpu", torch.float64)


def _sequences(B, T, starts):
    if starts is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, lo, hi) for lo, hi in zip(starts[:-1], starts[1:])]


def attention(q, k, v, dy=None, *, starts=None, scale=None):
    """dict(y, lse) and, with dy, dq, dk, dv."""
    q, k, v, dy = map(_d, (q, k, v, dy))
    B, T, Hq, D = q.shape
    Hk = k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out = {n: torch.full_like(q, math.nan) for n in ("y", "y_1", "y_2")}
    out["lse"] = torch.full_like(q[..., 0], math.nan)
    if dy is not None:
        for n, like in (("dq", q), ("dk", k), ("dv", k)):
            for m in ("", "_1", "_2"):
                out[n + m] = torch.full_like(like, math.nan)
        # what an error in D = dy . y, as large as |dy| . |y|, |dy| . y_1 or
        # sqrt(dy^2 . y_2^2), makes of dq and dk
        for m in ("_d", "_d1", "_d2"):
            out["dq" + m], out["dk" + m] = torch.full_like(q, math.nan), torch.full_like(k, math.nan)
    for b, lo, hi in _sequences(B, T, starts):
        if hi <= lo:
            continue
        for n in out:
            if n[:2] in ("dk", "dv"):
                out[n][b, lo:hi] = 0
        seen = torch.ones(hi - lo, hi - lo, dtype=torch.bool).tril()
        for h in range(Hq):
            g = h * Hk // Hq
            qq, kk, vv = q[b, lo:hi, h], k[b, lo:hi, g], v[b, lo:hi, g]
            z = scale * (qq @ kk.T)
            top = z.masked_fill(~seen, -math.inf).amax(-1, keepdim=True)
            e = torch.where(seen, torch.exp(z - top), 0.0)
            total = e.sum(-1, keepdim=True)
            p = e / total
            y = p @ vv
            out["y"][b, lo:hi, h] = y
            out["y_1"][b, lo:hi, h] = p @ vv.abs()
            out["y_2"][b, lo:hi, h] = torch.sqrt(p ** 2 @ vv ** 2)
            out["lse"][b, lo:hi, h] = (top + torch.log(total))[:, 0]
            if dy is None:
                continue
            gy = dy[b, lo:hi, h]
            ds = p * (gy @ vv.T - (gy * y).sum(-1, keepdim=True)) * scale
            dots = {"_d": (gy * y).abs().sum(-1, keepdim=True), "_d1": (gy.abs() * (p @ vv.abs())).sum(-1, keepdim=True),
                    "_d2": torch.sqrt((gy ** 2 * (p ** 2 @ vv ** 2)).sum(-1, keepdim=True))}
            for m, dot in dots.items():
                out["dq" + m][b, lo:hi, h] = scale * dot * (p @ kk.abs())
                out["dk" + m][b, lo:hi, g] += scale * (p * dot).T @ qq.abs()
            out["dq"][b, lo:hi, h] = ds @ kk
            out["dq_1"][b, lo:hi, h] = ds.abs() @ kk.abs()
            out["dq_2"][b, lo:hi, h] = torch.sqrt(ds ** 2 @ kk ** 2)
            out["dk"][b, lo:hi, g] += ds.T @ qq
            out["dk_1"][b, lo:hi, g] += ds.abs().T @ qq.abs()
            out["dk_2"][b, lo:hi, g] += ds.T ** 2 @ qq ** 2
            out["dv"][b, lo:hi, g] += p.T @ gy
            out["dv_1"][b, lo:hi, g] += p.T @ gy.abs()
            out["dv_2"][b, lo:hi, g] += p.T ** 2 @ gy ** 2
    if dy is not None:
        for n in ("dk_2", "dv_2"):
            out[n] = torch.sqrt(out[n])
    return out


def qk_norm(q, k, wq=None, wk=None, theta=None, positions=None, dq=None, dk=None, *, eps=1e-6, interleaved=False):
    """dict(q, k) and, with dq and dk, the gradients dq, dk, dwq, dwk."""
    theta = _d(theta)
    out = {}
    for n, x, w, dz in (("q", q, wq, dq), ("k", k, wk, dk)):
        x, w, dz = _d(x), _d(w), _d(dz)
        B, T, H, D = x.shape
        norm = torch.ones_like(x[..., :1]) if w is None else torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        xn = x / norm
        z = xn if w is None else xn * w
        M = torch.eye(D, dtype=torch.float64).expand(B, T, D, D).clone()   # the rotation as a matrix
        if theta is not None:
            R = 2 * theta.numel()
            pos = torch.arange(T).expand(B, T).double() if positions is None else _d(positions)
            angle = pos[..., None] * theta
            i = torch.arange(R // 2)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            M[..., a, a] = torch.cos(angle)
            M[..., a, b] = -torch.sin(angle)
            M[..., b, a] = torch.sin(angle)
            M[..., b, b] = torch.cos(angle)
        out[n] = torch.einsum("btij,bthj->bthi", M, z)
        if dz is not None:
            dn = torch.einsum("btij,bthi->bthj", M, dz)
            if w is None:
                out["d" + n] = dn
                continue
            out["dw" + n] = (dn * xn).sum((0, 1, 2))
            out["dw" + n + "_2"] = torch.sqrt(((dn * xn) ** 2).sum((0, 1, 2)))
            dn = dn * w
            out["d" + n] = (dn - xn * (dn * xn).mean(-1, keepdim=True)) / norm
    return out


def e4m3(x):
    """The e4m3 value nearest to x, ties to even, at most 448 in magnitude."""
    x = torch.as_tensor(x, dtype=torch.float64)
    size = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(torch.where(size > 0, size, 1.0))).clamp(min=-6) - 3)
    return torch.sign(x) * torch.round(size / step) * step


def quantise(x):
    """The values and the scale of [..., D] heads in 8 bits, by fp32's own
    product and quotients (which are part of the definition)."""
    x = x.detach().cpu().float()
    scale = x.abs().amax(-1) * torch.tensor(1 / 448.0, dtype=torch.float32)
    return e4m3((x / torch.where(scale > 0, scale, 1.0)[..., None]).double()), scale


def places(lens, counts, table, page, pages):
    """For each row the (page, offset) of its last counts[r] tokens, None where
    there is none."""
    out = []
    for r, (n, m) in enumerate(zip(lens, counts)):
        row = []
        for i in range(m):
            pos = n - m + i
            ok = 0 <= pos < len(table[r]) * page
            p = table[r][pos // page] if ok else -1
            row.append((p, pos % page) if 0 <= p < pages else None)
        out.append(row)
    return out


def decode(q, k_pages, v_pages, table, lens, *, scale=None):
    """y [B, T, Hq, D] over pages [pages, Hk, page, D] that hold fp64 values."""
    q, k_pages, v_pages = map(_d, (q, k_pages, v_pages))
    B, T, Hq, D = q.shape
    pages, Hk, page, _ = k_pages.shape
    scale = D ** -0.5 if scale is None else scale
    y, y1 = torch.zeros_like(q), torch.zeros_like(q)
    for b in range(B):
        for t in range(T):
            n = lens[b] - (T - 1 - t)
            seen = []
            for pos in range(min(max(n, 0), len(table[b]) * page)):
                p = table[b][pos // page]
                if 0 <= p < pages:
                    seen.append(p * page + pos % page)
            if not seen:
                continue
            at = torch.tensor(seen)
            K = k_pages.transpose(1, 2).reshape(-1, Hk, D)[at]
            V = v_pages.transpose(1, 2).reshape(-1, Hk, D)[at]
            for h in range(Hq):
                g = h * Hk // Hq
                w = torch.softmax(scale * (K[:, g] @ q[b, t, h]), 0)
                y[b, t, h] = w @ V[:, g]
                y1[b, t, h] = w @ V[:, g].abs()
    return {"y": y, "y_1": y1}

"""The backward pass of a block of routed experts in 64 bits, from what its forward
pass stored, and how far bfloat16 rounding on the way may move each gradient.

Tolerances are Frobenius norms.  A value stored in bfloat16 is off by H = 2^-8 of
itself, so a tensor by H of its norm; a product carries an error on with the other
operand's spectral norm, a sum of k rows with k^(1/2), a column sum of n rows with
n^(1/2), the norm's gradient with rho max |weight| (what is left of it is a projection).
Float32 sums count 2^-24 for each term and the norms of the magnitudes."""

import torch

H, U = 2.0 ** -8, 2.0 ** -24


def norm(t):
    return float(torch.linalg.vector_norm(t.double()))


def spectral(t):
    return float(torch.linalg.matrix_norm(t.double().cpu(), 2)) if t.numel() else 0.0


def bank_gradients(dout, n, e, w, v):
    """{dv, dn} as (gradient, tolerance): of the bank v (experts, out, in) and, through it, of its inputs n (tokens, in),
    for out_t = sum_j w_tj v_e(t,j) n_t.  Rounded on the way: w dout, each choice's row, their sum."""
    dout, n, w, v = dout.double(), n.double(), w.double(), v.double()
    (tokens, k), width = e.shape, n.shape[1]
    dy = w[:, :, None] * dout[:, None]
    dv, rows = torch.zeros_like(v), torch.zeros(tokens, k, width, dtype=torch.float64, device=n.device)
    dv_tol = rows_tol = 0.0
    for i in range(v.shape[0]):
        at = torch.nonzero(e == i)
        if not at.numel():
            continue
        t, j = at[:, 0], at[:, 1]
        part, its = dy[t, j], n[t]
        dv[i] = part.t().contiguous() @ its
        rows[t, j] = part @ v[i]
        off = (H + 2 * U) * norm(part)
        dv_tol += (off * spectral(its) + 2 * U * len(t) * norm(part) * norm(its)) ** 2
        rows_tol += (off * spectral(v[i]) + 2 * U * v.shape[1] * norm(part) * norm(v[i])) ** 2
    rows_tol = rows_tol ** 0.5
    rows_tol += H * (norm(rows) + rows_tol)
    dn, dn_tol = rows.sum(1), k ** 0.5 * (rows_tol + k * U * norm(rows))
    dn_tol += H * (norm(dn) + dn_tol)
    return {"dv": (dv, dv_tol ** 0.5), "dn": (dn, dn_tol)}


def block_gradients(dout, weight, router, v, h, mean, rstd, n, e, w, y):
    """{dx, dweight, dbias, drouter, dv} as (gradient, tolerance) of expert_step.py's block, whose forward pass left
    h, mean, rstd and n of the norm, the experts e and weights w of each token (tokens, k), and y (tokens, k, width)."""
    (tokens, k), width = e.shape, n.shape[1]
    out = bank_gradients(dout, n, e, w, v)
    dout, weight, router, h, n, w, y = (t.double() for t in (dout, weight, router, h, n, w, y))
    dn, dn_tol = out.pop("dn")
    each = y * dout[:, None]
    dw, dw_tol = each.sum(2), (width + 64) * U * each.abs().sum(2)
    dw_tol = dw_tol + 8 * U * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True))
    dl = torch.zeros(tokens, router.shape[1], dtype=torch.float64, device=n.device)
    dl_tol = norm(w * (dw_tol + (w * dw_tol).sum(1, keepdim=True)))
    dl.scatter_add_(1, e, w * (dw - (w * dw).sum(1, keepdim=True)))
    out["drouter"] = n.t().contiguous() @ dl, spectral(n) * dl_tol + tokens * U * norm(n) * norm(dl)
    dn_tol += spectral(router) * dl_tol + (router.shape[1] + 2) * U * (norm(dl) * norm(router) + norm(dn))
    dn = dn + dl @ router.t().contiguous()
    dn_tol += H * (norm(dn) + dn_tol)
    rho = rstd.double()[:, None]
    hh = (h - mean.double()[:, None]) * rho
    g = dn * weight
    dx = dout + rho * (g - g.mean(1, keepdim=True) - hh * (g * hh).mean(1, keepdim=True))
    gain = float(rho.max() * weight.abs().max()) * (1 + 1e-3)
    out["dx"] = dx, H * norm(dx) + (1 + H) * gain * (dn_tol + (width / 8 + 100) * U * norm(dn))
    columns = float(torch.linalg.vector_norm(hh, dim=0).max())
    out["dweight"] = (dn * hh).sum(0), columns * dn_tol + (tokens + 60) * U * norm((dn * hh).abs().sum(0))
    out["dbias"] = dn.sum(0), tokens ** 0.5 * dn_tol + (tokens + 60) * U * norm(dn.abs().sum(0))
    return out


def block_inputs(tokens, width, seed, device):
    """(x, dout) in bfloat16.  The gradient has a part that all tokens share, so that sums over tokens are no smaller
    than their terms."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, width, generator=g)
    dout = torch.randn(1, width, generator=g) + 0.3 * torch.randn(tokens, width, generator=g)
    return x.bfloat16().to(device), dout.bfloat16().to(device)

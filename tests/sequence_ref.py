"""Plain 64-bit forms of the sequence operators, with the error each result may
carry.

Every tolerance is built from the roundings that the kernels make: `u`, half a
step of a type, once per rounding to it, and n * 2^-24 for a sum of n terms in
fp32 (2^-23 where a tensor core adds, whose rounding may be a truncation)."""
import math

import torch

F32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half a step of a type's subnormal numbers: what a rounding may be off by
    below the smallest normal number, where steps no longer shrink with the
    value (fp16: steps of 2^-24 below 2^-14)."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def lookup(weight, tokens, scale, padding):
    V, D = weight.shape
    ok = (tokens != padding) & (tokens >= 0) & (tokens < V)
    rows = weight.double()[tokens.clamp(0, V - 1)] * scale
    return torch.where(ok[..., None], rows, 0.0)


def embed_grad(tokens, grad, V, scale, padding):
    """(gradient, the sum of its terms' magnitudes)."""
    t, g = tokens.reshape(-1), grad.double().reshape(-1, grad.shape[-1])
    ok = (t != padding) & (t >= 0) & (t < V)
    out = torch.zeros((V, g.shape[1]), dtype=torch.float64, device=g.device)
    mag = torch.zeros_like(out)
    out.index_add_(0, t[ok], g[ok])
    mag.index_add_(0, t[ok], g[ok].abs())
    return out * scale, mag * abs(scale)


class Norm:
    """Layer norm of rows x [M, D] in 64 bits.  `n`: additions behind an fp32 sum
    over a row (a thread's columns, then the tree over threads)."""

    def __init__(self, x, w, b, eps, n=96):
        x = x.double()
        M, D = x.shape
        self.w = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w.double()
        b = 0.0 if b is None else b.double()
        self.mean = x.mean(1)
        xc = x - self.mean[:, None]
        var = (xc * xc).mean(1)
        self.rstd = 1.0 / torch.sqrt(var + eps)
        self.xh = xc * self.rstd[:, None]
        self.y = self.xh * self.w + b
        mag = x.abs().mean(1)
        self.mean_err = n * F32 * mag
        # the centred values are off by the mean's error and one rounding; the
        # variance by the sum's roundings and the mean's error squared
        self.rstd_err = self.rstd * (0.5 * ((n + 4) * F32 + 2 * self.mean_err ** 2 * self.rstd ** 2) + 4 * F32)
        self.xh_err = (self.mean_err * self.rstd)[:, None] + self.xh.abs() * (
            self.rstd_err / self.rstd + 3 * F32)[:, None] + 2 * F32 * (mag * self.rstd)[:, None]
        self.y_err = self.xh_err * self.w.abs() + 2 * F32 * (self.xh * self.w).abs() + F32 * self.y.abs()
        self.n = n

    def back(self, gy, n_rows):
        """dx, dw, db and their errors; n_rows: fp32 additions over rows."""
        gy = gy.double()
        D = gy.shape[1]
        g = gy * self.w
        r = self.rstd[:, None]
        m0, m1 = g.mean(1, keepdim=True), (g * self.xh).mean(1, keepdim=True)
        dx = r * (g - m0 - self.xh * m1)
        m0_err = (self.n + 2) * F32 * g.abs().mean(1, keepdim=True)
        m1_err = (g.abs() * self.xh_err).mean(1, keepdim=True) + (self.n + 3) * F32 * (g * self.xh).abs().mean(
            1, keepdim=True)
        dx_err = r * (4 * F32 * (g.abs() + m0.abs() + (self.xh * m1).abs()) + m0_err + self.xh.abs() * m1_err
                      + self.xh_err * m1.abs()) + dx.abs() * (self.rstd_err[:, None] / r + 2 * F32)
        dw, db = (gy * self.xh).sum(0), gy.sum(0)
        dw_err = (gy.abs() * self.xh_err).sum(0) + (n_rows + 2) * F32 * (gy * self.xh).abs().sum(0)
        db_err = (n_rows + 2) * F32 * gy.abs().sum(0)
        return (dx, dx_err), (dw, dw_err), (db, db_err)


def attend(q, k, v, q_offsets, k_offsets, scale, mask=None, grad=None):
    """name -> (value, tolerance) of out, lse and, with grad, the gradients."""
    dtype, dev = q.dtype, q.device
    u, sub, (Tq, Hq, D), Hkv = half_step(dtype), least(dtype), q.shape, k.shape[1]
    G = Hq // Hkv
    qd, kd, vd = q.double(), k.double(), v.double()
    names = ["out", "lse"] + (["grad_q", "grad_k", "grad_v"] if grad is not None else [])
    shapes = dict(out=q.shape, lse=q.shape[:2], grad_q=q.shape, grad_k=k.shape, grad_v=v.shape)
    res = {n: [torch.zeros(shapes[n], dtype=torch.float64, device=dev) for _ in range(2)] for n in names}
    res["lse"][0].fill_(-math.inf)
    qo, ko = q_offsets.tolist(), k_offsets.tolist()
    for b in range(len(qo) - 1):
        keys = torch.arange(ko[b], ko[b + 1], device=dev)
        if mask is not None:
            keys = keys[mask[keys].bool()]
        n = keys.numel()
        if qo[b + 1] == qo[b] or n == 0:
            continue
        rows = slice(qo[b], qo[b + 1])
        for h in range(Hkv):
            K, V = kd[keys, h], vd[keys, h]
            gk = [torch.zeros_like(K) for _ in range(4)]  # grad_k, grad_v, their errors
            for hq in range(h * G, (h + 1) * G):
                Q = qd[rows, hq]
                s = Q @ K.T * scale
                # s is a tensor-core sum of D products, scaled in fp32; the exponential's argument and value round too
                ds_ = (D + 4) * 2 * F32 * (Q.abs() @ K.abs().T) * abs(scale) + 4 * F32 * s.abs()
                e = 2 * ds_.amax(1, keepdim=True) + (n + 64) * 2 * F32
                lse = torch.logsumexp(s, 1)
                p = torch.exp(s - lse[:, None])
                o = p @ V
                # p is rounded unnormalised, where its sum is 1 or more: the subnormal half step is not magnified
                o_err = (u + e) * (p @ V.abs()) + sub * V.abs().sum(0)
                res["out"][0][rows, hq], res["out"][1][rows, hq] = o, o_err + u * o.abs() + sub
                res["lse"][0][rows, hq] = lse
                res["lse"][1][rows, hq] = e[:, 0] + 8 * F32 * lse.abs() + 2 * F32 * s.abs().amax(1)
                if grad is None:
                    continue
                dO = grad.double()[rows, hq]
                dp = dO @ V.T
                delta = (dO * o).sum(1, keepdim=True)
                ds = p * (dp - delta)
                # the backward's p comes from the rounded lse; delta from the rounded out
                pe = p * (e + res["lse"][1][rows, hq][:, None])
                delta_err = (dO.abs() * (o_err + u * o.abs() + sub)).sum(1, keepdim=True) + (D + 2) * F32 * (dO * o).abs().sum(
                    1, keepdim=True)
                dp_err = (D + 2) * 2 * F32 * (dO.abs() @ V.abs().T)
                ds_err = pe * (dp - delta).abs() + p * (delta_err + dp_err) + (u + 4 * F32) * ds.abs() + sub
                nq = (Q.shape[0] * G + 8) * 2 * F32
                dq = ds @ K * scale
                res["grad_q"][0][rows, hq] = dq
                res["grad_q"][1][rows, hq] = (ds_err + (n + 8) * 2 * F32 * ds.abs()) @ K.abs() * abs(
                    scale) + (u + 4 * F32) * dq.abs() + sub
                gk[0] += ds.T @ Q * scale
                gk[2] += (ds_err + nq * ds.abs()).T @ Q.abs() * abs(scale)
                gk[1] += p.T @ dO
                gk[3] += (pe + (u + nq) * p + sub).T @ dO.abs()
            if grad is not None:
                res["grad_k"][0][keys, h], res["grad_v"][0][keys, h] = gk[0], gk[1]
                res["grad_k"][1][keys, h] = gk[2] + (u + 4 * F32) * gk[0].abs() + sub
                res["grad_v"][1][keys, h] = gk[3] + (u + 4 * F32) * gk[1].abs() + sub
    return res


def close(got, want, tol, what):
    """|got - want| <= tol elementwise; infinities equal."""
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    off = (got - want).abs()
    bad = ~inf & ~(off <= tol)
    if bad.any():
        i = tuple(int(x) for x in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first {i}: got {float(got[i])}, "
                             f"want {float(want[i])} +- {float(tol[i])}")

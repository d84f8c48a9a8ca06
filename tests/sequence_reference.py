"""float64 definitions of the operators over token sequences and of the optimizer step, with a bound of the
rounding error of each output.

A rounding to a type with unit eps (torch.finfo) is off by at most eps / 2 of the value. The kernels round each
probability and each dS once as an operand and each output once; everything else is fp32, taken as F32 = 1e-5 of
the sums of absolute values (a sum of up to a few thousand fp32 terms, the hardware exponential and logarithm).
Below a type's smallest normal value its steps stop shrinking: fp16 has steps of 2^-24 there, so a rounding is off
by up to 2^-25 whatever the value (bf16: 2^-134, of no account).
"""

import math

import torch

F32 = 1e-5
EXCLUDE = -1e30


def rounding(dtype, x):
    """Bound of the error of rounding values of size x to dtype."""
    f = torch.finfo(dtype)
    return torch.clamp(f.eps / 2 * x.abs(), min=f.smallest_normal * f.eps / 2)


# ------------------------------------------------------------------ norm and rotation
def _pair_index(d, rot, interleaved):
    """For each channel its partner, its angle and the sign of its partner's sine term."""
    other, angle, sign = list(range(d)), [0] * d, [0.0] * d
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        other[a], other[b], angle[a], angle[b], sign[a], sign[b] = b, a, i, i, -1.0, 1.0
    return other, angle, sign


def qk_norm(x, gamma, eps, cos=None, sin=None, positions=None, interleaved=False, dy=None):
    """{"y", "dx", "dgamma"} in float64, and bounds {"y_tol", ...} for tensors of x's type."""
    dt, dev, d = x.dtype, x.device, x.shape[-1]
    xd, w = x.double(), gamma.double()
    r = 1 / torch.sqrt((xd * xd).mean(-1, keepdim=True) + eps)
    unit = xd * r
    n = unit * w
    rot = 0 if cos is None else 2 * cos.shape[1]
    other, angle, sign = (torch.tensor(t, device=dev) for t in _pair_index(d, rot, interleaved))
    c = torch.ones(x.shape[0], x.shape[1], 1, d, dtype=torch.float64, device=dev)
    s = torch.zeros_like(c)
    if rot:
        at = torch.arange(x.shape[1], device=dev).expand(x.shape[0], -1) if positions is None else positions.long()
        turned = sign != 0
        c = torch.where(turned, cos.double()[at][..., angle][:, :, None], c)
        s = torch.where(turned, sin.double()[at][..., angle][:, :, None] * sign, s)
    y = n * c + n[..., other] * s
    out = dict(y=y, y_tol=rounding(dt, y) + F32 * (n.abs() + n[..., other].abs()))
    if dy is None:
        return out
    g = dy.double()
    g = g * c - g[..., other] * s  # the inverse turn
    gu = g * unit
    hw = g * w
    along = (hw * unit).mean(-1, keepdim=True)
    out["dgamma"] = gu.sum((0, 1, 2))
    dyo = dy.double().abs()
    mag = (dyo + dyo[..., other])
    out["dgamma_tol"] = F32 * (mag * unit.abs()).sum((0, 1, 2)) + 1e-30
    out["dx"] = r * (hw - unit * along)
    along_abs = (mag * w.abs() * unit.abs()).mean(-1, keepdim=True)
    out["dx_tol"] = rounding(dt, out["dx"]) + F32 * r * (mag * w.abs() + unit.abs() * along_abs)
    return out


# ------------------------------------------------------------------ attention with bucketed bias
def bias_attention(q, k, v, table, bmap, scale, causal=False, q_lens=None, kv_lens=None, q_start=None, dout=None):
    """{"out", "lse"} and with dout {"dq", "dk", "dv", "dtable"}, in float64, each with its "_tol"."""
    dt = q.dtype
    B, Lq, hq, d = q.shape
    Lk, hk = k.shape[1], k.shape[2]
    D, dev = bmap.numel() // 2, q.device
    assert 0 <= int(bmap.min()) and int(bmap.max()) < table.shape[0], "a bucket outside the table"
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device=dev)  # noqa: E731
    r = dict(out=z(B, Lq, hq, d), out_tol=z(B, Lq, hq, d), lse=z(B, hq, Lq) - math.inf, lse_tol=z(B, hq, Lq))
    if dout is not None:
        for n, s in (("dq", (B, Lq, hq, d)), ("dk", (B, Lk, hk, d)), ("dv", (B, Lk, hk, d)),
                     ("dtable", tuple(table.shape))):
            r[n], r[n + "_tol"] = z(*s), z(*s)
    for b in range(B):
        nq = Lq if q_lens is None else int(q_lens[b])
        nk = Lk if kv_lens is None else int(kv_lens[b])
        st = 0 if q_start is None else int(q_start[b])
        if nq == 0 or nk == 0:
            continue
        rel = torch.arange(nk, device=dev)[None] - st - torch.arange(nq, device=dev)[:, None]
        bucket = bmap.long()[rel.clamp(-D, D) + D]
        for h in range(hq):
            g = h // (hq // hk)
            Q, K, V = q[b, :nq, h].double(), k[b, :nk, g].double(), v[b, :nk, g].double()
            bias = table[:, h].double()[bucket]
            gone = bias <= EXCLUDE
            if causal:
                gone = gone | (rel > 0)
            s = torch.where(gone, -math.inf, Q @ K.T * scale + torch.where(gone, 0.0, bias))
            some = ~gone.all(1)
            top = torch.where(some, s.amax(1), 0.0)[:, None]
            e = torch.exp(s - top)
            total = torch.where(some, e.sum(1), 1.0)[:, None]
            P = e / total
            # a score's fp32 error moves its probability by as much, relatively
            ds_rel = F32 * (1 + Q.abs() @ K.abs().T * abs(scale) + torch.where(gone, 0.0, bias).abs())
            o = P @ V
            A = P @ V.abs()
            r["out"][b, :nq, h] = o
            worst = (P * ds_rel).sum(1, keepdim=True)
            o_tol = 1.01 * (rounding(dt, P) @ V.abs() + rounding(dt, o)) + (P * ds_rel) @ V.abs() + worst * A + F32 * A
            r["out_tol"][b, :nq, h] = o_tol
            r["lse"][b, h, :nq] = torch.where(some, top[:, 0] + torch.log(total[:, 0]), -math.inf)
            r["lse_tol"][b, h, :nq] = torch.where(some, worst[:, 0] + F32 * (1 + top[:, 0].abs()), 0.0)
            if dout is None:
                continue
            dO = dout[b, :nq, h].double()
            dP = dO @ V.T
            Di = (dO * o).sum(1, keepdim=True)
            dS = P * (dP - Di)
            P_tol = P * (2 * ds_rel + worst)
            D_tol = (dO.abs() * o_tol).sum(1, keepdim=True)
            mag = dO.abs() @ V.abs().T + (dO.abs() * A).sum(1, keepdim=True)
            dS_tol = P * D_tol + (P_tol + F32 * P) * mag
            round_dS = dS_tol + 1.01 * rounding(dt, dS.abs() + dS_tol)
            r["dq"][b, :nq, h] = dS @ K * scale
            r["dq_tol"][b, :nq, h] = round_dS @ K.abs() * abs(scale)
            r["dk"][b, :nk, g] += dS.T @ Q * scale
            r["dk_tol"][b, :nk, g] += round_dS.T @ Q.abs() * abs(scale)
            r["dv"][b, :nk, g] += P.T @ dO
            r["dv_tol"][b, :nk, g] += (1.01 * rounding(dt, P) + P_tol + F32 * P).T @ dO.abs()
            r["dtable"][:, h].index_add_(0, bucket.flatten(), dS.flatten())
            r["dtable_tol"][:, h].index_add_(0, bucket.flatten(), dS_tol.flatten())
    if dout is not None:
        for n in ("dq", "dk", "dv", "dtable"):
            r[n + "_tol"] = 1.01 * r[n + "_tol"] + rounding(dt, r[n]) + 1e-30
    return r


# ------------------------------------------------------------------ AdamW
def adamw(p, g, m, v, lr, b1, b2, eps, wd, step):
    """(p, m, v) after a step, float64 in and out."""
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    upd = (m / (1 - b1 ** step)) / (torch.sqrt(v / (1 - b2 ** step)) + eps)
    return p * (1 - lr * wd) - lr * upd, m, v

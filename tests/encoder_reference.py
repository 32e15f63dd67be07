"""Float64 forms of the sequence encoder's operators, written from their formulas, with bounds of what the
kernels' roundings may add.

Every value comes with a bound of its absolute error, term by term:
  half       relative half step of the stored type (results; bf16: the p and ds that enter second products)
  U * steps  float32 roundings of sums and exponents, U = 2^-24; a score's error moves p by as much relatively
"""
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def buckets(dist, bounds):
    return sum((dist >= b).long() for b in bounds) if bounds else torch.zeros_like(dist)


def attention(q, k, v, offsets, scale, bias=None, bounds=(), dout=None):
    """q [n, hq, d], k, v [n, hk, d] (any type, on the CPU).  Returns {name: (value, bound)} of out (and dq, dk, dv, dbias)."""
    half = HALF[q.dtype]
    mul = half if q.dtype == torch.bfloat16 else 0.0   # of p and ds as operands
    n, hq, d = q.shape
    hk = k.shape[1]
    G = hq // hk
    Q, K, V = (t.double().transpose(0, 1) for t in (q, k, v))
    res = {"out": [torch.zeros(hq, n, d, dtype=torch.float64) for _ in range(2)]}
    if dout is not None:
        DO = dout.double().transpose(0, 1)
        res.update(dq=[torch.zeros(hq, n, d, dtype=torch.float64) for _ in range(2)],
                   dk=[torch.zeros(hk, n, d, dtype=torch.float64) for _ in range(2)],
                   dv=[torch.zeros(hk, n, d, dtype=torch.float64) for _ in range(2)])
        if bias is not None:
            res["dbias"] = [torch.zeros(bias.shape, dtype=torch.float64) for _ in range(2)]
    offs = [min(max(int(o), 0), n) for o in offsets]
    for a, b in zip(offs[:-1], offs[1:]):
        if b <= a:
            continue
        L = b - a
        dist = torch.arange(L)[:, None] - torch.arange(L)
        bk = buckets(dist, bounds)
        for h in range(hq):
            g = h // G
            x, y, z = Q[h, a:b], K[g, a:b], V[g, a:b]
            S = x @ y.T * scale
            size = x.abs() @ y.abs().T * scale
            if bias is not None:
                B = bias.double()[:, h][bk]
                S = S + torch.where(B <= -1e30, -torch.inf, B)
                size = size + torch.where(B <= -1e30, 0.0, B.abs())
            S = S.masked_fill(dist < 0, -torch.inf)
            m = S.amax(1, keepdim=True).clamp(min=-1e300)
            E = (S - m).exp()
            z0 = E.sum(1, keepdim=True)
            P = E / z0.clamp(min=1e-300)
            lse = m + z0.clamp(min=1e-300).log()
            near = torch.where(P > 0, size, 0.0)
            # scores: d products and sums, the factor, the reference; the row's sum has the same once more
            rel = U * ((d + 8) * near + 8 * (lse.abs().clamp(max=1e30) + (S - lse).abs().nan_to_num(0.0, 0.0, 0.0)) + 2 * L + 8)
            rel = rel + (P * rel).sum(1, keepdim=True)
            O = P @ z
            eO = half * O.abs() + (P * (mul + rel + L * U)) @ z.abs()
            res["out"][0][h, a:b], res["out"][1][h, a:b] = O, eO
            if dout is None:
                continue
            do = DO[h, a:b]
            dP = do @ z.T
            D = (P * dP).sum(1, keepdim=True)
            dS = P * (dP - D)
            sizeP = do.abs() @ z.abs().T
            # D: exact up to float32 in dk and dbias; for dq from the rounded outputs
            eD = (P * (rel + L * U) * sizeP).sum(1, keepdim=True) + U * (d + 8) * (P * sizeP).sum(1, keepdim=True)
            eDq = eD + (do.abs() * eO).sum(1, keepdim=True)
            eS = P * (rel * (dP - D).abs() + U * (d + 8) * sizeP + U * 4 * D.abs())
            for name, e, w in (("dq", eDq, y), ("dk", eD, x)):
                T, eT = dS, (eS + P * e) + (mul + L * U) * dS.abs()
                if name == "dk":
                    T, eT = T.T, eT.T
                val = T @ w * scale
                at = h if name == "dq" else g
                res[name][0][at, a:b] += val
                res[name][1][at, a:b] += eT @ w.abs() * scale
            res["dv"][0][g, a:b] += P.T @ do
            res["dv"][1][g, a:b] += (P * (mul + rel + L * U)).T @ do.abs()
            if bias is not None:
                for c in range(bias.shape[0]):
                    pick = (bk == c) & (dist >= 0)
                    res["dbias"][0][c, h] += dS[pick].sum()
                    res["dbias"][1][c, h] += ((eS + P * eD)[pick].sum() + 64 * U * dS.abs()[pick].sum())
    out = {}
    for name, (val, e) in res.items():
        if name in ("dq", "dk", "dv"):
            e = e + half * val.abs()
        if name != "dbias":
            val, e = val.transpose(0, 1), e.transpose(0, 1)
        out[name] = (val, e)
    return out


def close(got, want, floor=1e-30):
    """Largest error in units of its bound."""
    val, e = want
    return float(((got.double().cpu() - val).abs() / (e + floor)).max()) if val.numel() else 0.0


def norm(x, residual, weight, eps, dy=None, dh=None):
    """{name: value} in float64 from the stored h, which is returned in the inputs' type."""
    h16 = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    h, w = h16.double(), weight.double()
    rstd = 1.0 / (h.square().mean(1, keepdim=True) + eps).sqrt()
    out = {"h": h16, "rstd": rstd[:, 0], "y": h * rstd * w}
    if dy is not None:
        g = dy.double() * w
        out["dx"] = rstd * (g - h * rstd.square() * (g * h).mean(1, keepdim=True)) + (0 if dh is None else dh.double())
        out["dweight"] = (dy.double() * h * rstd).sum(0)
    return out


def int8_rows(t):
    """(values, scale) of float64 rows: ties to even."""
    m = t.abs().amax(1, keepdim=True)
    return torch.where(m > 0, (127.0 * t / torch.where(m > 0, m, 1.0)).round(), 0.0).to(torch.int8), m[:, 0] / 127.0


def moved(tensors):
    """Tensors (or None) on the GPU."""
    return tuple(t if t is None else t.cuda() for t in tensors)

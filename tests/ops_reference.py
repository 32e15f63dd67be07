"""Plain float64 forms of the operators around the losses (item embedding, catalogue
log-probabilities, policy and preference losses), from the formulas in include/rece.h,
on the CPU, with the error bounds the GPU results are held to.

A rounding to type t is off by at most U[t] relative to the value."""
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
U32 = 2.0 ** -24
F64 = torch.float64


# ------------------------------------------------------------------ item embedding
def embed(table, ids, scale):
    keep = (ids >= 0) & (ids < table.shape[0])
    out = torch.zeros(ids.numel(), table.shape[1], dtype=F64)
    out[keep] = table.double()[ids[keep].long()] * scale
    return out


def embed_grad(ids, dout, C, scale):
    """(gradient, bound without the rounding to the output type).  A row of k terms is summed in
    float32: k - 1 additions, each off by U32 of a partial sum no larger than the sum of
    magnitudes, then one product with the scale."""
    keep = (ids >= 0) & (ids < C)
    g = torch.zeros(C, dout.shape[1], dtype=F64)
    mag = torch.zeros_like(g)
    k = torch.zeros(C, dtype=F64)
    at = ids[keep].long()
    g.index_add_(0, at, dout.double()[keep])
    mag.index_add_(0, at, dout.double()[keep].abs())
    k.index_add_(0, at, torch.ones(at.numel(), dtype=F64))
    return g * scale, (k[:, None] + 1) * U32 * 1.01 * mag * abs(scale)


# ------------------------------------------------------------------ log-probabilities
def logprob(X, Y, ids, T, dlogp=None, dent=None):
    """dict of logp, entropy, dX, dY and, for each, "e_..." the magnitude its error scales with."""
    C, d = Y.shape
    s = X.shape[0]
    keep = (ids >= 0) & (ids < C)
    a = ids[keep].long()
    Xk, Yd = X.double()[keep], Y.double()
    L = Xk @ Yd.T / T
    logq = torch.log_softmax(L, 1)
    q = logq.exp()
    H = -(torch.where(q > 0, q * logq, 0.0)).sum(1)
    n = torch.arange(a.numel())
    out = {}

    def full(v, shape):
        f = torch.zeros(shape, dtype=F64)
        f[keep] = v
        return f

    out["logp"] = full(logq[n, a], (s,))
    out["entropy"] = full(H, (s,))
    # A float32 logit: d products and d additions, each off by U32 of the sum of magnitudes, and
    # the factor log2(e) / T (two roundings); in nats.
    mag = Xk.abs() @ Yd.abs().T / T
    ex = (d + 4) * U32 * mag.amax(1) if a.numel() else torch.zeros(0, dtype=F64)
    # log-sum-exp: the logits' error, the reference and fma at the size of the largest logit, and a
    # sum of positive terms: 16 in a row, then one per block of 32 items, then the parts (at
    # most 1024 + a few), each exp2 off by 2 U32
    depth = 16 + C / 32 + 64 + 8
    elog = 2 * ex + (depth + 8 * (L.abs().amax(1) if a.numel() else 0.0) + 40) * U32
    out["e_logp"] = full(elog, (s,)) + 4 * U32 * out["logp"].abs()
    # sum p (x - m) has the same terms times their distance from the reference
    far = (L.amax(1) - L.amin(1)).clamp(max=200.0) + 1.0 if a.numel() else torch.zeros(0, dtype=F64)
    out["e_entropy"] = full(elog * (far + 2.0), (s,))
    if dlogp is None:
        return out
    g = dlogp.double()[keep][:, None]
    h = dent.double()[keep][:, None] if dent is not None else torch.zeros_like(g)
    G = -q * (g + h * (logq + H[:, None]))
    size = q * (g.abs() + h.abs() * (logq.abs() + H[:, None]))   # what a weight's error scales with
    hot = torch.zeros_like(G)
    hot[n, a] = 1.0
    G = (G + hot * g) / T
    size, hot = size / T, hot * g.abs() / T
    out["dX"] = full(G @ Yd, (s, d))
    out["dY"] = G.T @ Xk
    # exp2 of a logit and a log-sum-exp that are off, and the entropy's own error
    rel = (2 * ex + elog + 8 * U32)[:, None] + h.abs() * (out["e_entropy"][keep])[:, None] / (g.abs() + h.abs() + 1e-300)
    size_e = size * rel
    one = torch.ones_like(size)
    out["p_dX"] = full(size_e @ Yd.abs() + C * 2 * U32 * ((size + hot) @ Yd.abs()), (s, d))
    out["p_dY"] = size_e.T @ Xk.abs() + max(s, 1) * 2 * U32 * ((size + hot).T @ Xk.abs())
    # the weights rounded once to bf16 before the product (results that are bf16 themselves)
    r = U[torch.bfloat16]
    out["b_dX"] = full(r * (size @ Yd.abs()), (s, d))
    out["b_dY"] = r * (size.T @ Xk.abs())
    del one
    return out


# ------------------------------------------------------------------ policy loss
def seq_of_tokens(offsets, n):
    """Sequence of every token, -1 where it is in none (offsets clamped into [0, n])."""
    o = offsets.long().clamp(0, n)
    seq = torch.full((n,), -1, dtype=torch.long)
    for i in range(o.numel() - 1):
        seq[o[i]:o[i + 1]] = i
    return seq


def policy(logp, old, adv, offsets, cfg, ref=None, entropy=None, mask=None):
    """(loss, stats, dlogp, dentropy) in float64; gradients by autograd of the formula."""
    n, ns = logp.numel(), offsets.numel() - 1
    seq = seq_of_tokens(offsets, n)
    keep = seq >= 0
    if mask is not None:
        keep &= mask != 0
    at = torch.nonzero(keep)[:, 0]
    lp = logp.double()[at].requires_grad_(True)
    H = entropy.double()[at].requires_grad_(True) if entropy is not None else torch.zeros(at.numel(), dtype=F64)
    A = (adv[at] if cfg["token"] else adv[seq[at]]).double()
    r = (lp - old.double()[at]).exp()
    lo, hi = 1.0 - cfg["low"], 1.0 + cfg["high"]
    near = r.clamp(lo, hi)
    pg = -torch.minimum(r * A, near * A)
    kl = torch.zeros_like(pg)
    if ref is not None:
        u = ref.double()[at] - lp
        kl = u.exp() - u - 1
    total = pg + (cfg["kl"] * kl if cfg["kl"] else 0.0) - (cfg["ent"] * H if cfg["ent"] else 0.0)
    count = torch.zeros(ns, dtype=F64).index_add_(0, seq[at], torch.ones(at.numel(), dtype=F64))
    if cfg["reduction"] == "token":
        w = torch.full((at.numel(),), 1.0 / max(at.numel(), 1), dtype=F64)
    else:
        w = 1.0 / (count[seq[at]] * max(int((count > 0).sum()), 1))
    loss = (w * total).sum()
    dlp, dH = torch.zeros(n, dtype=F64), torch.zeros(n, dtype=F64)
    if at.numel():
        loss.backward()
        dlp[at] = lp.grad
        if entropy is not None and cfg["ent"]:
            dH[at] = H.grad
    mean = lambda v: float(v.detach().sum() / max(at.numel(), 1))  # noqa: E731
    clipped = ((A > 0) & (r > hi)) | ((A < 0) & (r < lo))
    stats = [mean(pg), mean(kl), mean(H), mean(clipped.double()), mean(r), float(at.numel())]
    return float(loss.detach()), stats, dlp, dH


# ------------------------------------------------------------------ preference loss
def preference(logp, ref, offsets, goffs, cfg, mask=None):
    """(loss, loss per group, rewards, dlogp) in float64; the gradient by autograd of the formula."""
    n, ns, G = logp.numel(), offsets.numel() - 1, goffs.numel() - 1
    seq = seq_of_tokens(offsets, n)
    keep = seq >= 0
    if mask is not None:
        keep &= mask != 0
    at = torch.nonzero(keep)[:, 0]
    lp = logp.double()[at].requires_grad_(True)
    v = lp - (ref.double()[at] if ref is not None else 0.0)
    h = torch.zeros(ns, dtype=F64).index_add(0, seq[at], v)
    if cfg["average"]:
        c = torch.zeros(ns, dtype=F64).index_add_(0, seq[at], torch.ones(at.numel(), dtype=F64))
        h = h / c.clamp(min=1)
    beta = cfg["beta"]
    o = goffs.long().clamp(0, ns)
    per_group = []
    for g in range(G):
        lo, hi = int(o[g]), int(o[g + 1])
        if hi - lo < 2:
            per_group.append(torch.zeros((), dtype=F64))
            continue
        z = beta * (h[lo] - h[lo + 1:hi]) - cfg["margin"]
        if cfg["kind"] == "softmax":
            per_group.append(torch.logsumexp(torch.cat([torch.zeros(1, dtype=F64), -z]), 0))
        elif cfg["kind"] == "sigmoid":
            ls = torch.nn.functional.logsigmoid
            per_group.append((-(1 - cfg["smoothing"]) * ls(z) - cfg["smoothing"] * ls(-z)).mean())
        elif cfg["kind"] == "ipo":
            per_group.append(((z / beta - 0.5 / beta) ** 2).mean())
        else:
            per_group.append(torch.relu(1 - z).mean())
    loss_pg = torch.stack(per_group)
    loss = loss_pg.mean()
    dlp = torch.zeros(n, dtype=F64)
    if at.numel() and loss.requires_grad:
        loss.backward()
        if lp.grad is not None:
            dlp[at] = lp.grad
    return float(loss.detach()), loss_pg.detach(), (beta * h).detach(), dlp

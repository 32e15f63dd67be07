"""Cases of the operators around the catalogue losses, for timing and for comparison.

Four operators, each as a user's program calls it:
  embed       rows of the item table as a model's inputs (scaled), and the table's gradient
  logprob     log-probability of one item per position under the softmax over the whole
              catalogue, its entropy, and the gradients of both for positions and items
  policy      clipped policy loss with a KL and an entropy term on ragged sequences, with
              the gradient of the log-probabilities
  preference  paired log ratios of sequences in groups (one preferred, the rest not), with
              the gradient of the log-probabilities

`run` is the plain form (elementary torch operations in 32 bits, 64 for long sums) where
`own` is false, and the framework's entry points where it is true.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the lookup of one small batch (4 sequences of 64 items): latency counts
        dict(name="embed_fwd_256", op="embed", n=256, C=2000, d=64, dtype="f32", train=False, alpha=0.0, pad=0.0),
        # a SASRec batch: 256 sequences of 200 items, popularity by Zipf's law, a quarter of it padding
        dict(name="embed_train_51200", op="embed", n=51200, C=30000, d=64, dtype="bf16", train=True, alpha=1.1, pad=0.25),
        # a catalogue of a million items: the dense gradient is what costs
        dict(name="embed_train_1m", op="embed", n=25600, C=1_000_000, d=128, dtype="bf16", train=True, alpha=1.0,
             pad=0.0),
        # serving: the probability of one chosen item for five users, a million items
        dict(name="logprob_fwd_5x1m", op="logprob", s=5, C=1_000_000, d=64, dtype="bf16", train=False, entropy=True,
             temperature=0.7, pad=0.0),
        # scoring of collected sequences (old and reference policies): forward only
        dict(name="logprob_fwd_2047x200k", op="logprob", s=2047, C=200_000, d=128, dtype="bf16", train=False,
             entropy=False, temperature=1.0, pad=0.1),
        # the smallest training step, float32 throughout
        dict(name="logprob_train_256x2000_f32", op="logprob", s=256, C=2000, d=64, dtype="f32", train=True,
             entropy=True, temperature=1.0, pad=0.1),
        # a SASRec batch, 51,200 positions on 30,000 items, no entropy term
        dict(name="logprob_train_51200x30000", op="logprob", s=51200, C=30000, d=64, dtype="bf16", train=True,
             entropy=False, temperature=1.0, pad=0.25),
        # a policy update with an entropy bonus, wide vectors, sizes that divide by nothing
        dict(name="logprob_train_4099x50021_d256", op="logprob", s=4099, C=50021, d=256, dtype="bf16", train=True,
             entropy=True, temperature=1.3, pad=0.1),
        # one small update: 16 sequences of a few items each
        dict(name="policy_16", op="policy", n_seq=16, mean_len=24, dtype="f32", kl=0.05, ent=0.01, per_token=False,
             reduction="sequence", masked=True),
        # a large one: 8,192 ragged sequences, about four million tokens
        dict(name="policy_8192", op="policy", n_seq=8192, mean_len=512, dtype="f32", kl=0.05, ent=0.0, per_token=False,
             reduction="token", masked=True),
        # pairs of single items (one shown and taken, one shown and not)
        dict(name="preference_256_items", op="preference", groups=256, rejected=1, mean_len=1, dtype="f32",
             kind="sigmoid", smoothing=0.1, average=False, masked=False),
        # one preferred sequence against up to seven, softmax over them, ragged lengths, stored in 16 bits
        dict(name="preference_2048x8", op="preference", groups=2048, rejected=7, mean_len=200, dtype="bf16",
             kind="softmax", smoothing=0.0, average=False, masked=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "logprob", "logprob", "policy", "preference"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "embed":
        return dict(op=op, n=_log_int(rng, 1, 51200), C=_log_int(rng, 500, 1_000_000), d=rng.choice([32, 64, 128]),
                    dtype=dtype, train=rng.random() < 0.7, alpha=rng.choice([0.0, 1.0, 1.1]),
                    pad=rng.choice([0.0, 0.1, 0.25]))
    if op == "logprob":
        d = rng.choice([32, 64, 128, 256])
        s, C = _log_int(rng, 1, 51200), _log_int(rng, 500, 1_000_000)
        most = (1 << 34) // d if dtype == "f32" else (1 << 36) // d
        most = min(most, 1_200_000_000)
        if s * C > most:
            s = max(1, most // C)
        return dict(op=op, s=s, C=C, d=d, dtype=dtype, train=rng.random() < 0.6, entropy=rng.random() < 0.5,
                    temperature=rng.choice([0.7, 1.0, 1.3]), pad=rng.choice([0.0, 0.1, 0.25]))
    if op == "policy":
        n_seq = _log_int(rng, 1, 8192)
        return dict(op=op, n_seq=n_seq, mean_len=_log_int(rng, 4, 512), dtype=dtype, kl=rng.choice([0.0, 0.05]),
                    ent=rng.choice([0.0, 0.01]), per_token=rng.random() < 0.3,
                    reduction=rng.choice(["token", "sequence"]), masked=rng.random() < 0.6)
    return dict(op=op, groups=_log_int(rng, 1, 2048), rejected=rng.choice([1, 1, 3, 7]), mean_len=_log_int(rng, 1, 200),
                dtype=dtype, kind=rng.choice(["sigmoid", "ipo", "hinge", "softmax"]), smoothing=rng.choice([0.0, 0.1]),
                average=rng.random() < 0.3, masked=rng.random() < 0.6)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ids(g, n, C, alpha, pad):
    """n item ids: uniform (alpha 0) or by a power law over a shuffled catalogue; a share `pad` of -1."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    if alpha > 0:
        cdf = torch.arange(1, C + 1, device="cuda", dtype=torch.float64).pow(-alpha).cumsum(0)
        ranks = torch.searchsorted(cdf, u * cdf[-1]).clamp_(max=C - 1)
        ids = torch.randperm(C, generator=g, device="cuda")[ranks]
    else:
        ids = (u * C).long().clamp_(max=C - 1)
    if pad > 0:
        ids = torch.where(torch.rand(n, generator=g, device="cuda") < pad, -1, ids)
    return ids.to(torch.int32)


def _rows(g, n, d, scale=1.0):
    return torch.randn(n, d, generator=g, device="cuda") * (scale * d ** -0.25)


def _offsets(g, n_seq, mean_len):
    """Ends of n_seq sequences with n_seq * mean_len tokens in all, and that number: every sequence one token
    where mean_len is 1, otherwise cut at random places (many short ones, a few long, some of one token or none)."""
    n = n_seq * mean_len
    if mean_len == 1:
        return torch.arange(n_seq + 1, device="cuda", dtype=torch.int32), n
    offs = torch.zeros(n_seq + 1, device="cuda", dtype=torch.int32)
    offs[1:n_seq] = torch.randint(0, n + 1, (n_seq - 1,), generator=g, device="cuda").sort().values.to(torch.int32)
    offs[n_seq] = n
    return offs, n


def _logps(g, n, spread):
    """Log-probabilities of a next item (mostly between -12 and 0) and a copy that moved a little."""
    a = -12.0 * torch.rand(n, generator=g, device="cuda").pow(1.5) - 0.01
    b = a + spread * torch.randn(n, generator=g, device="cuda")
    return a, b.clamp_(max=-1e-4)


def prepare(case, seed):
    g = _gen(seed)
    dt = _DT[case["dtype"]]
    st = {"case": case}
    op = case["op"]
    if op == "embed":
        n, C, d = case["n"], case["C"], case["d"]
        st["table"] = _rows(g, C, d).to(dt)
        st["ids"] = _ids(g, n, C, case["alpha"], case["pad"])
        st["scale"] = math.sqrt(d)
        if case["train"]:
            st["dout"] = (torch.randn(n, d, generator=g, device="cuda") * 1e-3).to(dt)
    elif op == "logprob":
        s, C, d = case["s"], case["C"], case["d"]
        Yf = _rows(g, C, d)
        st["ids"] = _ids(g, s, C, 1.0, case["pad"])
        # hidden states that point towards their item more or less, as a trained model's do
        lean = 2.0 * torch.rand(s, 1, generator=g, device="cuda")
        st["X"] = (_rows(g, s, d, 1.5) + lean * Yf[st["ids"].long().clamp(min=0)]).to(dt)
        st["Y"] = Yf.to(dt)
        if case["train"]:
            st["dlogp"] = torch.randn(s, generator=g, device="cuda") / s
            if case["entropy"]:
                st["dent"] = torch.full((s,), -0.01 / s, device="cuda")
    elif op == "policy":
        offs, n = _offsets(g, case["n_seq"], case["mean_len"])
        lp, old = _logps(g, n, 0.15)
        st["offsets"], st["logp"], st["old"] = offs, lp.to(dt), old.to(dt)
        if case["kl"] > 0:
            st["ref"] = (lp + 0.3 * torch.randn(n, generator=g, device="cuda")).clamp_(max=-1e-4).to(dt)
        if case["ent"] > 0:
            st["entropy"] = (6.0 * torch.rand(n, generator=g, device="cuda")).to(dt)
        st["adv"] = torch.randn(n if case["per_token"] else case["n_seq"], generator=g, device="cuda")
        if case["masked"]:
            st["mask"] = (torch.rand(n, generator=g, device="cuda") < 0.9).to(torch.uint8)
    else:
        n_seq = case["groups"] * (1 + case["rejected"])
        offs, n = _offsets(g, n_seq, case["mean_len"])
        lp, ref = _logps(g, n, 0.2)
        st["offsets"], st["logp"], st["ref"] = offs, lp.to(dt), ref.to(dt)
        # one preferred and 1 .. `rejected` others for each group
        extra = torch.randint(1, case["rejected"] + 1, (case["groups"],), generator=g, device="cuda")
        goffs = torch.zeros(case["groups"] + 1, device="cuda", dtype=torch.int64)
        goffs[1:] = (1 + extra).cumsum(0)
        st["goffsets"] = goffs.to(torch.int32)
        if case["masked"]:
            st["mask"] = (torch.rand(n, generator=g, device="cuda") < 0.9).to(torch.uint8)
    if own:
        st["op"] = _handle(case, st)
    return st


def _handle(case, st):
    import catalogue_cross_entropy_amd as rece
    op = case["op"]
    if op == "embed":
        return rece.ItemEmbedding(case["n"], case["C"], case["d"], dtype=case["dtype"], scale=st["scale"])
    if op == "logprob":
        return rece.LogProb(case["s"], case["C"], case["d"], dtype=case["dtype"], temperature=case["temperature"],
                            entropy=case["entropy"], bf16_grads=case["dtype"] == "bf16")
    if op == "policy":
        return rece.PolicyLoss(st["logp"].numel(), case["n_seq"], clip_low=0.2, clip_high=0.28, kl_coef=case["kl"],
                               entropy_coef=case["ent"], reduction=case["reduction"], token_advantage=case["per_token"],
                               dtype=case["dtype"])
    return rece.PreferenceLoss(st["logp"].numel(), st["offsets"].numel() - 1, case["groups"], beta=0.1,
                               kind=case["kind"], label_smoothing=case["smoothing"], average=case["average"],
                               dtype=case["dtype"])


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        h = state["op"]
        if op == "embed":
            out = {"out": h.forward(state["table"], state["ids"])}
            if case["train"]:
                out["dtable"] = h.backward(state["ids"], state["dout"])
            return out
        if op == "logprob":
            logp, ent, ws = h.forward(state["X"], state["Y"], state["ids"], need_grad=case["train"])
            out = {"logp": logp}
            if case["entropy"]:
                out["entropy"] = ent
            if case["train"]:
                out["dX"], out["dY"] = h.backward(state["X"], state["Y"], state["ids"], ws, state["dlogp"],
                                                  dentropy=state.get("dent"))
            return out
        if op == "policy":
            loss, stats, dlogp, dent = h.forward(state["logp"], state["old"], state["adv"], state["offsets"],
                                                 ref_logp=state.get("ref"), entropy=state.get("entropy"),
                                                 mask=state.get("mask"))
            out = {"loss": loss, "stats": stats, "dlogp": dlogp}
            if case["ent"] > 0:
                out["dentropy"] = dent
            return out
        loss, loss_pg, rewards, dlogp = h.forward(state["logp"], state["ref"], state["offsets"], state["goffsets"],
                                                  mask=state.get("mask"))
        return {"loss": loss, "loss_pg": loss_pg, "rewards": rewards, "dlogp": dlogp}
    return {"embed": _embed, "logprob": _logprob, "policy": _policy, "preference": _preference}[op](state, case)


def _embed(st, case):
    ids, C = st["ids"].long(), case["C"]
    valid = (ids >= 0) & (ids < C)
    at = torch.where(valid, ids, 0)
    rows = st["table"][at].float() * st["scale"]
    out = {"out": torch.where(valid[:, None], rows, 0.0).to(st["table"].dtype)}
    if case["train"]:
        add = torch.where(valid[:, None], st["dout"].float() * st["scale"], 0.0)
        dtable = torch.zeros(C, case["d"], device=ids.device)
        dtable.index_add_(0, at, add)
        out["dtable"] = dtable
    return out


def _logprob(st, case):
    dt = st["X"].dtype
    X, Y, ids = st["X"].float(), st["Y"].float(), st["ids"].long()
    valid = (ids >= 0) & (ids < case["C"])
    at = torch.where(valid, ids, 0)[:, None]
    L = torch.matmul(X, Y.t()) * (1.0 / case["temperature"])
    m = L.amax(1, keepdim=True)
    e = (L - m).exp()
    z = e.sum(1, keepdim=True)
    lse = m + z.log()
    logp = L.gather(1, at) - lse
    out = {"logp": torch.where(valid, logp[:, 0], 0.0)}
    ent = None
    if case["entropy"]:
        ent = lse - (e * L).sum(1, keepdim=True) / z
        out["entropy"] = torch.where(valid, ent[:, 0], 0.0)
    if case["train"]:
        g = torch.where(valid, st["dlogp"], 0.0)[:, None]
        P = e / z
        if case["entropy"]:
            h = torch.where(valid, st["dent"], 0.0)[:, None]
            G = -P * (g + h * (L - lse + ent))
        else:
            G = -P * g
        G.scatter_add_(1, at, g)
        G *= 1.0 / case["temperature"]
        out["dX"] = torch.matmul(G, Y).to(dt)
        out["dY"] = torch.matmul(G.t(), X).to(dt)
    return out


def _seq_of(offs, n):
    """Sequence of every token."""
    return torch.searchsorted(offs.long(), torch.arange(n, device=offs.device), right=True) - 1


def _seq_sum(v, offs):
    """Sum of v over every sequence: differences of a running sum in 64 bits."""
    c = torch.zeros(v.numel() + 1, device=v.device, dtype=torch.float64)
    c[1:] = v.double().cumsum(0)
    return c[offs[1:].long()] - c[offs[:-1].long()]


def _policy(st, case):
    n, n_seq = st["logp"].numel(), case["n_seq"]
    seq = _seq_of(st["offsets"], n)
    lp, old = st["logp"].float(), st["old"].float()
    keep = st["mask"].bool() if case["masked"] else torch.ones(n, dtype=torch.bool, device=lp.device)
    count = _seq_sum(keep, st["offsets"])
    tokens = count.sum()
    if case["reduction"] == "token":
        w = (1.0 / tokens.clamp(min=1.0)).expand(n)
    else:
        w = (1.0 / (count.clamp(min=1.0) * (count > 0).sum().clamp(min=1)))[seq]
    w = torch.where(keep, w.float(), 0.0)
    A = st["adv"] if case["per_token"] else st["adv"][seq]
    r = (lp - old).exp()
    clipped = ((A > 0) & (r > 1.0 + 0.28)) | ((A < 0) & (r < 1.0 - 0.2))
    pg = -torch.where(clipped, A * r.clamp(1.0 - 0.2, 1.0 + 0.28), A * r)
    dlp = torch.where(clipped, 0.0, -A * r)
    total = pg
    kl = torch.zeros_like(lp)
    if case["kl"] > 0:
        u = st["ref"].float() - lp
        eu = u.exp()
        kl = eu - u - 1.0
        total = total + case["kl"] * kl
        dlp = dlp + case["kl"] * (1.0 - eu)
    H = torch.zeros_like(lp)
    if case["ent"] > 0:
        H = st["entropy"].float()
        total = total - case["ent"] * H
    mean = lambda v: (torch.where(keep, v.double(), 0.0).sum() / tokens.clamp(min=1.0)).float()  # noqa: E731
    out = {"loss": (w.double() * torch.where(keep, total, 0.0).double()).sum().float().reshape(1),
           "stats": torch.stack([mean(pg), mean(kl), mean(H), mean(clipped), mean(r), tokens.float()]),
           "dlogp": (w * torch.where(keep, dlp, 0.0)).to(st["logp"].dtype)}
    if case["ent"] > 0:
        out["dentropy"] = (-case["ent"] * w).to(st["logp"].dtype)
    return out


def _softplus(x):
    return x.clamp(min=0.0) + torch.log1p(torch.exp(-x.abs()))


def _preference(st, case):
    n, n_seq, G, beta = st["logp"].numel(), st["offsets"].numel() - 1, case["groups"], 0.1
    dev = st["logp"].device
    seq = _seq_of(st["offsets"], n)
    keep = st["mask"].bool() if case["masked"] else torch.ones(n, dtype=torch.bool, device=dev)
    ratio = torch.where(keep, st["logp"].float() - st["ref"].float(), 0.0)
    h = _seq_sum(ratio, st["offsets"])
    share = torch.ones(n_seq, device=dev, dtype=torch.float64)
    if case["average"]:
        share = 1.0 / _seq_sum(keep, st["offsets"]).clamp(min=1.0)
        h = h * share
    goffs = st["goffsets"].long()
    i = torch.arange(n_seq, device=dev)
    grp = torch.searchsorted(goffs, i, right=True) - 1
    inside = grp < G
    grp = grp.clamp(max=G - 1)
    first = goffs[grp]
    other = inside & (i > first)
    others = _seq_sum(other, goffs)
    z = beta * (h[first] - h)
    if case["kind"] == "softmax":
        e = torch.where(other, (-z).exp(), 0.0)
        tot = 1.0 + _seq_sum(e, goffs)
        loss_pg = tot.log()
        dz = -e / tot[grp]
    else:
        eps = case["smoothing"]
        if case["kind"] == "sigmoid":
            l = (1.0 - eps) * _softplus(-z) + eps * _softplus(z)
            dz = torch.sigmoid(z) - (1.0 - eps)
        elif case["kind"] == "ipo":
            l = (z / beta - 0.5 / beta) ** 2
            dz = 2.0 * (z / beta - 0.5 / beta) / beta
        else:
            l = (1.0 - z).clamp(min=0.0)
            dz = -(z < 1.0).double()
        per = 1.0 / others.clamp(min=1.0)[grp]
        loss_pg = _seq_sum(torch.where(other, l * per, 0.0), goffs)
        dz = torch.where(other, dz * per, 0.0)
    dh = -beta * dz
    dh.index_add_(0, first, beta * dz)
    dh = torch.where(inside, dh, 0.0) * share / G
    return {"loss": loss_pg.mean().float().reshape(1), "loss_pg": loss_pg.float(), "rewards": (beta * h).float(),
            "dlogp": torch.where(keep, dh.float()[seq], 0.0).to(st["logp"].dtype)}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "embed":
        n, C, d = case["n"], case["C"], case["d"]
        b, f = 4 * n + min(n, C) * d * es + n * d * es, n * d
        if case["train"]:
            b, f = b + n * d * es + C * d * 4, f + 2 * n * d
        return {"bytes": b, "flops": f}
    if op == "logprob":
        s, C, d = case["s"], case["C"], case["d"]
        b, f = (s + C) * d * es + 4 * s * (3 if case["entropy"] else 2), 2 * s * C * d
        if case["train"]:
            b, f = b + (s + C) * d * es + 4 * s * (2 if case["entropy"] else 1), 3 * f
        return {"bytes": b, "flops": f}
    if op == "policy":
        n = case["n_seq"] * case["mean_len"]
        arrays = 3 + (case["kl"] > 0) + 2 * (case["ent"] > 0)
        return {"bytes": n * (arrays * es + (1 if case["masked"] else 0)) + (4 * n if case["per_token"] else 0)
                + 8 * case["n_seq"], "flops": 20 * n}
    n_seq = case["groups"] * (1 + case["rejected"])
    n = n_seq * case["mean_len"]
    return {"bytes": n * (3 * es + (1 if case["masked"] else 0)) + 8 * n_seq + 8 * case["groups"], "flops": 4 * n}


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    st = prepare(case, seed)
    f64 = {k: v.double() for k, v in st.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    op = case["op"]
    if op == "embed":
        keep = (st["ids"] >= 0) & (st["ids"] < case["C"])
        out = torch.zeros(case["n"], case["d"], device="cuda", dtype=torch.float64)
        out[keep] = f64["table"][st["ids"][keep].long()] * st["scale"]
        res = {"out": out}
        if case["train"]:
            # sums of equal ids by differences of a running sum over the sorted rows
            ids, order = torch.sort(st["ids"][keep].long(), stable=True)
            run_sum = torch.cat([torch.zeros(1, case["d"], device="cuda", dtype=torch.float64),
                                 (f64["dout"][keep][order] * st["scale"]).cumsum(0)])
            edges = torch.searchsorted(ids, torch.arange(case["C"] + 1, device="cuda"))
            res["dtable"] = run_sum[edges[1:]] - run_sum[edges[:-1]]
        return res
    if op == "logprob":
        s, C, T = case["s"], case["C"], case["temperature"]
        keep = torch.nonzero((st["ids"] >= 0) & (st["ids"] < C))[:, 0]
        a = st["ids"][keep].long()
        X, Y = f64["X"], f64["Y"]
        res = {"logp": torch.zeros(s, device="cuda", dtype=torch.float64)}
        if case["entropy"]:
            res["entropy"] = torch.zeros_like(res["logp"])
        if case["train"]:
            res["dX"], res["dY"] = torch.zeros_like(X), torch.zeros_like(Y)
        for lo in range(0, keep.numel(), 2048):
            rows, pick = keep[lo:lo + 2048], a[lo:lo + 2048]
            logq = torch.log_softmax(X[rows] @ Y.T / T, dim=1)
            at = torch.arange(rows.numel(), device="cuda")
            res["logp"][rows] = logq[at, pick]
            q = logq.exp()
            if case["entropy"]:
                H = -(q * logq).sum(1)
                res["entropy"][rows] = H
            if case["train"]:
                w = -q * f64["dlogp"][rows, None]
                if case["entropy"]:
                    w -= f64["dent"][rows, None] * q * (logq + H[:, None])
                w[at, pick] += f64["dlogp"][rows]
                res["dX"][rows] = w @ Y / T
                res["dY"] += w.T @ X[rows] / T
        return res
    lens = st["offsets"].long().diff()
    n = st["logp"].numel()
    seq = torch.repeat_interleave(torch.arange(lens.numel(), device="cuda"), lens)
    keep = st["mask"].double() if case["masked"] else torch.ones(n, device="cuda", dtype=torch.float64)

    def per_seq(v):
        return v.new_zeros(lens.numel()).scatter_add(0, seq, v)

    if op == "policy":
        lp = f64["logp"].requires_grad_(True)
        H = f64["entropy"].requires_grad_(True) if case["ent"] > 0 else torch.zeros_like(lp)
        A = f64["adv"] if case["per_token"] else f64["adv"][seq]
        ratio = (lp - f64["old"]).exp()
        near = torch.minimum(torch.maximum(ratio, ratio.new_tensor(0.8)), ratio.new_tensor(1.28))
        pg = -torch.minimum(ratio * A, near * A)
        kl = ((f64["ref"] - lp).exp() - (f64["ref"] - lp) - 1) if case["kl"] > 0 else torch.zeros_like(lp)
        each = (pg + case["kl"] * kl - case["ent"] * H) * keep
        if case["reduction"] == "token":
            loss = each.sum() / keep.sum().clamp(min=1)
        else:
            count = per_seq(keep)
            loss = (each / count.clamp(min=1)[seq]).sum() / (count > 0).sum().clamp(min=1)
        loss.backward()
        mean = lambda v: (v.detach() * keep).sum() / keep.sum().clamp(min=1)  # noqa: E731
        res = {"loss": loss.detach().reshape(1),
               "stats": torch.stack([mean(pg), mean(kl), mean(H), mean((near * A < ratio * A).double()), mean(ratio),
                                     keep.sum()]),
               "dlogp": lp.grad}
        if case["ent"] > 0:
            res["dentropy"] = H.grad
        return res
    lp = f64["logp"].requires_grad_(True)
    beta, G = 0.1, case["groups"]
    h = per_seq((lp - f64["ref"]) * keep)
    if case["average"]:
        h = h / per_seq(keep).clamp(min=1)
    # groups as rows of a padded table: column 0 preferred, the rest not
    first = st["goffsets"][:-1].long()
    size = st["goffsets"].long().diff()
    col = torch.arange(case["rejected"] + 1, device="cuda")
    there = col[None] < size[:, None]
    table = h[(first[:, None] + col[None]).clamp(max=lens.numel() - 1)]
    delta = table[:, :1] - table[:, 1:]
    there = there[:, 1:]
    if case["kind"] == "softmax":
        loss_pg = torch.logsumexp(torch.cat([torch.zeros(G, 1, device="cuda", dtype=torch.float64),
                                             torch.where(there, -beta * delta, -math.inf)], 1), 1)
    else:
        if case["kind"] == "sigmoid":
            e = case["smoothing"]
            each = -(1 - e) * torch.nn.functional.logsigmoid(beta * delta) - e * torch.nn.functional.logsigmoid(-beta * delta)
        elif case["kind"] == "ipo":
            each = (delta - 1 / (2 * beta)).square()
        else:
            each = torch.relu(1 - beta * delta)
        loss_pg = torch.where(there, each, 0.0).sum(1) / there.sum(1).clamp(min=1)
    loss = loss_pg.mean()
    loss.backward()
    return {"loss": loss.detach().reshape(1), "loss_pg": loss_pg.detach(), "rewards": beta * h.detach(), "dlogp": lp.grad}

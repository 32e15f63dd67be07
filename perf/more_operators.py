"""Cases of the operators of a sequence encoder and of 8-bit scoring, for timing and for comparison.

Four operators, each as a user's program calls it:
  attention   causal attention over packed sequences of different lengths, grouped heads, with a learned
              bias by buckets of the distance, and the gradients of all of them
  last        the same for the last token of every sequence, over a cache of keys and values
  norm        root-mean-square norm of a residual stream after the addition of a branch, with its gradients,
              or with the result in 8 bits and a scale for each row
  scores      scores of positions against items, both held in 8 bits with a scale for each row

`run` is the plain form (elementary torch operations in 32 bits, 64 for long sums and for values next to a
border) where `own` is false, and the framework's entry points where it is true.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one small batch of short histories, float32 throughout: latency counts
        dict(name="attention_train_16x12_f32", op="attention", n_seq=16, mean_len=12, heads=2, kv_heads=2, d=32,
             dtype="f32", buckets=32, train=True),
        # a SASRec batch: 256 histories of up to 200 or so items, two heads of 32
        dict(name="attention_train_256x150", op="attention", n_seq=256, mean_len=150, heads=2, kv_heads=2, d=32,
             dtype="bf16", buckets=32, train=True),
        # long histories, four query heads to a key head
        dict(name="attention_train_16x1021", op="attention", n_seq=16, mean_len=1021, heads=8, kv_heads=2, d=64,
             dtype="bf16", buckets=32, train=True),
        # whole prompts of a wide model, forward only, no bias
        dict(name="attention_fwd_3x2731_d128", op="attention", n_seq=3, mean_len=2731, heads=16, kv_heads=4, d=128,
             dtype="bf16", buckets=0, train=False),
        # serving: the next item of five users
        dict(name="last_5x200", op="last", n_seq=5, mean_len=200, heads=2, kv_heads=2, d=32, dtype="bf16", buckets=32),
        # one very long history: few rows, the work lies along the cache
        dict(name="last_1x65536_d128", op="last", n_seq=1, mean_len=65536, heads=8, kv_heads=2, d=128, dtype="bf16",
             buckets=0),
        # many users at once
        dict(name="last_2048x500", op="last", n_seq=2048, mean_len=500, heads=4, kv_heads=4, d=64, dtype="bf16",
             buckets=32),
        # a step of one small batch, in 8 bits for the product that follows
        dict(name="norm_int8_5x64", op="norm", n=5, d=64, dtype="bf16", int8=True, train=False),
        # the positions of a SASRec batch in training
        dict(name="norm_train_51200x256", op="norm", n=51200, d=256, dtype="bf16", int8=False, train=True),
        # a width that is no power of two, in 8 bits
        dict(name="norm_int8_16381x1000", op="norm", n=16381, d=1000, dtype="bf16", int8=True, train=False),
        # five users against a million items
        dict(name="scores_5x1m", op="scores", s=5, C=1_000_000, d=128, dtype="bf16"),
        # an evaluation batch against a large catalogue
        dict(name="scores_2047x100003", op="scores", s=2047, C=100_003, d=64, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "last", "norm", "scores"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("attention", "last"):
        kv = rng.choice([1, 2, 4])
        heads = kv * rng.choice([1, 1, 2, 4])
        d = rng.choice([32, 64, 128])
        n_seq = _log_int(rng, 1, 512)
        if op == "attention":
            mean = _log_int(rng, 1, 2048)
            # the plain form's scores, padded, stay below those of the largest listed case
            while n_seq * heads * (2 * mean) ** 2 > 1 << 28 or n_seq * mean > 40000:
                mean = mean * 3 // 4
            return dict(op=op, n_seq=n_seq, mean_len=mean, heads=heads, kv_heads=kv, d=d, dtype=dtype,
                        buckets=rng.choice([0, 16, 32]), train=rng.random() < 0.7)
        mean = _log_int(rng, 1, 65536)
        while n_seq * mean * kv * d > 1 << 27:
            mean = mean * 3 // 4
        return dict(op=op, n_seq=n_seq, mean_len=max(1, mean), heads=heads, kv_heads=kv, d=d, dtype=dtype,
                    buckets=rng.choice([0, 16, 32]))
    if op == "norm":
        d = 8 * _log_int(rng, 4, 512)
        n = max(1, min(_log_int(rng, 1, 51200), (1 << 24) // d))
        int8 = rng.random() < 0.5
        return dict(op=op, n=n, d=d, dtype=dtype, int8=int8, train=not int8 and rng.random() < 0.7)
    C, d = _log_int(rng, 100, 1_000_000), 16 * _log_int(rng, 2, 64)
    s = _log_int(rng, 1, 8192)
    while s * C > 1 << 27 or s * C * d > 1 << 35:
        s = s * 3 // 4
    while C * d > 1 << 28:
        d = d // 32 * 16
    return dict(op=op, s=max(1, s), C=C, d=d, dtype=dtype)


# ------------------------------------------------------------------ inputs
def bounds_of(buckets, most=128):
    """First distances of the buckets 1, 2, ...: one distance each in the lower half, by equal ratios up to `most`."""
    half = buckets // 2
    far = [math.ceil(half * (most / half) ** (k / half) - 1e-9) for k in range(1, half)]
    return list(range(1, half + 1)) + [max(b, half + 1 + k) for k, b in enumerate(far)]


def _offsets(g, n_seq, mean_len):
    """Ends of n_seq sequences with n_seq * mean_len tokens in all: lengths spread evenly from none to about twice the
    mean. On the host."""
    n = n_seq * mean_len
    ends = (torch.rand(n_seq, generator=g, dtype=torch.float64) + 1e-6).cumsum(0)
    offs = torch.zeros(n_seq + 1, dtype=torch.int64)
    offs[1:] = (ends / ends[-1] * n).round().long()
    return offs, n


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    st = {"case": case}
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    op = case["op"]
    if op in ("attention", "last"):
        hq, hk, d = case["heads"], case["kv_heads"], case["d"]
        offs, n = _offsets(torch.Generator().manual_seed(seed), case["n_seq"], case["mean_len"])
        st["max_len"] = int(offs.diff().max())
        st["offsets"] = offs.to(torch.int32).cuda()
        if case["buckets"]:
            bounds = bounds_of(case["buckets"])
            # a learned bias that falls with the distance
            slope = torch.linspace(1.0, -1.5, case["buckets"], device="cuda")
            st["bias"] = slope[:, None] + 0.3 * randn(case["buckets"], hq)
            st["bounds"], st["bounds_dev"] = bounds, torch.tensor(bounds, device="cuda")
        if op == "attention":
            # one projection gives all three; queries lean towards keys as a trained model's do
            x = (1.3 * randn(n, (hq + 2 * hk) * d)).to(dt)
            st["q"], st["k"], st["v"] = (x[:, a * d:b * d].view(n, b - a, d)
                                         for a, b in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
            if case["train"]:
                st["dout"] = (1e-3 * randn(n, hq, d)).to(dt)
        else:
            st["q"] = (1.3 * randn(case["n_seq"], hq, d)).to(dt)
            st["k"], st["v"] = ((1.3 * randn(n, hk, d)).to(dt) for _ in range(2))
            st["begin"], st["length"] = st["offsets"][:-1].clone(), st["offsets"].diff()
    elif op == "norm":
        n, d = case["n"], case["d"]
        st["x"] = randn(n, d).to(dt)
        # a residual stream whose rows differ in size, a few channels much larger than the rest
        wide = torch.where(torch.rand(d, generator=g, device="cuda") < 0.02, 12.0, 1.0)
        st["residual"] = (randn(n, d) * wide * (0.5 + 4.0 * torch.rand(n, 1, generator=g, device="cuda"))).to(dt)
        st["weight"] = 1.0 + 0.2 * randn(d)
        if case["train"]:
            st["dy"], st["dh"] = ((1e-3 * randn(n, d)).to(dt) for _ in range(2))
    else:
        s, C, d = case["s"], case["C"], case["d"]
        for name, rows in (("x", s), ("y", C)):
            v = randn(rows, d)
            m = v.abs().amax(1, keepdim=True)
            st[name + "8"] = (127.0 * v / m).round().to(torch.int8)
            st["s" + name] = m[:, 0] / 127.0
    if own:
        st["op"] = _handle(case, st)
    return st


def _handle(case, st):
    import catalogue_cross_entropy_amd as rece
    op = case["op"]
    if op == "attention":
        return rece.SequenceAttention(st["q"].shape[0], case["n_seq"], case["heads"], case["d"], kv_heads=case["kv_heads"],
                                      dtype=case["dtype"], bounds=st.get("bounds"))
    if op == "last":
        return rece.LastAttention(case["n_seq"], st["k"].shape[0], case["heads"], case["d"], st["max_len"],
                                  kv_heads=case["kv_heads"], dtype=case["dtype"], bounds=st.get("bounds"))
    if op == "norm":
        return rece.ResidualNorm(case["n"], case["d"], eps=1e-6, dtype=case["dtype"])
    return rece.Int8Scores(case["s"], case["C"], case["d"], dtype=case["dtype"])


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"attention": _attention, "last": _last, "norm": _norm, "scores": _scores}[op](state, case)
    h = state["op"]
    if op == "attention":
        q, k, v, offs, bias = state["q"], state["k"], state["v"], state["offsets"], state.get("bias")
        o, ws = h.forward(q, k, v, offs, bias=bias, need_grad=case["train"])
        out = {"out": o}
        if case["train"]:
            out["dq"], out["dk"], out["dv"], dbias = h.backward(q, k, v, offs, o, ws, state["dout"], bias=bias)
            if dbias is not None:
                out["dbias"] = dbias
        return out
    if op == "last":
        return {"out": h.forward(state["q"], state["k"], state["v"], state["begin"], state["length"],
                                 bias=state.get("bias"))}
    if op == "norm":
        if case["int8"]:
            y8, scale, s = h.forward_int8(state["x"], state["residual"], state["weight"])
            return {"y": y8 * scale[:, None], "h": s}
        y, s, rstd = h.forward(state["x"], state["residual"], state["weight"])
        out = {"y": y, "h": s}
        if case["train"]:
            out["dx"], out["dweight"] = h.backward(state["dy"], s, state["weight"], rstd, dh=state["dh"])
        return out
    return {"scores": h.forward(state["x8"], state["sx"], state["y8"], state["sy"])}


def _padded(offs, L):
    """[n_seq, L] index of every token in a padded batch, and where there is one."""
    at = offs[:-1].long()[:, None] + torch.arange(L, device=offs.device)
    there = at < offs[1:].long()[:, None]
    return torch.where(there, at, 0), there


def _bias_by_distance(st, L):
    """[L, heads]: the bias of every distance."""
    return st["bias"][torch.searchsorted(st["bounds_dev"], torch.arange(L, device="cuda"), right=True)]


def _attention(st, case):
    hq, hk, d, L, dt = case["heads"], case["kv_heads"], case["d"], st["max_len"], st["q"].dtype
    n, scale = st["q"].shape[0], 1.0 / math.sqrt(d)
    at, there = _padded(st["offsets"], L)
    of = torch.arange(hq, device="cuda") // (hq // hk)      # the key head of a query head
    q = st["q"][at].float().transpose(1, 2)                 # [n_seq, heads, L, d]
    k = st["k"][at].float().transpose(1, 2)[:, of]
    v = st["v"][at].float().transpose(1, 2)[:, of]
    pos = torch.arange(L, device="cuda")
    dist = pos[:, None] - pos
    S = torch.matmul(q, k.transpose(2, 3)) * scale
    if case["buckets"]:
        S += _bias_by_distance(st, L)[dist.clamp(min=0)].permute(2, 0, 1)
    S.masked_fill_(dist < 0, -math.inf)
    P = (S - S.amax(3, keepdim=True)).exp_()
    P /= P.sum(3, keepdim=True)
    o = torch.matmul(P, v)
    out = {"out": st["q"].new_zeros(n, hq, d)}
    out["out"][at[there]] = o.transpose(1, 2)[there].to(dt)
    if not case["train"]:
        return out
    do = torch.where(there[:, None, :, None], st["dout"][at].float().transpose(1, 2), 0.0)
    dP = torch.matmul(do, v.transpose(2, 3))
    dS = P * (dP - (P * dP).sum(3, keepdim=True))
    group = lambda t: t.unflatten(1, (hk, hq // hk)).sum(2)  # noqa: E731
    grads = {"dq": torch.matmul(dS, k) * scale, "dk": group(torch.matmul(dS.transpose(2, 3), q)) * scale,
             "dv": group(torch.matmul(P.transpose(2, 3), do))}
    for name, t in grads.items():
        out[name] = st["q"].new_zeros(n, t.shape[1], d)
        out[name][at[there]] = t.transpose(1, 2)[there].to(dt)
    if case["buckets"]:
        # rows shifted so that a column holds one distance, and summed
        T = torch.cat([dS.sum(0).flip(2), dS.new_zeros(hq, L, L)], 2).reshape(hq, 2 * L * L)
        by_dist = T[:, :L * (2 * L - 1)].reshape(hq, L, 2 * L - 1).sum(1, dtype=torch.float64)[:, L - 1:]
        bucket = torch.searchsorted(st["bounds_dev"], pos, right=True)
        chosen = (bucket[:, None] == torch.arange(case["buckets"], device="cuda")).double()
        out["dbias"] = torch.matmul(by_dist, chosen).t().float().contiguous()
    return out


def _last(st, case):
    hq, hk, d, L = case["heads"], case["kv_heads"], case["d"], st["max_len"]
    at = st["begin"].long()[:, None] + torch.arange(L, device="cuda")
    back = st["length"].long()[:, None] - 1 - torch.arange(L, device="cuda")   # distance to the last token
    there = back >= 0
    at = torch.where(there, at, 0)
    q = st["q"].float().unflatten(1, (hk, hq // hk))
    k = st["k"][at].float().transpose(1, 2)
    v = st["v"][at].float().transpose(1, 2)
    S = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    if case["buckets"]:
        S += _bias_by_distance(st, L)[back.clamp(min=0)].permute(0, 2, 1).unflatten(1, (hk, hq // hk))
    S = torch.where(there[:, None, None], S, -math.inf)
    e = (S - S.amax(3, keepdim=True).clamp(min=-1e30)).exp()
    o = torch.matmul(e, v) / e.sum(3, keepdim=True).clamp(min=1e-30)
    return {"out": o.flatten(1, 2).to(st["q"].dtype)}


def _norm(st, case):
    dt, w = st["x"].dtype, st["weight"]
    h = (st["x"].float() + st["residual"].float()).to(dt)
    hf = h.float()
    rstd = 1.0 / (hf.square().mean(1, keepdim=True) + 1e-6).sqrt()
    if case["int8"]:
        t = hf.double() * w.double()
        m = t.abs().amax(1, keepdim=True)
        y8 = (127.0 * t / torch.where(m > 0, m, 1.0)).round()      # in 64 bits: values next to a half
        return {"y": y8.float() * (m.float() * rstd / 127.0), "h": h}
    out = {"y": (hf * rstd * w).to(dt), "h": h}
    if case["train"]:
        dy = st["dy"].float()
        g = dy * w
        c = (g * hf).mean(1, keepdim=True) * rstd.square()
        out["dx"] = (st["dh"].float() + rstd * (g - hf * c)).to(dt)
        out["dweight"] = (dy * hf * rstd).sum(0, dtype=torch.float64).float()
    return out


def _scores(st, case):
    acc = torch.matmul(st["x8"].float(), st["y8"].float().t())
    return {"scores": (acc * st["sx"][:, None] * st["sy"]).to(_DT[case["dtype"]])}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("attention", "last"):
        hq, hk, d, n_seq, mean = case["heads"], case["kv_heads"], case["d"], case["n_seq"], case["mean_len"]
        n = n_seq * mean
        table = 4 * case["buckets"] * hq
        if op == "last":
            return {"bytes": 2 * n * hk * d * es + 2 * n_seq * hq * d * es + 8 * n_seq + table, "flops": 4 * n * hq * d}
        # lengths spread evenly: the mean of their squares is 4/3 of the mean's
        pairs = hq * n * (mean * (4 / 3 if n_seq > 1 else 1) + 1) / 2
        b, f = n * d * es * (2 * hq + 2 * hk) + 4 * n_seq + table, 4 * d * pairs
        if case["train"]:
            b, f = b + n * d * es * (2 * hq + 2 * hk) + table, f + 10 * d * pairs
        return {"bytes": int(b), "flops": int(f)}
    if op == "norm":
        n, d = case["n"], case["d"]
        if case["int8"]:
            return {"bytes": 3 * n * d * es + n * d + 4 * n + 4 * d, "flops": 8 * n * d}
        b, f = 4 * n * d * es + 4 * d, 6 * n * d
        if case["train"]:
            b, f = b + 3 * n * d * es + 4 * d, f + 12 * n * d
        return {"bytes": b, "flops": f}
    s, C, d = case["s"], case["C"], case["d"]
    return {"bytes": (s + C) * (d + 4) + s * C * es, "flops": 2 * s * C * d}


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("attention", "last"):
        hq, hk, d = case["heads"], case["kv_heads"], case["d"]
        offs = st["offsets"].tolist()
        grad = case.get("train", False)
        q, k, v = (st[x].double().requires_grad_(grad) for x in ("q", "k", "v"))
        bias = st["bias"].double().requires_grad_(grad) if case["buckets"] else None
        rows = []
        for u, (a, b) in enumerate(zip(offs[:-1], offs[1:])):
            if a == b:
                if op == "last":
                    rows.append(torch.zeros(1, hq, d, device="cuda", dtype=torch.float64))
                continue
            mine = q[a:b] if op == "attention" else q[u:u + 1]
            i = torch.arange(b - a, device="cuda")[-mine.shape[0]:]
            t = i[:, None] - torch.arange(b - a, device="cuda")
            heads = []
            for j in range(hq):
                s = mine[:, j] @ k[a:b, j * hk // hq].T / d ** 0.5
                if bias is not None:
                    s = s + bias[:, j][sum((t >= x).long() for x in st["bounds"])]
                heads.append(torch.softmax(s.masked_fill(t < 0, -math.inf), 1) @ v[a:b, j * hk // hq])
            o = torch.stack(heads, 1)
            rows.append(o.detach())
            if grad:
                (o * st["dout"][a:b].double()).sum().backward()
        res = {"out": torch.cat(rows)}
        if grad:
            res.update(dq=q.grad, dk=k.grad, dv=v.grad)
            if bias is not None:
                res["dbias"] = bias.grad
        return res
    if op == "norm":
        # the sum as it is stored is what everything after it reads
        h = (st["x"].double() + st["residual"].double()).to(st["x"].dtype).double().requires_grad_(True)
        w = st["weight"].double().requires_grad_(True)
        y = h / torch.linalg.vector_norm(h, dim=1, keepdim=True).square().div(case["d"]).add(1e-6).sqrt() * w
        res = {"h": h.detach()}
        if case["int8"]:
            top = (h * w).abs().amax(1, keepdim=True).detach()
            step = torch.round(127.0 * (h * w).detach() / top.clamp(min=1e-300))
            res["y"] = step * y.detach().abs().amax(1, keepdim=True) / 127
            return res
        res["y"] = y.detach()
        if case["train"]:
            ((y * st["dy"].double()).sum() + (h * st["dh"].double()).sum()).backward()
            res.update(dx=h.grad, dweight=w.grad)
        return res
    scaled = {x: st[x + "8"].double() * st["s" + x].double()[:, None] for x in ("x", "y")}
    return {"scores": scaled["x"] @ scaled["y"].T}

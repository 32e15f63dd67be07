"""The encoder's operators in a run, as a next-item model uses them: items embedded, blocks of normed attention over packed
histories, log-probabilities over the catalogue, and back; then serving: the last tokens over the same cache, and the
catalogue scored in 8 bits."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece
from encoder_reference import buckets

pytestmark = pytest.mark.gpu

LENS, C, HQ, HK, D = [5, 1, 0, 37, 90], 300, 4, 2, 16
W, N = HQ * D, sum(LENS)


def parameters(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return {"table": r(C, W) * W ** -0.5, "w1": 1 + 0.2 * r(W), "w2": 1 + 0.2 * r(W), "qkv": r(W, (HQ + 2 * HK) * D) * W ** -0.5,
            "proj": r(W, W) * W ** -0.5, "bias": 0.5 * r(16, HQ)}


def batch(seed=0):
    g = torch.Generator().manual_seed(seed + 1)
    ids = torch.randint(0, C, (N,), generator=g)
    ids[7] = -1
    return ids, torch.randint(0, C, (N,), generator=g)


def plain(p, ids, target, bounds, eps=1e-6):
    """Everything in float64 with elementary operations; returns the log-probabilities."""
    norm = lambda h, w: h * (h.square().mean(1, keepdim=True) + eps).rsqrt() * w  # noqa: E731
    e = torch.where((ids >= 0)[:, None], p["table"][ids.clamp(min=0)] * W ** 0.5, 0.0)
    x = norm(e, p["w1"]) @ p["qkv"]
    q, k, v = x[:, :W].view(N, HQ, D), x[:, W:W + HK * D].view(N, HK, D), x[:, W + HK * D:].view(N, HK, D)
    rows, at = [], 0
    for n in LENS:
        t = torch.arange(n)[:, None] - torch.arange(n)
        o = []
        for h in range(HQ):
            s = q[at:at + n, h] @ k[at:at + n, h // (HQ // HK)].T * D ** -0.5 + p["bias"][:, h][buckets(t, bounds)]
            o.append(torch.softmax(s.masked_fill(t < 0, -torch.inf), 1) @ v[at:at + n, h // (HQ // HK)] if n else s[:, :0])
        rows.append(torch.cat(o, 1) if n else torch.zeros(0, W, dtype=torch.float64))
        at += n
    h2 = torch.cat(rows) @ p["proj"] + e
    y = norm(h2, p["w2"])
    return torch.log_softmax(y @ p["table"].T, 1)[torch.arange(N), target]


def ours(p, ids, target, offs, ops, dtype):
    embed, norm, att, lp = ops
    to = lambda t: t.to(dtype)  # noqa: E731
    e = rece.embed(p["table"], ids, embed)
    y, _ = rece.residual_norm(e, None, p["w1"], norm)
    a = rece.attention_qkv(y @ to(p["qkv"]), offs, att, bias=p["bias"])
    y2, _ = rece.residual_norm(a.reshape(N, W) @ to(p["proj"]), e, p["w2"], norm)
    return rece.log_probs(y2, p["table"], target, lp)


def operators(name):
    return (rece.ItemEmbedding(N, C, W, dtype=name, scale=W ** 0.5), rece.ResidualNorm(N, W, dtype=name),
            rece.SequenceAttention(N, len(LENS), HQ, D, kv_heads=HK, dtype=name, bounds=rece.log_buckets(16, 60)),
            rece.LogProb(N, C, W, dtype=name))


@pytest.mark.parametrize("name,tol", [("f32", 2e-5), ("bf16", 6e-2)])
def test_block_and_its_gradients(name, tol):
    """float32: a dozen sums of up to 300 terms in a row, each off by some 1e-7 of its terms.  bf16: ten roundings in a row
    forward and as many back, each by up to 2^-8."""
    dtype = torch.float32 if name == "f32" else torch.bfloat16
    p = parameters()
    # the table is the input of two operators in its own type; what the float64 form takes is what they read
    for k in ("table", "qkv", "proj"):
        p[k] = p[k].to(dtype).double()
    ids, target = batch()
    ref = {k: v.clone().requires_grad_(True) for k, v in p.items()}
    want = plain(ref, ids, target, rece.log_buckets(16, 60))
    want.sum().backward()
    ops = operators(name)
    dev = {k: v.to(dtype if k in ("table", "qkv", "proj") else torch.float32).cuda().requires_grad_(True) for k, v in p.items()}
    offs = torch.tensor([0] + LENS).cumsum(0).to(torch.int32).cuda()
    got = ours(dev, ids.to(torch.int32).cuda(), target.to(torch.int32).cuda(), offs, ops, dtype)
    got.sum().backward()
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert rel(got.detach(), want.detach()) < tol
    for k in p:
        off = rel(dev[k].grad, ref[k].grad)
        print(f"  {k}: {off:.2e}")
        assert off < tol, k
    with torch.no_grad():
        again = ours(dev, ids.to(torch.int32).cuda(), target.to(torch.int32).cuda(), offs, ops, dtype)
    assert torch.equal(again, got)


def test_gradients_against_differences():
    """Differences of the float64 form along a direction against the kernels' gradient along it."""
    p = parameters(3)
    for k in ("table", "qkv", "proj"):
        p[k] = p[k].float().double()
    ids, target = batch(3)
    ops = operators("f32")
    dev = {k: v.float().cuda().requires_grad_(True) for k, v in p.items()}
    offs = torch.tensor([0] + LENS).cumsum(0).to(torch.int32).cuda()
    ours(dev, ids.to(torch.int32).cuda(), target.to(torch.int32).cuda(), offs, ops, torch.float32).sum().backward()
    g = torch.Generator().manual_seed(9)
    for k in p:
        v = torch.randn(p[k].shape, generator=g, dtype=torch.float64)
        step = 1e-6
        sides = [float(plain({**p, k: p[k] + s * step * v}, ids, target, rece.log_buckets(16, 60)).sum()) for s in (1, -1)]
        slope = float((dev[k].grad.double().cpu() * v).sum())
        scale = float(dev[k].grad.norm()) * float(v.norm())
        assert abs(slope - (sides[0] - sides[1]) / (2 * step)) < 1e-4 * scale / v.numel() ** 0.5 + 1e-6 * abs(slope), k


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_last_tokens_agree_with_whole_histories(name):
    dtype = torch.float32 if name == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(4)
    q, k, v = ((torch.randn(N, h, D, generator=g)).to(dtype).cuda() for h in (HQ, HK, HK))
    offs = torch.tensor([0] + LENS).cumsum(0).to(torch.int32).cuda()
    bias = torch.randn(16, HQ, generator=g).cuda()
    bounds = rece.log_buckets(16, 60)
    whole, _ = rece.SequenceAttention(N, len(LENS), HQ, D, kv_heads=HK, dtype=name, bounds=bounds).forward(
        q, k, v, offs, bias=bias, need_grad=False)
    length = offs.diff()
    last = (offs[1:] - 1).long().clamp(min=0)
    out = rece.LastAttention(len(LENS), N, HQ, D, max(LENS), kv_heads=HK, dtype=name, bounds=bounds).forward(
        q[last].contiguous(), k, v, offs[:-1].contiguous(), length, bias=bias)
    there = length > 0
    # two orders of the same sums, each rounded (bf16: p as well, to 2^-8 of it, and the result)
    tol = 1e-5 if name == "f32" else 4 * 2.0 ** -8 * float(v.abs().max())
    assert (out[there].float() - whole[last][there].float()).abs().max() < tol
    assert (out[~there] == 0).all()


def test_catalogue_scored_in_8_bits():
    """Norm with 8-bit rows into scores against a table laid out once: the integer product of what was stored, and near
    the scores in float32."""
    g = torch.Generator().manual_seed(5)
    h, r = (torch.randn(37, W, generator=g).bfloat16().cuda() for _ in range(2))
    w = (1 + 0.2 * torch.randn(W, generator=g)).cuda()
    table = torch.randn(5003, W, generator=g).bfloat16().cuda()
    y8, sy = rece.quantize_rows(table)
    norm = rece.ResidualNorm(37, W)
    x8, sx, s = norm.forward_int8(h, r, w)
    scores = rece.Int8Scores(37, 5003, W, dtype="f32").forward(x8, sx, y8, sy)
    want = (x8.cpu().double() @ y8.cpu().double().T) * sx.cpu().double()[:, None] * sy.cpu().double()
    assert ((scores.cpu().double() - want).abs() <= 3 * 2.0 ** -24 * want.abs()).all()
    y, _, _ = norm.forward(h, r, w)
    full = y.float() @ table.float().T
    # both sides rounded to half a step of 1/127 of a row's largest: independent errors of W products
    step = (sx[:, None] * table.float().norm(dim=1) + y.float().norm(dim=1, keepdim=True) * sy) / 12 ** 0.5
    assert ((scores - full).abs() < 8 * step + 0.02 * full.abs()).all()


def test_separate_tensors_through_autograd():
    """Gradients of some inputs only, through gradients that are slices of others', a second pass adding up."""
    g = torch.Generator().manual_seed(6)
    op = rece.SequenceAttention(N, len(LENS), HQ, D, kv_heads=HK, dtype="f32", bounds=rece.log_buckets(16, 60))
    offs = torch.tensor([0] + LENS).cumsum(0).to(torch.int32).cuda()
    q, k, v = (torch.randn(N, h, D, generator=g).cuda() for h in (HQ, HK, HK))
    bias = torch.randn(16, HQ, generator=g).cuda()
    weight = torch.randn(N, HQ, 3 * D, generator=g).cuda()
    out, ws = op.forward(q, k, v, offs, bias=bias)
    want = op.backward(q, k, v, offs, out, ws, weight[..., D:2 * D].contiguous(), bias=bias)
    for chosen in ((0,), (1, 3), (2,), (3,), (0, 1, 2, 3)):
        t = [x.clone().requires_grad_(i in chosen) for i, x in enumerate((q, k, v, bias))]
        for passes in (1, 2):
            o = rece.attention(*t[:3], offs, op, bias=t[3])
            # the gradient of a concatenation reaches the call as a slice
            (torch.cat([torch.zeros_like(o), o, torch.zeros_like(o)], 2) * weight).sum().backward()
            for i, x in enumerate(t):
                assert (x.grad is None) == (i not in chosen)
                if i in chosen:
                    assert torch.equal(x.grad, passes * want[i])


@pytest.mark.parametrize("use", ["y", "h", "both"])
def test_norm_through_autograd(use):
    g = torch.Generator().manual_seed(7)
    x, r, cy, ch = (torch.randn(20, 72, generator=g, dtype=torch.float64) for _ in range(4))
    w = 1 + 0.2 * torch.randn(72, generator=g, dtype=torch.float64)
    ref = [t.float().double().requires_grad_(True) for t in (x, r, w)]
    h = ref[0] + ref[1]
    y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * ref[2]
    loss = (y * cy.float().double()).sum() * (use != "h") + (h * ch.float().double()).sum() * (use != "y")
    loss.backward()
    dev = [t.float().cuda().requires_grad_(True) for t in (x, r, w)]
    y, h = rece.residual_norm(*dev, rece.ResidualNorm(20, 72, dtype="f32"))
    loss = (y * cy.float().cuda()).sum() if use == "y" else (h * ch.float().cuda()).sum() if use == "h" else \
        (y * cy.float().cuda()).sum() + (h * ch.float().cuda()).sum()
    loss.backward()
    for a, b in zip(dev, ref):
        if use == "h" and a is dev[2]:
            assert a.grad is None
        else:
            assert (a.grad.double().cpu() - b.grad).abs().max() < 1e-5 * max(1.0, float(b.grad.abs().max()))

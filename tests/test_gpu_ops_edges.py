"""The operators where their paths meet: sizes on either side of every change of kernel, arrays that begin at any
element, two calls at once, a graph's second backward pass."""
import numpy as np
import pytest
import torch

import catalogue_cross_entropy_amd as rece
import ops_reference as R
import test_gpu_embed as TE
import test_gpu_logprob as TL
import test_gpu_policy as TP

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# the sort: one workgroup, then 1, 2 and 4 records per thread, then the longer sort
@pytest.mark.parametrize("n", [4096, 4097, 65536, 65537, 131072, 131073, 262144, 262145])
def test_embed_gradient_at_the_sorts_sizes(n):
    C, d = 5003, 32
    table, ids, dout = TE._case(n, C, d, "bf16", "heavy", seed=n)
    ids[::7] = -1
    print(f"[gpu] embed gradient n={n}", flush=True)
    op = rece.ItemEmbedding(n, C, d, dtype="bf16", scale=1.5)
    grad, bound = R.embed_grad(ids, dout, C, 1.5)
    got = op.backward(ids.cuda(), dout.cuda())
    assert bool(((got.cpu().double() - grad).abs() <= bound).all())
    assert torch.equal(op.backward(ids.cuda(), dout.cuda()), got)


def _against_plain(s, C, d, dtype, entropy, pad, bf16_grads=False):
    X, Y, ids, dlogp, dent, bad = TL._case(s, C, d, dtype, seed=s + C + d, pad=pad, peak=1.0)
    if not entropy:
        dent = None
    print(f"[gpu] logprob s={s} C={C} d={d} {dtype} entropy={entropy}", flush=True)
    logp, ent, dX, dY = TL._run(X, Y, ids, dlogp, dent, 0.9, entropy, bf16_grads)
    w = R.logprob(X, Y, ids, 0.9, dlogp, dent)
    assert bool(((logp.double() - w["logp"]).abs() <= w["e_logp"]).all())
    if entropy:
        assert bool(((ent.double() - w["entropy"]).abs() <= w["e_entropy"]).all())
    u = R.U[torch.bfloat16] if bf16_grads else R.U32
    for name, got in (("dX", dX), ("dY", dY)):
        bound = w["p_" + name] + (w["b_" + name] if bf16_grads else 0.0)
        bound = bound + u * (w[name].abs() + bound) + 1e-30
        assert bool(((got.double() - w[name]).abs() <= bound).all()), name


@pytest.mark.parametrize("s,C,d,dtype,entropy,pad", [
    # joins by a workgroup, a wave, a thread per position
    (256, 300, 32, "bf16", True, 0.1), (257, 300, 32, "f32", False, 0.1),
    (8192, 90, 32, "bf16", True, 0.1), (8193, 90, 32, "bf16", False, 0.1), (8193, 90, 32, "f32", True, 0.0),
    # the waves of a workgroup share 32 or 64 positions, and the size after
    (32, 9000, 64, "f32", False, 0.0), (33, 9000, 64, "f32", True, 0.0), (64, 9000, 64, "bf16", False, 0.2),
    (65, 9000, 64, "bf16", True, 0.0), (32, 9000, 128, "bf16", False, 0.0), (33, 9000, 128, "bf16", True, 0.0),
    # as many blocks of items as workgroups, and one more
    (70, 131072, 32, "bf16", False, 0.3), (70, 131073, 32, "bf16", True, 0.3),
    # ids of one packing step and one more
    (64, 65, 32, "bf16", False, 0.5), (65, 65, 32, "bf16", False, 0.5),
])
def test_logprob_at_the_changes_of_kernel(s, C, d, dtype, entropy, pad):
    _against_plain(s, C, d, dtype, entropy, pad)


@pytest.mark.parametrize("lead", [1, 2, 3])
def test_logprob_ids_at_any_element(lead):
    s, C, d = 600, 500, 64
    X, Y, ids, dlogp, _, _ = TL._case(s, C, d, "bf16", seed=lead, pad=0.3, peak=1.0)
    long = torch.cat([torch.full((lead,), 3, dtype=torch.int32), ids]).cuda()
    op = rece.LogProb(s, C, d, dtype="bf16")
    X, Y = X.cuda(), Y.cuda()
    a, _, wa = op.forward(X, Y, long[lead:])
    b, _, wb = op.forward(X, Y, ids.cuda())
    assert torch.equal(a, b)
    for x, y in zip(op.backward(X, Y, long[lead:], wa, dlogp.cuda()), op.backward(X, Y, ids.cuda(), wb, dlogp.cuda())):
        assert torch.equal(x, y)


def test_logprob_second_backward_of_one_forward():
    """The gradients of one forward pass may be taken again (another dlogp, the same bits for the same one)."""
    for entropy in (False, True):
        s, C, d = 300, 700, 64
        X, Y, ids, dlogp, dent, _ = TL._case(s, C, d, "bf16", seed=8, pad=0.1, peak=1.0)
        op = rece.LogProb(s, C, d, dtype="bf16", entropy=entropy)
        X, Y, ids, dlogp = X.cuda(), Y.cuda(), ids.cuda(), dlogp.cuda()
        dent = dent.cuda() if entropy else None
        _, _, ws = op.forward(X, Y, ids)
        first = op.backward(X, Y, ids, ws, dlogp, dentropy=dent)
        op.backward(X, Y, ids, ws, -3.0 * dlogp, dentropy=dent)
        for a, b in zip(first, op.backward(X, Y, ids, ws, dlogp, dentropy=dent)):
            assert torch.equal(a, b)
    X, Y = X.requires_grad_(), Y.requires_grad_()
    logp, ent = rece.log_probs(X, Y, ids, op)
    loss = (logp * dlogp).sum() + (ent * dent).sum()
    gx, gy = torch.autograd.grad(loss, (X, Y), retain_graph=True)
    hx, hy = torch.autograd.grad(loss, (X, Y))
    assert torch.equal(gx, hx) and torch.equal(gy, hy)


@pytest.mark.parametrize("reduction,token", [("token", False), ("sequence", False), ("sequence", True), ("token", True)])
def test_policy_more_sequences_in_a_tile_than_lds_holds(reduction, token):
    TP.test_policy_against_plain(20000, 15000, "f32", 0.05, 0.02, token, reduction, True, 3, 5)


@pytest.mark.parametrize("n_seq", [1, 3000])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_policy_no_tokens(n_seq, reduction):
    op = rece.PolicyLoss(0, n_seq, reduction=reduction)
    none = torch.empty(0, device="cuda")
    loss, stats, dlp, _ = op.forward(none, none, torch.ones(n_seq, device="cuda"),
                                     torch.zeros(n_seq + 1, dtype=torch.int32, device="cuda"))
    assert float(loss) == 0.0 and stats.tolist() == [0.0] * 6 and dlp.numel() == 0


def test_policy_extreme_ratios():
    """e^(logp - old) of 0, infinity and everything between; NaN stays NaN.  The policy term of one token, against
    the formula in float64: an exact difference, an exponential (its instruction's last place, two roundings), the
    weight's division, three products."""
    inf = float("inf")
    diff = torch.tensor([0.0, -inf, 1e-7, -1e-7, 0.3, -0.3, 5.0, -5.0, 60.0, -60.0, 80.0, -85.0, 100.0, -200.0])
    n = diff.numel()
    for A in (1.0, -1.0):
        for small in (True, False):
            reps = 1 if small else 1000
            lp = diff.repeat(reps)
            N = lp.numel()
            op = rece.PolicyLoss(N, N, clip_low=0.2, clip_high=1e30)
            args = (torch.zeros(N).cuda(), torch.full((N,), A).cuda(), torch.arange(N + 1, dtype=torch.int32).cuda())
            _, _, dlp, _ = op.forward(lp.cuda(), *args)
            r = lp.double().exp()
            clipped = (r < 0.8) if A < 0 else (r > 1e30)
            want = torch.where(clipped, 0.0, -A * r / N)
            got = dlp.cpu().double()
            fine = (r < 3e38) & (r > 1e-36)
            err = (got - want).abs()
            rel = 9 * R.U32   # whatever the exponent's size: its rounding is corrected for
            assert bool((err <= rel * want.abs())[fine].all()), (A, small)
            assert bool((got.isinf() | (want == 0) | (want.abs() * N < 3.5e38))[r >= 3.5e38].all())
            assert bool((got.abs() <= 1e-35)[r <= 1e-36].all())
    lp = torch.zeros(9000)
    lp[77] = float("nan")
    op = rece.PolicyLoss(9000, 1)
    loss, _, dlp, _ = op.forward(lp.cuda(), torch.zeros(9000).cuda(), torch.ones(1).cuda(),
                                 torch.tensor([0, 9000], dtype=torch.int32).cuda())
    assert np.isnan(float(loss)) and bool(dlp[77].isnan()) and not bool(dlp[:77].isnan().any())


@pytest.mark.parametrize("n", [4000, 40000])
def test_policy_clips_on_the_right_side_of_its_bounds(n):
    """Differences a few steps around log(0.8) and log(1.2): clipped exactly where the float64 ratio is beyond the
    (float32) bounds.  old is 0, so the differences are the values themselves."""
    low, high = float(np.float32(0.2)), float(np.float32(0.2))
    half = n // 2
    at = np.concatenate([np.full(half, np.log1p(-low), np.float32), np.full(n - half, np.log1p(high), np.float32)])
    bits = at.view(np.int32) + np.random.default_rng(0).integers(-6, 7, n, dtype=np.int32)
    lp = torch.from_numpy(bits.view(np.float32).copy())
    A = torch.cat([torch.full((half,), -1.0), torch.ones(n - half)])
    r = lp.double().exp()
    clipped = torch.where(A > 0, r > 1 + high, r < 1 - low)
    assert 0.3 * n < int(clipped.sum()) < 0.7 * n
    op = rece.PolicyLoss(n, 1, clip_low=0.2, clip_high=0.2, token_advantage=True)
    _, stats, dlp, _ = op.forward(lp.cuda(), torch.zeros(n).cuda(), A.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda())
    assert torch.equal(dlp.cpu() == 0, clipped)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,n_seq,G", [(40000, 150, 50), (6000, 600, 20), (2400, 600, 200), (900, 900, 300)])
def test_preference_views_at_odd_addresses(n, n_seq, G, dtype):
    """Token arrays that begin at any element give what copies of them give, but for the order of the float64 sums."""
    g = torch.Generator().manual_seed(n)
    lp, ref, _ = (t.cuda() for t in TP._tokens(g, n + 3, dtype))
    mask = (torch.rand(n + 3, generator=g) < 0.6).to(torch.uint8).cuda()
    offs = TP._offsets(g, n_seq, n).cuda()
    goffs = (torch.arange(G + 1) * (n_seq // G)).to(torch.int32).cuda()
    op = rece.PreferenceLoss(n, n_seq, G, kind="softmax", dtype=dtype, average=True)
    a = op.forward(lp[3:], ref[3:], offs, goffs, mask=mask[3:])
    b = op.forward(lp[3:].clone(), ref[3:].clone(), offs, goffs, mask=mask[3:].clone())
    for x, y, u in zip(a, b, (R.U32, R.U32, R.U32, R.U[DT[dtype]])):
        # equal in float64 to far below a step: at most one step apart after the rounding
        assert bool(((x.double() - y.double()).abs() <= 2.01 * u * y.double().abs() + 1e-30).all())


def test_two_calls_at_once():
    """One operator object on two streams at once, each call with its own workspace, gives the bits of calls one after
    the other."""
    s, C, d, n, n_seq = 900, 5000, 64, 30000, 400
    g = torch.Generator().manual_seed(21)
    lpop = rece.LogProb(s, C, d, dtype="bf16")
    emb = rece.ItemEmbedding(9000, C, d, dtype="bf16")
    pol = rece.PolicyLoss(n, n_seq, kl_coef=0.1, reduction="sequence")
    pref = rece.PreferenceLoss(n, n_seq, 100, kind="softmax")
    goffs = (torch.arange(101) * 4).to(torch.int32).cuda()
    sets = []
    for q in range(2):
        X, Y, ids, dlogp, _, _ = TL._case(s, C, d, "bf16", seed=q, pad=0.2, peak=1.0)
        _, eids, dout = TE._case(9000, C, d, "bf16", "heavy", seed=q)
        lp, old, ref = (t.cuda() for t in TP._tokens(g, n, "f32"))
        sets.append(dict(X=X.cuda(), Y=Y.cuda(), ids=ids.cuda(), dlogp=dlogp.cuda(), eids=eids.cuda(), dout=dout.cuda(), lp=lp,
                         old=old, ref=ref, offs=TP._offsets(g, n_seq, n).cuda(), adv=torch.randn(n_seq, generator=g).cuda()))

    def run(t):
        logp, _, ws = lpop.forward(t["X"], t["Y"], t["ids"])
        grads = lpop.backward(t["X"], t["Y"], t["ids"], ws, t["dlogp"])
        return (logp,) + tuple(grads) + (emb.backward(t["eids"], t["dout"]),) + \
            pol.forward(t["lp"], t["old"], t["adv"], t["offs"], ref_logp=t["ref"])[:3] + \
            pref.forward(t["lp"], t["ref"], t["offs"], goffs)

    want = [run(t) for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for t, st in zip(sets, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(run(t))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_embed_gradient_of_many_rows():
    """More rows than a launch has threads for at 32 a piece of 8: gradients of ones are counts, exact in float32."""
    n, C, d = (1 << 27) + 4099, 1000, 8
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(-1, C, (n,), generator=g, device="cuda", dtype=torch.int32)
    op = rece.ItemEmbedding(n, C, d, dtype="bf16")
    got = op.backward(ids, torch.ones(n, d, dtype=torch.bfloat16, device="cuda"))
    want = torch.bincount(ids.clamp(min=-1).long() + 1, minlength=C + 1)[1:].float()
    assert torch.equal(got, want[:, None].expand(C, d).contiguous())


@pytest.mark.parametrize("G,K,n,dtype,kind,smoothing,average,masked,margin,with_ref", [
    (8193, 1, 30000, "f32", "sigmoid", 0.1, False, True, 0.2, True), (8200, 3, 50000, "bf16", "softmax", 0.0, False, True, 0.0, True),
    (8193, 3, 190000, "f32", "softmax", 0.0, True, True, 0.3, True), (8193, 1, 200000, "bf16", "ipo", 0.0, True, False, 0.0, True),
    (9000, 1, 20000, "f32", "hinge", 0.0, False, False, 0.1, False), (2048, 1, 5000, "bf16", "sigmoid", 0.0, False, True, 0.0, True),
    (2047, 1, 5000, "bf16", "sigmoid", 0.0, False, True, 0.0, True),
])
def test_preference_many_small_groups(G, K, n, dtype, kind, smoothing, average, masked, margin, with_ref):
    TP.test_preference_against_plain(G, K, n, dtype, kind, smoothing, average, masked, margin, with_ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("per", [1, 9])
def test_preference_groups_are_the_same_in_a_large_call(per, kind, dtype):
    """The first groups of 12,000 give what a call of a few gives: rewards and losses to a step, gradients (times the
    ratio of the numbers of groups) too."""
    big, few, K = 12000, 30, 2
    g = torch.Generator().manual_seed(per)
    lp, ref, _ = (t.cuda() for t in TP._tokens(g, big * K * per, dtype))
    offs = (torch.arange(big * K + 1) * per).to(torch.int32).cuda()
    goffs = (torch.arange(big + 1) * K).to(torch.int32).cuda()
    n = few * K * per
    a = rece.PreferenceLoss(big * K * per, big * K, big, kind=kind, dtype=dtype).forward(lp, ref, offs, goffs)
    b = rece.PreferenceLoss(n, few * K, few, kind=kind, dtype=dtype).forward(
        lp[:n].clone(), ref[:n].clone(), offs[:few * K + 1].clone(), goffs[:few + 1].clone())
    for x, y in ((a[1][:few], b[1]), (a[2][:few * K], b[2])):
        assert bool(((x.double() - y.double()).abs() <= 2.01 * R.U32 * y.double().abs()).all())
    u = R.U[DT[dtype]]
    x, y = a[3][:n].double() * (big / few), b[3].double()
    assert bool(((x - y).abs() <= 2.1 * u * y.abs()).all())

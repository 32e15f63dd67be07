"""Calls of the operators that their documentation allows: the smallest tables, streams given explicitly, results
changed in place, gradients that arrive at any address, scoring without gradients."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 4096, 4097, 70000, 300000])
@pytest.mark.parametrize("C,d", [(1, 8), (2, 8), (1, 16), (3, 24)])
@pytest.mark.parametrize("bf16_grads", [False, True])
def test_embed_gradient_of_a_small_table_is_cleared(n, C, d, bf16_grads):
    """Every row of the gradient is written, however few there are and whatever lay there: ids that are all padding
    leave zeros, one id its row alone."""
    op = rece.ItemEmbedding(n, C, d, bf16_grads=bf16_grads)
    dout = torch.ones(n, d, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    gdt = torch.bfloat16 if bf16_grads else torch.float32
    print(f"[gpu] embed gradient n={n} C={C} d={d} bf16_grads={bf16_grads}", flush=True)
    got = op.backward(ids, dout, dtable=torch.full((C, d), float("nan"), dtype=gdt, device="cuda"))
    assert not bool(got.any())
    ids[n // 2] = C - 1
    got = op.backward(ids, dout, dtable=torch.full((C, d), float("nan"), dtype=gdt, device="cuda"))
    assert bool((got[C - 1] == 1).all()) and not bool(got[:C - 1].any())


def _stream_calls():
    """(name, call(stream) -> results, workspace dropped or not) of every operator, with inputs that stay alive."""
    g = torch.Generator().manual_seed(31)
    s, C, d, n, n_seq = 700, 3000, 64, 40000, 1500
    f = lambda *shape: torch.randn(*shape, generator=g)  # noqa: E731
    X, Y = f(s, d).bfloat16().cuda(), f(C, d).bfloat16().cuda()
    ids = torch.randint(-1, C, (s,), generator=g).to(torch.int32).cuda()
    dlogp = f(s).cuda()
    eids = torch.randint(0, C, (9000,), generator=g).to(torch.int32).cuda()
    dout = f(9000, d).bfloat16().cuda()
    lp, old = (-6.0 * torch.rand(n, generator=g)).cuda(), (-6.0 * torch.rand(n, generator=g)).cuda()
    offs = torch.sort(torch.randint(0, n + 1, (n_seq + 1,), generator=g)).values.to(torch.int32).cuda()
    goffs = torch.tensor([0, 800, n_seq], dtype=torch.int32).cuda()   # groups whose sums lie in the workspace
    adv = f(n_seq).cuda()
    emb = rece.ItemEmbedding(9000, C, d)
    lpo = rece.LogProb(s, C, d)
    pol = rece.PolicyLoss(n, n_seq, reduction="sequence")
    prf = rece.PreferenceLoss(n, n_seq, 2, kind="softmax")

    def logprob(stream):
        logp, _, ws = lpo.forward(X, Y, ids, stream=stream)
        return (logp,) + tuple(lpo.backward(X, Y, ids, ws, dlogp, stream=stream))

    return [("embed rows", lambda st: (emb.forward(Y, eids, stream=st),)),
            ("embed gradient", lambda st: (emb.backward(eids, dout, stream=st),)),
            ("log-probabilities", logprob),
            ("log-probabilities alone", lambda st: lpo.forward(X, Y, ids, need_grad=False, stream=st)[:1]),
            ("policy", lambda st: pol.forward(lp, old, adv, offs, stream=st)[:3]),
            ("preference", lambda st: prf.forward(lp, old, offs, goffs, stream=st))]


def _busy(stream):
    """Some milliseconds of work on a stream."""
    with torch.cuda.stream(stream):
        a = torch.zeros(4096, 4096, dtype=torch.bfloat16, device="cuda")
        for _ in range(40):
            a = a @ a
        return a


def test_a_given_streams_workspace_is_not_handed_out_while_in_use():
    """A call enqueued on a busy stream, then tensors of every size filled on the current one before it runs."""
    side = torch.cuda.Stream()
    for name, call in _stream_calls():
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        print(f"[gpu] {name} on another stream", flush=True)
        hold = _busy(side)
        got = call(side)
        junk = [torch.full((1 << k,), 0xFF, dtype=torch.uint8, device="cuda") for k in range(8, 25) for _ in range(4)]
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        del junk, hold


def test_a_given_streams_results_lie_in_memory_of_its_own():
    """Memory freed on the current stream while that still writes it (a queue of work, then fills) is not taken for
    what the given stream writes at once."""
    side = torch.cuda.Stream()
    for name, call in _stream_calls():
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        print(f"[gpu] {name} into memory freed on another stream", flush=True)
        hold = _busy(torch.cuda.current_stream())
        junk = [torch.full((t.numel() * t.element_size(),), 0xFF, dtype=torch.uint8, device="cuda") for t in want for _ in range(8)]
        del junk
        got = call(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        del hold


def test_a_given_stream_may_be_the_current_one_and_must_be_the_devices():
    for name, call in _stream_calls():
        want = call(None)
        assert all(torch.equal(a, b) for a, b in zip(call(torch.cuda.current_stream()), want)), name
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name

    class Elsewhere:
        device = torch.device("cuda", 99)
        cuda_stream = 0

    for name, call in _stream_calls():
        with pytest.raises(ValueError):
            call(Elsewhere())


def _losses():
    """The two losses through autograd: (name, call(logp) -> results, number of tokens)."""
    n, n_seq = 600, 12
    g = torch.Generator().manual_seed(41)
    ref = (-6.0 * torch.rand(n, generator=g)).cuda()
    offs = (torch.arange(n_seq + 1) * (n // n_seq)).to(torch.int32).cuda()
    goffs = (torch.arange(5) * 3).to(torch.int32).cuda()
    adv = torch.randn(n_seq, generator=g).cuda()
    pol, prf = rece.PolicyLoss(n, n_seq), rece.PreferenceLoss(n, n_seq, 4)
    lp = ref + 0.1 * torch.randn(n, generator=g).cuda()
    return lp, [("policy", lambda t: rece.policy_loss(t, ref, adv, offs, pol)),
                ("preference", lambda t: rece.preference_loss(t, ref, offs, goffs, prf))]


def test_losses_may_be_changed_in_place():
    """loss /= steps, loss += other, and the other results too; the gradient follows."""
    lp, calls = _losses()
    for name, call in calls:
        a = lp.clone().requires_grad_(True)
        call(a)[0].backward()
        b = lp.clone().requires_grad_(True)
        loss, *rest = call(b)
        assert loss.shape == ()
        value = float(loss.detach())
        loss /= 4
        loss += b.detach().sum() * 0
        for t in rest:
            t *= 2
        assert float(loss.detach()) == value / 4
        loss.backward()
        assert torch.equal(b.grad, a.grad / 4), name


def test_scoring_without_gradients_makes_no_gradients(monkeypatch):
    """Under no_grad (and with inputs that need none) the functions ask for no gradient, with a parameter as the table
    too, take the smaller workspace, and give the same values."""
    s, C, d = 3000, 2000, 64
    g = torch.Generator().manual_seed(42)
    X = torch.randn(s, d, generator=g).bfloat16().cuda()
    table = torch.nn.Parameter(torch.randn(C, d, generator=g).bfloat16().cuda())
    ids = torch.randint(-1, C, (s,), generator=g).to(torch.int32).cuda()
    asked = []

    def watch(cls, key):
        real = cls.forward

        def forward(self, *args, **kw):
            asked.append(kw.get(key, True))
            return real(self, *args, **kw)
        monkeypatch.setattr(cls, "forward", forward)

    watch(rece.LogProb, "need_grad")
    watch(rece.PolicyLoss, "grads")
    watch(rece.PreferenceLoss, "grads")
    for entropy in (False, True):
        op = rece.LogProb(s, C, d, entropy=entropy)
        both = lambda y: rece.log_probs(X, y, ids, op) if entropy else (rece.log_probs(X, y, ids, op),)  # noqa: E731
        want = both(table)
        assert asked.pop() is True and all(t.requires_grad for t in want)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        with torch.no_grad():
            got = both(table)
        assert torch.cuda.max_memory_allocated() - before <= op.workspace_bytes_no_grad + 8 * s + 4096
        assert asked.pop() is False and not any(t.requires_grad for t in got)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(both(table.detach()), want)) and asked.pop() is False
        with torch.inference_mode():
            both(table)
        assert asked.pop() is False
    lp, calls = _losses()
    for name, call in calls:
        want = call(lp.clone().requires_grad_(True))
        assert asked.pop() is True and want[0].requires_grad
        with torch.no_grad():
            got = call(lp.clone().requires_grad_(True))
        plain = call(lp)
        assert asked == [False, False]
        asked.clear()
        for r in (got, plain):
            assert r[0].shape == () and not r[0].requires_grad and all(torch.equal(a, b) for a, b in zip(r, want)), name


@pytest.mark.parametrize("lead", [1, 3, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_embed_gradient_that_begins_anywhere(lead, dtype):
    """The rows as a part of a longer vector: their gradient is a part of its gradient, at any address."""
    n, C, d = 300, 40, 32
    g = torch.Generator().manual_seed(lead)
    ids = torch.randint(-1, C, (n,), generator=g).to(torch.int32).cuda()
    w = torch.randn(lead + n * d, generator=g).to(dtype).cuda()
    op = rece.ItemEmbedding(n, C, d, dtype="f32" if dtype is torch.float32 else "bf16", bf16_grads=dtype is torch.bfloat16)
    table = torch.randn(C, d, generator=g).to(dtype).cuda().requires_grad_(True)
    head = torch.zeros(lead, dtype=dtype, device="cuda", requires_grad=True)
    (torch.cat([head, rece.embed(table, ids, op).flatten()]) * w).sum().backward()
    assert torch.equal(table.grad, op.backward(ids, w[lead:].clone().view(n, d)))
    assert torch.equal(head.grad, w[:lead])


def test_a_given_stream_inside_a_captured_graph():
    """A capture that forks to another stream, calls the operators on it and joins again: replays between eager work give
    the eager results."""
    for name, call in _stream_calls():
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        print(f"[gpu] {name} captured on a forked stream", flush=True)
        main, fork = torch.cuda.Stream(), torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        main.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(main):
            with torch.cuda.graph(graph, stream=main):
                fork.wait_stream(main)
                got = call(fork)
                main.wait_stream(fork)
        for r in range(3):
            for t in got:
                t.fill_(3.0)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (name, r)
            assert all(torch.equal(a, b) for a, b in zip(call(None), want)), (name, r)

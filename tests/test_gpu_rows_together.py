"""The row operators as a program uses them: a training step of a tensor-parallel model
over virtual ranks, captured graphs, streams, and refusals with device tensors."""

import pytest
import torch

from ring_all_reduce_schedule_amd import binding as B
from tests import rows_ref as R
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

P, TOK, HID, FFN, VOCAB, EPS = 4, 48, 96, 160, 211, 1e-5


def weights(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, s=1.0):
        return s * torch.randn(shape, device="cuda", generator=g)

    def scale():
        return 1 + 0.1 * n(HID)
    return dict(table=n(VOCAB, HID, s=0.3), n1=scale(), up=[n(HID, FFN // P, s=0.1) for _ in range(P)],
                down=[n(FFN // P, HID, s=0.1) for _ in range(P)], n2=scale(),
                head=[n(VOCAB // P + (r < VOCAB % P), HID, s=0.1) for r in range(P)])


def library_step(w, ids, targets):
    """Loss and gradients: the ranks' products by torch, everything where they meet by the library."""
    f = dict(device="cuda", dtype=torch.float32)
    b = B.ra_chunk_bounds(VOCAB, P)
    tables = [w["table"][b[r]:b[r + 1]].contiguous() for r in range(P)]
    emb = torch.empty((TOK, HID), **f)
    B.ra_embedding(tables, ids, [emb], scale=2.0)
    x1, r1 = [torch.empty((TOK, HID), **f) for _ in range(P)], torch.empty(TOK, **f)
    B.ra_allreduce_rmsnorm([emb], w["n1"], EPS, x1[:1], rstd=r1)            # p = 1: a plain norm
    for r in range(1, P):
        x1[r].copy_(x1[0])
    a = [x1[r] @ w["up"][r] for r in range(P)]
    part = [torch.relu(a[r]) @ w["down"][r] for r in range(P)]
    h2, x2, r2 = torch.empty((TOK, HID), **f), [torch.empty((TOK, HID), **f) for _ in range(P)], torch.empty(TOK, **f)
    B.ra_allreduce_rmsnorm(part, w["n2"], EPS, x2, residual=emb, residual_out=h2, rstd=r2)
    logits = [x2[r] @ w["head"][r].t() for r in range(P)]
    loss = torch.empty(TOK, **f)
    B.ra_cross_entropy(logits, targets, loss, grads=logits, grad_scale=1.0 / TOK)     # logits become gradients
    g = dict(head=[logits[r].t() @ x2[r] for r in range(P)])
    dx2 = [logits[r] @ w["head"][r] for r in range(P)]
    g["n2"], dh2, dpart = torch.empty(HID, **f), torch.empty((TOK, HID), **f), [torch.empty((TOK, HID), **f) for _ in range(P)]
    B.ra_allreduce_rmsnorm_backward(dx2, h2, r2, w["n2"], dh2, dxs=dpart, dweight=g["n2"])
    da = [(dpart[r] @ w["down"][r].t()) * (a[r] > 0) for r in range(P)]
    g["down"] = [torch.relu(a[r]).t() @ dpart[r] for r in range(P)]
    g["up"] = [x1[r].t() @ da[r] for r in range(P)]
    dx1 = [da[r] @ w["up"][r].t() for r in range(P)]
    g["n1"], demb = torch.empty(HID, **f), torch.empty((TOK, HID), **f)
    B.ra_allreduce_rmsnorm_backward(dx1, emb, r1, w["n1"], demb, dh_in=dh2, dweight=g["n1"])
    dt = [torch.empty_like(t) for t in tables]
    B.ra_embedding_backward(demb, ids, dt, scale=2.0)
    g["table"] = torch.cat(dt)
    return loss, g


def exact_step(w, ids, targets):
    w = {k: [t.double().cpu().requires_grad_() for t in v] if isinstance(v, list) else v.double().cpu().requires_grad_()
         for k, v in w.items()}
    ids, targets = ids.cpu(), targets.cpu()

    def norm(h, s):
        return h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * s
    emb = torch.where((ids >= 0).unsqueeze(1), w["table"][ids.clamp_min(0)] * 2.0, 0.0)
    x1 = norm(emb, w["n1"])
    h2 = emb + sum(torch.relu(x1 @ u) @ d for u, d in zip(w["up"], w["down"]))
    z = norm(h2, w["n2"]) @ torch.cat(w["head"]).t()
    live = targets >= 0
    loss = torch.where(live, torch.logsumexp(z, 1) - z.gather(1, targets.clamp_min(0).unsqueeze(1)).squeeze(1), 0.0)
    (loss.sum() / TOK).backward()
    return loss.detach(), {k: [t.grad for t in v] if isinstance(v, list) else v.grad for k, v in w.items()}


def batch(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, VOCAB, (TOK,), device="cuda", generator=g)
    ids[5], ids[6:12] = -1, 7
    targets = torch.randint(0, VOCAB, (TOK,), device="cuda", generator=g)
    targets[3] = -100
    return ids, targets


def compare(loss, g, want):
    # float32 chains of some ten products of up to 211 terms: 2^-24 times about 1000 of the norm
    tol = 1000 * R.U

    def near(a, b):
        b = b.cuda()
        assert float((a.double() - b).norm()) <= tol * float(b.norm())
    near(loss, want[0])
    for k, v in g.items():
        for a, b in zip(v, want[1][k]) if isinstance(v, list) else [(v, want[1][k])]:
            near(a, b)


def test_training_step_of_a_tensor_parallel_model():
    require_gpu()
    w = weights(1)
    ids, targets = batch(2)
    compare(*library_step(w, ids, targets), exact_step(w, ids, targets))


def test_training_step_in_a_graph():
    """Captured once and replayed on other batches, with eager steps between the replays."""
    require_gpu()
    w = weights(3)
    ids, targets = batch(4)
    library_step(w, ids, targets)                    # the libraries' first calls, outside the capture
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    print("[case] capture of a training step", flush=True)
    with torch.cuda.graph(graph, stream=s):
        loss, g = library_step(w, ids, targets)
    for seed in (4, 5, 6):
        i, t = batch(seed)
        ids.copy_(i)
        targets.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        eager = library_step(w, i, t)
        torch.cuda.synchronize()
        want = exact_step(w, i, t)
        compare(loss, g, want)
        compare(*eager, want)


def backward_pair(seed):
    """Calls that take workspace, on inputs of their own."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dys = [torch.randn((700, 520), device="cuda", generator=g) for _ in range(3)]
    h = torch.randn((700, 520), device="cuda", generator=g)
    ids = torch.randint(0, 50, (5000,), device="cuda", generator=g)
    dy = torch.randn((5000, 24), device="cuda", generator=g)
    x = torch.randn((3, 60000), device="cuda", generator=g)
    y = torch.tensor([1, 7, 59999], device="cuda")
    out = dict(dh=torch.empty_like(h), dw=torch.empty(520, device="cuda"), dt=torch.empty((50, 24), device="cuda"),
               loss=torch.empty(3, device="cuda"), dx=torch.empty_like(x))

    def run():
        B.ra_allreduce_rmsnorm_backward(dys, h, torch.ones(700, device="cuda"), torch.ones(520, device="cuda"),
                                        out["dh"], dweight=out["dw"])
        B.ra_embedding_backward(dy, ids, [out["dt"]])
        B.ra_cross_entropy([x], y, out["loss"], grads=[out["dx"]])
    return run, out


def test_two_graphs_replayed_side_by_side():
    """Each graph owns its scratch memory, so that replays on two streams do not meet."""
    require_gpu()
    runs = [backward_pair(k) for k in (1, 2)]
    want = []
    for run, out in runs:
        run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in out.items()})
    graphs, streams = [], [torch.cuda.Stream() for _ in runs]
    for (run, _), s in zip(runs, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            run()
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(4):
        for _, out in runs:
            for v in out.values():
                v.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(runs, want):
            for k in w:
                assert torch.equal(out[k], w[k]), k


def test_calls_on_two_streams_at_once():
    require_gpu()
    runs = [backward_pair(k) for k in (3, 4)]
    want = []
    for run, out in runs:
        run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in out.items()})
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(10):
        for (run, _), s in zip(runs, streams):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for (_, out), w in zip(runs, want):
        for k in w:
            assert torch.equal(out[k], w[k]), k


def test_a_stream_given_by_argument():
    """The call and its scratch memory are on that stream, behind the work already there."""
    require_gpu()
    s = torch.cuda.Stream()
    dy, ids = torch.zeros((300, 64), device="cuda"), torch.arange(300, device="cuda") % 7
    d = torch.empty((7, 64), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.randn((4096, 4096), device="cuda")
        for _ in range(10):
            big = big @ big * 1e-2
        dy.fill_(1.0)
    B.ra_embedding_backward(dy, ids, [d], stream=s)
    s.synchronize()
    want = torch.bincount(ids, minlength=7).float().unsqueeze(1).expand(7, 64)
    assert torch.equal(d, want)


def test_workspace_of_the_callers():
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(8)
    dy, ids = torch.randn((9000, 40), device="cuda", generator=g), torch.randint(0, 90, (9000,), device="cuda", generator=g)
    a, b = torch.empty((90, 40), device="cuda"), torch.empty((90, 40), device="cuda")
    n = B.ra_embedding_backward_workspace(9000, 90, 40)
    flat = torch.full((n + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    B.ra_embedding_backward(dy, ids, [a])
    B.ra_embedding_backward(dy, ids, [b], workspace=flat[:n])
    assert torch.equal(a, b) and bool((flat[n:] == 0xAB).all())
    with pytest.raises(B.RaError) as e:
        B.ra_embedding_backward(dy, ids, [b], workspace=flat[:n - 16])
    assert e.value.code == B.RA_ERR_INVALID_ARG


def test_binding_refuses_what_does_not_fit():
    require_gpu()
    f = dict(device="cuda")
    x, w, o = torch.zeros((4, 16), **f), torch.ones(16, **f), torch.zeros((4, 16), **f)
    ids, r = torch.zeros(4, dtype=torch.int64, **f), torch.zeros(4, **f)
    q = torch.zeros((4, 16), dtype=torch.float8_e4m3fn, **f)
    wide = torch.zeros((4, 32), **f)
    for err, call in [
        (ValueError, lambda: B.ra_allreduce_rmsnorm([x, x[:2]], w, 1e-5, [o])),
        (ValueError, lambda: B.ra_allreduce_rmsnorm([wide[:, :16]], w, 1e-5, [o])),
        (ValueError, lambda: B.ra_allreduce_rmsnorm([x], w, 1e-5, [wide[:, ::2]])),
        (ValueError, lambda: B.ra_allreduce_rmsnorm([x], torch.ones(7, **f), 1e-5, [o])),
        (ValueError, lambda: B.ra_allreduce_rmsnorm([x], w, 1e-5, [])),
        (ValueError, lambda: B.ra_allreduce_rmsnorm([x], w, 1e-5, [o[:3]])),
        (TypeError, lambda: B.ra_allreduce_rmsnorm([x], w.half(), 1e-5, [o])),
        (TypeError, lambda: B.ra_allreduce_rmsnorm([x], w, 1e-5, [o], residual=x, residual_out=o.half())),
        (ValueError, lambda: B.ra_allreduce_rmsnorm([x], w, 1e-5, [o], residual=x.cpu())),
        (ValueError, lambda: B.ra_allreduce_rmsnorm([x], w, 1e-5, [q])),
        (ValueError, lambda: B.ra_allreduce_rmsnorm([x], w, 1e-5, [q], scales=[torch.zeros(3, **f)])),
        (TypeError, lambda: B.ra_allreduce_rmsnorm([x], w, 1e-5, [q], scales=[torch.zeros(4, **f).half()])),
        (TypeError, lambda: B.ra_allreduce_rmsnorm([x], w, 1e-5, [o], rstd=r.double())),
        (TypeError, lambda: B.ra_allreduce_rmsnorm_backward([x], o, r, w, o.half())),
        (TypeError, lambda: B.ra_allreduce_rmsnorm_backward([x], o, r, w, wide[:2].clone().view(4, 16), dxs=[o.half()])),
        (ValueError, lambda: B.ra_cross_entropy([x], ids[:3], loss=r)),
        (TypeError, lambda: B.ra_cross_entropy([x], ids.float(), loss=r)),
        (ValueError, lambda: B.ra_cross_entropy([x], ids, loss=r[:3])),
        (ValueError, lambda: B.ra_cross_entropy([x, wide], ids, loss=r)),
        (ValueError, lambda: B.ra_cross_entropy([x], ids, loss=r, grads=[wide])),
        (TypeError, lambda: B.ra_cross_entropy([x], ids, loss=r, grads=[o.half()])),
        (TypeError, lambda: B.ra_embedding([x], ids, [o.half()])),
        (ValueError, lambda: B.ra_embedding([x], ids, [o[:2]])),
        (ValueError, lambda: B.ra_embedding([x, wide], ids, [o])),
        (ValueError, lambda: B.ra_embedding_backward(o[:2], ids, [x])),
        (B.RaError, lambda: B.ra_embedding_backward(o.half(), ids, [x.bfloat16()])),
        (B.RaError, lambda: B.ra_allreduce_rmsnorm([x], w, 0.0, [o])),
        (B.RaError, lambda: B.ra_cross_entropy([x], ids, loss=r, valid=17)),
    ]:
        with pytest.raises(err):
            call()
    torch.cuda.synchronize()


def test_rank_buffers_in_place_of_lists():
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(10)

    def n(*shape):
        return torch.randn(shape, device="cuda", generator=g)
    bufs, w, ids = [n(6, 24) for _ in range(3)], n(24), torch.tensor([0, 5, 5, 2, -1, 8], device="cuda")
    logits, tables, h, r = [n(6, 4) for _ in range(3)], [n(3, 24) for _ in range(3)], n(6, 24), n(6).abs()

    def run(wrap):
        out = [[torch.empty(6, 24, device="cuda") for _ in range(3)] for _ in range(3)]
        grads, dt = [torch.empty(6, 4, device="cuda") for _ in range(3)], [torch.empty(3, 24, device="cuda") for _ in range(3)]
        dh = torch.empty(6, 24, device="cuda")
        B.ra_allreduce_rmsnorm(wrap(bufs), w, 1e-5, wrap(out[0]))
        B.ra_allreduce_rmsnorm_backward(wrap(bufs), h, r, w, dh, dxs=wrap(out[1]))
        B.ra_embedding(wrap(tables), ids, wrap(out[2]))
        B.ra_embedding_backward(h, ids, wrap(dt))
        B.ra_cross_entropy(wrap(logits), ids, lse=r.clone(), grads=wrap(grads))
        lse = torch.empty(6, device="cuda")
        B.ra_cross_entropy(wrap(logits), ids, lse=lse)
        again = [torch.empty(6, 4, device="cuda") for _ in range(3)]
        B.ra_cross_entropy_backward(wrap(logits), ids, lse, wrap(again))
        return out[0] + out[1] + out[2] + grads + dt + again + [dh]
    assert all(torch.equal(a, b) for a, b in zip(run(list), run(B.RankBuffers)))


def test_a_sum_and_its_norm_agree_with_the_all_reduce():
    """Integers small enough that every order and rounding gives the same sum: the norm's h is
    what ra_allreduce leaves."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(9)
    bufs = [torch.randint(-8, 9, (37, 260), device="cuda", generator=g).to(torch.bfloat16) for _ in range(8)]
    h, y = torch.empty_like(bufs[0]), torch.empty_like(bufs[0])
    B.ra_allreduce_rmsnorm(bufs, torch.ones(260, dtype=torch.bfloat16, device="cuda"), 1e-5, [y], residual_out=h)
    B.ra_allreduce(bufs)
    B.ra_stream_status()
    assert all(torch.equal(b, h) for b in bufs)

"""The router's load-balancing loss, z loss, counts and their gradient against the definitions in 64
bits (tests/mx4_reference.py), on an MI355X; the formula itself against differences on the CPU.

Bars.  Counts: equal.  p_te carries (|l - max| + 32) roundings of 2^-24 relative (the rounded
exponent, exp, the row's sum and division), |l| <= 128 here; a mean over T tokens adds at most
D = 700 additions (a lane's rows, the lanes', the blocks').  Both are positive sums, so mean_prob and
the losses are within C = (2 * 128 + 32 + 700) 2^-24 = 6e-5 relative.  A gradient element is within
C of the sum of its terms' magnitudes, plus half a step of the output type.
"""
import numpy as np
import pytest
import torch

import moe_inputs as mi
import sparse_moe_expert_router_amd as moe
from tests import mx4_reference as ref

DEV = "cuda"
gpu = pytest.mark.gpu
FAKE = 1 << 20
C = (2 * 128 + 32 + 700) * 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------------------------------
# without a GPU

def test_reference_gradient_matches_differences():
    """Central differences of the losses with the counts held, and of sum(dw * renormalised weights)."""
    r = np.random.default_rng(0)
    T, E, k = 7, 6, 3
    l = r.normal(size=(T, E)) * 2
    idx = np.argsort(-l, axis=1)[:, :k]
    mask = np.array([1, 1, 0, 1, 1, 1, 1])
    _, counts, _ = ref.balance(l, idx, mask)
    f = counts / counts.sum()
    g = np.array([0.7, 0.3])
    dw = r.normal(size=(T, k))

    def weights(x):
        e = np.exp(np.take_along_axis(x, idx, 1))
        return e / e.sum(1, keepdims=True)

    def value(x):
        p, lse = ref.softmax(x[mask == 1])
        return (g[0] * E * f @ p.mean(0) + g[1] * np.mean(lse ** 2) + np.sum(weights(x) * dw * mask[:, None]))

    d, _ = ref.balance_grad(l, idx, counts, g, weights(l), dw, mask)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((value(a) - value(b)) / (2 * h) - d[t, e]) < 1e-8


def test_even_load_has_loss_one():
    l = np.zeros((8, 4))
    idx = np.array([[t % 4] for t in range(8)])
    loss, counts, P = ref.balance(l, idx)
    assert loss[0] == 1 and counts.tolist() == [2] * 4 and np.allclose(P, .25) and np.isclose(loss[1], np.log(4) ** 2)


def test_argument_checks():
    L = moe.lib()
    assert L.moe_balance_workspace_bytes(0, 8) == L.moe_balance_workspace_bytes(8, 513) == 0
    assert L.moe_balance_workspace_bytes(32768, 512) > L.moe_balance_workspace_bytes(8, 8) > 0

    def fwd(l=FAKE, lt=0, T=8, E=16, idx=FAKE, k=2, mask=None, loss=FAKE, c=FAKE, p=FAKE, ws=FAKE, n=1 << 30):
        return L.moe_balance_loss(l, lt, T, E, idx, k, mask, loss, c, p, ws, n, None)

    def bwd(l=FAKE, lt=0, T=8, E=16, idx=FAKE, k=2, mask=None, c=FAKE, dl=FAKE, w=None, dw=None, g=FAKE, gt=0):
        return L.moe_balance_loss_backward(l, lt, T, E, idx, k, mask, c, dl, w, dw, g, gt, None)

    both = (dict(l=None), dict(l=FAKE + 4), dict(lt=2), dict(lt=4), dict(T=0), dict(T=32769), dict(E=0), dict(E=513),
            dict(k=0), dict(k=17), dict(E=128, k=65), dict(idx=None), dict(idx=FAKE + 4), dict(mask=FAKE + 1),
            dict(c=None), dict(c=FAKE + 4))
    for bad in both + (dict(loss=None), dict(loss=FAKE + 4), dict(p=None), dict(ws=None)):
        assert fwd(**bad) == moe.EINVAL, bad
    assert fwd(n=16) == moe.EWORKSPACE
    for bad in both + (dict(dl=None), dict(w=FAKE), dict(dw=FAKE), dict(w=FAKE, dw=FAKE + 4), dict(g=None), dict(gt=2),
                       dict(gt=3)):
        assert bwd(**bad) == moe.EINVAL, bad


def test_binding_refuses_wrong_tensors():
    l, i = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.balance_loss(l, i)                                 # not on a GPU
    with pytest.raises(TypeError):
        moe.balance_loss(l.half(), i)
    with pytest.raises(ValueError):
        moe.balance_loss_backward(l[0], i, i, l)


# ------------------------------------------------------------------------------------------
# on the GPU

def batch(T, E, k, dtype, mask=None, seed=0, scale=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed + 17 * T + E)
    l = torch.randn((T, E), generator=g, device=DEV) * scale
    idx = torch.topk(l, k, 1).indices.to(torch.int32)
    w = torch.softmax(torch.gather(l, 1, idx.long()), 1)
    dw = torch.randn((T, k), generator=g, device=DEV)
    m = None if mask is None else torch.rand(T, generator=g, device=DEV) < mask
    return l.to(dtype), idx, w, dw, m


def check(l, idx, w, dw, m, g=(0.7, 0.3), grad_dtype=None):
    # losses of float64 logits are those of the logits rounded to fp32
    lv = f64(l.float() if l.dtype == torch.float64 else l)
    loss, counts, P = moe.balance_loss(l, idx, mask=m)
    dl = torch.tensor(g, device=DEV)
    d = moe.balance_loss_backward(l, idx, counts, dl, topk_w=w, d_topk_w=dw, mask=m, grad_dtype=grad_dtype)
    torch.cuda.synchronize()
    iv, mv = idx.cpu().numpy(), None if m is None else m.cpu().numpy()
    rloss, rcounts, rP = ref.balance(lv, iv, mv)
    assert np.array_equal(counts.cpu().numpy(), rcounts)
    np.testing.assert_allclose(f64(P), rP, rtol=C, atol=1e-37)
    np.testing.assert_allclose(f64(loss), rloss, rtol=2 * C, atol=1e-37)
    rd, mag = ref.balance_grad(lv, iv, rcounts, f64(dl), None if w is None else w.cpu().numpy(),
                               None if dw is None else dw.cpu().numpy(), mv)
    assert (np.abs(f64(d) - rd) <= C * mag + HALF[d.dtype] * (np.abs(rd) + C * mag) + 1e-37).all()
    if mv is not None:
        assert (f64(d)[~mv.astype(bool)] == 0).all()
    return d


SHAPES = [(1, 1, 1), (1, 8, 2), (2, 3, 3), (5, 13, 4), (8, 128, 8), (63, 16, 16), (64, 17, 1), (65, 64, 6), (100, 65, 5),
          (130, 128, 64), (77, 129, 9), (300, 256, 22), (259, 257, 3), (500, 512, 22), (33, 511, 64), (4099, 40, 5)]


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float64])
@pytest.mark.parametrize("T,E,k", SHAPES, ids=["T%d-E%d-k%d" % s for s in SHAPES])
def test_loss_and_gradient(T, E, k, dtype):
    check(*batch(T, E, k, dtype))


@gpu
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (64, 12, 3), (700, 128, 8), (90, 250, 4)])
def test_padding_holds_anything(T, E, k):
    """Masked tokens' logits are NaN, infinite or the type's lowest value, their weights NaN."""
    l, idx, w, dw, m = batch(T, E, k, torch.float32, mask=0.6)
    off = ~m
    l[off] = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).min],
                          device=DEV).repeat(-(-E // 4))[:E]
    w[off] = float("nan")
    dw[off] = float("inf")
    check(l, idx, w, dw, m)
    check(l, idx, w, dw, m.to(torch.uint8) * 255)


@gpu
def test_no_token_counts():
    l, idx, w, dw, m = batch(40, 24, 3, torch.float32, mask=0.0)
    l[:] = float("nan")
    d = check(l, idx, w, dw, m)
    assert not d.any()
    l2, idx, w, dw, _ = batch(40, 24, 3, torch.float32)
    l2[:] = -float("inf")                                       # no expert is open to any token
    d = check(l2, idx, w, dw, None)
    assert not d.any()


@gpu
def test_masked_experts():
    """Experts closed by -inf or by the type's lowest value; a token with one open expert, a token with
    none (it counts as padding)."""
    l, idx, w, dw, _ = batch(50, 32, 4, torch.float32)
    l[:, 5] = -float("inf")
    l[:, 9] = torch.finfo(torch.float32).min
    l[7] = -float("inf")
    l[7, 3] = 2.0
    l[11] = -float("inf")
    d = check(l, idx, w, dw, None)
    assert not d[11].any() and torch.isfinite(d).all()


@gpu
def test_nan_token_spoils_only_what_it_enters():
    """A NaN or +inf in a token that counts: its gradient row and the means are NaN, the counts and the
    other rows are not."""
    for bad in (float("nan"), float("inf")):
        l, idx, w, dw, _ = batch(50, 32, 4, torch.float32)
        _, counts, _ = moe.balance_loss(l, idx)
        l[7, 3] = bad
        loss, c2, P = moe.balance_loss(l, idx)
        d = moe.balance_loss_backward(l, idx, c2, torch.ones(2, device=DEV))
        torch.cuda.synchronize()
        assert torch.equal(counts, c2) and torch.isnan(loss).all() and torch.isnan(P).all()
        assert torch.isnan(d[7]).all() and torch.isfinite(torch.cat((d[:7], d[8:]))).all()


@gpu
def test_repeated_and_wild_ids():
    """An id that a token names several times, and ids outside [0, E) (clamped)."""
    l, idx, w, dw, _ = batch(60, 16, 5, torch.float32)
    idx[3] = 7
    idx[4, 1:4] = idx[4, 0]
    idx[5, 0], idx[5, 1], idx[6, 2] = -3, 99, 2 ** 31 - 1
    d = check(l, idx, w, dw, None)
    for _ in range(3):
        assert torch.equal(d, check(l, idx, w, dw, None))


@gpu
def test_large_logits():
    l, idx, w, dw, _ = batch(64, 64, 4, torch.float32, scale=1.0)
    l = (l * 1e4).clamp(-1e5, 1e5)                              # softmax is one-hot, lse^2 large
    loss, counts, P = moe.balance_loss(l, idx)
    torch.cuda.synchronize()
    rloss, _, rP = ref.balance(f64(l), idx.cpu().numpy())
    np.testing.assert_allclose(f64(loss), rloss, rtol=C)
    np.testing.assert_allclose(f64(P), rP, rtol=C, atol=1e-37)


@gpu
def test_without_weights_and_with_another_gradient_type():
    l, idx, w, dw, m = batch(200, 96, 6, torch.float32, mask=0.8)
    check(l, idx, None, None, m)
    assert check(l, idx, w, dw, m, grad_dtype=torch.bfloat16).dtype == torch.bfloat16
    l, idx, w, dw, m = batch(200, 96, 6, torch.bfloat16, mask=0.8)
    assert check(l, idx, w, dw, m).dtype == torch.bfloat16
    assert check(l, idx, w, dw, m, grad_dtype=torch.float32).dtype == torch.float32


@gpu
def test_largest_batch():
    l, idx, w, dw, m = batch(32768, 128, 8, torch.float32, mask=0.9)
    lv, iv, mv = f64(l), idx.cpu().numpy(), m.cpu().numpy()
    loss, counts, P = moe.balance_loss(l, idx, mask=m)
    d = moe.balance_loss_backward(l, idx, counts, torch.ones(2, device=DEV), topk_w=w, d_topk_w=dw, mask=m)
    torch.cuda.synchronize()
    rloss, rcounts, rP = ref.balance(lv, iv, mv)
    assert np.array_equal(counts.cpu().numpy(), rcounts)
    np.testing.assert_allclose(f64(P), rP, rtol=C)
    np.testing.assert_allclose(f64(loss), rloss, rtol=2 * C)
    at = np.r_[0:200, 32600:32768]
    rd, mag = ref.balance_grad(lv[at], iv[at], rcounts, np.ones(2), w.cpu().numpy()[at], dw.cpu().numpy()[at], mv[at])
    assert (np.abs(f64(d)[at] - rd) <= (C + 2 ** -24) * mag + 1e-37).all()


@gpu
def test_gradient_against_differences_of_the_loss_kernel():
    """The kernel's own loss at l +- h, counts as they are (no id changes), against its gradient: the
    difference is exact to h^2 and to the loss's rounding 2 C |loss| / (2 h)."""
    T, E, k = 6, 24, 3
    l, idx, _, _, _ = batch(T, E, k, torch.float32, scale=1.0)
    loss, counts, _ = moe.balance_loss(l, idx)
    h = 2.0 ** -4
    for which in (0, 1):
        g = torch.zeros(2, device=DEV)
        g[which] = 1.0
        d = f64(moe.balance_loss_backward(l, idx, counts, g))
        for t, e in ((0, 0), (2, 5), (5, 23), (3, int(idx[3, 0]))):
            a, b = l.clone(), l.clone()
            a[t, e] += h
            b[t, e] -= h
            va, vb = (float(moe.balance_loss(v, idx)[0][which]) for v in (a, b))
            # third derivatives of both losses along a logit are below 12 E max(f) and 12 (1 + |lse|)
            third = 12 * (E if which == 0 else 8) / T
            assert abs((va - vb) / (2 * h) - d[t, e]) <= h * h / 6 * third + 2 * 2.0 ** -20 * float(loss[which]) / h


@gpu
def test_run_with_the_router():
    """As a trainer uses them: route (its workspace keeps the fp64 logits), loss on those, gradient
    with the routing weights' gradient."""
    w = mi.workload("gemma_decode", T=70)
    wr, _ = mi.make_router(w, 0, DEV)
    x = mi.make_x(w, 0, T=70, device=DEV)
    ws = moe.alloc_workspace(int(moe.lib().moe_route_workspace_bytes(70, w.E)))
    idx, wts = moe.route(x, wr, None, w.k, ws=ws)
    logits = ws[:70 * w.E * 8].view(torch.float64).view(70, w.E)
    exact = f64(x) @ f64(wr).T
    torch.cuda.synchronize()
    np.testing.assert_allclose(f64(logits), exact, rtol=1e-9, atol=1e-9)
    assert np.array_equal(np.argsort(-exact, axis=1, kind="stable")[:, :w.k], idx.cpu().numpy())
    check(logits, idx, wts, torch.randn_like(wts), None)
    counts, *_ = moe.permute(idx, w.E)
    assert torch.equal(moe.balance_loss(logits, idx)[1], counts)


@gpu
def test_replays_in_a_graph_and_on_another_stream():
    for T, E, k in ((9, 40, 4), (3000, 128, 8)):
        l, idx, w, dw, m = batch(T, E, k, torch.float32, mask=0.7)
        ws = moe.alloc_workspace(int(moe.lib().moe_balance_workspace_bytes(T, E)))
        dl = torch.tensor([.5, .25], device=DEV)

        def step(ws=None):
            loss, counts, P = moe.balance_loss(l, idx, mask=m, ws=ws)
            return loss, counts, P, moe.balance_loss_backward(l, idx, counts, dl, topk_w=w, d_topk_w=dw, mask=m)

        s = torch.cuda.Stream()
        want = step()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, other))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step(ws)
        for i in range(4):
            if i == 2:
                l.copy_(l.flip(0))
            want = step()
            ws.fill_(255)
            for t in got:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got)), i


@gpu
def test_two_batches_at_once():
    """Losses and gradients of two batches on two streams, each call with a workspace of its own."""
    batches = [batch(3000, 128, 8, torch.float32), batch(700, 250, 5, torch.float32, seed=1)]
    dl = torch.tensor([.5, .25], device=DEV)

    def step(b):
        l, idx, w, dw, _ = b
        loss, counts, P = moe.balance_loss(l, idx)
        return loss, counts, P, moe.balance_loss_backward(l, idx, counts, dl, topk_w=w, d_topk_w=dw)

    want = [step(b) for b in batches]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in batches], [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(batches[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, want[i]))

"""The expert router on the GPU against a plain 64-bit restatement: experts,
counts and orders exactly, weights, loss and gradients to bounds counted from
the kernels' 32-bit roundings."""
import numpy as np
import pytest
import torch

import activation_sparse_gated_epilogue_b200 as sge
from tests._util import to_f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def route_np(l, k, renorm, mask):
    """numpy float64 restatement; l [N][E] float64."""
    n, e = l.shape
    ids, w = np.full((n, k), -1), np.zeros((n, k))
    p, live = np.zeros((n, e)), np.zeros(n, bool)
    for t in range(n):
        if mask is not None and not mask[t]:
            continue
        if np.isnan(l[t]).any() or (l[t] == np.inf).any():
            p[t], live[t] = np.nan, True
            continue
        if not (l[t] > -np.inf).any():
            continue
        live[t] = True
        x = np.exp(l[t] - l[t].max())
        p[t] = x / x.sum()
        top = [i for i in np.argsort(-l[t], kind="stable")[:k] if l[t][i] > -np.inf]
        ids[t, :len(top)] = top
        w[t, :len(top)] = p[t][top] / (p[t][top].sum() if renorm else 1.0)
    flat = ids.reshape(-1)
    counts = np.bincount(flat[flat >= 0], minlength=e)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    by = np.argsort(np.where(flat >= 0, flat, e), kind="stable")
    pos = np.full(n * k, -1)
    pos[by[:offsets[-1]]] = np.arange(offsets[-1])
    order = np.where(np.arange(n * k) < offsets[-1], by, -1)
    loss = e * np.sum(counts / max(1, counts.sum()) * p.sum(0) / max(1, live.sum()))
    return ids, w, counts, offsets, pos.reshape(n, k), order, loss, int(live.sum()), p


def grad_np(r, k, renorm, dloss, dw):
    ids, w, counts, _, _, _, _, live, p = r
    n, e = p.shape
    dp = np.broadcast_to(dloss * e * counts / max(1, counts.sum()) / max(1, live), (n, e)).copy()
    dl = np.zeros((n, e))
    size = np.zeros((n, e))     # magnitude of the terms that were added
    for t in range(n):
        there = ids[t] >= 0
        at, g = ids[t][there], np.where(there, dw[t], 0.0)[there]
        if not renorm:
            np.add.at(dp[t], at, g)
        dot = np.sum(p[t] * dp[t])
        dl[t] = p[t] * (dp[t] - dot)
        size[t] = p[t] * (np.abs(dp[t]) + np.sum(p[t] * np.abs(dp[t])))
        if renorm:
            wt = w[t][there]
            np.add.at(dl[t], at, wt * (g - np.sum(wt * g)))
            np.add.at(size[t], at, wt * (np.abs(g) + np.sum(wt * np.abs(g))))
    return dl, size


def check(cuda_device, logits, k, renorm, mask=None, seed=0):
    n, e = logits.shape
    l64 = logits.double().numpy()
    r = route_np(l64, k, renorm, None if mask is None else mask.numpy())
    ids, w, counts, offsets, pos, order, loss, live, p = r
    dev_l = logits.to(cuda_device)
    dev_m = None if mask is None else mask.to(cuda_device)
    got = sge.moe_route_fwd(dev_l, k, renorm=renorm, mask=dev_m)
    for name, want in (("ids", ids), ("counts", counts), ("offsets", offsets), ("pos", pos), ("order", order)):
        np.testing.assert_array_equal(getattr(got, name).cpu().numpy(), want, err_msg=name)
    assert int(got.n_live) == live
    # p: the exponent's argument is one fp32 subtraction (error U * |l - max|, at most U * 200 where p is
    # not 0 in fp32), expf 2 ulp (4U), the sum of positive terms log2(32) + 8 roundings of at most U
    # each with the same relative error of its terms, division and product 2U
    spread = np.where(np.isfinite(l64), l64, 0).max(1, initial=0) - np.where(np.isfinite(l64), l64, 0).min(1, initial=0)
    rel = (2 * (np.minimum(spread, 200.0) + 4) + 20) * U
    tiny = 2.0 ** -120
    assert np.all(np.abs(to_f64(got.w) - w) <= rel[:, None] * w + tiny)
    worst = rel.max(initial=0.0)
    if np.isnan(loss):
        assert np.isnan(float(got.loss))
    else:
        # sums over a warp's rows and over 32 warps in fp32: at most rows + 32 further roundings
        rows = -(-n // (32 * 148)) + 32
        assert abs(float(got.loss) - loss) <= (worst + (rows + 2) * U) * loss + tiny
    rng = np.random.default_rng(seed)
    dw = torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32))
    dloss = torch.tensor([0.37])
    dl, size = grad_np(r, k, renorm, float(dloss), dw.double().numpy())
    g = to_f64(sge.moe_route_bwd(dev_l, got, dloss.to(cuda_device), dw.to(cuda_device), mask=dev_m))
    out = 2.0 ** -8 if logits.dtype == torch.bfloat16 else 0.0
    fine = ~np.isnan(dl)
    np.testing.assert_array_equal(np.isnan(g), ~fine)
    bound = (2 * worst + 60 * U) * size + out * np.abs(dl) + tiny
    assert np.all(np.abs(g - dl)[fine] <= bound[fine])
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("n,e,k", [(1, 1, 1), (1, 2, 2), (1, 64, 8), (2, 7, 3), (31, 32, 4), (32, 33, 1),
                                   (33, 65, 5), (64, 128, 16), (65, 129, 8), (300, 8, 2), (257, 256, 8),
                                   (1000, 40, 6), (5000, 16, 2)])
def test_route_and_its_gradient(cuda_device, dtype, renorm, n, e, k):
    g = torch.Generator().manual_seed(n + e + k)
    logits = (torch.randn(n, e, generator=g) * 2 + torch.randn(1, e, generator=g)).to(dtype)
    mask = (torch.rand(n, generator=g) < 0.8).to(torch.uint8) if n % 2 else None
    check(cuda_device, logits, k, renorm, mask)


@pytest.mark.parametrize("renorm", [True, False])
def test_route_ties_go_to_the_lower_index(cuda_device, renorm):
    g = torch.Generator().manual_seed(3)
    logits = torch.randint(-2, 3, (200, 70), generator=g).float()
    logits[0] = 0.0
    logits[1] = torch.where(torch.arange(70) % 2 == 0, 0.0, -0.0)    # equal values
    got = check(cuda_device, logits, 6, renorm)
    assert got.ids[0].tolist() == got.ids[1].tolist() == [0, 1, 2, 3, 4, 5]


@pytest.mark.parametrize("renorm", [True, False])
def test_route_masked_infinite_and_lowest_logits(cuda_device, renorm):
    n, e, k = 60, 20, 4
    logits = torch.randn(n, e, generator=torch.Generator().manual_seed(5))
    mask = torch.ones(n, dtype=torch.uint8)
    low = torch.finfo(torch.float32).min
    logits[1] = -float("inf")                 # nothing left
    logits[2, 3:] = -float("inf")             # fewer than k
    logits[3] = low                           # the type's lowest value is a number like any other
    logits[4, ::2] = low
    logits[5, 1:] = -float("inf")
    mask[6:9] = 0
    logits[6] = float("nan")                  # in masked places: not read
    logits[7] = float("inf")
    logits[8] = -float("inf")
    logits[9] = torch.linspace(-90, 90, e)
    logits[10] = torch.linspace(-3e38, 3e38, e)    # its step passes fp32: the row is not finite
    assert not torch.isfinite(logits[10]).all()
    got = check(cuda_device, logits, k, renorm, mask)
    assert got.ids[1].tolist() == [-1] * 4 and got.ids[2].tolist()[3] == -1
    assert torch.isnan(got.loss).all()
    logits[10] = (torch.arange(e) - 9.5) * 3e37
    assert torch.isfinite(check(cuda_device, logits, k, renorm, mask).loss).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_route_live_row_that_is_not_finite(cuda_device, bad):
    logits = torch.randn(50, 9, generator=torch.Generator().manual_seed(6))
    logits[17, 4] = bad
    got = check(cuda_device, logits, 2, True)
    assert got.ids[17].tolist() == [-1, -1] and torch.isnan(got.loss).all()


def test_route_no_live_token_and_no_token(cuda_device):
    logits = torch.randn(40, 12)
    check(cuda_device, logits, 3, True, torch.zeros(40, dtype=torch.uint8))
    r = sge.moe_route_fwd(torch.randn(0, 12, device=cuda_device), 3)
    assert r.counts.tolist() == [0] * 12 and r.offsets.tolist() == [0] * 13
    assert float(r.loss) == 0 and int(r.n_live) == 0
    assert sge.moe_route_bwd(torch.randn(0, 12, device=cuda_device), r).shape == (0, 12)


def test_route_gradient_against_differences(cuda_device):
    """The gradient of 0.37 * loss + <dw, w> against central differences of
    the 64-bit restatement (step 1e-5: truncation 1e-10, cancellation 1e-11)."""
    n, e, k = 6, 5, 2
    g = torch.Generator().manual_seed(8)
    logits, dw = torch.randn(n, e, generator=g), torch.randn(n, k, generator=g)
    for renorm in (True, False):
        dev = logits.to(cuda_device)
        r = sge.moe_route_fwd(dev, k, renorm=renorm)
        got = to_f64(sge.moe_route_bwd(dev, r, torch.full((1,), 0.37, device=cuda_device), dw.to(cuda_device)))

        def value(l):
            s = route_np(l, k, renorm, None)
            return 0.37 * s[6] + np.sum(s[1] * dw.double().numpy())

        for t in range(n):
            for i in range(e):
                step = np.zeros((n, e))
                step[t, i] = 1e-5
                want = (value(logits.double().numpy() + step) - value(logits.double().numpy() - step)) / 2e-5
                assert abs(got[t, i] - want) <= 1e-6 * max(1.0, abs(want))


def test_route_parts_of_the_gradient(cuda_device):
    logits = torch.randn(70, 10, generator=torch.Generator().manual_seed(9)).to(cuda_device)
    r = sge.moe_route_fwd(logits, 2)
    zero, one = torch.zeros(1, device=cuda_device), torch.ones(1, device=cuda_device)
    dw = torch.randn(70, 2, device=cuda_device)
    assert (sge.moe_route_bwd(logits, r) == 0).all()
    assert torch.equal(sge.moe_route_bwd(logits, r, dw=dw), sge.moe_route_bwd(logits, r, zero, dw))
    assert torch.equal(sge.moe_route_bwd(logits, r, one), sge.moe_route_bwd(logits, r, one, torch.zeros_like(dw)))


def test_route_repeats_graphs_and_streams(cuda_device):
    logits = torch.randn(3000, 100, device=cuda_device)
    dw = torch.randn(3000, 4, device=cuda_device)
    one = torch.ones(1, device=cuda_device)

    def both(stream=None):
        r = sge.moe_route_fwd(logits, 4, stream=stream)
        return [r.ids, r.w, r.counts, r.offsets, r.pos, r.order, r.loss,
                sge.moe_route_bwd(logits, r, one, dw, stream=stream)]

    want = both()
    same = lambda got: all(torch.equal(a, b) for a, b in zip(got, want))  # noqa: E731
    assert same(both())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    torch.cuda.current_stream().wait_stream(side)
    assert same(got)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = both()
    graph.replay()
    assert same(got)
    graph.replay()
    assert same(got)


def test_route_refusals(cuda_device):
    logits = torch.randn(8, 16, device=cuda_device)
    with pytest.raises(sge.LibraryError):
        sge.moe_route_fwd(logits, 17)
    with pytest.raises(sge.LibraryError):
        sge.moe_route_fwd(logits, 0)
    with pytest.raises(sge.LibraryError, match="experts"):
        sge.moe_route_fwd(torch.randn(8, 257, device=cuda_device), 2)
    with pytest.raises(ValueError, match="mask"):
        sge.moe_route_fwd(logits, 2, mask=torch.ones(8, device=cuda_device))
    with pytest.raises(ValueError):
        sge.moe_route_fwd(logits.half(), 2)
    r = sge.moe_route_fwd(logits, 2)
    with pytest.raises(ValueError, match="shape"):
        sge.moe_route_bwd(logits[:4], r)
    with pytest.raises(ValueError, match="dw"):
        sge.moe_route_bwd(logits, r, dw=torch.zeros(8, 3, device=cuda_device))


def test_route_of_the_callers_own_tensors(cuda_device):
    """A MoeRoute of separate tensors gets the same results as one of
    MoeRoute.empty, and is checked tensor by tensor."""
    n, e, k = 37, 11, 3
    logits = torch.randn(n, e, device=cuda_device)
    want = sge.moe_route_fwd(logits, k)
    i = lambda *s: torch.full(s, 7, dtype=torch.int32, device=cuda_device)  # noqa: E731
    f = lambda *s: torch.full(s, 7.0, device=cuda_device)  # noqa: E731
    own = sge.MoeRoute(i(n, k), f(n, k), i(e), i(e + 1), i(n, k), i(n * k), f(1), i(1))
    got = sge.moe_route_fwd(logits, k, out=own)
    assert got is own
    for name in sge.MoeRoute.NAMES:
        assert torch.equal(getattr(got, name), getattr(want, name)), name
    dw, one = torch.randn(n, k, device=cuda_device), torch.ones(1, device=cuda_device)
    assert torch.equal(sge.moe_route_bwd(logits, own, one, dw), sge.moe_route_bwd(logits, want, one, dw))
    bad = sge.MoeRoute(i(n, k), f(n, k), i(e), i(e), i(n, k), i(n * k), f(1), i(1))
    with pytest.raises(ValueError, match="offsets"):
        sge.moe_route_fwd(logits, k, out=bad)
    with pytest.raises(ValueError, match="shape"):
        sge.moe_route_fwd(logits, k + 1, out=want)


def route_wide(l, k, renorm, mask):
    """route_np over whole tensors, for long batches (no NaN or +inf)."""
    n, e = l.shape
    l = l.double()
    if mask is not None:
        l = torch.where(mask[:, None] != 0, l, -torch.inf)
    live = (l > -torch.inf).any(1)
    p = torch.where(live[:, None], torch.softmax(l, 1), 0.0)
    value, ids = torch.sort(l, dim=1, descending=True, stable=True)
    there = value[:, :k] > -torch.inf
    ids = torch.where(there, ids[:, :k], -1)
    w = torch.where(there, p.gather(1, ids.clamp(min=0)), 0.0)
    if renorm:
        w = torch.where(there, w / w.sum(1, keepdim=True).clamp(min=1e-300), 0.0)
    flat = ids.reshape(-1)
    counts = torch.bincount(flat[flat >= 0], minlength=e)
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    by = torch.sort(torch.where(flat >= 0, flat, e), stable=True)[1]
    place = torch.arange(n * k, device=l.device)
    there = place < offsets[-1]
    pos = torch.full_like(by, -1)
    pos[by] = torch.where(there, place, -1)
    order = torch.where(there, by, -1)
    n_live = live.sum()
    f = counts.double() / counts.sum().clamp(min=1)
    loss = e * (f * p.sum(0)).sum() / n_live.clamp(min=1)
    return dict(ids=ids, w=w, counts=counts, offsets=offsets, pos=pos.view(n, k), order=order, loss=loss,
                n_live=n_live), p, f


# rows a warp: 5 (the places beyond the four that stay in registers), 9, 64, 65
# and 64 + 64 + 1 (where the probability sums are folded)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,e,k,renorm", [(18945, 7, 1, True), (40000, 100, 16, False), (303104, 33, 2, True),
                                          (303105, 64, 4, False), (606209, 5, 3, True), (20001, 256, 8, False),
                                          (303200, 256, 8, True), (310000, 131, 2, False)])
def test_route_of_long_batches(cuda_device, dtype, n, e, k, renorm):
    g = torch.Generator(device=cuda_device).manual_seed(n)
    logits = torch.randn(n, e, generator=g, device=cuda_device) + torch.randn(1, e, generator=g, device=cuda_device)
    logits[::11, : e // 2] = -torch.inf       # fewer experts, for some fewer than k
    logits[5::1000] = -torch.inf              # none
    logits = logits.to(dtype)
    mask = (torch.rand(n, generator=g, device=cuda_device) < 0.9).to(torch.uint8)
    want, p, f = route_wide(logits, k, renorm, mask)
    got = sge.moe_route_fwd(logits, k, renorm=renorm, mask=mask)
    for name in ("ids", "counts", "offsets", "pos", "order"):
        assert torch.equal(getattr(got, name).long(), want[name]), name
    assert int(got.n_live) == int(want["n_live"])
    # as in check(): an fp32 subtraction (|l - max| <= 20 here), expf, the sum, division and product
    assert float(logits[logits > -torch.inf].abs().max()) < 10
    rel, tiny = (2 * (20 + 4) + 20) * U, 2.0 ** -120
    assert bool(((got.w.double() - want["w"]).abs() <= rel * want["w"] + tiny).all())
    # a probability sum: at most 64 rows and 32 warps in fp32, the rest in 64 bits
    assert abs(float(got.loss) - float(want["loss"])) <= (rel + (64 + 32 + 2) * U) * float(want["loss"])
    dw = torch.randn(n, k, generator=g, device=cuda_device)
    dloss = torch.tensor([0.37], device=cuda_device)
    dl = sge.moe_route_bwd(logits, got, dloss, dw, mask=mask).double()
    there, at = want["ids"] >= 0, want["ids"].clamp(min=0)
    dw64 = torch.where(there, dw.double(), 0.0)
    share = (0.37 * e * f / want["n_live"]).expand(n, e)
    live = (p.sum(1, keepdim=True) > 0).double()
    added = torch.zeros_like(p).scatter_add_(1, at, dw64) if not renorm else torch.zeros_like(p)
    dp = share * live + added
    # dloss is an fp32 number, 0.37 within U
    ref = p * (dp - (p * dp).sum(1, keepdim=True))
    size = p * ((share * live + added.abs()) + (p * (share * live + added.abs())).sum(1, keepdim=True))
    if renorm:
        w = want["w"]
        ref = ref.scatter_add(1, at, w * (dw64 - (w * dw64).sum(1, keepdim=True)))
        size = size.scatter_add(1, at, w * (dw64.abs() + (w * dw64.abs()).sum(1, keepdim=True)))
    out = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert bool(((dl - ref).abs() <= (2 * rel + 61 * U) * size + out * ref.abs() + tiny).all())


@pytest.mark.parametrize("n,e", [(2 ** 24 + 3, 5), (2 ** 22 + 1, 7)])
def test_route_loss_of_very_long_batches(cuda_device, n, e):
    """Equal logits: every token takes expert 0 and the loss is 1.  Each p is
    1 / e within two roundings, a sum of 64 of them within 64, every other sum
    is in 64 bits (fp32 sums of a warp's 3543 rows were off by 588 roundings)."""
    r = sge.moe_route_fwd(torch.zeros(n, e, device=cuda_device), 1)
    assert r.counts.tolist() == [n] + [0] * (e - 1) and int(r.n_live) == n
    assert torch.equal(r.pos.view(-1), torch.arange(n, device=cuda_device, dtype=torch.int32))
    assert torch.equal(r.order, torch.arange(n, device=cuda_device, dtype=torch.int32))
    assert abs(float(r.loss) - 1) <= (2 + 64 + 2) * U


def test_refused_route_leaves_its_output_as_it_was(cuda_device):
    """The gradient after a refused call is that of the route that is there."""
    logits = torch.randn(9, 6, device=cuda_device)
    r = sge.moe_route_fwd(logits, 2, renorm=True)
    dw = torch.randn(9, 2, device=cuda_device)
    want = sge.moe_route_bwd(logits, r, dw=dw)
    with pytest.raises(ValueError):
        sge.moe_route_fwd(logits, 3, renorm=False, out=r)
    with pytest.raises(ValueError):
        sge.moe_route_fwd(logits.half(), 2, renorm=False, out=r)
    with pytest.raises(sge.LibraryError, match="workspace"):
        sge.moe_route_fwd(logits, 2, renorm=False, out=r, workspace=torch.empty(16, dtype=torch.uint8, device=cuda_device))
    assert r.renorm and torch.equal(sge.moe_route_bwd(logits, r, dw=dw), want)

"""The feed-forward block on 8-bit weights, dense and over experts, on the
GPU against a plain restatement: the integers by their 32-bit definition,
everything after them in 64 bits.

Bound: the block sums are exact; adding them in fp32 costs at most one
rounding per term of F / 16 partial sums (the finest split any path uses) plus
32 for reductions, scales and weights, each at most U of the sum of the
magnitudes; a bf16 result adds 2^-8 of every expert's part and 2^-8 of y."""
import numpy as np
import pytest
import torch

import activation_sparse_gated_epilogue_b200 as sge
from tests._util import to_f64
from tests.test_gpu_int8 import quant_np, rows_np, upload

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
GROUP = 128


def f32_product(q, s, wq, sw):
    acc = (q.astype(np.float64) @ wq.astype(np.float64).T).astype(np.float32)
    return acc * s[:, None] * sw        # fp32, in this order


def block_np(x, wg, wu, wd):
    """(y, sum of magnitudes) of one block; weights as (integers, scales)."""
    q, s = quant_np(x)
    g, u = f32_product(q, s, *wg), f32_product(q, s, *wu)
    with np.errstate(invalid="ignore"):
        h = np.where(np.isnan(g), g, np.maximum(g, 0)) * u
    n, f = h.shape
    y, mag = 0.0, 0.0
    for c in range(0, f, GROUP):
        hq, hs = quant_np(h[:, c:c + GROUP])
        w = wd[0][:, c:c + GROUP].astype(np.float64)
        y = y + (hq.astype(np.float64) @ w.T) * hs.astype(np.float64)[:, None]
        mag = mag + (np.abs(hq).astype(np.float64) @ np.abs(w).T) * hs.astype(np.float64)[:, None]
    return y * wd[1].astype(np.float64), mag * wd[1].astype(np.float64)


class Experts:
    def __init__(self, rng, e, d, f, dev):
        self.e, self.d, self.f = e, d, f
        self.np, self.dev = [], []
        for rows, cols in ((f, d), (f, d), (d, f)):
            q, s, full = rows_np(rng, e * rows, cols, cols ** -0.5)
            self.np.append((q.reshape(e, rows, cols), s.reshape(e, rows)))
            self.dev.append(upload(full, s, cols, dev))

    def block(self, i, x):
        return block_np(x, *((q[i], s[i]) for q, s in self.np))


def tokens(rng, n, d, dtype):
    x = rng.standard_normal((n, d)) * np.exp(0.5 * rng.standard_normal((n, 1)))
    return torch.from_numpy(x).to(dtype)


def assert_close(y, want, mag, f, dtype, parts=None):
    out = 2.0 ** -8 * (np.abs(want) + (parts if parts is not None else 0)) if dtype == torch.bfloat16 else 0.0
    bound = (f / 16 + 32) * U * mag * (1 + 2.0 ** -8) + out + 1e-30
    bad = ~(np.abs(to_f64(y) - want) <= bound)
    assert not bad.any(), (np.abs(to_f64(y) - want)[bad][:3], bound[bad][:3], int(bad.sum()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d,f", [(1, 8, 8), (1, 256, 1024), (2, 264, 136), (5, 64, 128), (8, 512, 2048),
                                   (9, 200, 264), (33, 136, 520), (64, 256, 1024), (128, 512, 384),
                                   (129, 256, 640), (257, 384, 896), (600, 264, 1000), (300, 1024, 256),
                                   (2600, 1000, 264), (1300, 2048, 136)])
def test_dense_block(cuda_device, dtype, n, d, f):
    rng = np.random.default_rng(n + d + f)
    ex = Experts(rng, 1, d, f, cuda_device)
    x = tokens(rng, n, d, dtype)
    want, mag = ex.block(0, x.float().numpy())
    buf = torch.full((n * d + 512,), 7.0, dtype=dtype, device=cuda_device)
    y = buf[256:256 + n * d].view(n, d)
    diag = sge.new_diag(cuda_device)
    sge.int8_ffn_fwd(x.to(cuda_device), *ex.dev, y=y, diag=diag)
    torch.cuda.synchronize()
    assert_close(y, want, mag, f, dtype)
    assert (buf[:256] == 7).all() and (buf[256 + n * d:] == 7).all() and int(diag[3]) == 0


def run_experts(cuda_device, n, d, f, e, k, dtype, ids=None, seed=0, x=None):
    rng = np.random.default_rng(seed + n + d + f + e)
    ex = Experts(rng, e, d, f, cuda_device)
    x = tokens(rng, n, d, dtype) if x is None else x
    logits = torch.from_numpy(rng.standard_normal((n, e)).astype(np.float32))
    if ids is not None:                  # logits that choose these experts
        logits = torch.full((n, e), -float("inf"))
        for t in range(n):
            for j, i in enumerate(ids[t]):
                if i >= 0:
                    logits[t, i] = 1.0 - 0.25 * j
    r = sge.moe_route_fwd(logits.to(cuda_device), k)
    diag = sge.new_diag(cuda_device)
    y = sge.moe_int8_ffn_fwd(x.to(cuda_device), *ex.dev, r.w, r.offsets, r.pos, diag=diag)
    torch.cuda.synchronize()
    chosen, w = r.ids.cpu().numpy(), to_f64(r.w)
    want, mag, parts = np.zeros((n, d)), np.zeros((n, d)), np.zeros((n, d))
    for i in range(e):
        t, j = np.nonzero(chosen == i)
        if len(t):
            z, m = ex.block(i, x.float().numpy()[t])
            np.add.at(want, t, w[t, j][:, None] * z)
            np.add.at(mag, t, w[t, j][:, None] * m)
            np.add.at(parts, t, w[t, j][:, None] * np.abs(z))
    if ids is not None:
        assert chosen.tolist() == [list(a) for a in ids]
    assert int(diag[3]) == 0
    return y, want, mag, parts


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d,f,e,k", [(1, 64, 128, 2, 1), (1, 256, 512, 64, 8), (3, 136, 200, 5, 5),
                                       (4, 1024, 256, 32, 4), (17, 64, 136, 3, 2), (100, 256, 256, 8, 2),
                                       (300, 128, 384, 4, 2), (500, 264, 264, 256, 3), (1200, 128, 256, 3, 1),
                                       (700, 256, 520, 2, 2), (1300, 1544, 264, 2, 2), (2, 136, 264, 1, 1),
                                       (8, 64, 264, 16, 4), (7, 72, 136, 100, 16), (50, 64, 136, 1, 1)])
def test_experts(cuda_device, dtype, n, d, f, e, k):
    y, want, mag, parts = run_experts(cuda_device, n, d, f, e, k, dtype)
    assert_close(y, want, mag, f, dtype, parts)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 6, 40, 700])
def test_experts_uneven_loads_and_tokens_without_one(cuda_device, dtype, n):
    """All tokens on one expert, experts without any, tokens without any."""
    ids = [[2, -1] if t % 3 else [2, 4] for t in range(n)]
    ids[n // 2] = [-1, -1]
    y, want, mag, parts = run_experts(cuda_device, n, 128, 264, 5, 2, dtype, ids)
    assert_close(y, want, mag, 264, dtype, parts)
    assert (y[n // 2] == 0).all()


@pytest.mark.parametrize("n", [3, 20, 300])
def test_tokens_that_are_not_finite_or_zero(cuda_device, n):
    rng = np.random.default_rng(1)
    x = tokens(rng, n, 128, torch.float32)
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 9] = float("nan")
    ex = Experts(rng, 1, 128, 256, cuda_device)
    y = sge.int8_ffn_fwd(x.to(cuda_device), *ex.dev)
    assert (y[0] == 0).all() and torch.isnan(y[1:3]).all() and torch.isfinite(y[3:]).all()
    y, want, _, _ = run_experts(cuda_device, n, 128, 256, 4, 2, torch.float32, x=x)
    assert torch.isnan(y[1:3]).all() and torch.isfinite(y[3:]).all() and (y[0] == 0).all()


@pytest.mark.parametrize("n", [4, 30, 600])
def test_places_and_bounds_out_of_range_are_left_out(cuda_device, n):
    """A plan that does not fit: nothing outside the buffers is touched (the
    kernels clamp the bounds and skip the places), tokens with good places
    keep their values."""
    rng = np.random.default_rng(2)
    d, f, e, k = 64, 128, 3, 2
    ex = Experts(rng, e, d, f, cuda_device)
    x = tokens(rng, n, d, torch.float32).to(cuda_device)
    r = sge.moe_route_fwd(torch.randn(n, e, device=cuda_device), k)
    good = sge.moe_int8_ffn_fwd(x, *ex.dev, r.w, r.offsets, r.pos)
    pos = r.pos.clone()
    pos[0] = torch.tensor([n * k, 2 ** 31 - 1], dtype=torch.int32)
    pos[1] = torch.tensor([-5, -2 ** 31], dtype=torch.int32)
    y = sge.moe_int8_ffn_fwd(x, *ex.dev, r.w, r.offsets, pos)
    assert (y[:2] == 0).all() and torch.equal(y[2:], good[2:])
    for bad in ([0, n * k, 1, 7 * n], [-9, 2 ** 31 - 1, -2 ** 31, 5], [n * k] * 4):
        sge.moe_int8_ffn_fwd(x, *ex.dev, r.w, torch.tensor(bad, dtype=torch.int32, device=cuda_device), r.pos)
    torch.cuda.synchronize()
    assert torch.equal(sge.moe_int8_ffn_fwd(x, *ex.dev, r.w, r.offsets, r.pos), good)


@pytest.mark.parametrize("n", [2, 50, 700])
def test_repeats_workspaces_graphs_and_streams(cuda_device, n):
    rng = np.random.default_rng(3)
    d, f, e, k = 128, 256, 4, 2
    ex, one = Experts(rng, e, d, f, cuda_device), Experts(rng, 1, d, f, cuda_device)
    x = tokens(rng, n, d, torch.bfloat16).to(cuda_device)
    logits = torch.randn(n, e, device=cuda_device)

    def both(stream=None, ws=(None, None)):
        r = sge.moe_route_fwd(logits, k, stream=stream)
        return (sge.moe_int8_ffn_fwd(x, *ex.dev, r.w, r.offsets, r.pos, workspace=ws[0], stream=stream),
                sge.int8_ffn_fwd(x, *one.dev, workspace=ws[1], stream=stream))

    want = both()
    same = lambda got: torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])  # noqa: E731
    assert same(both())
    # a workspace that held other bytes
    ws = [torch.full_like(sge.int8_ffn_workspace(n, d, f, a, b, x.dtype, cuda_device), 255) for a, b in ((e, k), (1, 1))]
    assert same(both(ws=ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    torch.cuda.current_stream().wait_stream(side)
    assert same(got)
    torch.cuda.synchronize()
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(ws=ws)
    with torch.cuda.graph(graph2):       # the same workspaces, replayed in turn
        got2 = both(ws=ws)
    for g, out in ((graph, got), (graph2, got2), (graph, got)):
        g.replay()
        torch.cuda.synchronize()
        assert same(out)


def test_refusals(cuda_device):
    rng = np.random.default_rng(4)
    ex = Experts(rng, 2, 64, 128, cuda_device)
    one = Experts(rng, 1, 64, 128, cuda_device)
    x = torch.randn(4, 64, device=cuda_device)
    r = sge.moe_route_fwd(torch.randn(4, 2, device=cuda_device), 1)
    with pytest.raises(ValueError, match="rows"):
        sge.int8_ffn_fwd(x, *ex.dev)
    with pytest.raises(ValueError, match="columns"):
        sge.int8_ffn_fwd(x[:, :56].contiguous(), *one.dev)
    with pytest.raises(ValueError, match="pos"):
        sge.moe_int8_ffn_fwd(x, *ex.dev, r.w, r.offsets, r.pos[:3].contiguous())
    with pytest.raises(sge.LibraryError, match="workspace"):
        sge.int8_ffn_fwd(x, *one.dev, workspace=torch.empty(256, dtype=torch.uint8, device=cuda_device))
    with pytest.raises(ValueError, match="CUDA"):
        sge.int8_ffn_fwd(x.cpu(), *one.dev)
    assert sge.int8_ffn_fwd(x[:0], *one.dev).shape == (0, 64)


@pytest.mark.parametrize("n,d,f,e,k", [(300, 128, 384, 4, 2), (700, 256, 520, 2, 2), (1300, 1544, 264, 2, 2),
                                       (1200, 128, 256, 3, 1), (50, 64, 136, 1, 1), (4, 1024, 256, 32, 4),
                                       (40, 128, 2056, 4, 2), (300, 128, 384, 16, 8)])
def test_experts_results_are_rounded_once(cuda_device, n, d, f, e, k):
    """A bf16 y is the rounding of an fp32 sum over the experts on every path:
    whole and split down products, single CTAs and pairs, few tokens."""
    y, want, mag, _ = run_experts(cuda_device, n, d, f, e, k, torch.bfloat16)
    assert_close(y, want, mag, f, torch.bfloat16)


def guarded_call(ex, x, w, offsets, pos, fill):
    """moe_int8_ffn_fwd with y and the workspace inside larger buffers, whose
    other bytes must stay; the workspace is full of `fill` bytes."""
    n, d, e = x.shape[0], x.shape[1], ex.e
    need = sge.int8_ffn_workspace(n, d, ex.f, e, w.shape[1], x.dtype, x.device).numel()
    ws = torch.full((need + 512,), fill, dtype=torch.uint8, device=x.device)
    y = torch.full((n * d + 512,), 7.0, dtype=x.dtype, device=x.device)
    sge.moe_int8_ffn_fwd(x, *ex.dev, w, offsets, pos, y=y[256:256 + n * d].view(n, d), workspace=ws[256:256 + need])
    assert (ws[:256] == fill).all() and (ws[256 + need:] == fill).all()
    assert (y[:256] == 7).all() and (y[256 + n * d:] == 7).all()
    return y[256:256 + n * d].view(n, d).clone()


def as_bounds(values, rows, device):
    """Bounds as given, and the ascending ones that they stand for."""
    made = np.maximum.accumulate(np.clip(np.array(values, np.int64), 0, rows))
    return (torch.tensor(values, dtype=torch.int32, device=device),
            torch.tensor(made.tolist(), dtype=torch.int32, device=device))


@pytest.mark.parametrize("n,d", [(3, 64), (30, 64), (600, 64), (3000, 512)])
def test_bounds_out_of_order_stand_for_ascending_ones(cuda_device, n, d):
    """On every path (few tokens, single CTAs, pairs) an expert's rows begin
    where those of the experts before it end."""
    rng = np.random.default_rng(5)
    f, e, k = 128, 3, 2
    ex = Experts(rng, e, d, f, cuda_device)
    x = tokens(rng, n, d, torch.float32).to(cuda_device)
    r = sge.moe_route_fwd(torch.randn(n, e, device=cuda_device), k)
    rows = n * k
    for values in ([0, rows, 1, rows], [0, rows // 2, rows // 3, rows], [0, -5, rows, 7 * n],
                   [0, 2 ** 31 - 1, -2 ** 31, 5], [0, 1, 0, rows]):
        bad, good = as_bounds(values, rows, cuda_device)
        want = guarded_call(ex, x, r.w, good, r.pos, 0)
        for fill in (0, 255):
            assert torch.equal(guarded_call(ex, x, r.w, bad, r.pos, fill), want), values


@pytest.mark.parametrize("n,d", [(3, 64), (30, 64), (600, 64), (3000, 512)])
def test_places_in_no_experts_rows_add_nothing(cuda_device, n, d):
    """Bounds that leave rows out at either end: on every path a token's sum is
    over the places that an expert has, whatever the workspace held."""
    rng = np.random.default_rng(6)
    f, e, k = 128, 3, 2
    ex = Experts(rng, e, d, f, cuda_device)
    x = tokens(rng, n, d, torch.float32).to(cuda_device)
    r = sge.moe_route_fwd(torch.randn(n, e, device=cuda_device), k)
    rows = n * k
    pos, w, x64 = r.pos.cpu().numpy(), to_f64(r.w), x.cpu().numpy()
    for values in ([rows // 4, rows // 2, rows // 2, 3 * rows // 4], [0, 1, 1, 1], [rows] * 4, [0] * 4,
                   [rows // 2, 0, rows // 3, rows // 2 + 1]):
        bounds, ascending = as_bounds(values, rows, cuda_device)
        want, mag = np.zeros((n, d)), np.zeros((n, d))
        lo = ascending.tolist()
        for i in range(e):
            t, j = np.nonzero((pos >= lo[i]) & (pos < lo[i + 1]))
            if len(t):
                z, m = ex.block(i, x64[t])
                np.add.at(want, t, w[t, j][:, None] * z)
                np.add.at(mag, t, w[t, j][:, None] * m)
        for fill in (0, 255):
            y = guarded_call(ex, x, r.w, bounds, r.pos, fill)
            assert_close(y, want, mag, f, torch.float32)


def test_refusals_are_value_errors(cuda_device):
    ex = Experts(np.random.default_rng(4), 2, 64, 128, cuda_device)
    x = torch.randn(4, 64, device=cuda_device)
    r = sge.moe_route_fwd(torch.randn(4, 2, device=cuda_device), 1)
    with pytest.raises(ValueError, match="dtype"):
        sge.moe_int8_ffn_fwd(x.half(), *ex.dev, r.w, r.offsets, r.pos)
    with pytest.raises(ValueError, match="w must"):
        sge.moe_int8_ffn_fwd(x, *ex.dev, r.w.view(-1), r.offsets, r.pos)
    for offsets in (r.offsets[0], r.offsets[:1], r.offsets[None]):
        with pytest.raises(ValueError, match="offsets"):
            sge.moe_int8_ffn_fwd(x, *ex.dev, r.w, offsets, r.pos)

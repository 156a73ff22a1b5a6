"""The router, the 8-bit products and the blocks of the framework together,
as a serving loop and as a training step use them; two calls at once; the
debug build; the bounded waits of the 8-bit engine."""
import ctypes
import os
import subprocess
import sys
import time

import numpy as np
import pytest
import torch

import activation_sparse_gated_epilogue_b200 as sge
from activation_sparse_gated_epilogue_b200 import build as sge_build
from activation_sparse_gated_epilogue_b200 import synth
from tests._util import BF16_TOL, to_f64
from tests.test_gpu_debug import SGE_FLAG_BOUNDS, library_at
from tests.test_gpu_int8_ffn import Experts, assert_close, run_experts, tokens
from tests.test_gpu_timeout import _selftest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 5, 200])
def test_serving_loop_in_a_graph(cuda_device, n):
    """One captured step (router product in 8 bits, route, experts), replayed
    on new tokens, equals the same calls made one by one."""
    rng = np.random.default_rng(n)
    d, f, e, k = 256, 384, 8, 2
    ex = Experts(rng, e, d, f, cuda_device)
    w_router = sge.int8_quant_rows(torch.from_numpy(rng.standard_normal((e, d)).astype(np.float32)).to(cuda_device))
    x = torch.zeros(n, d, dtype=torch.bfloat16, device=cuda_device)

    def step(x):
        logits = sge.int8_linear(sge.int8_quant_rows(x), w_router, torch.float32)
        r = sge.moe_route_fwd(logits, k)
        return r, sge.moe_int8_ffn_fwd(x, *ex.dev, r.w, r.offsets, r.pos)

    step(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, y = step(x)
    for s in range(3):
        new = tokens(np.random.default_rng(100 + s), n, d, torch.bfloat16)
        x.copy_(new)
        graph.replay()
        r2, y2 = step(new.to(cuda_device))
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(r.ids, r2.ids) and torch.equal(r.loss, r2.loss)


def test_training_step_of_experts(cuda_device):
    """Router forward; each expert's tokens through twell_gate_pack,
    hybrid_pack, hybrid_ffn_fwd and _bwd; router backward.  The gradient of
    <dy, y> + dloss * balance loss with respect to the logits against 64-bit
    autograd of the same formula (the bf16 bar of the blocks)."""
    n, e, k, d, f, tile = 600, 3, 2, 256, 1024, 128
    cfg = synth.CONFIGS["ffn_0p5b_bf16"].with_(n_tokens=n, d_model=d, d_ff=f, rho=0.05)
    inps = [synth.make_inputs(cfg.with_(seed=s)) for s in range(e)]
    x = inps[0].x.to(cuda_device)
    weights = [[getattr(i, name).to(cuda_device) for name in ("wg_t", "wu_t", "wd")] for i in inps]
    g = torch.Generator().manual_seed(1)
    logits = torch.randn(n, e, generator=g)
    dy = torch.randn(n, d, generator=g).to(torch.bfloat16)
    dloss = torch.tensor([2.0])
    route = sge.moe_route_fwd(logits.to(cuda_device), k)
    offsets, order = route.offsets.tolist(), route.order.long()
    y_of = torch.zeros(n * k, d, device=cuda_device)
    dx = torch.zeros(n, d, device=cuda_device)
    for i, (wg, wu, wd) in enumerate(weights):
        at = order[offsets[i]:offsets[i + 1]]
        xe = x[at // k]
        hy = sge.hybrid_pack(sge.twell_gate_pack(xe, wg, tile, tile), 64, len(at))
        y_of[at] = sge.hybrid_ffn_fwd(xe, hy, wu, wd, wd.t().contiguous()).float()
        dye = (route.w.view(-1)[at][:, None] * dy.to(cuda_device)[at // k].float()).to(torch.bfloat16)
        dxe = sge.hybrid_ffn_bwd(xe, dye, hy, wg, wu, wd)[0]
        dx.index_add_(0, at // k, dxe.float())
    dw = (y_of.view(n, k, d) * dy.to(cuda_device).float()[:, None]).sum(2)
    dlogits = sge.moe_route_bwd(logits.to(cuda_device), route, dloss.to(cuda_device), dw)

    x64 = x.cpu().double().requires_grad_()
    l64 = logits.double().requires_grad_()
    ids = torch.argsort(-l64.detach(), dim=1, stable=True)[:, :k]
    w64 = torch.softmax(l64.gather(1, ids), 1)
    counts = torch.bincount(ids.reshape(-1), minlength=e).double()
    p = torch.softmax(l64, 1)
    total = dloss.item() * e * (counts / counts.sum() * p.mean(0)).sum()
    for i, (wg, wu, wd) in enumerate(weights):
        wg, wu, wd = (t.cpu().double() for t in (wg, wu, wd))
        block = (torch.relu(x64 @ wg.T) * (x64 @ wu.T)) @ wd
        share = (w64 * (ids == i)).sum(1, keepdim=True)
        total = total + (share * block * dy.double()).sum()
    total.backward()
    for got, want in ((dlogits, l64.grad), (dx, x64.grad)):
        want = want.numpy()
        assert np.abs(to_f64(got) - want).max() <= BF16_TOL * np.abs(want).max()


def test_two_calls_at_once(cuda_device):
    """Calls on two streams, each with its own workspace, do not disturb one
    another: the results equal those of calls made alone."""
    rng = np.random.default_rng(7)
    sizes = [(700, 256, 520, 4, 2), (6, 128, 264, 8, 4)]
    made = []
    for n, d, f, e, k in sizes:
        ex = Experts(rng, e, d, f, cuda_device)
        x = tokens(rng, n, d, torch.bfloat16).to(cuda_device)
        logits = torch.randn(n, e, device=cuda_device)
        made.append((ex, x, logits, k))

    def call(ex, x, logits, k, stream=None):
        r = sge.moe_route_fwd(logits, k, stream=stream)
        return sge.moe_int8_ffn_fwd(x, *ex.dev, r.w, r.offsets, r.pos, stream=stream)

    want = [call(*m) for m in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(20):
        got.append([call(*m, stream=s) for m, s in zip(made, streams)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for pair in got for a, b in zip(pair, want))


def test_first_calls_of_a_process_in_a_capture(cuda_device):
    """Nothing that a first call sets up (limits, attributes, occupancy) breaks
    the capture of a graph: a fresh process captures before it calls anything."""
    code = """
import torch
import activation_sparse_gated_epilogue_b200 as sge
def rows(r, c):
    return sge.Int8Rows(torch.randint(-127, 128, (r, c), dtype=torch.int8, device="cuda"),
                        torch.rand(r, device="cuda") * 0.01, c)
x, logits = torch.randn(3000, 1024, device="cuda"), torch.randn(3000, 64, device="cuda")
w, block = rows(512, 1024), [rows(512, 1024), rows(512, 1024), rows(1024, 512)]
def run():
    r = sge.moe_route_fwd(logits, 4)
    q = sge.int8_quant_rows(x)
    tw = sge.twell_gate_pack_int8(q, w, 128, 128)
    return [sge.int8_linear(q, w, torch.float32), sge.int8_ffn_fwd(x, *block), r.order, tw.count,
            sge.moe_route_bwd(logits, r, torch.ones_like(r.loss))]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, run()))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert done.returncode == 0, done.stderr[-2000:]


def test_debug_build_gives_the_same_bits_and_flags_bad_plans(cuda_device):
    path = sge_build.LIB_DEBUG
    assert os.path.exists(path)
    rng = np.random.default_rng(8)
    d, f, e, k = 1024, 264, 5, 2
    ex = Experts(rng, e, d, f, cuda_device)
    one = torch.ones(1, device=cuda_device)
    for n in (3, 40, 3000):            # few tokens, single CTAs, CTA pairs
        x = tokens(rng, n, d, torch.float32).to(cuda_device)
        logits = torch.randn(n, e, device=cuda_device)
        dw = torch.randn(n, k, device=cuda_device)

        def run():
            r = sge.moe_route_fwd(logits, k)
            return [sge.moe_int8_ffn_fwd(x, *ex.dev, r.w, r.offsets, r.pos),
                    sge.moe_route_bwd(logits, r, one, dw), r.pos, r.offsets, r.w]

        want = run()
        with library_at(path):
            sge.debug_flags(clear=True)
            got = run()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            assert sge.debug_flags(clear=True) == 0
            pos = want[2].clone()
            pos[0, 0] = n * k + 3
            y = sge.moe_int8_ffn_fwd(x, *ex.dev, want[4], want[3], pos)
            torch.cuda.synchronize()
            assert sge.debug_flags(clear=True) & SGE_FLAG_BOUNDS
            assert torch.equal(y[1:], want[0][1:])


@pytest.mark.parametrize("pair", [2, 3])
def test_bounded_wait_of_the_8_bit_engine_runs_out(cuda_device, pair):
    """A stage barrier that can never complete (its copies are in bounds): the
    wait runs out, the kernel reports it, drains and returns."""
    st = _selftest()
    m, n, k = 512, 512, 512
    a = torch.zeros(m, k, dtype=torch.int8, device=cuda_device)
    b = torch.zeros(n, k, dtype=torch.int8, device=cuda_device)
    diag = sge.new_diag(cuda_device)
    tiles = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    stream = ctypes.c_void_p(torch.cuda.current_stream(cuda_device).cuda_stream)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert st.sge_selftest_wait_timeout(pair, ctypes.c_void_p(a.data_ptr()), ctypes.c_void_p(b.data_ptr()), m, n, k,
                                        ctypes.c_void_p(diag.data_ptr()), ctypes.c_void_p(tiles.data_ptr()),
                                        stream) == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    assert int(diag[3]) & 1 and int(tiles) == 0
    y, want, mag, parts = run_experts(cuda_device, 300, 128, 256, 3, 2, torch.float32)
    assert_close(y, want, mag, 256, torch.float32, parts)


@pytest.mark.parametrize("pair", [4, 5, 6, 7])
def test_bounded_waits_of_the_blocks_products_run_out(cuda_device, pair):
    """The same for the shapes of the feed-forward block: two B loads a stage
    (4, 5: single CTA, pairs), and the block-by-block sums (6, 7), whose epilogue
    waits on the stages and has copies of its scales in flight."""
    st = _selftest()
    m, n, k = 512, 512, 2048
    a = torch.zeros(m, k, dtype=torch.int8, device=cuda_device)
    b = torch.zeros(n, k, dtype=torch.int8, device=cuda_device)
    diag = sge.new_diag(cuda_device)
    tiles = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    stream = ctypes.c_void_p(torch.cuda.current_stream(cuda_device).cuda_stream)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert st.sge_selftest_wait_timeout(pair, ctypes.c_void_p(a.data_ptr()), ctypes.c_void_p(b.data_ptr()), m, n, k,
                                        ctypes.c_void_p(diag.data_ptr()), ctypes.c_void_p(tiles.data_ptr()),
                                        stream) == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    assert int(diag[3]) & 1 and int(tiles) == 0
    for tokens_n, d, f in ((300, 128, 1280), (3000, 512, 1280)):     # single CTAs, pairs
        y, want, mag, _ = run_experts(cuda_device, tokens_n, d, f, 3, 2, torch.float32)
        assert_close(y, want, mag, f, torch.float32)

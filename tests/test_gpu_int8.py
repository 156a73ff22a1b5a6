"""8-bit integer products on the GPU against plain 64-bit restatements: the
quantiser, int8_linear and twell_gate_pack_int8.

Integers are compared exactly.  An fp32 output is the exact integer sum after
three roundings (to fp32, times a scale, times a scale), a bf16 output after
one more: |y - y64| <= (3 * 2^-24 [+ 2^-8]) |y64| with a margin of 2^-20 for
the products of these small terms."""
import numpy as np
import pytest
import torch

import activation_sparse_gated_epilogue_b200 as sge
from activation_sparse_gated_epilogue_b200 import synth
from tests._util import to_f64, twell_host

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -100


def quant_np(x: np.ndarray):
    """int8 rows and fp32 scales of fp32 rows, numpy fp32 arithmetic."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(-1, keepdims=True)
        bad = ~np.isfinite(x).all(-1, keepdims=True)
        zero = (amax < TINY) | bad
        inv = np.where(zero, np.float32(0), np.float32(127) / np.where(zero, np.float32(1), amax))
        q = np.where(zero, np.float32(0), np.rint(np.where(bad, np.float32(0), x) * inv.astype(np.float32)))
        scale = np.where(bad, np.float32(np.nan), np.where(amax < TINY, np.float32(0), amax / np.float32(127)))
    return q.astype(np.int8), scale[..., 0].astype(np.float32)


def rows_np(rng, rows, cols, std=1.0, mean=0.0):
    """Random int8 rows as an Int8Rows whose padding bytes are not zero."""
    q, s = quant_np(rng.standard_normal((rows, cols)) * std + mean)
    pad = -cols % 16
    full = np.concatenate([q, rng.integers(-127, 128, (rows, pad)).astype(np.int8)], 1)
    return q, s, full


def upload(full, s, cols, dev):
    return sge.Int8Rows(torch.from_numpy(full).to(dev), torch.from_numpy(s).to(dev), cols)


def product64(xq, sx, wq, sw):
    return (xq.astype(np.float64) @ wq.astype(np.float64).T) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d", [(1, 1), (1, 8), (3, 7), (5, 16), (9, 130), (33, 2048), (8, 2056), (2, 5001),
                                 (7, 4096), (1, 20000)])
def test_quant_rows_gives_the_defined_integers(cuda_device, dtype, n, d):
    g = torch.Generator().manual_seed(n * 7 + d)
    x = (torch.randn(n, d, generator=g) * torch.exp(torch.randn(n, 1, generator=g) * 3)).to(dtype)
    q, s = quant_np(x.float().numpy())
    got = sge.int8_quant_rows(x.to(cuda_device))
    np.testing.assert_array_equal(got.q.cpu().numpy()[:, :d], q)
    np.testing.assert_array_equal(got.q.cpu().numpy()[:, d:], 0)
    np.testing.assert_array_equal(got.scale.cpu().numpy(), s)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quant_rows_special_rows(cuda_device, dtype):
    x = torch.ones(9, 40)
    x[0] = 0.0
    x[1] = -0.0
    x[2, 3] = float("inf")
    x[3, 39] = float("-inf")
    x[4, 0] = float("nan")
    x[5] = 2.0 ** -101          # below the smallest magnitude that is kept
    x[6] = torch.linspace(-1, 1, 40) * 2.0 ** -99
    x[7] = torch.linspace(-1, 1, 40) * 3.0e38
    x[8] = torch.arange(40) - 127.0 + 0.5    # ties
    x = x.to(dtype)
    q, s = quant_np(x.float().numpy())
    got = sge.int8_quant_rows(x.to(cuda_device))
    np.testing.assert_array_equal(got.q.cpu().numpy()[:, :40], q)
    np.testing.assert_array_equal(got.scale.cpu().numpy(), s)
    assert np.isnan(s[2:5]).all() and (s[[0, 1, 5]] == 0).all()


@pytest.mark.parametrize("ld,off", [(72, 0), (72, 8), (67, 0)])
def test_quant_rows_of_strided_rows(cuda_device, ld, off):
    base = torch.randn(11, ld, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(cuda_device)
    x = base[:, off:off + 56]
    q, s = quant_np(x.float().cpu().numpy())
    got = sge.int8_quant_rows(x)
    np.testing.assert_array_equal(got.q.cpu().numpy()[:, :56], q)
    np.testing.assert_array_equal(got.scale.cpu().numpy(), s)


def assert_scaled(y, y64, dtype):
    rel = 3 * 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    assert np.all(np.abs(to_f64(y) - y64) <= rel * (1 + 2.0 ** -20) * np.abs(y64))


LINEAR = [(1, 64, 64), (1, 1, 1), (2, 2048, 300), (3, 33, 17), (8, 1000, 129), (9, 128, 64), (17, 250, 1000),
          (64, 2048, 512), (65, 96, 65), (128, 400, 256), (129, 129, 200), (200, 2049, 511), (256, 256, 256),
          (257, 1024, 777), (300, 100, 8), (513, 513, 513), (1000, 2560, 300), (2049, 130, 1025)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d,m", LINEAR)
def test_linear_matches_the_exact_product(cuda_device, dtype, n, d, m):
    rng = np.random.default_rng(n + 3 * d + 5 * m)
    xq, sx, xf = rows_np(rng, n, d)
    wq, sw, wf = rows_np(rng, m, d, d ** -0.5)
    diag = sge.new_diag(cuda_device)
    # the output lies inside a larger buffer whose other bytes must stay
    buf = torch.full((n * m + 512,), 7.0, dtype=dtype, device=cuda_device)
    y = buf[256:256 + n * m].view(n, m)
    sge.int8_linear(upload(xf, sx, d, cuda_device), upload(wf, sw, d, cuda_device), dtype, y=y, diag=diag)
    torch.cuda.synchronize()
    assert_scaled(y, product64(xq, sx, wq, sw), dtype)
    assert (buf[:256] == 7).all() and (buf[256 + n * m:] == 7).all()
    assert int(diag[3]) == 0


@pytest.mark.parametrize("n", [1, 4, 40, 300])
def test_linear_extreme_integers_are_exact(cuda_device, n):
    """Sums at the 32-bit bound: all products +-127 * 127."""
    d, m = 16384, 160
    sign = torch.where(torch.arange(m) % 2 == 0, 1, -1).to(torch.int8)
    x = torch.full((n, d), 127, dtype=torch.int8, device=cuda_device)
    w = (torch.full((m, d), 127, dtype=torch.int8) * sign[:, None]).to(cuda_device)
    one = lambda k: torch.ones(k, device=cuda_device)  # noqa: E731
    y = sge.int8_linear(sge.Int8Rows(x, one(n), d), sge.Int8Rows(w, one(m), d), torch.float32)
    want = (sign.double() * 127 * 127 * d).expand(n, m)
    assert torch.equal(y.cpu().double(), want.float().double())


@pytest.mark.parametrize("n", [1, 2, 40, 300])
def test_linear_longest_rows_of_the_lowest_integer(cuda_device, n):
    """k = 131071 products of -128 * -128, the largest sum that is allowed."""
    d, m = 131071, 40
    low = lambda r: sge.Int8Rows(torch.full((r, d + 1), -128, dtype=torch.int8, device=cuda_device),  # noqa: E731
                                 torch.ones(r, device=cuda_device), d)
    y = sge.int8_linear(low(n), low(m), torch.float32)
    assert (y.double() == torch.tensor(128.0 * 128 * d).float().double().item()).all()


def test_linear_row_that_is_not_finite_gives_nan(cuda_device):
    x = torch.randn(5, 64, device=cuda_device)
    x[2, 7] = float("inf")
    x[4, 0] = float("nan")
    x[1] = 0
    wq = sge.int8_quant_rows(torch.randn(32, 64, device=cuda_device))
    y = sge.int8_linear(sge.int8_quant_rows(x), wq, torch.float32)
    nan = torch.isnan(y).all(1).tolist()
    assert nan == [False, False, True, False, True]
    assert (y[1] == 0).all() and torch.isfinite(y[[0, 1, 3]]).all()


def test_offsets_past_32_bits(cuda_device):
    """Outputs and inputs of more than 2^31 elements: the last rows and
    columns, and the first ones, which a wrapped offset would overwrite."""
    n, d, m = 33000, 64, 66000
    x = torch.randn(n, d, device=cuda_device)
    w = torch.randn(m, d, device=cuda_device)
    xq, wq = sge.int8_quant_rows(x), sge.int8_quant_rows(w)
    y = sge.int8_linear(xq, wq, torch.bfloat16)
    host = lambda r: (r.q.cpu().numpy(), r.scale.cpu().numpy())  # noqa: E731
    (q, s), (p, t) = host(xq), host(wq)
    for rows in (slice(0, 3), slice(16000, 16003), slice(n - 3, n)):
        for cols in (slice(0, 300), slice(m - 300, m)):
            assert_scaled(y[rows, cols], product64(q[rows], s[rows], p[cols], t[cols]), torch.bfloat16)
    big = y[:, :65536].contiguous()                     # 2^31 elements and more to quantise
    got = sge.int8_quant_rows(big)
    for rows in (slice(0, 2), slice(n - 2, n)):
        q, s = quant_np(big[rows].float().cpu().numpy())
        np.testing.assert_array_equal(got.q[rows].cpu().numpy(), q)
        np.testing.assert_array_equal(got.scale[rows].cpu().numpy(), s)


def test_linear_empty_batch_and_repeats(cuda_device):
    wq = sge.int8_quant_rows(torch.randn(32, 64, device=cuda_device))
    x = sge.int8_quant_rows(torch.randn(300, 64, device=cuda_device))
    assert torch.equal(sge.int8_linear(x, wq), sge.int8_linear(x, wq))
    e = sge.int8_quant_rows(torch.randn(0, 64, device=cuda_device))
    assert sge.int8_linear(e, wq).shape == (0, 32)


def test_quant_and_linear_captured_in_a_graph_and_on_another_stream(cuda_device):
    x = torch.randn(70, 264, device=cuda_device)
    wq = sge.int8_quant_rows(torch.randn(96, 264, device=cuda_device))
    want = sge.int8_linear(sge.int8_quant_rows(x), wq, torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sge.int8_linear(sge.int8_quant_rows(x, stream=side), wq, torch.float32, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    keep = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        y = sge.int8_linear(sge.int8_quant_rows(keep), wq, torch.float32)
    keep.copy_(x)
    graph.replay()
    assert torch.equal(y, want)


def twell_np(g, tile, cap):
    n, f = g.shape
    on = (g > 0).reshape(n, f // tile, tile)
    count = on.sum(2)
    idx = np.sort(np.where(on, np.arange(tile), tile), 2)[:, :, :cap]
    return count, idx


@pytest.mark.parametrize("tile,cap", [(16, 16), (16, 3), (32, 32), (32, 5), (64, 64), (128, 128), (128, 8)])
@pytest.mark.parametrize("n,d,f", [(1, 64, 128), (7, 100, 384), (64, 2048, 1024), (129, 257, 128),
                                   (257, 512, 640), (600, 96, 1152)])
def test_gate_pack_int8(cuda_device, tile, cap, n, d, f):
    rng = np.random.default_rng(tile + cap + n)
    xq, sx, xf = rows_np(rng, n, d, mean=0.3)
    wq, sw, wf = rows_np(rng, f, d, d ** -0.5, -2.0 / d)
    sw[::7] = 0.0                       # a channel of zeros is never active
    g = product64(xq, sx, wq, sw)
    count, idx = twell_np(g, tile, cap)
    out = sge.TwELL(*(torch.full((n, f // tile) + t, 77, dtype=k, device=cuda_device) for t, k in
                      (((), torch.uint8), ((cap,), torch.uint8), ((cap,), torch.bfloat16))), tile, cap)
    diag = sge.new_diag(cuda_device)
    sge.twell_gate_pack_int8(upload(xf, sx, d, cuda_device), upload(wf, sw, d, cuda_device), tile, cap, out=out,
                             diag=diag)
    c, i, v = twell_host(out)
    np.testing.assert_array_equal(c, count)
    keep = idx < tile
    np.testing.assert_array_equal(i[keep], idx[keep])
    r, b, k = np.nonzero(keep)
    want = g[r, b * tile + idx[r, b, k]]
    assert np.all(np.abs(v[keep] - want) <= (2.0 ** -8 + 4 * 2.0 ** -24) * want)
    assert (i[~keep] == 77).all() and (v[~keep] == 77).all()      # slots past the count: untouched
    assert int(diag[0]) == int((count > cap).sum()) and int(diag[3]) == 0


def test_gate_pack_int8_feeds_the_up_down_calls(cuda_device):
    """quantise -> 8-bit gate -> routed up/down, the sparse forward with an
    8-bit gate, against the same formula in 64 bits (bf16 bar of the up/down
    calls: h rounded to bf16, y rounded to bf16)."""
    cfg = synth.CONFIGS["ffn_0p5b_bf16"].with_(n_tokens=300, d_model=256, d_ff=1024, rho=0.05, seed=4)
    inp = synth.make_inputs(cfg)
    x, wg, wu, wd = (getattr(inp, k).to(cuda_device) for k in ("x", "wg_t", "wu_t", "wd"))
    xq, wq = sge.int8_quant_rows(x), sge.int8_quant_rows(wg)
    tw = sge.twell_gate_pack_int8(xq, wq, 128, 128)
    y = sge.twell_hybrid_up_down(x, tw, wu, wd, wd.t().contiguous(), 16, 64)
    y2 = sge.twell_fused_up_down(x, tw, wu, wd)
    (q1, s1), (q2, s2) = quant_np(x.float().cpu().numpy()), quant_np(wg.float().cpu().numpy())
    a = np.maximum(product64(q1, s1, q2, s2), 0)
    want = (a * (to_f64(x) @ to_f64(wu).T)) @ to_f64(wd)
    top = np.abs(want).max()
    for got in (y, y2):
        assert np.abs(to_f64(got) - want).max() / top <= 2e-2


def test_refusals(cuda_device):
    x = torch.randn(4, 64, device=cuda_device)
    xq = sge.int8_quant_rows(x)
    with pytest.raises(ValueError, match="columns"):
        sge.int8_linear(xq, sge.int8_quant_rows(torch.randn(4, 72, device=cuda_device)))
    with pytest.raises(ValueError, match="pitch"):
        sge.int8_linear(xq, sge.Int8Rows(xq.q[:, :8].contiguous(), xq.scale, 8))
    with pytest.raises(ValueError):
        sge.int8_quant_rows(x.half())
    with pytest.raises(ValueError, match="contiguous rows"):
        sge.int8_quant_rows(x.t())
    with pytest.raises(sge.LibraryError, match="tile"):
        sge.twell_gate_pack_int8(xq, sge.int8_quant_rows(torch.randn(96, 64, device=cuda_device)), 48, 48)


# tiles of 128 rows on the 148 SMs: 64 columns while that gives every SM at most
# one, 128 columns while those do, pairs beyond; on each, short and ragged sizes
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d,m", [(1000, 300, 1100), (3, 64, 9472), (18900, 65, 33),          # 64 columns
                                   (3, 64, 9473), (200, 129, 4801), (2000, 96, 1000),          # 128 columns
                                   (700, 129, 3300), (257, 256, 6500), (19000, 65, 33), (5000, 100, 500)])  # pairs
def test_linear_on_every_tile_shape(cuda_device, dtype, n, d, m):
    test_linear_matches_the_exact_product(cuda_device, dtype, n, d, m)


@pytest.mark.parametrize("tile,cap", [(16, 5), (128, 128)])
@pytest.mark.parametrize("n,d,f", [(1300, 96, 1152), (2049, 96, 1280), (140, 257, 9600), (18944, 40, 128),
                                   (18945, 40, 128)])
def test_gate_pack_int8_on_every_tile_shape(cuda_device, tile, cap, n, d, f):
    test_gate_pack_int8(cuda_device, tile, cap, n, d, f)


def test_linear_longest_rows_of_the_lowest_integer_on_pairs(cuda_device):
    n, d, m = 300, 131071, 6500
    low = lambda r: sge.Int8Rows(torch.full((r, d + 1), -128, dtype=torch.int8, device=cuda_device),  # noqa: E731
                                 torch.ones(r, device=cuda_device), d)
    y = sge.int8_linear(low(n), low(m), torch.float32)
    assert (y.double() == torch.tensor(128.0 * 128 * d).float().double().item()).all()

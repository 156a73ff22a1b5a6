"""The feed-forward block on 8-bit weights at the lengths it is built for: long
hidden rows on every path, buffers past 2^31 bytes, as many experts as there may
be.  Which path a case takes is part of it: the need that the call itself names
tells few tokens (no partial results) and the number of splits of the down
product; CTA pairs are told by the rule in `pairs`."""
import ctypes

import numpy as np
import pytest
import torch

import activation_sparse_gated_epilogue_b200 as sge
from activation_sparse_gated_epilogue_b200.binding import library
from tests.test_gpu_int8_ffn import Experts, assert_close, run_experts, tokens

pytestmark = pytest.mark.gpu
FEW = 0


def down_splits(n, d, f, e, k, routed):
    """FEW, or the parts of the down product, from the workspace's need."""
    lib, p = library(), ctypes.c_void_p(4096)
    args = ([p] * 11 + [n, d, f, e, k]) if routed else ([p] * 8 + [n, d, f])
    call = lib.moe_int8_ffn_fwd if routed else lib.int8_ffn_fwd
    assert call(*args, sge.SGE_F32, p, 0, None, None) == 1     # refused: a workspace of 0 bytes
    need = int(lib.sge_last_error().decode().split(",")[1].split()[0])
    up = lambda b, to: -(-b // to) * to  # noqa: E731
    rows, blocks = (n * k if routed else n), -(-f // 128)
    fixed = sum(up(b, 256) for b in (rows * up(d, 16), rows * 4, rows * up(f, 16), rows * blocks * 4))
    z = need - fixed
    if z == 0:
        return FEW if routed else None      # dense: few tokens, or y is written by the down product
    splits = z // (rows * d * 4)
    assert splits >= 1 and up(splits * rows * d * 4, 256) == z
    return splits


def pairs(rows, d, e):
    return rows // e > 512 and rows // 256 * -(-d // 256) >= 40


# hidden blocks of 128 in a tile of the down product: 25 on pairs; 17, 9 and 8 or
# fewer (split) on single CTAs; three pieces of a row on the few-token kernels
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d,f,splits,paired", [(2600, 1000, 3080, None, True), (600, 1928, 2056, None, False),
                                                 (40, 128, 16400, 15, False), (200, 264, 4104, 7, False),
                                                 (1, 256, 4104, None, False), (2, 136, 6152, None, False)])
def test_dense_block_with_long_hidden_rows(cuda_device, dtype, n, d, f, splits, paired):
    assert down_splits(n, d, f, 1, 1, False) == splits and pairs(n, d, 1) == paired
    rng = np.random.default_rng(n + d + f)
    ex = Experts(rng, 1, d, f, cuda_device)
    x = tokens(rng, n, d, dtype)
    want, mag = ex.block(0, x.float().numpy())
    diag = sge.new_diag(cuda_device)
    y = sge.int8_ffn_fwd(x.to(cuda_device), *ex.dev, diag=diag)
    torch.cuda.synchronize()
    assert_close(y, want, mag, f, dtype)
    assert int(diag[3]) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("uneven", [False, True])
@pytest.mark.parametrize("n,d,f,e,k,splits,paired", [(2600, 520, 3080, 3, 2, 1, True), (600, 776, 2056, 4, 2, 1, False),
                                                     (40, 128, 2056, 4, 2, 4, False), (60, 264, 8200, 5, 3, 8, False),
                                                     (4, 256, 4104, 32, 4, FEW, False), (8, 128, 6152, 8, 2, FEW, False),
                                                     (1, 264, 4104, 4, 3, FEW, False)])
def test_experts_with_long_hidden_rows(cuda_device, dtype, uneven, n, d, f, e, k, splits, paired):
    """Even loads, and nearly all tokens on one expert (some with fewer experts
    than they may have, one expert without any)."""
    assert down_splits(n, d, f, e, k, True) == splits and pairs(n * k, d, e) == paired
    ids = None
    if uneven:
        others = [i for i in range(e) if i != 2]
        ids = [([2] + (others[:k - 1] if t % 7 == 0 else [-1] * (k - 1)))[:k] for t in range(n)]
    y, want, mag, _ = run_experts(cuda_device, n, d, f, e, k, dtype, ids)
    assert_close(y, want, mag, f, dtype)


def test_256_experts_on_cta_pairs(cuda_device):
    n, d, f, e = 140000, 64, 136, 256
    assert pairs(n, d, e) and down_splits(n, d, f, e, 1, True) == 1
    y, want, mag, _ = run_experts(cuda_device, n, d, f, e, 1, torch.bfloat16)
    assert_close(y, want, mag, f, torch.bfloat16)


def test_block_offsets_past_32_bits(cuda_device):
    """Hidden rows and experts' results of more than 2^31 bytes: the tokens at
    either end, around the byte 2^31 of both buffers, and where the second
    expert's rows begin."""
    n, d, f, e = 270000, 2048, 8192, 2
    assert pairs(n, d, e) and down_splits(n, d, f, e, 1, True) == 1
    rng = np.random.default_rng(9)
    ex = Experts.__new__(Experts)
    ex.e, ex.d, ex.f, ex.np, ex.dev = e, d, f, [], []
    for rows, cols in ((f, d), (f, d), (d, f)):
        q = rng.integers(-127, 128, (e, rows, cols), dtype=np.int8)
        s = (rng.random((e, rows)) * cols ** -0.5 / 64).astype(np.float32)
        ex.np.append((q, s))
        ex.dev.append(sge.Int8Rows(torch.from_numpy(q.reshape(-1, cols)).to(cuda_device),
                                   torch.from_numpy(s.reshape(-1)).to(cuda_device), cols))
    g = torch.Generator(device=cuda_device).manual_seed(9)
    x = torch.randn(n, d, generator=g, device=cuda_device).to(torch.bfloat16)
    r = sge.moe_route_fwd(torch.randn(n, e, generator=g, device=cuda_device), 1)
    y = sge.moe_int8_ffn_fwd(x, *ex.dev, r.w, r.offsets, r.pos)
    cut, edge = r.offsets[1].item(), 2 ** 31 // f
    places = [0, 1, cut - 1, cut, edge - 1, edge, edge + 1, n - 2, n - 1]
    for p in places:
        t = int(r.order[p])
        want, mag = ex.block(0 if p < cut else 1, x[t:t + 1].float().cpu().numpy())
        assert_close(y[t:t + 1], want, mag, f, torch.bfloat16)

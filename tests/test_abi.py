"""The C-ABI library loads without a GPU, exports every symbol include/sge.h
declares, and rejects bad arguments on the host before any launch."""
import ctypes
import os
import re
import subprocess

import pytest

import activation_sparse_gated_epilogue_b200 as sge
from activation_sparse_gated_epilogue_b200 import build as sge_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sge.h")


SELFTEST_HEADER = os.path.join(ROOT, "include", "sge_selftest.h")


def declared_functions(header=HEADER):
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^[A-Za-z_][\w\s\*]*?\b([a-z_][a-z0-9_]*)\s*\(", text, flags=re.M)
    return sorted(set(n for n in names if n not in ("defined",)))


@pytest.fixture(scope="module")
def lib():
    sge_build.build()
    return sge.library()


def test_header_declares_entry_points():
    names = declared_functions()
    for want in ("twell_gate_pack", "twell_fused_up_down", "dense_ffn_fwd", "sge_last_error"):
        assert want in names


def test_library_exports_every_declared_symbol(lib):
    out = subprocess.run(["nm", "-D", "--defined-only", sge.library_path()],
                         capture_output=True, text=True, check=True).stdout
    exported = set(line.split()[-1] for line in out.splitlines() if line.strip())
    for name in declared_functions():
        assert name in exported, name
        assert getattr(lib, name) is not None


def test_every_header_is_covered():
    """include/ holds the product library's header and the self-test
    library's; the tests below check both."""
    headers = sorted(os.listdir(os.path.join(ROOT, "include")))
    assert headers == ["sge.h", "sge_selftest.h"], headers


def test_selftest_library_exports_its_declared_symbols(lib):
    path = sge_build.SELFTEST_LIB
    out = subprocess.run(["nm", "-D", "--defined-only", path], capture_output=True, text=True,
                         check=True).stdout
    exported = set(line.split()[-1] for line in out.splitlines() if line.strip())
    names = declared_functions(SELFTEST_HEADER)
    assert names == ["sge_selftest_wait_timeout"]
    st = ctypes.CDLL(path)
    for name in names:
        assert name in exported, name
        assert getattr(st, name) is not None


def test_debug_library_exports_the_same_symbols(lib):
    """libsge_debug.so (the index-checking build) exports every symbol of
    the header, like the release library; the release build's
    sge_debug_flags answers -1 without touching the device."""
    path = sge_build.build_debug()
    out = subprocess.run(["nm", "-D", "--defined-only", path], capture_output=True, text=True,
                         check=True).stdout
    exported = set(line.split()[-1] for line in out.splitlines() if line.strip())
    for name in declared_functions():
        assert name in exported, name
    lib.sge_debug_flags.restype = ctypes.c_int
    lib.sge_debug_flags.argtypes = [ctypes.c_int]
    assert lib.sge_debug_flags(0) == -1


def test_selftest_rejects_bad_arguments(lib):
    st = ctypes.CDLL(sge_build.SELFTEST_LIB)
    P = ctypes.c_void_p
    st.sge_selftest_wait_timeout.argtypes = [ctypes.c_int, P, P, ctypes.c_int64, ctypes.c_int64,
                                             ctypes.c_int64, P, P, P]
    p = P(4096)
    assert st.sge_selftest_wait_timeout(0, None, p, 256, 256, 256, p, p, None) == 1
    assert st.sge_selftest_wait_timeout(1, p, p, 256, 256, 32, p, p, None) == 1    # k < 64


def test_version_and_error_string(lib):
    assert lib.sge_version() >= 100
    assert isinstance(lib.sge_last_error(), bytes)


def _gate(lib, **kw):
    a = dict(x=None, w=None, n=8, d=64, f=256, dt=sge.SGE_BF16, tile=128, cap=128,
             count=None, idx=None, val=None, diag=None, stream=None)
    a.update(kw)
    return lib.twell_gate_pack(a["x"], a["w"], a["n"], a["d"], a["f"], a["dt"], a["tile"], a["cap"],
                               a["count"], a["idx"], a["val"], a["diag"], a["stream"])


def test_bad_arguments_are_rejected_on_host(lib):
    assert _gate(lib, d=60) == 1                  # d % 8
    assert _gate(lib, tile=48) == 2               # unsupported tile
    assert _gate(lib, f=200, tile=64) == 1        # T does not divide F
    assert _gate(lib, cap=0) == 1
    assert _gate(lib, cap=129) == 1
    assert _gate(lib, n=-1) == 1
    assert _gate(lib) == 1                        # null pointers
    assert b"null" in lib.sge_last_error()
    assert _gate(lib, dt=7, x=ctypes.c_void_p(16), w=ctypes.c_void_p(16), count=ctypes.c_void_p(16),
                 idx=ctypes.c_void_p(16), val=ctypes.c_void_p(16)) == 2
    assert _gate(lib, x=ctypes.c_void_p(17), w=ctypes.c_void_p(16), count=ctypes.c_void_p(16),
                 idx=ctypes.c_void_p(16), val=ctypes.c_void_p(16)) == 1   # misaligned
    assert b"aligned" in lib.sge_last_error()


def test_empty_input_is_a_no_op(lib):
    assert _gate(lib, n=0) == 0
    assert lib.twell_fused_up_down(None, None, None, None, None, None, 64, None, 0, 64, 256,
                                   sge.SGE_BF16, 128, 128, None, 0, None, None) == 0
    assert lib.dense_ffn_fwd(None, None, None, None, None, None, 0, 64, 256, None, None) == 0


def test_fused_rejects_bad_arguments(lib):
    assert lib.twell_fused_up_down(None, None, None, None, None, None, 12, None, 8, 12, 256,
                                   sge.SGE_BF16, 128, 128, None, 0, None, None) == 1
    assert lib.twell_fused_up_down(None, None, None, None, None, None, 64, None, 8, 64, 256,
                                   sge.SGE_BF16, 128, 128, None, 0, None, None) == 1
    p = ctypes.c_void_p(16)
    # a workspace smaller than the query's answer is rejected
    assert lib.twell_fused_up_down(p, p, p, p, p, p, 64, p, 1000, 64, 256, sge.SGE_BF16, 128, 128,
                                   p, 64, None, None) == 1
    assert b"workspace" in lib.sge_last_error()
    assert lib.twell_fused_up_down_workspace_bytes(1000, 64) >= 16 + 5 * 1000
    assert lib.twell_fused_up_down_workspace_bytes(1000, 64) % 256 == 0
    # the workspace must be 256-byte aligned
    ws = lib.twell_fused_up_down_workspace_bytes(1000, 64)
    assert lib.twell_fused_up_down(p, p, p, p, p, p, 64, p, 1000, 64, 256, sge.SGE_BF16, 128, 128,
                                   ctypes.c_void_p(4096 + 16), ws, None, None) == 1
    assert b"aligned" in lib.sge_last_error()
    # the weights' row stride: at least d_model, a multiple of 8
    for ldw in (32, 60, 68):
        assert lib.twell_fused_up_down(p, p, p, p, p, p, ldw, p, 1000, 64, 256, sge.SGE_BF16, 128,
                                       128, ctypes.c_void_p(4096), ws, None, None) == 1
        assert b"ldw" in lib.sge_last_error()
    assert lib.dense_ffn_fwd(None, None, None, None, None, None, 8, 64, 100, None, None) == 1


def test_interleave_rejects_bad_arguments(lib):
    p = ctypes.c_void_p(4096)
    assert lib.sge_interleave_up_down(None, None, None, 0, 64, sge.SGE_BF16, None) == 0  # F = 0
    assert lib.sge_interleave_up_down(None, p, p, 8, 64, sge.SGE_BF16, None) == 1
    assert b"null" in lib.sge_last_error()
    assert lib.sge_interleave_up_down(p, p, p, 8, 0, sge.SGE_BF16, None) == 1
    assert lib.sge_interleave_up_down(p, p, p, 8, 64, 7, None) == 2
    # the output may not overlap an input
    assert lib.sge_interleave_up_down(ctypes.c_void_p(4096), ctypes.c_void_p(1 << 20),
                                      ctypes.c_void_p(4096 + 512), 8, 64, sge.SGE_BF16, None) == 1
    assert b"overlaps" in lib.sge_last_error()


def test_binding_refuses_cpu_tensors():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sge.twell_gate_pack(x, torch.zeros(128, 64, dtype=torch.bfloat16), 128, 128)


def _routed(lib, **kw):
    p = ctypes.c_void_p(4096)
    a = dict(x=p, count=p, idx=p, val=p, wu=p, wd=p, ldw=64, wd_t=p, y=p, n=1000, d=64, f=256,
             tile=128, cap=128, k=16, s_max=64, ws=p, ws_bytes=1 << 40, diag=None, stream=None)
    a.update(kw)
    return lib.twell_hybrid_up_down(a["x"], a["count"], a["idx"], a["val"], a["wu"], a["wd"],
                                    a["ldw"], a["wd_t"], a["y"], a["n"], a["d"], a["f"], a["tile"],
                                    a["cap"], a["k"], a["s_max"], a["ws"], a["ws_bytes"], a["diag"],
                                    a["stream"])


def test_routed_rejects_bad_arguments(lib):
    assert _routed(lib, n=0, x=None, ws=None) == 0          # empty input: no-op
    assert _routed(lib, k=-1) == 1
    assert b"capacity" in lib.sge_last_error()
    assert _routed(lib, s_max=-3) == 1
    assert _routed(lib, wd_t=None) == 1                      # the spill needs W_down^T
    assert b"null" in lib.sge_last_error()
    assert _routed(lib, f=260, tile=20, cap=20) == 1         # F % 8
    assert _routed(lib, d=60, ldw=64) == 1                   # d % 8
    need = lib.twell_hybrid_up_down_workspace_bytes(1000, 64, 256, 64)
    assert _routed(lib, ws_bytes=need - 1) == 1
    assert b"workspace" in lib.sge_last_error()
    assert _routed(lib, ws=ctypes.c_void_p(4096 + 128), ws_bytes=need) == 1
    assert b"aligned" in lib.sge_last_error()
    # the spill operands grow the workspace with S_max
    small = lib.twell_hybrid_up_down_workspace_bytes(1000, 64, 256, 0)
    assert need >= small + 64 * (64 + 2 * 256) * 2
    assert lib.twell_hybrid_up_down_workspace_bytes(1000, 64, 256, -1) == 0


def test_transpose_up_gate_rejects_bad_arguments(lib):
    p = ctypes.c_void_p(4096)
    assert lib.sge_transpose_up_gate(p, p, p, 100, 64, None) == 1     # F % 8
    assert lib.sge_transpose_up_gate(p, None, p, 128, 64, None) == 1
    assert b"null" in lib.sge_last_error()
    assert lib.sge_transpose_up_gate(ctypes.c_void_p(4100), p, p, 128, 64, None) == 1
    assert b"aligned" in lib.sge_last_error()


def _quant(lib, **kw):
    p = ctypes.c_void_p(4096)
    a = dict(x=p, ldx=64, rows=8, cols=64, dt=sge.SGE_BF16, q=p, ldq=64, scale=p)
    a.update(kw)
    return lib.int8_quant_rows(a["x"], a["ldx"], a["rows"], a["cols"], a["dt"], a["q"], a["ldq"], a["scale"], None)


def test_int8_quant_rejects_bad_arguments(lib):
    assert _quant(lib, rows=0, x=None, q=None, scale=None) == 0
    assert _quant(lib, rows=-1) == 1
    assert _quant(lib, cols=0) == 1
    assert _quant(lib, dt=7) == 2
    assert _quant(lib, ldx=63) == 1
    assert b"ldx" in lib.sge_last_error()
    assert _quant(lib, ldq=72) == 1
    assert _quant(lib, ldq=48) == 1
    assert b"ldq" in lib.sge_last_error()
    assert _quant(lib, q=None) == 1
    assert b"null" in lib.sge_last_error()
    assert _quant(lib, scale=ctypes.c_void_p(4098)) == 1
    assert b"aligned" in lib.sge_last_error()
    assert _quant(lib, rows=1 << 31) == 2
    assert _quant(lib, cols=1 << 30, ldx=1 << 30, ldq=1 << 30) == 2


def _linear(lib, **kw):
    p = ctypes.c_void_p(4096)
    a = dict(xq=p, ldx=64, sx=p, wq=p, ldw=64, sw=p, y=p, n=8, m=32, k=64, dt=sge.SGE_BF16, diag=None)
    a.update(kw)
    return lib.int8_linear(a["xq"], a["ldx"], a["sx"], a["wq"], a["ldw"], a["sw"], a["y"], a["n"], a["m"],
                           a["k"], a["dt"], a["diag"], None)


def test_int8_linear_rejects_bad_arguments(lib):
    assert _linear(lib, n=0, xq=None, y=None) == 0
    assert _linear(lib, n=-1) == 1
    assert _linear(lib, m=0) == 1
    assert _linear(lib, k=0) == 1
    assert _linear(lib, dt=2) == 2
    assert _linear(lib, k=65) == 1                     # pitch below the row
    assert _linear(lib, ldx=72) == 1
    assert _linear(lib, ldw=68) == 1
    assert b"pitches" in lib.sge_last_error()
    assert _linear(lib, k=131072, ldx=1 << 18, ldw=1 << 18) == 2
    assert b"32-bit sums" in lib.sge_last_error()
    assert _linear(lib, n=1 << 30) == 2
    assert _linear(lib, sw=None) == 1
    assert _linear(lib, y=None) == 1
    assert _linear(lib, y=ctypes.c_void_p(4104)) == 1
    assert b"aligned" in lib.sge_last_error()


def test_twell_gate_pack_int8_rejects_bad_arguments(lib):
    p = ctypes.c_void_p(4096)

    def call(n=8, d=64, f=256, ld=64, tile=128, cap=128, xq=p, count=p, idx=p, val=p):
        return lib.twell_gate_pack_int8(xq, ld, p, p, ld, p, n, d, f, tile, cap, count, idx, val, None, None)

    assert call(n=0, xq=None, count=None) == 0
    assert call(tile=48, cap=48) == 2
    assert call(f=200) == 1
    assert call(cap=0) == 1
    assert call(cap=129) == 1
    assert call(d=65) == 1                             # pitch
    assert call(xq=None) == 1
    assert call(val=None) == 1
    assert call(idx=ctypes.c_void_p(4097)) == 1
    assert call(d=200000, ld=200000) == 2


def _route(lib, bwd=False, **kw):
    p = ctypes.c_void_p(4096)
    a = dict(logits=p, mask=None, n=100, e=16, k=2, dt=sge.SGE_F32, ids=p, w=p, counts=p, offsets=p, pos=p,
             order=p, loss=p, live=p, ws=p, ws_bytes=1 << 30, dlogits=p)
    a.update(kw)
    head = (a["logits"], a["mask"], a["n"], a["e"], a["k"], 1, a["dt"], a["ids"], a["w"], a["counts"], a["offsets"])
    if bwd:
        return lib.moe_route_bwd(*head, a["live"], None, None, a["dlogits"], None)
    return lib.moe_route_fwd(*head, a["pos"], a["order"], a["loss"], a["live"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("bwd", [False, True])
def test_moe_route_rejects_bad_arguments(lib, bwd):
    assert _route(lib, bwd, n=-1) == 1
    assert _route(lib, bwd, e=0) == 1
    assert _route(lib, bwd, k=0) == 1
    assert _route(lib, bwd, k=17) == 1                 # above E
    assert _route(lib, bwd, e=300) == 2
    assert _route(lib, bwd, e=64, k=17) == 2
    assert _route(lib, bwd, dt=5) == 2
    assert _route(lib, bwd, n=1 << 29) == 2
    assert _route(lib, bwd, logits=None) == 1
    assert _route(lib, bwd, counts=None) == 1
    assert b"null" in lib.sge_last_error()
    assert _route(lib, bwd, ids=ctypes.c_void_p(4100)) == 1
    assert b"aligned" in lib.sge_last_error()
    if bwd:
        assert _route(lib, bwd, n=0, logits=None) == 0
    else:
        need = lib.moe_route_workspace_bytes(100, 16)
        assert need > 0 and need % 256 == 0
        assert _route(lib, ws_bytes=need - 1) == 1
        assert b"workspace" in lib.sge_last_error()
        assert _route(lib, ws=ctypes.c_void_p(4096 + 16)) == 1
        assert lib.moe_route_workspace_bytes(100, 257) == 0


def _ffn(lib, routed, **kw):
    p = ctypes.c_void_p(4096)
    a = dict(x=p, wg=p, sg=p, w=p, offsets=p, pos=p, y=p, n=10, d=64, f=128, e=4, k=2, dt=sge.SGE_BF16, ws=p,
             ws_bytes=1 << 40)
    a.update(kw)
    head = (a["x"], a["wg"], a["sg"], p, p, p, p)
    tail = (a["dt"], a["ws"], a["ws_bytes"], None, None)
    if routed:
        return lib.moe_int8_ffn_fwd(*head, a["w"], a["offsets"], a["pos"], a["y"], a["n"], a["d"], a["f"], a["e"],
                                    a["k"], *tail)
    return lib.int8_ffn_fwd(*head, a["y"], a["n"], a["d"], a["f"], *tail)


@pytest.mark.parametrize("routed", [False, True])
def test_int8_ffn_rejects_bad_arguments(lib, routed):
    assert _ffn(lib, routed, n=0, x=None, y=None, ws=None) == 0
    assert _ffn(lib, routed, n=-1) == 1
    assert _ffn(lib, routed, d=0) == 1
    assert _ffn(lib, routed, d=60) == 1
    assert _ffn(lib, routed, f=100) == 1
    assert _ffn(lib, routed, dt=4) == 2
    assert _ffn(lib, routed, d=200000) == 2
    assert _ffn(lib, routed, n=1 << 30) == 2
    assert _ffn(lib, routed, x=None) == 1
    assert b"null" in lib.sge_last_error()
    assert _ffn(lib, routed, y=ctypes.c_void_p(4104)) == 1
    assert b"aligned" in lib.sge_last_error()
    assert _ffn(lib, routed, ws=ctypes.c_void_p(4096 + 64)) == 1
    assert _ffn(lib, routed, ws_bytes=256) == 1
    assert b"workspace" in lib.sge_last_error()
    if routed:
        assert _ffn(lib, routed, e=0) == 1
        assert _ffn(lib, routed, k=5) == 1
        assert _ffn(lib, routed, e=257) == 2
        assert _ffn(lib, routed, e=64, k=17) == 2
        assert _ffn(lib, routed, w=None) == 1
        assert _ffn(lib, routed, offsets=None) == 1
        assert _ffn(lib, routed, pos=ctypes.c_void_p(4100)) == 1
    need = lib.int8_ffn_workspace_bytes(10, 64, 128, 4, 2, sge.SGE_BF16)
    assert need > 0 and need % 256 == 0
    assert lib.int8_ffn_workspace_bytes(10, 60, 128, 4, 2, sge.SGE_BF16) == 0


def test_binding_of_the_8_bit_operators_and_the_router_refuses_cpu_tensors():
    import torch
    x = torch.zeros(4, 64)
    rows = sge.Int8Rows.empty(4, 64, "cpu")
    assert rows.q.shape == (4, 64) and rows.scale.shape == (4,) and rows.rows == 4
    route = sge.MoeRoute.empty(4, 8, 2, "cpu")
    assert route.ids.shape == route.w.shape == route.pos.shape == (4, 2) and route.w.dtype == torch.float32
    assert route.offsets.shape == (9,) and route.order.shape == (8,) and route.top_k == 2
    ends = [getattr(route, a).data_ptr() for a in sge.MoeRoute.NAMES]
    assert all(p % 4 == 0 for p in ends) and len(set(ends)) == 8
    for call in (lambda: sge.int8_quant_rows(x), lambda: sge.int8_linear(rows, rows),
                 lambda: sge.twell_gate_pack_int8(rows, rows, 16, 16), lambda: sge.moe_route_fwd(x, 2),
                 lambda: sge.moe_route_bwd(x[:, :8], route), lambda: sge.int8_ffn_fwd(x, rows, rows, rows),
                 lambda: sge.moe_int8_ffn_fwd(x, rows, rows, rows, route.w, route.offsets, route.pos)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("d,f,e,k", [(2048, 8192, 1, 1), (2048, 2048, 16, 2), (1024, 1024, 32, 4), (136, 4096, 3, 2),
                                     (2560, 10240, 1, 1), (64, 16384, 256, 8), (8, 8, 1, 1)])
def test_workspace_of_a_batch_serves_every_smaller_one(lib, d, f, e, k):
    """The largest need of any batch up to n, by the call's own check of the
    workspace, is what the size query gives for n."""
    p = ctypes.c_void_p(4096)

    def too_small(n, nbytes):
        code = (lib.moe_int8_ffn_fwd(p, p, p, p, p, p, p, p, p, p, p, n, d, f, e, k, sge.SGE_BF16, p, nbytes, None, None)
                if e > 1 else lib.int8_ffn_fwd(p, p, p, p, p, p, p, p, n, d, f, sge.SGE_BF16, p, nbytes, None, None))
        return code == 1 and b"workspace" in lib.sge_last_error()

    sizes = list(range(1, 1100)) + list(range(1100, 9000, 41))
    given = [lib.int8_ffn_workspace_bytes(n, d, f, e, k, sge.SGE_BF16) for n in sizes]
    assert given == sorted(given)
    for n, nbytes in zip(sizes, given):
        # the message of a call that gets 0 bytes names its need
        assert too_small(n, 0)
        need = int(lib.sge_last_error().decode().split(",")[1].split()[0])
        assert 0 < need <= nbytes
    route = [lib.moe_route_workspace_bytes(n, max(e, 2)) for n in sizes]
    assert route == sorted(route)


def test_int8_ffn_workspace_refuses_other_dtypes(lib):
    import torch
    with pytest.raises(ValueError, match="dtype"):
        sge.int8_ffn_workspace(8, 64, 128, 1, 1, torch.float16, "cpu")


def test_numbers_kept_for_each_device_are_made_without_a_race(tmp_path):
    """Threads that ask for one device's number at once, under the thread
    sanitiser."""
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text("""
#include <thread>
#include <vector>
#include "sge_host.h"
int main() {
  sge::PerDevice kept;
  std::vector<std::thread> threads;
  std::atomic<int> wrong{0};
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&] {
      for (int dev = -1; dev < 66; ++dev)
        for (int i = 0; i < 2; ++i)
          if (kept.get(dev, [dev] { return dev + 100; }) != dev + 100) ++wrong;
    });
  for (auto& t : threads) t.join();
  return wrong;
}
""")
    csrc = os.path.join(ROOT, "activation_sparse_gated_epilogue_b200", "csrc")
    made = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=thread", "-I", csrc, "-I", "/usr/local/cuda/include",
                           str(src), "-o", str(exe), "-ldl", "-pthread"], capture_output=True, text=True)
    if "cannot find" in made.stderr and "tsan" in made.stderr:
        pytest.skip("no thread sanitiser here")
    assert made.returncode == 0, made.stderr[-2000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    if "unexpected memory mapping" in run.stderr:
        pytest.skip("the thread sanitiser cannot run here")
    assert run.returncode == 0 and "data race" not in run.stderr, run.stderr[-2000:]

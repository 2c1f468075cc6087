"""C-ABI checks that need no GPU: the library builds, loads, exports every
function ``include/tcg.h`` declares, and rejects bad arguments on the host
before touching the device.  Nothing here launches a kernel."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def tcg():
    from blackwell_tensor_core_swizzled_gb300 import build
    build.build()
    import blackwell_tensor_core_swizzled_gb300 as m
    return m


def _declared():
    text = open(os.path.join(ROOT, "include", "tcg.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(tcg_[a-z0-9_]+)\s*\(", text)))


def test_header_declares_the_four_gemms():
    names = _declared()
    for n in ("tcg_gemm_f16", "tcg_gemm_bf16", "tcg_gemm_tf32", "tcg_gemm_mxf8_blockscaled"):
        assert n in names


def test_every_declared_symbol_is_exported(tcg):
    lib = ctypes.CDLL(tcg.LIB_PATH)
    missing = [n for n in _declared() if not hasattr(lib, n)]
    assert not missing, missing
    assert sorted(tcg.EXPORTED) == _declared()


def test_status_strings(tcg):
    for s in range(0, -7, -1):
        assert tcg.status_string(s) != "unknown status"


def _call(tcg, name, M=256, N=256, K=64, A=0x10000, am=0, lda=0, B=0x20000, bm=0, ldb=0, D=0x30000,
          dt=2, ldd=0, acc=0):
    return tcg.raw_call(f"tcg_gemm_{name}", M, N, K, A, am, lda, B, bm, ldb, D, dt, ldd, acc, None)


def test_host_validation_rejects_bad_arguments(tcg):
    assert _call(tcg, "bf16", M=-1) == tcg.ERR_INVALID
    assert _call(tcg, "bf16", A=None) == tcg.ERR_INVALID
    assert _call(tcg, "bf16", D=None) == tcg.ERR_INVALID
    assert _call(tcg, "bf16", am=7) == tcg.ERR_INVALID
    assert _call(tcg, "bf16", lda=32) == tcg.ERR_INVALID            # lda < K
    assert _call(tcg, "bf16", ldd=100) == tcg.ERR_INVALID           # ldd < N
    assert _call(tcg, "bf16", A=0x10008) == tcg.ERR_ALIGNMENT       # TMA base alignment
    assert _call(tcg, "bf16", K=60, lda=60) == tcg.ERR_ALIGNMENT    # 120-byte rows
    assert _call(tcg, "bf16", acc=1, dt=1) == tcg.ERR_UNSUPPORTED   # bf16 with f16 accumulation
    assert _call(tcg, "f16", acc=1, dt=2) == tcg.ERR_UNSUPPORTED    # f16 accumulation needs f16 out
    assert _call(tcg, "tf32", dt=5) == tcg.ERR_INVALID
    # generic entry point: split_k below -1 (stream-K) is not a mode
    rc = tcg.gemm(256, 256, 64, 1, 0x10000, 0, 0, 0x20000, 0, 0, 0x30000, 2, 0, 0, split_k=-2, stream=0, check=False)
    assert rc == tcg.ERR_INVALID
    # mxf8 without scales
    rc = tcg.raw_call("tcg_gemm_mxf8_blockscaled", 64, 64, 64, 0x10000, 0, 0, 0x20000, 0, 0, None, None,
                      0x30000, 2, 0, 0, None)
    assert rc == tcg.ERR_INVALID
    # cp probe: shape codes 0..11 (4..11 decompressing), walk inside the image
    for shape in (-1, 12):
        assert tcg.raw_call("tcg_probe_cp", 0x10000, 512, shape, 0, 16, 128, 0, 0x20000, None) == tcg.ERR_INVALID
    assert tcg.raw_call("tcg_probe_cp", 0x10000, 256, 9, 0, 16, 128, 0, 0x20000, None) == tcg.ERR_INVALID
    # cp probe: a 4-row 4x256b walk whose 8-row blocks are not backed whole
    # (192 of the 256 bytes its two 16-byte columns organise) is rejected
    assert tcg.raw_call("tcg_probe_cp", 0x10000, 48, 3, 0, 128, 256, 0, 0x20000, None) == tcg.ERR_INVALID
    assert tcg.raw_call("tcg_probe_cp", 0x10000, 64, 3, 0, 128, 256, 0, 0x20000, None) != tcg.ERR_INVALID
    # MMA image probe: mode 4 is TF32 MN-major only, and a walk that could
    # leave its 96 KiB region under either stride assignment is rejected
    def op(major, sw, ldo, sdo, starts=(0,), nbytes=4096):
        return tcg.probe_operand(0x10000, nbytes, major, ldo, sdo, sw, starts)
    ok_a, ok_b = op(0, 3, 16, 1024), op(0, 3, 16, 1024)
    assert tcg.raw_call("tcg_probe_mma_image", ok_a, ok_b, 1, 64, 1, 0x30000, None) == tcg.ERR_NO_DEVICE
    assert tcg.raw_call("tcg_probe_mma_image", op(1, 4, 4096, 512), ok_b, 1, 64, 1, 0x30000,
                        None) == tcg.ERR_UNSUPPORTED
    assert tcg.raw_call("tcg_probe_mma_image", op(1, 3, 4096, 1024), ok_b, 2, 64, 1, 0x30000,
                        None) == tcg.ERR_UNSUPPORTED                                   # TF32 MN-major needs mode 4
    assert tcg.raw_call("tcg_probe_mma_image", op(1, 0, 128, 8192), ok_b, 1, 64, 1, 0x30000,
                        None) == tcg.ERR_INVALID                                       # 15 chunks x 8 KiB
    assert tcg.raw_call("tcg_probe_mma_image", op(0, 3, 16, 1024, starts=(8,)), ok_b, 1, 64, 1, 0x30000,
                        None) == tcg.ERR_INVALID                                       # origin not 16-byte aligned
    assert tcg.raw_call("tcg_probe_mma_image", ok_a, ok_b, 1, 72, 1, 0x30000, None) == tcg.ERR_INVALID
    assert tcg.raw_call("tcg_probe_mma_image", op(0, 3, 16, 1024, nbytes=200 * 1024), ok_b, 1, 64, 1, 0x30000,
                        None) == tcg.ERR_INVALID
    # trace request: buffer and count go together; null + 0 cancels
    assert tcg.raw_call("tcg_trace_next", None, 4) == tcg.ERR_INVALID
    assert tcg.raw_call("tcg_trace_next", 0x10000, 0) == tcg.ERR_INVALID
    assert tcg.raw_call("tcg_trace_next", 0x10004, 4) == tcg.ERR_ALIGNMENT
    assert tcg.raw_call("tcg_trace_next", None, 0) == tcg.OK
    # .ws probe: N must be one of the weight-stationary widths 64 / 128 / 256
    for n in (32, 96, 512):
        assert tcg.raw_call("tcg_probe_mma_tile_ws", 0x10000, 0x20000, n, 64, 0, 0x30000, None) == tcg.ERR_INVALID
    # split-access probe: repeat counts 1/2/4/8 and the four in-bounds immediates only
    for num, il, ic in ((3, 16, 8), (16, 16, 8), (4, 16, 4), (4, 0, 8), (4, 8, 0), (8, 32, 0)):
        assert tcg.raw_call("tcg_probe_ld_split", 0x10000, num, il, ic, 0x20000, 0x30000, None) == tcg.ERR_INVALID
    assert tcg.raw_call("tcg_probe_ld_split", None, 4, 16, 8, 0x20000, 0x30000, None) == tcg.ERR_INVALID
    # stmatrix probe: x1 / x2 / x4 only
    for count in (0, 3, 8):
        assert tcg.raw_call("tcg_probe_stmatrix", 0x10000, 0x20000, count, 0, 0x30000, None) == tcg.ERR_INVALID


def test_generic_entry_point_rejects_unknown_epilogue(tcg):
    for ep in (-1, 3):
        rc = tcg.gemm(256, 256, 64, tcg.IN_BF16, 0x10000, 0, 64, 0x20000, 0, 64, 0x30000, 2, 256,
                      check=False, epilogue=ep, stream=0)
        assert rc == tcg.ERR_INVALID


def test_chain_validation_before_any_device_work(tcg):
    # tcg_gemm_chain(in, M, N1, N2, K, A, lda, B1, ldb1, B2, ldb2, E, e_type, lde, stream)
    def call(in_type=1, M=64, N1=32, N2=64, K=64, A=0x10000, lda=64, B1=0x20000, ldb1=64, B2=0x30000, ldb2=32,
             E=0x40000, et=0, lde=64):
        return tcg.raw_call("tcg_gemm_chain", in_type, M, N1, N2, K, A, lda, B1, ldb1, B2, ldb2, E, et, lde, None)
    assert call(in_type=2) == tcg.ERR_INVALID                 # tf32: 16-bit operands only
    for n1 in (0, 8, 40, 272):
        assert call(N1=n1) == tcg.ERR_INVALID                 # N1 a multiple of 16 in [16, 256]
    assert call(M=-1) == tcg.ERR_INVALID
    assert call(et=5) == tcg.ERR_INVALID
    assert call(E=None) == tcg.ERR_INVALID
    assert call(lde=32) == tcg.ERR_INVALID                    # lde < N2
    assert call(E=0x40008) == tcg.ERR_ALIGNMENT               # E base
    assert call(et=2, lde=68) == tcg.ERR_ALIGNMENT            # 136-byte rows of E
    assert call(A=0x10008) == tcg.ERR_ALIGNMENT
    assert call(lda=60) == tcg.ERR_INVALID                    # lda < K
    assert call(ldb2=16) == tcg.ERR_INVALID                   # ldb2 < N1
    assert call(M=0, A=None, B1=None, B2=None, E=None) == tcg.OK
    assert call(N2=0, A=None, B1=None, B2=None, E=None) == tcg.OK


def test_empty_problems_are_noops(tcg):
    # M == 0 or N == 0 returns before any device work, even with null pointers
    assert _call(tcg, "bf16", M=0, A=None, B=None, D=None) == tcg.OK
    assert _call(tcg, "f16", N=0, A=None, B=None, D=None) == tcg.OK


def test_scale_image_sizes(tcg):
    # [K step][tile][chunk][512 B]: K=8192 -> 256 blocks -> 64 steps
    assert tcg.mxf8_scale_image_bytes(8192, 8192, 128) == 64 * 64 * 512
    assert tcg.mxf8_scale_image_bytes(8192, 8192, 224) == 64 * 37 * 2 * 512
    assert tcg.mxf8_scale_image_bytes(300, 96, 128) == 1 * 3 * 512
    assert tcg.mxf8_scale_image_bytes(8192, 8192, 256) == 64 * 32 * 2 * 512
    # N = 256 tiles for one CTA and for a pair (a pair's MN-major B half tile
    # is one whole 128-byte swizzle span of E4M3); pairs with K-major B over
    # at least 300 tiles of 256 x 384 take those
    for cg in (0, 1, 2):
        assert tcg.mxf8_tile_n(8192, 8192, 8192, tcg.K_MAJOR, cg) == 256
        assert tcg.mxf8_tile_n(8192, 8192, 8192, tcg.MN_MAJOR, cg) == 256
        for fmt in (tcg.IN_E5M2, tcg.IN_E3M2, tcg.IN_E2M3):
            assert tcg.tile_n(fmt, 8192, 8192, 8192, tcg.K_MAJOR, cg) == 256
        # packed FP4 pairs with K-major B over at least 300 tiles of 256 x 384
        for fmt in (tcg.IN_E2M1, tcg.IN_NVF4):
            assert tcg.tile_n(fmt, 8192, 8192, 8192, tcg.K_MAJOR, cg) == (256 if cg == 1 else 384)
    assert tcg.tile_n(tcg.IN_E2M1, 4096, 4096, 4096, tcg.K_MAJOR, 2) == 256      # 16 x 11 = 176 tiles
    assert tcg.tile_n(tcg.IN_NVF4, 2600, 10668, 256, tcg.K_MAJOR, 0) == 384      # 11 x 28 = 308
    assert tcg.tile_n(tcg.IN_BF16, 8192, 8192, 8192, tcg.K_MAJOR, 0) == tcg.ERR_INVALID
    assert tcg.scale_image_bytes(tcg.IN_E2M1, 8192, 8192, 384) == 32 * 22 * 3 * 2 * 512


@pytest.mark.skipif(os.environ.get("CUDA_VISIBLE_DEVICES_FORCE_GPU") is not None, reason="GPU present")
def test_fails_loudly_without_a_device(tcg):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _call(tcg, "bf16") == tcg.ERR_NO_DEVICE
    with pytest.raises(tcg.TcgError):
        tcg.gemm_bf16(256, 256, 64, 0x10000, 0, 0, 0x20000, 0, 0, 0x30000, 2, 0, 0, stream=0)


def test_moe_validation_before_any_device_work(tcg):
    def sort(T=4, topk=2, E=8, ex=0x10000, off=0x20000, pos=0x30000, src=0x40000):
        return tcg.raw_call("tcg_moe_sort", T, topk, E, ex, off, pos, src, None)
    assert sort(T=-1) == tcg.ERR_INVALID
    assert sort(topk=0) == tcg.ERR_INVALID
    assert sort(E=0) == tcg.ERR_INVALID
    assert sort(E=1025) == tcg.ERR_UNSUPPORTED
    assert sort(T=1 << 28, topk=8) == tcg.ERR_UNSUPPORTED
    assert sort(T=(1 << 62), topk=8) == tcg.ERR_UNSUPPORTED
    for p in ("ex", "off", "pos", "src"):
        assert sort(**{p: None}) == tcg.ERR_INVALID
        assert sort(**{p: 0x10002}) == tcg.ERR_ALIGNMENT
    assert sort(T=0, off=None) == tcg.ERR_INVALID

    def disp(t=2, T=4, topk=2, H=64, X=0x10000, ldx=0, pos=0x20000, Xs=0x30000, ldxs=0):
        return tcg.raw_call("tcg_moe_dispatch", t, T, topk, H, X, ldx, pos, Xs, ldxs, None)
    assert disp(t=3) == tcg.ERR_INVALID
    assert disp(H=-1) == tcg.ERR_INVALID
    assert disp(topk=65) == tcg.ERR_UNSUPPORTED
    assert disp(ldx=63) == tcg.ERR_INVALID
    assert disp(ldxs=63) == tcg.ERR_INVALID
    assert disp(X=None) == tcg.ERR_INVALID
    assert disp(X=0x10001) == tcg.ERR_ALIGNMENT
    assert disp(t=0, Xs=0x30002) == tcg.ERR_ALIGNMENT
    assert disp(pos=0x20002) == tcg.ERR_ALIGNMENT
    assert disp(T=0, X=None, Xs=None, pos=None) == tcg.OK
    assert disp(H=0, X=None, Xs=None, pos=None) == tcg.OK

    def comb(t=2, T=4, topk=2, H=64, Ys=0x10000, ldys=0, pos=0x20000, w=0x30000, Y=0x40000, ldy=0):
        return tcg.raw_call("tcg_moe_combine", t, T, topk, H, Ys, ldys, pos, w, Y, ldy, None)
    assert comb(Ys=None) == tcg.ERR_INVALID
    assert comb(ldy=8) == tcg.ERR_INVALID
    assert comb(w=0x30002) == tcg.ERR_ALIGNMENT
    assert comb(T=0, Ys=None, Y=None, pos=None, w=None) == tcg.OK

    def grad(t=2, T=4, topk=2, H=64, dY=0x10000, Ys=0x20000, pos=0x30000, w=0x40000, dYs=0x50000, dw=0x60000):
        return tcg.raw_call("tcg_moe_combine_grad", t, T, topk, H, dY, 0, Ys, 0, pos, w, dYs, 0, dw, None)
    assert grad(Ys=None) == tcg.ERR_INVALID                  # Ys and dweight go together
    assert grad(dw=None) == tcg.ERR_INVALID
    assert grad(dYs=None) == tcg.ERR_INVALID
    assert grad(dw=0x60002) == tcg.ERR_ALIGNMENT
    assert grad(T=0, dY=None, Ys=None, dYs=None, dw=None) == tcg.OK


def test_grouped_validation_before_any_device_work(tcg):
    def call(t=1, R=64, N=64, K=64, G=4, A=0x10000, lda=0, off=0x20000, B=0x30000, major=0, ldb=0, sb=0, D=0x40000,
             dt=2, ldd=0):
        return tcg.raw_call("tcg_gemm_grouped", t, R, N, K, G, A, lda, off, B, major, ldb, sb, D, dt, ldd, None)
    assert call(t=2) == tcg.ERR_INVALID                       # 16-bit operands only
    assert call(R=-1) == tcg.ERR_INVALID
    assert call(G=0) == tcg.ERR_INVALID
    assert call(G=1025) == tcg.ERR_UNSUPPORTED
    assert call(R=1 << 30) == tcg.ERR_UNSUPPORTED
    assert call(major=2) == tcg.ERR_INVALID
    assert call(dt=3) == tcg.ERR_INVALID
    for p in ("A", "off", "B", "D"):
        assert call(**{p: None}) == tcg.ERR_INVALID
    assert call(lda=56) == tcg.ERR_INVALID
    assert call(ldb=56) == tcg.ERR_INVALID
    assert call(ldd=56) == tcg.ERR_INVALID
    assert call(sb=-8) == tcg.ERR_INVALID
    assert call(K=60) == tcg.ERR_ALIGNMENT                    # packed rows of 120 bytes
    assert call(N=60, major=1) == tcg.ERR_ALIGNMENT
    assert call(sb=64 * 64 + 4) == tcg.ERR_ALIGNMENT
    assert call(A=0x10008) == tcg.ERR_ALIGNMENT
    assert call(off=0x20002) == tcg.ERR_ALIGNMENT
    assert call(D=0x40001) == tcg.ERR_ALIGNMENT
    assert call(R=0, A=None, off=None, B=None, D=None) == tcg.OK
    assert call(N=0, A=None, off=None, B=None, D=None) == tcg.OK

    def wgrad(t=1, R=64, N=64, K=64, G=4, DY=0x10000, lddy=0, A=0x20000, lda=0, off=0x30000, DW=0x40000, dt=0,
              lddw=0, sw=0):
        return tcg.raw_call("tcg_gemm_grouped_wgrad", t, R, N, K, G, DY, lddy, A, lda, off, DW, dt, lddw, sw, None)
    assert wgrad(t=3) == tcg.ERR_INVALID
    assert wgrad(K=-1) == tcg.ERR_INVALID
    for p in ("DY", "A", "off", "DW"):
        assert wgrad(**{p: None}) == tcg.ERR_INVALID
    assert wgrad(lddw=32) == tcg.ERR_INVALID
    assert wgrad(sw=-1) == tcg.ERR_INVALID
    assert wgrad(DW=0x40002) == tcg.ERR_ALIGNMENT
    assert wgrad(N=60) == tcg.ERR_ALIGNMENT
    assert wgrad(lda=68) == tcg.ERR_ALIGNMENT
    assert wgrad(N=0, DY=None, A=None, off=None, DW=None) == tcg.OK


def test_gemv_w4_validation_before_any_device_work(tcg):
    def call(fmt=0, t=1, R=2, N=64, K=256, A=0x10000, lda=0, B=0x20000, scale=0x30000, D=0x40000, dt=2, ldd=0,
             group=64, **kw):
        return tcg.gemv_w4(fmt, t, R, N, K, A, lda, B, scale, D, dt, ldd, group=group, check=False, stream=0, **kw)
    assert tcg.raw_call("tcg_gemv_w4", None, None) == tcg.ERR_INVALID
    assert call(fmt=3) == tcg.ERR_INVALID
    assert call(t=2) == tcg.ERR_INVALID
    assert call(dt=4) == tcg.ERR_INVALID
    assert call(R=-1) == tcg.ERR_INVALID
    assert call(groups=0) == tcg.ERR_INVALID
    assert call(groups=2) == tcg.ERR_INVALID                  # groups need offsets
    assert call(groups=1025, offsets=0x50000) == tcg.ERR_UNSUPPORTED
    assert call(group=0) == tcg.ERR_INVALID
    assert call(group=16) == tcg.ERR_UNSUPPORTED
    assert call(fmt=1, group=64) == tcg.ERR_INVALID           # MXFP4: 32
    assert call(fmt=2, group=32) == tcg.ERR_INVALID           # NVFP4: 16
    assert call(fmt=1, group=0, zero=0x60000) == tcg.ERR_INVALID
    assert call(K=80, group=32) == tcg.ERR_ALIGNMENT
    assert call(K=96, group=64) == tcg.ERR_ALIGNMENT          # half a group
    for p in ("A", "B", "scale", "D"):
        assert call(**{p: None}) == tcg.ERR_INVALID
    assert call(lda=248) == tcg.ERR_INVALID
    assert call(ldb=224) == tcg.ERR_INVALID
    assert call(ld_scale=3) == tcg.ERR_INVALID
    assert call(ldd=63) == tcg.ERR_INVALID
    assert call(stride_b=-32) == tcg.ERR_INVALID
    assert call(lda=260) == tcg.ERR_ALIGNMENT
    assert call(ldb=272) == tcg.ERR_ALIGNMENT
    assert call(stride_b=16) == tcg.ERR_ALIGNMENT
    assert call(A=0x10008) == tcg.ERR_ALIGNMENT
    assert call(B=0x20008) == tcg.ERR_ALIGNMENT
    assert call(scale=0x30001) == tcg.ERR_ALIGNMENT
    assert call(alpha=0x50002) == tcg.ERR_ALIGNMENT
    assert call(D=0x40001) == tcg.ERR_ALIGNMENT
    assert call(R=0, A=None, B=None, scale=None, D=None) == tcg.OK
    assert call(N=0, A=None, B=None, scale=None, D=None) == tcg.OK


def test_none_and_addresses_are_not_asked_for_data_ptr(tcg):
    """A call passes up to four None scales and any pointer as an address: none
    of them goes through a raised AttributeError."""
    events = []

    def trace(frame, event, arg):
        events.append(event)
        return trace

    class Tensor:
        def data_ptr(self):
            return 0x30000

    before = sys.gettrace()
    sys.settrace(trace)
    try:
        got = [tcg._ptr(None), tcg._ptr(0), tcg._ptr(0x20000), tcg._ptr(Tensor())]
    finally:
        sys.settrace(before)
    assert got == [None, 0, 0x20000, 0x30000]
    assert "exception" not in events
    with pytest.raises(AttributeError):
        tcg._ptr(object())


def test_a_failed_setup_is_tried_again(tmp_path):
    """What the library does once for each device is done again after an error,
    once after success, and apart for each device and thread."""
    csrc = os.path.join(ROOT, "blackwell_tensor_core_swizzled_gb300", "csrc")
    src = tmp_path / "once.cpp"
    src.write_text(r"""
#include <thread>
#include <vector>
#include "once.h"
enum Err { Ok = 0, NoMemory = 2 };
int main() {
  tcg::OncePerDevice<Err> once;
  int calls = 0;
  Err result = NoMemory;
  auto setup = [&] { ++calls; return result; };
  if (once(1, setup) != NoMemory || once(1, setup) != NoMemory || calls != 2) return 1;
  result = Ok;
  if (once(1, setup) != Ok || once(1, setup) != Ok || calls != 3) return 2;
  if (once(2, setup) != Ok || calls != 4) return 3;
  std::vector<std::thread> all;
  for (int i = 0; i < 8; ++i) all.emplace_back([&] { once(3, setup); });
  for (auto& t : all) t.join();
  return calls == 5 ? 0 : 4;
}
""")
    exe = tmp_path / "once"
    subprocess.run(["g++", "-std=c++17", "-pthread", "-I", csrc, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_moe_refuses_sizes_whose_product_overflows(tcg):
    for T, topk in ((1 << 62, 8), (1 << 61, 64), ((1 << 63) - 1, 64), (1 << 30, 1), (1 << 29, 2)):
        big = (T, topk, 64)
        assert tcg.raw_call("tcg_moe_dispatch", 2, *big, 0x10000, 0, 0x20000, 0x30000, 0, None) == tcg.ERR_UNSUPPORTED
        assert tcg.raw_call("tcg_moe_combine", 2, *big, 0x10000, 0, 0x20000, None, 0x40000, 0,
                            None) == tcg.ERR_UNSUPPORTED
        assert tcg.raw_call("tcg_moe_combine_grad", 2, *big, 0x10000, 0, None, 0, 0x20000, None, 0x50000, 0, None,
                            None) == tcg.ERR_UNSUPPORTED

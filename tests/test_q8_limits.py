"""The 8-bit calls at the largest sizes they take: no launch of more threads
than HIP takes, and nothing left out (tests/sanitize/q8_limits.cpp with the
planner under AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU); the
sizes that still fit a card, on the GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "newton_schulz_04_amd", "csrc")
ROCM = "/opt/rocm"


def test_launches_of_the_largest_sizes(tmp_path):
    gxx = shutil.which("g++")
    if not gxx or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")):
        pytest.skip("g++ or the HIP headers are missing")
    exe = str(tmp_path / "q8_limits")
    subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
                    f"-I{ROCM}/include", f"-I{ROOT}/include", f"-I{CSRC}", os.path.join(CSRC, "ns_q8_api.cpp"),
                    os.path.join(HERE, "sanitize", "q8_limits.cpp"), "-o", exe, f"-L{ROCM}/lib",
                    f"-Wl,-rpath,{ROCM}/lib", "-lamdhip64"], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1", HIP_VISIBLE_DEVICES="")
    r = subprocess.run([exe], env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    assert "q8_limits ok" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr


def test_sizes_up_to_their_bounds():
    """What the header says of each product's sizes: rows up to 2^24, row
    lengths up to 2^21, matmul's sums up to NS_Q8_MAX_K."""
    from newton_schulz_04_amd import _q8
    rows, length, at = 1 << 24, 1 << 21, 0x10000000
    L = _q8.lib()

    def status(op, tokens, out, inp):
        n = out if op == 0 else inp
        layer = _q8.LayerStruct(tokens=tokens, out_features=out, in_features=inp, xq=at, ld_xq=inp, x_scale=at, wq=at,
                                ld_wq=inp, w_scale=at, dy=at, ld_dy=out, out=at, ld_out=n)
        need = ctypes.c_size_t(0)
        return L.ns_q8_workspace_bytes(op, (_q8.LayerStruct * 1)(layer), 1, 0, ctypes.byref(need))

    for op, most in ((0, (rows, length, _q8.Q8_MAX_K)), (1, (rows, length, length)), (2, (rows, length, length))):
        for axis in range(3):
            size = [40, 40, 40]
            size[axis] = most[axis]
            assert status(op, *size) == 0
            size[axis] += 1
            assert status(op, *size) == 1
    # 2^17 x 127 tiles of 128 x 128 are fewer than 2^24, 2^17 x 128 are not
    assert status(0, rows, 127 * 128, 40) == 0 and status(0, rows, 127 * 128 + 1, 40) == 1
    # a gradient without tokens has no dY whose rows would bound its own
    assert status(2, 0, rows, 40) == 0


@pytest.mark.gpu
def test_quantize_matrices_of_the_most_rows():
    """Four matrices of 2^24 rows: as many workgroups as one launch cannot take."""
    import newton_schulz_04_amd as ns
    rows = 1 << 24
    x = [torch.randn((rows, 8), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").bfloat16()
         for i in range(4)]
    pairs = ns.quantize_rows(x)
    back = ns.dequantize_rows(pairs)
    for v, (q, s), b in zip(x, pairs, back):
        want_s = (v.abs().amax(1).double() / 127).float().clamp_min(2.0 ** -126)
        assert torch.equal(s, want_s)
        assert torch.equal(q, (v.double() / want_s.double()[:, None]).round().to(torch.int8))
        assert torch.equal(b, (q.double() * want_s.double()[:, None]).float().bfloat16())


@pytest.mark.gpu
def test_a_gradient_without_tokens_of_the_most_rows():
    """2^24 x 1024: a layer without tokens scales 32 GiB of gradient."""
    import newton_schulz_04_amd as ns
    rows = 1 << 24
    g = torch.full((rows, 1024), 2.0, dtype=torch.bfloat16, device="cuda")
    dy = torch.empty((0, rows), dtype=torch.bfloat16, device="cuda")
    x = (torch.empty((0, 1024), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))
    ns.q8_grad_weight([dy], [x], [g], beta=0.5)
    assert bool((g.view(-1, 1 << 20).amin(1) == 1).all()) and bool((g.view(-1, 1 << 20).amax(1) == 1).all())

"""The 8-bit operators' one-time set-up on a device, with failing calls faked on the host: the library's own
objects are linked again with one function replaced."""
import ctypes
import os
import subprocess

import pytest

import sgemm_row_major_gb300 as sg


def linked_with(tmp_path, symbol, c_source):
    """libsgemm with the function `symbol` (its mangled name) replaced by __wrap_<symbol> of `c_source`."""
    from sgemm_row_major_gb300 import build, fp8
    build.build()
    objs = [os.path.join(build.BUILD_DIR, os.path.basename(s) + ".o") for s in build.sources()]
    if not all(os.path.exists(o) for o in objs):
        pytest.skip("the library's objects are not here")
    src, out = str(tmp_path / "fake.c"), str(tmp_path / "libsgemm_fake.so")
    with open(src, "w") as f:
        f.write(c_source)
    subprocess.run([build.nvcc(), *build.ARCH, "-shared", "-Xcompiler", "-fPIC", "-Xlinker", "--wrap=" + symbol, "-o", out, src, *objs,
                    "-cudart", "static"], check=True, capture_output=True)
    return fp8._declare(sg._declare(ctypes.CDLL(out)))


def product_of_ones(lib, n=64):
    """The status of lib.sgemm() on n x n matrices of ones, and its result."""
    import torch
    a, c = torch.ones(n, n, device="cuda"), torch.zeros(n, n, device="cuda")
    st = lib.sgemm(b"N", b"N", n, n, n, 1.0, a.data_ptr(), n, a.data_ptr(), n, 0.0, c.data_ptr(), n, None)
    torch.cuda.synchronize()
    return st, c


def quantize(lib):
    import torch
    x = torch.full((4, 256), 448.0, device="cuda")
    q, s = torch.zeros(4, 256, dtype=torch.uint8, device="cuda"), torch.zeros(4, 2, device="cuda")
    st = lib.sgemm_fp8_quantize(4, 256, x.data_ptr(), 0, 256, 0, 1, 128, q.data_ptr(), 256, s.data_ptr(), 2, None)
    torch.cuda.synchronize()
    return st, s


@pytest.mark.gpu
def test_a_failed_setup_of_8_bit_kernels_leaves_the_others_alone(tmp_path):
    """Only 8-bit calls set up 8-bit kernels: where that fails they report it, and are set up by a later call, while an
    FP32 product neither waits for it nor fails with it."""
    name = "_ZN10sgemm_impl17prepare_fp8_shortEv"
    lib = linked_with(tmp_path, name, f"""
        int fake_calls, fake_error = 1;
        int __real_{name}(void);
        int __wrap_{name}(void) {{ ++fake_calls; return fake_error ? fake_error : __real_{name}(); }}
    """)
    calls, error = ctypes.c_int.in_dll(lib, "fake_calls"), ctypes.c_int.in_dll(lib, "fake_error")
    st, c = product_of_ones(lib)
    assert st == 0 and bool((c == 64.0).all()) and calls.value == 0
    assert quantize(lib)[0] == sg.STATUS["ERR_CUDA"] and lib.sgemm_last_cuda_error() == 1 and calls.value == 1
    st, c = product_of_ones(lib)
    assert st == 0 and bool((c == 64.0).all())
    error.value = 0
    for _ in range(2):
        st, s = quantize(lib)
        assert st == 0 and bool((s == 1.0).all()) and calls.value == 2


@pytest.mark.gpu
def test_a_product_without_clusters(tmp_path):
    """Where no CTA pair can run, a product takes the short-side kernel with whole tiles; only forced pairs and shares
    of K are refused."""
    import torch
    name = "_ZN10sgemm_impl20tc_pair_max_clustersEPi"
    lib = linked_with(tmp_path, name, f"int __wrap_{name}(int *n) {{ *n = 0; return 1; }}")
    from sgemm_row_major_gb300.fp8 import MatrixStruct
    M, N, K = 300, 260, 1000
    ones = torch.full((300, 1008), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    sa, sb = torch.full((300, 8), 2.0, device="cuda"), torch.full((3, 8), 0.5, device="cuda")
    a, b = MatrixStruct(ones.data_ptr(), 1008, sa.data_ptr(), 8, 0, 1, 128), MatrixStruct(ones.data_ptr(), 1008, sb.data_ptr(), 8, 0, 128, 128)
    d = torch.zeros(M, N, device="cuda")
    args = (b"N", b"T", M, N, K, 1.0, a, b, 0.0, None, N, d.data_ptr(), N, 0)
    plan = sg.PlanStruct()
    assert lib.sgemm_fp8_plan(*args, 0, ctypes.byref(plan)) == 0 and (plan.variant, plan.split_k) == (33, 1)
    assert lib.sgemm_fp8(*args, None) == 0
    torch.cuda.synchronize()
    assert bool((d == float(K)).all())
    for forced in ((32, 0, 0), (33, 0, 2)):
        assert lib.sgemm_fp8_set_override(*forced) == 0
        assert lib.sgemm_fp8(*args, None) == sg.STATUS["ERR_UNSUPPORTED"]
    assert lib.sgemm_fp8_set_override(0, 0, 0) == 0

"""The elementwise pass of the BF16 layers' gradients where rows are many and columns few."""
import ctypes
import os
import subprocess

import pytest

import sgemm_row_major_gb300 as sg
from fp8_util import strided
from linear_util import check_all, linear_grad_ref
from test_fp8_debug import both, dbg  # noqa: F401 (fixtures)
from test_linear import kept_of, rand


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    """shape(rows, cols, activation, dbias, clusters): (columns of a CTA, CTAs that share the rows, whether a cluster adds the sums) on
    152 SMs."""
    from sgemm_row_major_gb300 import build
    library = build.build()
    d = tmp_path_factory.mktemp("shape")
    src, out = str(d / "shape.cu"), str(d / "libshape.so")
    with open(src, "w") as f:
        f.write("""
            #include "linear_internal.h"
            extern "C" void shape(long long rows, int cols, int act, int dbias, int clusters, int* out) {
              sgemm_impl::LinearGradParams p;
              static float sums;
              p.rows = rows;
              p.cols = cols;
              p.act = act;
              p.dbias = dbias ? &sums : nullptr;
              sgemm_impl::shape_linear_grad(&p, clusters != 0, 152);
              out[0] = p.strip;
              out[1] = p.row_blocks;
              out[2] = p.joined;
            }
        """)
    folder, name = os.path.split(library)
    subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-shared", "-o", out, src, "-L" + folder, "-l:" + name, "-Xlinker", "-rpath=" + folder],
                   check=True, capture_output=True)
    f = ctypes.CDLL(out).shape
    f.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]

    def call(rows, cols, activation, dbias, clusters=True):
        got = (ctypes.c_int * 3)()
        f(rows, cols, activation, dbias, clusters, got)
        return tuple(got)
    return call


def test_sums_do_not_leave_the_chip_idle(shape):
    """A pass over many rows has at least as many CTAs as the chip has SMs, whether the sums are wanted or not; over few rows a
    cluster adds them, with no second kernel."""
    for rows, activations in ((8193, (2,)), (16384, (1, 4)), (32769, (0, 2)), (65536, (0, 3)), (1 << 20, (0, 2))):
        for cols in (1, 64, 200, 256, 512, 1000, 1024, 1216, 1217, 4096, 5000, 40000):
            for activation in activations:
                for clusters in (True, False):
                    for dbias in (0, 1):
                        strip, blocks, joined = shape(rows, cols, activation, dbias, clusters)
                        assert -(-cols // strip) * blocks >= 152, (rows, cols, activation, dbias, clusters)
                        assert 32 * (blocks - 1) < rows and blocks <= 65535 and (not joined or blocks <= 8)
    for rows, activation in ((1, 0), (31, 2), (256, 2), (1000, 1), (8192, 3), (32768, 0)):
        for cols in (1, 64, 200, 1024):
            strip, blocks, joined = shape(rows, cols, activation, 1)
            assert (strip, joined) == (64, 1) and blocks <= min(8, -(-rows // 32))


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["bf16", "fp8"])
@pytest.mark.parametrize("activation", [None, "relu", "gelu"])
@pytest.mark.parametrize("T,O", [(513, 8), (8200, 8), (16384, 64), (33000, 64), (65536, 200), (8193, 1216), (5000, 1217)])
def test_many_rows_of_few_columns(T, O, activation, how):
    import torch
    if activation is None and how == "fp8":
        pytest.skip("nothing is kept without an activation")
    dy, x, w = rand(1, T, O, std=0.1), rand(2, T, 24), rand(3, O, 24)
    pre = kept_of(rand(4, T, O), how) if activation else None
    for d in (dy, strided(dy, 3, 1)):
        got = sg.linear_bf16_backward(d, x, w, pre, activation, dbias=True, dweight_dtype=torch.float32)
        check_all(got, linear_grad_ref(dy, x, w, pre, activation))
        again = sg.linear_bf16_backward(d, x, w, pre, activation, dbias=True, dweight_dtype=torch.float32)
        assert all(torch.equal(p, q) for p, q in zip(got, again))
    assert sg.sgemm_sync_status() == 0


@pytest.mark.gpu
def test_many_rows_of_few_columns_in_bounds(both):  # noqa: F811
    for T, O in ((8200, 8), (33000, 64), (33000, 200), (8193, 1216)):
        dy, a = rand(1, T, O), rand(2, T, O)
        for d, pre in ((dy, a), (strided(dy, 3, 1), sg.quantize_fp8(a))):
            both(lambda: tuple(sg.linear_bf16_backward(d, None, None, pre, "gelu", dx=False, dweight=False, dbias=True)), (T, O))
            both(lambda: tuple(sg.linear_bf16_backward(d, None, None, dx=False, dweight=False, dbias=True)), (T, O))

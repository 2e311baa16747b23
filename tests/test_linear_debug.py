"""The BF16 layers through the bounds-checking build (libsgemm_debug.so), and their one-time set-up with failing calls faked on
the host."""
import ctypes

import pytest

import sgemm_row_major_gb300 as sg
from fp8_util import strided
from linear_util import ACTS
from test_fp8_debug import both, dbg  # noqa: F401 (fixtures)
from test_fp8_setup import linked_with, product_of_ones, quantize
from test_linear import KERNELS, rand, strided_codes

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 1), (3, 7, 5), (17, 130, 33), (130, 520, 264), (257, 600, 129), (300, 72, 713)]


@pytest.fixture
def force(dbg):  # noqa: F811
    """force(kernel, tile, split) in both builds, for one test."""
    from sgemm_row_major_gb300 import linear
    linear._declare(dbg)

    def set_(variant="AUTO", tile=0, split=0):
        sg.sgemm_linear_set_override(variant, tile, split)
        assert dbg.sgemm_linear_set_override({"AUTO": 0, "LINEAR_PAIR": 40, "LINEAR_SHORT": 41}[variant], tile, split) == 0
    yield set_
    set_()


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: f"{k[0]}{k[1]}_{k[2]}")
def test_every_kernel(both, force, kernel):  # noqa: F811
    import torch
    force(*kernel)
    for i, (T, I, O) in enumerate(SHAPES):
        pad, offset = ((0, 0), (8, 0), (3, 1))[i % 3]
        x, w, u, r, dy, a = (strided(v, pad, offset) for v in (rand(1, T, I), rand(2, O, I), rand(3, O, I), rand(4, T, O), rand(5, T, O), rand(6, T, O)))
        b = rand(7, 1, O)[0]
        for k, save in enumerate((None, "bf16", "fp8")):
            act = ACTS[(i + k) % 5]
            dtype = (torch.bfloat16, torch.float32)[k % 2]
            out = torch.zeros(T, O, dtype=dtype, device="cuda")
            both(lambda: tuple(sg.linear_bf16(x, w, b, act, r, save=save, out=strided(out, pad, offset))), (T, I, O, save))
            both(lambda: tuple(sg.linear_bf16(x, w, None, act, save=save, out_dtype=dtype)), (T, I, O, save))
            both(lambda: tuple(sg.gated_bf16(x, w, u, act, save=save)), (T, I, O, save))
        q, qx = sg.quantize_fp8(a), sg.quantize_fp8(x)
        odd = sg.Fp8Matrix(strided_codes(q.data, 3, 1), strided(q.scale, 1))
        for pre, xx in ((a, x), (q, qx), (odd, x)):
            both(lambda: tuple(sg.linear_bf16_backward(dy, xx, w, pre, "silu", dbias=True, dweight_dtype=torch.float32)), (T, I, O))
            both(lambda: tuple(sg.gated_bf16_backward(dy, xx, w, u, pre, pre, "gelu", h=True)), (T, I, O))
        both(lambda: tuple(sg.linear_bf16_backward(dy, x, w, dbias=True)), (T, I, O))


def test_wide_gradients(both):  # noqa: F811
    """Strips of 256 columns with the sums in a second kernel, rows that end inside a chunk."""
    for T, O in ((3000, 5000), (2500, 6004), (700, 40000)):
        dy, a, b = rand(1, T, O), rand(2, T, O), rand(3, T, O)
        q = sg.quantize_fp8(a)
        for pre in (a, q):
            both(lambda: tuple(sg.linear_bf16_backward(dy, None, None, pre, "gelu", dx=False, dweight=False, dbias=True)), (T, O))
        both(lambda: tuple(sg.gated_bf16_backward(dy, None, None, None, a, b, dx=False, dweights=False, h=True)), (T, O))


def layer_of_ones(lib, T=64, I=64, O=64):
    """The status of lib.sgemm_linear() on ones, and its result."""
    import torch
    from sgemm_row_major_gb300 import linear
    linear._declare(lib)
    x, w = torch.ones(T, I, dtype=torch.bfloat16, device="cuda"), torch.ones(O, I, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(T, O, device="cuda")
    st = lib.sgemm_linear(T, I, O, x.data_ptr(), I, w.data_ptr(), I, None, 0, None, 0, None, y.data_ptr(), O, 0, None)
    torch.cuda.synchronize()
    return st, y


def test_a_failed_setup_leaves_the_others_alone(tmp_path):
    """Only calls of this part set up its kernels: where that fails they report it and are set up by a later call, while FP32
    and 8-bit calls neither wait for it nor fail with it."""
    name = "_ZN10sgemm_impl20prepare_linear_shortEv"
    lib = linked_with(tmp_path, name, f"""
        int fake_calls, fake_error = 1;
        int __real_{name}(void);
        int __wrap_{name}(void) {{ ++fake_calls; return fake_error ? fake_error : __real_{name}(); }}
    """)
    calls, error = ctypes.c_int.in_dll(lib, "fake_calls"), ctypes.c_int.in_dll(lib, "fake_error")
    st, c = product_of_ones(lib)
    assert st == 0 and bool((c == 64.0).all()) and quantize(lib)[0] == 0 and calls.value == 0
    assert layer_of_ones(lib)[0] == sg.STATUS["ERR_CUDA"] and lib.sgemm_last_cuda_error() == 1 and calls.value == 1
    assert product_of_ones(lib)[0] == 0 and quantize(lib)[0] == 0
    error.value = 0
    for _ in range(2):
        st, y = layer_of_ones(lib)
        assert st == 0 and bool((y == 64.0).all()) and calls.value == 2


def test_without_clusters(tmp_path):
    """Where no CTA pair can run, every call takes the short-side kernel with whole tiles; only forced pairs and shares of K
    are refused."""
    import torch
    name = "_ZN10sgemm_impl20tc_pair_max_clustersEPi"
    lib = linked_with(tmp_path, name, f"int __wrap_{name}(int *n) {{ *n = 0; return 1; }}")
    for T, I, O in ((1, 1000, 300), (300, 1000, 260)):
        st, y = layer_of_ones(lib, T, I, O)
        assert st == 0 and bool((y == float(I)).all())
    from sgemm_row_major_gb300.linear import KeptStruct
    T, I, O = 200, 264, 136
    one = lambda r, c: torch.ones(r, c, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    dy, x, w, pre = one(T, O), one(T, I), one(O, I), one(T, O)
    dx, dw, db = torch.zeros(T, I, dtype=torch.bfloat16, device="cuda"), torch.zeros(O, I, device="cuda"), torch.zeros(O, device="cuda")
    assert lib.sgemm_linear_backward(T, I, O, dy.data_ptr(), O, KeptStruct(x.data_ptr(), I, None, 1), w.data_ptr(), I, 1, KeptStruct(pre.data_ptr(), O, None, 1),
                                     dx.data_ptr(), I, dw.data_ptr(), I, 0, db.data_ptr(), None) == 0
    torch.cuda.synchronize()
    assert bool((dx == O).all()) and bool((dw == T).all()) and bool((db == T).all())
    for forced in ((40, 0, 0), (41, 0, 2)):
        assert lib.sgemm_linear_set_override(*forced) == 0
        assert layer_of_ones(lib)[0] == sg.STATUS["ERR_UNSUPPORTED"]
    assert lib.sgemm_linear_set_override(0, 0, 0) == 0

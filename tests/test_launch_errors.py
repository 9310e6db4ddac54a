"""A kernel launch that fails makes its call fail: the library's calls with a
runtime whose launches are counted, not made, and one of which fails. No GPU
is used; a process of its own loads the stand-ins of the runtime's
launch functions before the library."""
import subprocess
import sys

import pytest
from conftest import ROOT

SHIM = """
static int n, at, last;
void shim_reset(int fail_at) { n = 0; at = fail_at; last = 0; }
int shim_launches(void) { return n; }
int __hipPushCallConfiguration(void) { return 0; }
int __hipPopCallConfiguration(void) { return 0; }
int hipLaunchKernel(void) { return n++ == at ? (last = 701) : 0; }
int hipGetLastError(void) { int e = last; last = 0; return e; }
"""

RUN = """
import ctypes, itertools, sys
shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
from unstructured_sparse_feedforward_amd import binding as B
lib, P, R = B.load_library(), 1 << 20, ctypes.byref

def check(what, call):
    '''Every launch of the call in turn fails.'''
    shim.shim_reset(-1)
    st = call()
    n = shim.shim_launches()
    if st != B.SFFN_OK or n < 1:
        print(what, "status", st, "launches", n)
    for i in range(n):
        shim.shim_reset(i)
        st = call()
        if st != B.SFFN_E_HIP:
            print(what, "launch", i, "of", n, "failed, status", st)

which = sys.argv[2]
if which == "route":
    for E, (groups, top), T, bias, sig, norm in itertools.product(
            (8, 64, 100, 128, 256, 500, 512, 1000, 1024), ((1, 1), (4, 2)), (1, 5000, 20000),
            (None, P), (0, 1), (0, 1)):
        D = B.SffnRouteDesc(E, 4, groups, top, 1, sig, norm, 1.0)
        what = ("route", E, groups, T, bias, sig, norm)
        check(what, lambda: lib.sffn_route(R(D), P, 0, T, E, bias, None, P, P, None))
        check(what, lambda: lib.sffn_route_backward(R(D), P, P, 0, T, E, P, None, P << 20, 0, E, None))
elif which == "norm":
    COLS = (1, 8, 500, 1000, 2000, 4000, 8000, 16000)
    for rows, cols, out in itertools.product((1, 700, 9000), COLS, (0, 1, 3)):
        a = B.SffnNorm(P, P, P, P, P << 20, P if out == 3 else None, P, cols, cols, cols, cols, 0, 0, 0, out)
        check(("norm", rows, cols, out), lambda: lib.sffn_rms_norm(R(a), rows, cols, 1e-6, None, None))
    for rows, cols, ds, dw in itertools.product((0, 1, 700, 9000), COLS, (P, P << 20), (None, P << 21)):
        if rows == 0 and dw is None:
            continue
        a = B.SffnNormGrad(P, P << 10, None, P, P, ds, dw, cols, cols, cols, cols, 0, 0, 0, 0, 0)
        check(("norm grad", rows, cols, ds, dw),
              lambda: lib.sffn_rms_norm_backward(R(a), rows, cols, P, 1 << 30, None))
elif which == "mx":
    for dt, rows, cols in itertools.product((0, 1), (1, 700), (1, 3000)):
        w = ("mx", dt, rows, cols)
        for t in (0, 1):
            check(w, lambda: lib.sffn_mx_quantize(P, dt, rows, cols, cols, t, P, P, None))
        check(w, lambda: lib.sffn_mx8_quantize(P, dt, rows, cols, cols, P, P, None))
        for f in (lib.sffn_mx_dequantize, lib.sffn_mx8_dequantize):
            check(w, lambda: f(P, P, rows, cols, P, dt, cols, None))
    for f, dt, M, N, K in itertools.product((lib.sffn_mx_matmul, lib.sffn_mx8_matmul), (0, 1),
                                            (1, 10, 100, 1000, 8192), (1, 2000, 5632, 16384),
                                            (0, 64, 2048, 8192)):
        check(("product", dt, M, N, K), lambda: f(P, P, M, P, P, N, K, P, dt, N, None))
else:
    for T, E, k, mx, gated in itertools.product((1, 3, 200), (8, 64, 256), (1, 4), (1, 2), (0, 1)):
        D = B.SffnMoeDesc(d=256, d_ff=96, n_experts=E, top_k=k, gated=gated, normalize=1, weights=mx)
        s = P if mx == 2 else None
        w = B.SffnMoeWeights(router=P, gate=P, up=P if gated else None, down=P, gate_scales=s,
                             up_scales=s if gated else None, down_scales=s)
        what = ("experts", T, E, k, mx, gated)
        check(what, lambda: lib.sffn_moe_forward(R(D), P, R(w), T, None, P, P, P, P, 1 << 30, None))
        w.router = None
        check(what, lambda: lib.sffn_moe_forward_chosen(R(D), P, R(w), T, None, P, P, P, P, 1 << 30, None))
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("shim")
    (d / "shim.c").write_text(SHIM)
    subprocess.run(["gcc", "-shared", "-fPIC", str(d / "shim.c"), "-o", str(d / "shim.so")], check=True)
    return str(d / "shim.so")


@pytest.mark.parametrize("which", ["route", "norm", "mx", "experts"])
def test_failed_launch_is_an_error(shim, which):
    r = subprocess.run([sys.executable, "-c", RUN, shim, which], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout == "", r.stdout[:2000]

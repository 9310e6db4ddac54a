"""Results in the place of operands: a call whose result shares some of an
operand's memory, but not row by row, is refused (workgroups would write what
others have yet to read), and no other call is. Launches are counted, not made
(the stand-ins of test_launch_errors.py); the oracle compares the bytes of the
two matrices."""
import subprocess
import sys

from conftest import ROOT
from test_launch_errors import shim  # noqa: F401  (the fixture)

RUN = """
import ctypes, random, sys
shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
from unstructured_sparse_feedforward_amd import binding as B
lib, P, R = B.load_library(), 1 << 20, ctypes.byref
rng = random.Random(7)
SIZE = (4, 2)

class Place:
    def __init__(self, rows, cols, dtype, ld, at):
        self.rows, self.cols, self.dtype, self.ld, self.at = rows, cols, dtype, ld, at
    def bytes(self):
        e = SIZE[self.dtype]
        return {self.at + i * self.ld * e + j for i in range(self.rows) for j in range(self.cols * e)}
    def meets(self, o):
        '''0: apart, 1: the same rows in the same places, 2: otherwise'''
        if not self.bytes() & o.bytes():
            return 0
        same = self.at == o.at and self.dtype == o.dtype and (self.rows == 1 or self.ld == o.ld)
        return 1 if same else 2

def near(rows, cols, others):
    '''A matrix that may be one of the others, a view beside it, or anything near it.'''
    o = rng.choice(others) if others else None
    if o is None or rng.random() < 0.2:
        d = rng.randrange(2)
        return Place(rows, cols, d, cols + rng.randrange(2 * cols + 4), P + 4 * rng.randrange(60))
    if rng.random() < 0.3:
        return Place(rows, cols, o.dtype, o.ld, o.at)
    d = o.dtype if rng.random() < 0.8 else 1 - o.dtype
    ld = o.ld if rng.random() < 0.7 else cols + rng.randrange(2 * cols + 4)
    at = o.at + 4 * rng.choice((0, 0, cols, -cols, o.ld, -o.ld, rng.randrange(-80, 80)))
    return Place(rows, cols, d, ld, max(at, P))

seen = {}
def check(what, status, bad, *places):
    want = B.SFFN_E_ARG if bad else B.SFFN_OK
    seen[what, bad] = seen.get((what, bad), 0) + 1
    if status != want:
        print(what, "status", status, "not", want, [vars(p) for p in places if p])

for n in range(20000):
    rows, cols = rng.choice((1, 2, 3, 5)), rng.choice((1, 4, 9))
    x = near(rows, cols, [])
    res = near(rows, cols, [x]) if rng.random() < 0.7 else None
    ro = None
    if res:
        ro = near(rows, cols, [x, res])
        ro.dtype = res.dtype
    mx8 = rng.random() < 0.1
    if mx8:
        out = Place(rows, 64, 1, 64, P // 128 * 128 + 16 * rng.randrange(60))       # 128 bytes a row
    else:
        out = near(rows, cols, [p for p in (x, res, ro) if p])
    a = B.SffnNorm(x.at, res and res.at, ro and ro.at, None, out.at, P << 10 if mx8 else None, None,
                   x.ld, res.ld if res else 0, ro.ld if ro else 0, out.ld, x.dtype,
                   res.dtype if res else 0, 0, 3 if mx8 else out.dtype)
    bad = out.meets(x) == 2 or mx8 and out.meets(x) > 0
    if res:
        bad = (bad or ro.meets(x) == 2 or ro.meets(res) == 2 or out.meets(res) == 2 or out.meets(ro) > 0
               or mx8 and out.meets(res) > 0)
    shim.shim_reset(-1)
    check("norm", lib.sffn_rms_norm(R(a), rows, cols, 1e-6, None, None), bad, x, res, ro, out)

    dy = near(rows, cols, [])
    s = near(rows, cols, [dy])
    di = near(rows, cols, [dy, s]) if rng.random() < 0.6 else None
    ds = near(rows, cols, [p for p in (dy, s, di) if p])
    a = B.SffnNormGrad(dy.at, s.at, di and di.at, P << 11, P << 12, ds.at, P << 13, dy.ld, s.ld,
                       di.ld if di else 0, ds.ld, dy.dtype, s.dtype, di.dtype if di else 0, 0, ds.dtype)
    bad = any(p is not None and ds.meets(p) == 2 for p in (dy, s, di))
    if rng.random() < 0.2:       # the weight and its gradient, float32 or bfloat16 and float32
        wd = rng.randrange(2)
        a.weight, a.weight_dtype, a.dweight = P << 13, wd, (P << 13) + 4 * rng.randrange(-12, 13)
        bad = bad or a.weight < a.dweight + 4 * cols and a.dweight < a.weight + cols * SIZE[wd]
    check("norm grad", lib.sffn_rms_norm_backward(R(a), rows, cols, P << 14, 1 << 20, None), bad, dy, s,
          di, ds)

    l = near(rows, cols, [])
    dl = near(rows, cols, [l])
    D = B.SffnRouteDesc(cols, 1, 1, 1, 1, 0, 1, 1.0)
    check("route grad", lib.sffn_route_backward(R(D), P << 11, l.at, l.dtype, rows, l.ld, P << 12, None,
                                                dl.at, dl.dtype, dl.ld, None), dl.meets(l) == 2, l, dl)
for what in ("norm", "norm grad", "route grad"):
    for bad in (False, True):
        assert seen[what, bad] > 1000, seen
"""


def test_in_place_or_apart(shim):  # noqa: F811
    r = subprocess.run([sys.executable, "-c", RUN, shim], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout == "", r.stdout[:3000]

"""The products of 8-bit with 4-bit matrices copy operands into rings in LDS
and wait for them by hand, as the 4-bit products do: these tests compile
their file to gfx950 assembly (no GPU) and check that every such wait leaves
no copy of the slot it is for in flight, on every path, and that slots are
read and written in turn."""
import pytest

from test_asm_ring_waits import _asm, _kernels, Code, _ring

# by template arguments: a stage's copies, the stages in flight after the
# prologue's copies, the copies of it that the prologue leaves out, what is
# left after the last steady wait before the ring's end
KERNELS = {
    "mx8_few_kernel": {"Li4": (5, 2, 0), "Li8": (5, 2, 0)},
    "mx8_mid_kernel": {"Li1ELi2": (10, 2, 0), "Li2ELi2": (14, 2, 0)},
    "mx8_big_kernel": {"Li2ELi2ELi3": (8, 3, 3), "Li2ELi4ELi2": (10, 2, 5),
                       "Li4ELi4ELi3": (14, 3, 5)},
}


def _faults(code, name, per, slots, missing):
    """A wait with n operations left, of which at most n can be copies, is right
    for a slot if more copies than n came after the slot's: of the copies issued
    so far (per a stage, in order) those of the stage that is read next have to
    lie before the last n."""
    big = name == "mx8_big_kernel"
    w = code.waits()
    bad = []
    # the first wait: all but `missing` copies of `slots` stages are out, and the
    # oldest stage has to have landed
    first = code.copies_until(0, set(w))
    for i, n in first.items():
        if n == {0}:            # (a wave without a share goes to the last wait)
            if code.ins[i][1] != 0:
                bad.append(("empty", i))
        elif n != {slots * per - missing} or code.ins[i][1] != (slots - 1) * per - missing:
            bad.append(("first", i, n, code.ins[i][1]))
    starts = {i for i, n in first.items() if n != {0}}
    if len(starts) != 1:
        return bad + [("first waits", starts)]
    # every other: a stage's copies since the last one, and again all but the
    # next stage's left (of the large tiles a stage earlier: their wait is for the
    # next stage, in the middle of one)
    left = (slots - 2 if big else slots - 1) * per
    for i in w:
        for s in code.succ[i]:
            for j, n in code.copies_until(s, set(w)).items():
                want = {missing} if big and i in starts else {per}
                if code.ins[j][1] == 0 and not (big and slots == 2):
                    continue    # everything has landed
                if code.ins[j][1] == 0 and n != want:
                    continue
                if n != want or code.ins[j][1] != left:
                    bad.append(("between", i, j, n, code.ins[j][1]))
    if not any(code.ins[i][1] == 0 for i in w):
        bad.append(("no last wait",))
    if any(k[0] == "load" for k in code.ins):
        bad.append(("loads into registers",))
    return bad


def test_rings(tmp_path):
    lines = _asm(tmp_path, "mx8_gemm")
    checked = 0
    for name, kinds in KERNELS.items():
        codes = _kernels(lines, name)
        assert len(codes) == 2 * len(kinds), sorted(codes)      # two result types each
        for args, code in codes.items():
            key = next(k for k in kinds if args.startswith(k + "E"))
            assert not _faults(code, name, *kinds[key]), (name, args)
            if name != "mx8_big_kernel":     # (there the halves of a stage overlap)
                assert not code.order_faults(), (name, args)
            checked += 1
    assert checked == 14


@pytest.mark.parametrize("per", [4, 5])
def test_the_check(per):
    """On a plain ring; one copy more or less a pass or before it is found."""
    assert not _faults(Code(_ring(per)), "mx8_few_kernel", per, 2, 0)
    for kw in (dict(body=per - 1), dict(body=per + 1), dict(first=2 * per - 1),
               dict(first=2 * per + 1)):
        assert _faults(Code(_ring(per, **kw)), "mx8_few_kernel", per, 2, 0)

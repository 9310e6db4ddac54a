"""The MXFP4 products and the expert layer's hidden kernel copy operands into
rings in LDS and wait for them by hand: s_waitcnt vmcnt(N) before a slot is
read, N being the vector-memory operations that were issued after the
slot's copies. A compiler that merged, dropped or moved one of those
operations would make such a wait return too early, and the slot would be
read before its copies have landed.

These tests compile the two files to gfx950 assembly (no GPU) and check
that, on every path of every kernel's control-flow graph:
  * the products issue one stage's copies, no more and no fewer, between two
    waits, and the stages' number of them before the first;
  * in the hidden kernel, of the N youngest operations at a wait, no more
    are copies than the steps that may be in flight have;
  * a slot is read after its wait and before the wait that frees it, and
    copies are issued after that one.
"""
import os
import re
import subprocess

import pytest

from unstructured_sparse_feedforward_amd import build as B

WINDOW = 64        # the counter's largest value, and 0


def _asm(tmp_path, name):
    try:
        cc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    out = tmp_path / (name + ".s")
    cmd = [cc, *[f for f in B.FLAGS if f != "-fPIC"], "--cuda-device-only", "-S",
           os.path.join(B.CSRC, name + ".hip"), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return out.read_text().split("\n")


class Code:
    """A kernel's instructions, each one of
    ('copy',), ('load',), ('store',)   vector memory: into LDS, into registers, out
    ('wait', vm or None, lgkm or None, explicit)
    ('read',) ('write',) ('barrier',)  of LDS
    ('op',)
    and succ[i], the instructions that may follow i. A wait that the source
    asks for stands behind a scheduling barrier."""

    def __init__(self, lines):
        self.ins, self.text, labels, prev, jumps = [], [], {}, "", []
        for l in lines:
            t = l.strip()
            m = re.match(r"^(\.LBB\d+_\d+):", t)
            if m:
                labels[m.group(1)] = len(self.ins)
            elif t.startswith("; sched_barrier mask(0x00000000)"):
                prev = "barrier"
            elif t and t[0] not in ";." and not t.endswith(":"):
                self.ins.append(self._kind(t, prev == "barrier"))
                self.text.append(t)
                m = re.match(r"s_c?branch\w* (\.LBB\d+_\d+)", t)
                jumps.append((m.group(1) if m else None,
                              not re.match(r"s_(branch|endpgm|setpc)", t)))
                prev = ""
        assert not any(re.match(r"s_(setpc|swappc|getpc)", l.strip()) for l in lines), "a call"
        self.succ = []
        for i, (to, falls) in enumerate(jumps):
            s = [labels[to]] if to else []
            if falls and i + 1 < len(jumps):
                s.append(i + 1)
            self.succ.append(s)

    @staticmethod
    def _kind(t, marked):
        op = t.split()[0]
        if op == "s_waitcnt":
            vm, lg = re.search(r"vmcnt\((\d+)\)", t), re.search(r"lgkmcnt\((\d+)\)", t)
            return ("wait", int(vm.group(1)) if vm else None, int(lg.group(1)) if lg else None,
                    marked)
        if re.match(r"(global|buffer|flat|scratch)_load", op):
            return ("copy",) if re.search(r"\blds\b", t) else ("load",)
        if re.match(r"(global|buffer|flat|scratch)_(store|atomic)", op):
            return ("store",)
        if op.startswith("ds_read"):
            return ("read",)
        if op.startswith("ds_write"):
            return ("write",)
        return ("barrier",) if op == "s_barrier" else ("op",)

    def waits(self):
        """The explicit waits for vector memory, by index."""
        return [i for i, k in enumerate(self.ins) if k[0] == "wait" and k[3] and k[1] is not None]

    def copies_until(self, start, stops):
        """The numbers of copies on the paths from `start` to the first of
        `stops`: {stop: set of numbers}."""
        found, seen, stack = {}, set(), [(start, 0)]
        while stack:
            i, n = stack.pop()
            if (i, n) in seen or n > WINDOW:
                continue
            seen.add((i, n))
            if i in stops:
                found.setdefault(i, set()).add(n)
                continue
            n += self.ins[i][0] == "copy"
            stack.extend((s, n) for s in self.succ[i])
        return found

    def young_copies(self):
        """For each instruction the most copies among the j youngest
        operations in flight before it, j = 0 .. WINDOW, over all paths."""
        at = [None] * len(self.ins)
        at[0] = (0,) * (WINDOW + 1)
        todo = [0]
        while todo:
            i = todo.pop()
            v, k = at[i], self.ins[i]
            if k[0] == "copy":
                v = (0,) + tuple(x + 1 for x in v[:-1])
            elif k[0] in ("load", "store"):
                v = (0,) + v[:-1]
            elif k[0] == "wait" and k[1] is not None:
                v = v[:k[1]] + (v[k[1]],) * (WINDOW + 1 - k[1])
            for s in self.succ[i]:
                w = v if at[s] is None else tuple(map(max, v, at[s]))
                if w != at[s]:
                    at[s] = w
                    todo.append(s)
        return at

    def _follow(self, i, flags):
        """The instructions that may follow i, with what is known of scalar
        pairs there. The compiler joins the sides of an if and else through
        such a pair: set to 0 or -1, masked into vcc, branched on."""
        t, known = self.text[i], dict(flags)
        m = re.match(r"s_cbranch_vcc(n?)z", t)
        if m and "vcc" in known:
            taken = (known["vcc"] != 0) == (m.group(1) == "n")
            return [(self.succ[i][0 if taken else 1], flags)]
        m = re.match(r"(\w+) (vcc|s\[\d+:\d+\]|s\d+)(?:, (.*))?$", t.split(";")[0].strip())
        if m and not t.startswith(("s_cmp", "s_bitcmp")):
            op, dst, src = m.groups()
            value = None
            if op == "s_mov_b64" and src in ("0", "-1"):
                value = int(src)
            q = re.fullmatch(r"exec, (s\[\d+:\d+\])", src or "")
            if op in ("s_andn2_b64", "s_and_b64") and q and q.group(1) in known:
                value = known[q.group(1)] if op == "s_and_b64" else -1 - known[q.group(1)]
            a = [int(v) for v in re.findall(r"\d+", dst)]
            for k in list(known):       # what the destination overlaps
                b = [int(v) for v in re.findall(r"\d+", k)]
                if k == dst or (a and b and a[0] <= b[-1] and b[0] <= a[-1]):
                    del known[k]
            if value is not None:
                known[dst] = value
        elif "vcc" in t and t.startswith(("v_", "s_mov", "s_and", "s_or")):
            known.pop("vcc", None)
        return [(s, frozenset(known.items())) for s in self.succ[i]]

    def order_faults(self):
        """Copies between a slot's wait and the wait for its reads (one for
        LDS, to which the compiler may add what it waits for itself), and
        reads from there to the next slot's wait, or to a write or barrier,
        which end a ring's use."""
        slot = {i for i in self.waits() if self.ins[i][2] is None}
        freed = {i for i, k in enumerate(self.ins) if k[0] == "wait" and k[3] and k[2] == 0}
        end = {i for i, k in enumerate(self.ins) if k[0] in ("write", "barrier")}

        def reach(start, stops, wrong):
            stack, seen, met = [(s, frozenset()) for s in self.succ[start]], set(), set()
            while stack:
                i, flags = stack.pop()
                if (i, flags) in seen:
                    continue
                seen.add((i, flags))
                if i in stops:
                    met.add(i)
                elif self.ins[i][0] == wrong:
                    bad.append((start, i, wrong))
                else:
                    stack.extend(self._follow(i, flags))
            return met
        bad = []
        for w in slot:
            for f in reach(w, freed | slot | end, "copy"):
                if f in freed:
                    reach(f, slot | freed | end, "read")
        return bad


def _kernels(lines, name):
    """{template arguments: Code} of a kernel's instantiations."""
    out = {}
    starts = [i for i, l in enumerate(lines) if re.match(r"^_Z\w+:", l)]
    for a, b in zip(starts, starts[1:] + [len(lines)]):
        m = re.match(r"^_Z\w*?" + name + r"I(\w+?)EEvNS", lines[a])
        if not m:
            continue
        end = next(i for i in range(a, b) if lines[i].startswith(".Lfunc_end"))
        out[m.group(1)] = Code(lines[a + 1:end])
    return out


# stage's copies, slots, the steady wait's operations left, the first wait's
PRODUCTS = {
    "mx_few_kernel": {"Li4": (4, 2, 4, 4), "Li8": (4, 2, 4, 4)},
    "mx_mid_kernel": {"Li1": (8, 2, 8, 8), "Li2": (10, 2, 10, 10)},
    "mx_big_kernel": {"Li2ELi3": (8, 3, 8, 11), "Li4ELi4": (10, 4, 20, 25)},
}


def _product_faults(code, per, slots, left, left0):
    """What is wrong with a product kernel's waits."""
    bad, w = [], code.waits()
    steady = [i for i in w if code.ins[i][1] == left]
    first = [i for i in w if code.ins[i][1] == left0]
    final = [i for i in w if code.ins[i][1] == 0]
    if len(steady) != 1 or len(first) != 1 or not final or len(set(steady + first + final)) != len(w):
        return [("waits", [code.ins[i] for i in w])]
    # before the first wait: it leaves all but one stage's copies
    n = code.copies_until(0, set(first)).get(first[0])
    if n != {left0 + per}:
        bad.append(("before the first wait", n))
    n = code.copies_until(0, set(steady)).get(steady[0])
    if n != {slots * per}:
        bad.append(("before the steady wait", n))
    n = {m for s in code.succ[steady[0]]
         for m in code.copies_until(s, set(steady)).get(steady[0], set())}
    if n != {per}:
        bad.append(("between steady waits", n))
    # nothing else that the counter counts down stands in the loop but stores
    if any(k[0] == "load" for k in code.ins):
        bad.append(("loads into registers",))
    return bad


def test_product_rings(tmp_path):
    lines = _asm(tmp_path, "mx_gemm")
    checked = 0
    for name, kinds in PRODUCTS.items():
        codes = _kernels(lines, name)
        assert len(codes) == 2 * len(kinds), sorted(codes)      # two result types each
        for args, code in codes.items():
            key = next(k for k in kinds if args.startswith(k + "E"))
            assert not _product_faults(code, *kinds[key]), (name, args)
            if name != "mx_big_kernel":     # (there the halves of a stage overlap)
                assert not code.order_faults(), (name, args)
            checked += 1
    assert checked == 12


# operations left at a wait: copies that may be among them. A step of codes is
# two copies of rows, two scale loads and, staged, a copy of x, or four loads
# of it for 16 tokens; of bf16 two copies and two loads for 16 tokens; three
# and five steps are in a ring.
HIDDEN = {1: {10: 6, 16: 4, 24: 4}, 0: {16: 8, 24: 8}}


def _hidden_faults(code, mx, blocks):
    bad = []
    want = {n for n in HIDDEN[mx] if blocks == 2 or n != 24}
    w = code.waits()
    if not want <= {code.ins[i][1] for i in w}:
        bad.append(("waits", sorted({code.ins[i][1] for i in w})))
    young = code.young_copies()
    for i in w:
        n = code.ins[i][1]
        if n in want and young[i][n] > HIDDEN[mx][n]:
            bad.append((i, n, young[i][n]))
    return bad + code.order_faults()


def test_hidden_rings(tmp_path):
    codes = _kernels(_asm(tmp_path, "moe"), "moe_hidden_kernel")
    assert len(codes) == 12, sorted(codes)
    for args, code in codes.items():
        m = re.fullmatch(r"Lb([01])ELb[01]ELb[01]ELi([12])E", args)
        assert m, args
        assert not _hidden_faults(code, int(m.group(1)), int(m.group(2))), args


# ---------------------------------------------------------------- the checks themselves

_W = ["; sched_barrier mask(0x00000000)", "s_waitcnt vmcnt(%d)"]
_COPY = "buffer_load_dwordx4 v4, s[20:23], 0 offen lds"
_FREE = ["; sched_barrier mask(0x00000000)", "s_waitcnt lgkmcnt(0)"]


def _ring(per=4, slots=2, body=None, first=None):
    """A product's loop in assembly, with `body` copies a pass."""
    return ([_COPY] * (slots * per if first is None else first) + [".LBB0_1:", _W[0], _W[1] % (per * (slots - 1)),
            "ds_read_b128 v[0:3], v8"] + _FREE + [_COPY] * (per if body is None else body)
            + ["v_mfma_f32 a0", "s_cbranch_scc1 .LBB0_1", _W[0], _W[1] % 0, "s_endpgm"])


def test_the_check_on_a_product():
    assert not _product_faults(Code(_ring()), 4, 2, 4, 4) and not Code(_ring()).order_faults()
    for body, first in ((3, None), (5, None), (None, 7), (None, 9)):
        assert _product_faults(Code(_ring(body=body, first=first)), 4, 2, 4, 4)
    # a copy before the slot's reads are done, a read after
    t = _ring()
    at = t.index("ds_read_b128 v[0:3], v8")
    assert Code(t[:at] + [_COPY] + t[at:]).order_faults()
    assert Code(t[:-4] + ["ds_read_b128 v[0:3], v8"] + t[-4:]).order_faults()
    # a register load in the loop
    assert _product_faults(Code(t[:at] + ["global_load_dword v1, v2, s[0:1]"] + t[at:]), 4, 2, 4, 4)


def test_the_check_on_hidden_steps():
    load = "global_load_dwordx4 v[0:3], v8, s[0:1]"

    def steps(mx, step, left):
        d = 3 if mx else 5
        return Code(step * d + [".LBB0_1:", _W[0], _W[1] % left, "ds_read_b128 v[0:3], v8"] + _FREE
                    + step + ["s_cbranch_scc1 .LBB0_1", "s_endpgm"])

    def faults(mx, step, left):
        c = steps(mx, step, left)
        i = c.waits()[0]
        return c.young_copies()[i][left] > HIDDEN[mx][left]
    assert not faults(0, [_COPY] * 2 + [load] * 2, 16)
    assert not faults(1, [_COPY] * 2 + [load] * 2 + [_COPY], 10)
    # loads of x merged or gone: with enough of them the wait leaves a copy of
    # the step it is for
    assert faults(0, [_COPY] * 2 + [load], 16)
    assert faults(1, [_COPY] * 2 + [load] + [_COPY], 10)
    assert faults(1, [_COPY] * 2 + [load] * 3, 16)

"""How a CTA pair of the head-loss products ends when a wait has given up: the host build of the rule
(csrc/pair_exit.cuh) in a model of the pair's barriers, over every point at which the two producers can
have stopped, and the order of the steps in the kernel's source.

The model: the MMAs have consumed iterations [0, c). A producer fills iteration j once the MMAs that read
j - STAGES are done, so CTA r has issued n_r in [c, c + STAGES] iterations. Iteration j's barrier completes
when the first CTA has armed it (which it does as it issues j) and both CTAs' copies of j have landed."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ternary_weight_matmul_b200", "csrc")
STAGES = 5


class Exit(ctypes.Structure):
    _fields_ = [("start", ctypes.c_uint32), ("to", ctypes.c_uint32), ("drain", ctypes.c_uint32)]


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("pair_exit")
    src, out = d / "rule.cpp", d / "rule.so"
    src.write_text('#include "pair_exit.cuh"\n'
                   'extern "C" mmf::PairExit rule(uint32_t a, uint32_t b, uint32_t s) { return mmf::pair_exit(a, b, s); }\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(out), str(src)], check=True)
    f = ctypes.CDLL(str(out)).rule
    f.restype, f.argtypes = Exit, [ctypes.c_uint32] * 3
    return lambda mine, other: (lambda e: (e.start, e.to, e.drain))(f(mine, other, STAGES))


def points():
    for c in (0, 1, 3, 5, 12):
        for n0 in range(c, c + STAGES + 1):
            for n1 in range(c, c + STAGES + 1):
                yield c, n0, n1


def end_of(c, n, plans):
    """(copies that may still be in flight at the end, barriers waited for that can never complete, slots
    filled before their last reader was done) when CTA r ends by plans[r] = (start, to) issued and the first
    CTA waits for the barriers [drain, end)."""
    done = list(n)
    early = []
    for r in (0, 1):
        start, to = plans[r][:2]
        early += [j for j in range(start, to) if j >= c + STAGES]
        done[r] = max(done[r], to)
    drain, end = plans[2]
    waited = [j for j in range(drain, end)]
    never = [j for j in waited if j >= done[0] or j >= done[1]]
    settled = set(range(c)) | {j for j in waited if j not in never}
    flying = [(r, j) for r in (0, 1) for j in range(done[r]) if j not in settled]
    return flying, never, early


def test_both_ctas_end_with_every_copy_landed(rule):
    for c, n0, n1 in points():
        p0, p1 = rule(n0, n1), rule(n1, n0)
        assert p0[0] == n0 and p1[0] == n1 and p0[1] == p1[1] == max(n0, n1)
        assert end_of(c, (n0, n1), (p0, p1, (p0[2], p0[1]))) == ([], [], []), (c, n0, n1)


def test_the_model_sees_a_first_cta_that_only_waits_for_its_own_stages():
    """Draining what the first CTA armed, without agreeing on anything, loses copies when the other CTA is
    ahead and waits for barriers that never complete when it is behind."""
    lost = stuck = 0
    for c, n0, n1 in points():
        flying, never, _ = end_of(c, (n0, n1), ((n0, n0), (n1, n1), (max(n0 - STAGES, 0), n0)))
        lost += bool(flying and n1 > n0)
        stuck += bool(never and n1 < n0)
        assert not (n0 == n1 and (flying or never))
    assert lost and stuck


def test_kernel_ends_by_the_rule():
    code = open(os.path.join(CSRC, "head_loss.cuh")).read()
    code = re.sub(r"//[^\n]*", "", code)
    assert int(re.search(r"constexpr int STAGES = (\d+);", code).group(1)) == STAGES
    kernel = code[code.index("head_loss_kernel("):code.index("tmem_dealloc_pair(tmem")]
    publish = kernel.index("st_cluster_u32(in_cta(")
    teardown = kernel[kernel.rindex("mbar_wait_drain(drain, 0u)"):]
    steps = ["cluster_sync();", "& kGaveUp)", "pair_exit(", "fill(T", "mbar_wait_drain(&full[", "cluster_sync();"]
    at = -1
    for s in steps:
        at = teardown.index(s, at + 1)
    assert publish < kernel.rindex("mbar_wait_drain(drain, 0u)")
    # no other place waits for the copies' barriers on the way out
    assert kernel.count("mbar_wait_drain(&full[") == 1

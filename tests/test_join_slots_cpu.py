"""The joins of a workgroup's waves (csrc/join_slots.h, csrc/ffn_internal.h):
one barrier per join is enough only if consecutive joins of a kernel never
share a slot.  The slot function is the kernels' own, compiled here for the
host; which joins a kernel makes is read from its source."""
import os
import re
import subprocess

import pytest

from tensor_gemm_reduce_lds_amd import build as B

WAVES = 16
KERNELS = {"norm_forward_kernel": ("block_norm.hip", [1]), "norm_backward_kernel": ("block_norm.hip", [3, 1]),
           "quantize_kernel": ("gemm_q8.hip", [1])}


def _kernel_joins(name):
    """(MOST of the kernel's slots, numbers of values of its joins)."""
    text = open(os.path.join(B.CSRC, KERNELS[name][0])).read()
    body = text[re.search(r"__global__[^;{]*\b%s\(" % name, text).start():]
    body = body[:body.index("\n}\n")]
    most = re.findall(r"__shared__ JoinSlots<(\d+)> (\w+);", body)
    joins = re.findall(r"block_join<\w+, THREADS, (\d+)>\(\w+, (\w+), turn\)", body)
    assert len(most) == 1 and joins and {s for _, s in joins} == {most[0][1]}
    assert len(joins) == body.count("block_join")
    return int(most[0][0]), sorted({int(n) for n, _ in joins}, reverse=True)


def _slots(at, turn, values):
    return [at(turn, n, w) for n in range(values) for w in range(WAVES)]


def _clashes(at, values):
    """Consecutive joins, of any two of these numbers of values, that share a slot."""
    return [(a, b, t) for a in values for b in values for t in (0, 1)
            if set(_slots(at(a), t, a)) & set(_slots(at(b), t ^ 1, b))]


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    """{MOST: (floats, {(turn, n, wave): slot})} from the header, by the host compiler."""
    d = tmp_path_factory.mktemp("slots")
    src = ["#include <stdio.h>", '#include "join_slots.h"', "using gemm_rs::ffn::JoinSlots;",
           "template <int M> void show() {",
           '  printf("%d -1 0 0 %d\\n", M, (int)(sizeof(JoinSlots<M>) / sizeof(float)));',
           "  for (int t = 0; t < 2; ++t) for (int n = 0; n < M; ++n) for (int w = 0; w < JoinSlots<M>::kWaves; ++w)",
           '    printf("%d %d %d %d %d\\n", M, t, n, w, JoinSlots<M>::at(t, n, w)); }',
           "static_assert(JoinSlots<3>::at(1, 0, 0) == JoinSlots<3>::kFloats / 2, \"a constant expression\");",
           "int main() { show<1>(); show<2>(); show<3>(); return 0; }"]
    (d / "slots.cc").write_text("\n".join(src))
    subprocess.run(["g++", "-std=c++17", "-I", B.CSRC, str(d / "slots.cc"), "-o", str(d / "slots")], check=True)
    out = {}
    for line in subprocess.run([str(d / "slots")], check=True, capture_output=True, text=True).stdout.splitlines():
        m, t, n, w, v = (int(x) for x in line.split())
        if t < 0:
            out[m] = (v, {})
        else:
            out[m][1][t, n, w] = v
    return out


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_consecutive_joins_never_share_a_slot(kernel, compiled):
    most, values = _kernel_joins(kernel)
    assert values == KERNELS[kernel][1]
    floats, table = compiled[most]
    at = lambda values: lambda t, n, w: table[t, n, w]  # noqa: E731
    for t in (0, 1):
        for v in values:
            s = _slots(at(v), t, v)
            assert len(set(s)) == len(s) and min(s) >= 0 and max(s) < floats
    assert _clashes(at, values) == []


def test_halves_that_depend_on_the_number_of_values_would_clash():
    """Halves at 16 floats per value of the join itself, which looks right for
    each join alone, share slots where joins of 3 and of 1 value alternate."""
    at = lambda values: lambda t, n, w: t * values * WAVES + n * WAVES + w  # noqa: E731
    assert _clashes(at, [1]) == [] and _clashes(at, [3]) == []
    assert (3, 1, 0) in _clashes(at, [3, 1])

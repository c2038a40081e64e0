"""Which kernel a size takes (csrc/ffn_rules.h, compiled here for the host)."""
import os
import re
import subprocess

import pytest

import ffn_cases as C
from tensor_gemm_reduce_lds_amd import build as B

HEADER = os.path.join(B.CSRC, "ffn_rules.h")


def _choices(prefix):
    """The enumerators of a rule, in order, without the last (their number)."""
    body = re.search(r"enum \w+ \{([^}]*\b%sChoices\b)" % prefix, open(HEADER).read()).group(1)
    return [n.strip() for n in body.replace("\n", " ").split(",") if n.strip()][:-1]


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """Values of expressions over the header."""
    d = tmp_path_factory.mktemp("rules")

    def values(expressions):
        src = ["#include <stdio.h>", '#include "ffn_rules.h"', "using namespace gemm_rs::ffn;", "int main() {"]
        src += ['  printf("%%d\\n", (int)(%s));' % e for e in expressions] + ["  return 0; }"]
        (d / "ask.cc").write_text("\n".join(src))
        subprocess.run(["g++", "-std=c++17", "-I", B.CSRC, str(d / "ask.cc"), "-o", str(d / "ask")], check=True)
        return [int(v) for v in subprocess.run([str(d / "ask")], check=True, capture_output=True, text=True).stdout.split()]
    return values


@pytest.mark.parametrize("prefix,cases,call", [
    ("kQ8", C.Q8, lambda c: "q8_choice(%d, %d)" % c[1:3]),
    ("kQuant", C.QUANT, lambda c: "quant_choice(%d, %d)" % c[1:]),
    ("kRows", C.ROWS, lambda c: "rows_choice(%d, %d, %d, %d)" % (sum(c[1]), c[3], c[2], len(c[1])))],
    ids=["q8", "quantize", "grouped rows"])
def test_the_cases_reach_every_kernel(prefix, cases, call, ask):
    names = _choices(prefix)
    got = [names[v] for v in ask([call(c) for c in cases])]
    assert got == [c[0] for c in cases]
    assert set(got) == set(names)


def test_the_weight_gradients_cases_reach_every_kernel(ask):
    calls = ["tn_choice(%d, %d, %d, %d)" % (sum(s), k, n, len(s)) for _, _, s, n, k in C.TN]
    large, parts = ask(c + ".large" for c in calls), ask(c + ".parts" for c in calls)
    assert [(bool(a), b > 1) for a, b in zip(large, parts)] == [c[:2] for c in C.TN]
    assert {c[:2] for c in C.TN} == {(True, False), (False, False), (False, True)}
    # both clauses of the rule for large tiles, and an expert with fewer steps of 64 rows than parts
    tiles = ["%d" % (len(s) * (-(-k // 256)) * (-(-n // 256))) for big, _, s, n, k in C.TN if big]
    assert any(int(t) >= 1024 for t in tiles) and any(int(t) < 1024 for t in tiles)
    assert any(b > 1 and any(0 < r <= 64 * (b - 1) for r in c[2]) and 0 in c[2] for b, c in zip(parts, C.TN))


def test_parts_of_fewer_rows_fit_the_plans_workspace(ask):
    """A plan allocates for the parts of its most rows; a call of fewer has no more."""
    for k, n, e in ((264, 136, 2), (72, 200, 4), (1296, 304, 2), (768, 512, 8)):
        parts = ask("tn_choice(%d, %d, %d, %d).parts" % (r, k, n, e) for r in range(0, 20000, 97))
        assert all(a <= b for a, b in zip(parts, parts[1:]))

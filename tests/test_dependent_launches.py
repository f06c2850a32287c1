"""Kernels that may begin before the one in front of them has ended (griddepcontrol): what an earlier
kernel of the same call leaves in the workspace is read by ordinary loads. The non-coherent ones
(__ldg, const __restrict__) are for data that nothing writes while the kernel lives."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "io_aware_exact_07_gb300", "csrc")
# what kernels of one call write for one another
BETWEEN = ("row_sums", "key_tiles", "dkdv_part", "dsum", "diag_sums", "line_sums", "far_sums",
           "pieces", "o_part", "lse_part", "headers")


def _functions(text):
    """(name, parameters, body) of every function with a body at the left margin's depth."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\b(?!__launch_bounds__|if\b|for\b|while\b)(\w+)\s*\(([^;{}]*)\)\s*\{", text):
        depth, i = 1, m.end()
        while depth and i < len(text):
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), m.group(2), text[m.end():i]


def _waiting():
    out = []
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh")):
            with open(os.path.join(CSRC, f)) as h:
                found = list(_functions(h.read()))
            calls = {n: b for n, _, b in found}
            for n, p, b in found:
                if "pdl_wait()" in b and n not in ("pdl_wait",) and "_kernel" in n:
                    helpers = "".join(calls[c] for c in set(re.findall(r"\b(\w+)\(", b))
                                      if c in calls and c != n)
                    out.append((f, n, p, b + helpers))
    return out


KERNELS = _waiting()


def test_the_kernels_that_wait_are_found():
    names = {n for _, n, _, _ in KERNELS}
    assert {"rel_near_kernel", "rel_sums_kernel", "rel_table_kernel", "dkdv_merge_kernel",
            "fa_decode_combine_kernel", "fa_paged_step_merge_kernel",
            "fa_paged_chunk_merge_kernel"} <= names


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: k[1])
def test_workspaces_are_read_by_ordinary_loads(kernel):
    f, name, params, body = kernel
    assert "__restrict__" not in params
    for m in re.finditer(r"__ldg\(", body):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(body[i], 0)
            i += 1
        where = body[m.end():i - 1]
        # the pointers that it names, and where these come from
        for _ in range(3):
            for v in set(re.findall(r"\b[A-Za-z_]\w*\b(?!\s*\.)", where)):
                for d in re.findall(r"\*\s*%s\s*=\s*([^;]+);" % v, body):
                    if d not in where:
                        where += " " + d
        bad = [b for b in BETWEEN if re.search(r"\b%s\b" % b, where)]
        assert not bad, f"{f} {name}: __ldg of {bad}"

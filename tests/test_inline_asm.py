"""Inline assembly of the kernels (CPU, by reading the sources): no statement writes a register that its operands
do not declare, so that the compiler never holds a value of its own there."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dlrm_sparse_embedding_amd", "csrc")
STATEMENT = re.compile(r"\basm\s*(?:volatile)?\s*\(\s*((?:\"(?:[^\"\\]|\\.)*\"\s*)+)")
NAMED = re.compile(r"\b(m0|exec|vcc|scc|flat_scratch|[sva]\d+|[sva]\[\d+)", re.I)


def templates(path):
    text = re.sub(r"//[^\n]*", "", open(path).read())
    return [m.group(1) for m in STATEMENT.finditer(text)]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.h*")) + glob.glob(os.path.join(CSRC, "*.cpp"))),
                         ids=os.path.basename)
def test_no_register_by_name(path):
    for t in templates(path):
        assert not NAMED.search(t), t


def test_the_pattern_sees_statements():
    assert NAMED.search('"s_mov_b32 m0, %1\\n\\ts_mov_b64 %0, %3"') and NAMED.search('"v_mov_b32 v12, %0"')
    assert not NAMED.search('"global_load_lds_dwordx4 %2, %0"') and not NAMED.search('"s_waitcnt vmcnt(0)"')
    assert len(templates(os.path.join(CSRC, "k_prefix.hip"))) >= 4

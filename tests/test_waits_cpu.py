"""The bounded waits of the prompt kernels, as far as their source shows them: no
thread that gave up may leave others waiting without a limit."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_linear_attention_decode_b200", "csrc")
TENSOR_CORE = [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if "elect_one()" in open(p).read()]


def _code(path):
    """The file without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


def test_there_is_something_to_look_at():
    assert {os.path.basename(p) for p in TENSOR_CORE} >= {"stq_attn.cu", "stq_chunk.cu"}


@pytest.mark.parametrize("path", TENSOR_CORE, ids=os.path.basename)
def test_named_barriers_carry_the_verdict(path):
    """A barrier of some of the warps has no limit, so whoever gave up before it comes to it too and tells the others."""
    assert not re.search(r"\b(bar|barrier(\.cta)?)\.(sync|arrive)\b", _code(path))


@pytest.mark.parametrize("path", TENSOR_CORE, ids=os.path.basename)
def test_a_warp_that_issues_products_gives_up_as_one(path):
    """elect.sync wants the whole warp: where it is used, lanes leave a loop only by a verdict that all of them share."""
    code = _code(path)
    lines = [line.strip() for line in code[code.index("elect_one()"):code.rindex("elect_one()")].splitlines() if line.strip()]
    assert any("__all_sync(" in line for line in lines)
    for before, line in zip(lines, lines[1:]):
        assert "break;" not in line or "__all_sync(" in before or (line == "if (!ok) break;" and before == "}"), line


@pytest.mark.parametrize("path", [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if "barrier_init(" in open(p).read()],
                         ids=os.path.basename)
def test_barriers_are_64_bit_words(path):
    """An mbarrier is a 64-bit word on its own boundary: a word declared as one, and nothing that another purpose laid down."""
    code = _code(path)
    words = {re.match(r"\w+", name.strip()).group() for names in re.findall(r"unsigned long long ([^;()=]+);", code) for name in names.split(",")}
    code = re.sub(r"const auto (init|wait) = [^\n]*", "", code)  # these take an unsigned long long &
    used = [a or b for a, b in re.findall(r"(?:barrier_init|tc_commit|barrier_arrive)\(smem_addr\(&sm\.(\w+)|\bwait\(sm\.(\w+)", code)] + re.findall(r"\binit\(sm\.(\w+)", code)
    assert used or "bar0 = smem_addr(&sm.full[" in code
    assert set(used) <= words

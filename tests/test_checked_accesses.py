"""What the checked build tests before it touches memory: in the sources of the
operators between a block's linears, every indexed access to one of the buffers
named here stands under a bounds check (in_range, or a helper that ends in it) in the
lines before it.  The checks themselves run on the GPU; that they are there can be
read."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "float8_mixed_precision_gb300", "csrc")
CHECK = re.compile(r"in_range\(|\.holds\(|held\(|inside")
# lines that a check may stand ahead of its access; in these functions it opens a longer stretch
LINES, MORE = 7, {f: 17 for f in ("load8", "store8", "fill", "cols_walk_kernel")}

# file: {function: accesses}
ACCESSES = {
    "f8_rope.cu": {
        "rope_kernel": [r"a\.pos\[", r"a\.freqs\[", r"V \*>\(x \+ c0\)"],
        "holds": [r"return"],
    },
    "f8_act.cu": {
        "load8": [r"\bq\[at \+ e\]", r"\(p \+ at\)"],
        "store8": [r"\bq\[at \+ e\]", r"\(p \+ at\)"],
        "act_bwd_kernel": [r"\bparts\[", r"\bcarry\["],
        "act_reduce_kernel": [r"\bparts\[", r"\bcarry\[", r"\(out\)\[col\]"],
    },
    "f8_resnorm_rows.cuh": {
        "fill": [r"bulk_load\(to \+ i \* pitch_a"],
        "ragged": [r"\ba\[i\]\[", r"\br\[i\]\["],
        "tail": [r"\ba\[i\]\[", r"\br\[i\]\["],
        "take_typed": [r"uint4 \*>\(p \+ at \+ c\)", r"__ldg\(p \+ at \+ vec_col", r"__ldg\(p \+ at \+ elem_col"],
        "give_sums": [r"sums \+ at"],
        "give_param": [r"float \*>\(p\) \+ row"],
    },
    "f8_resnorm.cu": {
        "param": [r"\(p\)\[i\]"],
        "put_param": [r"\(p\)\[i\]"],
        "stat": [r"\bstats\["],
        "put_stat": [r"\bstats\["],
        "bwd_walk_kernel": [r"\bconsts\["],
        "cols_walk_kernel": [r"\bends\[", r"parts \+ chunk"],
        "reduce_kernel": [r"s \+= p\["],
    },
}
CASES = [(f, fn) for f, fns in ACCESSES.items() for fn in fns]


def _body(text: str, name: str) -> list:
    """The lines of the function `name`, its definition's braces matched."""
    for m in re.finditer(r"\b%s\(" % name, text):
        at, depth = m.end(), 1
        while depth:                                   # the parameters
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        rest = re.match(r"\s*(const\s*)?\{", text[at:])
        if rest is None:
            continue
        start = at = at + rest.end()
        depth = 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        return text[start:at].split("\n")
    raise AssertionError(f"no function {name}")


@pytest.mark.parametrize("source, function", CASES, ids=lambda v: v)
def test_accesses_are_checked(source, function):
    with open(os.path.join(CSRC, source)) as f:
        lines = _body(re.sub(r"//[^\n]*", "", f.read()), function)
    for access in ACCESSES[source][function]:
        at = [i for i, line in enumerate(lines) if re.search(access, line)]
        assert at, f"{source}: {function} has no {access}"
        for i in at:
            ahead = "\n".join(lines[max(0, i - MORE.get(function, LINES)):i + 1])
            assert CHECK.search(ahead), f"{source}: {function}: {lines[i].strip()}"


def test_statistics_go_through_their_checks():
    with open(os.path.join(CSRC, "f8_resnorm.cu")) as f:
        text = f.read()
    assert re.search(r"\bc\.stats\[", text) is None and text.count("c.stat(") >= 12 and text.count("c.put_stat(") == 8


def test_forward_kernels_that_no_call_reaches():
    """The residual norm's rule for widths of no whole vectors is a template argument: a mode chosen at run time would
    build the kernels of both for every kind of parameter, half of them never launched."""
    with open(os.path.join(CSRC, "f8_resnorm.cu")) as f:
        text = f.read()
    assert "by_mode<bf.value ? rows::kShift : rows::kRagged>" in text and "by_mode<rows::kShift>" in text
    assert re.search(r"by_mode\(", re.sub(r"by_mode\(int64_t cols", "", text)) is None

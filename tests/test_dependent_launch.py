"""Kernels launched behind another one start while it still writes; they may read
what it writes only after their grid_wait().  The compiler has to see it that
way too: through a `const ... __restrict__` parameter it may take a load for
invariant and move it above the wait or through a cache that is not kept
coherent.  Checked in the sources, as the schedule of one build proves nothing."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "vocab_wide_token_gb300", "csrc")


def _sources():
    out = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        text = open(path).read()
        out[os.path.basename(path)] = re.sub(r"//[^\n]*", "", text)
    return out


def _balanced(text, at, opening, closing):
    """The end of the bracket that opens at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == opening) - (text[i] == closing)
        if depth == 0:
            return i
    raise AssertionError("unbalanced")


def _kernels():
    """(file, name, parameters, body) of every kernel that waits for the one before it."""
    found = []
    for name, text in _sources().items():
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\s*(?=\())?", text):
            at = m.end()
            if text[at] == "(":  # the launch bounds
                at = _balanced(text, at, "(", ")") + 1
            head = re.match(r"\s*(\w+)\s*\(", text[at:])
            start = at + head.end() - 1
            end = _balanced(text, start, "(", ")")
            body = text.index("{", end)
            stop = _balanced(text, body, "{", "}")
            if "grid_wait()" in text[body:stop]:
                found.append((name, head.group(1), text[start + 1:end], text[body:stop]))
    return found


KERNELS = _kernels()


def test_every_kernel_launched_behind_another_waits():
    waiting = {k[1] for k in KERNELS}
    launched = set()
    for text in _sources().values():
        for m in re.finditer(r"launch_behind\(\s*(\w+)", text):
            launched.add(m.group(1))
    # `kernel` is the variable that takes one of filtered_backward_kernel's instances
    named = (launched - {"kernel", "void"}) | {"filtered_backward_kernel"}
    assert named == waiting and waiting


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: k[1])
def test_no_parameter_is_taken_for_constant(kernel):
    _, _, parameters, _ = kernel
    for p in re.split(r",(?![^<]*>)", parameters):
        assert not ("const" in p and "__restrict__" in p), p.strip()


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: k[1])
def test_pointers_are_read_through_the_wait(kernel):
    """Every pointer parameter that is read is taken through after_wait() behind
    the wait, and the plain one not used again."""
    _, name, parameters, body = kernel
    wait = body.index("grid_wait()")
    for p in re.split(r",(?![^<]*>)", parameters):
        if "const" not in p or "*" not in p:
            continue
        var = re.search(r"(\w+)\s*$", p).group(1)
        uses = [m.start() for m in re.finditer(rf"\b{var}\b", body)]
        taken = re.search(rf"\b{var}\s*=\s*after_wait\({var}\);", body)
        assert taken and taken.start() > wait and min(uses) == taken.start(), (name, var)


@pytest.mark.parametrize("function", ["fold_records", "for_each_group", "unit_squares", "scale_unit"])
def test_helpers_that_read_a_predecessors_output(function):
    """The functions that these kernels read records, group maxima and gradients
    with promise the compiler nothing either, nor use the read-only path."""
    for text in _sources().values():
        for m in re.finditer(rf"\b{function}\(", text):
            end = _balanced(text, m.end() - 1, "(", ")")
            if re.match(r"\s*\{", text[end + 1:]):
                body = text[end:_balanced(text, text.index("{", end), "{", "}")]
                assert "__restrict__" not in text[m.start():end] and "__ldg" not in body
                return
    pytest.fail(f"{function} is not defined")

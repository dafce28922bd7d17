"""Kernels launched behind another one that take their arguments as a structure: what the one
before may have written is read through after_wait(), as test_dependent_launch.py asks of
pointer parameters."""
import re

import pytest

from test_dependent_launch import _sources

READ = [("adamw.cu", "o.lr_at"), ("adamw.cu", "o.step_at"), ("adamw.cu", "o.seed_at"), ("adamw.cu", "o.norm"),
        ("adamw.cu", "at.g"), ("fp8.cu", "a.x"), ("fp8.cu", "a.W_scale"), ("fp8.cu", "a.q_scale"),
        ("beams.cu", "a.scores"), ("beams.cu", "a.f.records"), ("beams.cu", "a.f.group_max"),
        ("beams.cu", "a.f.logits"), ("reorder.cu", "a.parents"), ("reorder.cu", "s.in")]


@pytest.mark.parametrize("file,pointer", READ)
def test_pointers_of_structures_are_read_through_the_wait(file, pointer):
    text = _sources()[file]
    name = re.escape(pointer)
    assert re.search(rf"after_wait\({name}\)", text)
    read = rf"static_cast<[^<>]*>\({name}\)|\*{name}\b|\b{name}(\[| \+)"
    assert not re.search(read, text), re.search(read, text).group(0)

"""The lists of sources that the summaries of the model-side operators' kernels
are tied to hold every file that their kernels are compiled from: what a listed
file includes, at any depth (no GPU needed)."""
import json
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ring_allreduce_reduction_02_amd", "csrc")


@pytest.mark.parametrize("name", ["model_operators", "more_operators"])
def test_included_files_are_listed(name):
    listed = json.load(open(os.path.join(ROOT, "profiles", name + "_sources.json")))["kernel_sources"]
    todo, seen = list(listed), set()
    while todo:
        f = todo.pop()
        if f not in seen:
            seen.add(f)
            text = open(os.path.join(CSRC, f)).read()
            todo += [i for i in re.findall(r'^\s*#\s*include\s+"([^"]+)"', text, re.M) if os.path.exists(os.path.join(CSRC, i))]
    assert seen == set(listed) and len(set(listed)) == len(listed)

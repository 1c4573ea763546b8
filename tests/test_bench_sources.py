"""Recorded counter readings hold for the sources that they were taken on."""
import os
import re

import bench

CSRC = os.path.join(os.path.dirname(os.path.abspath(bench.__file__)), "activation_sparse_ffn_layer_amd", "csrc")


def included(name, seen):
    seen.add(name)
    with open(os.path.join(CSRC, name)) as f:
        for n in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
            if n not in seen and os.path.exists(os.path.join(CSRC, n)):
                included(n, seen)
    return seen


def test_the_hash_covers_what_the_stack_is_built_from():
    assert included("pi_lib.hip", set()) == set(bench.STACK_SOURCES)

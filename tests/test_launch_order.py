"""Every kernel launches its dependents only behind its own wait for what is
ahead of it, so that a dependent that reads early runs beside the kernel directly
ahead alone."""
import glob
import os
import re

import pytest

from linear_attention_decode_04_gb300 import build as B

WAIT = re.compile(r"griddepcontrol\.wait|\bgriddep_wait\(\)")
TRIGGER = r"griddepcontrol\.launch_dependents|\bgriddep_launch_dependents\(\)"


def functions(text):
    """(head, body) of the functions of a source"""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__(?:global|device)__[^;{}=]*?\([^{};]*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(0), text[m.end():i]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(B.CSRC, "*.cu*"))), ids=os.path.basename)
def test_dependents_start_behind_the_wait(path):
    found = list(functions(open(path).read()))
    # device functions that launch dependents count where kernels call them
    helpers = [re.search(r"(\w+)\s*\(", head[head.rindex("__"):]).group(1) for head, body in found
               if "__device__" in head and re.search(TRIGGER, body)]
    trigger = re.compile("|".join([TRIGGER] + [rf"\b{h}(?:<\w+>)?\(" for h in helpers]))
    for head, body in found:
        first = trigger.search(body)
        if "__global__" in head and first:
            assert WAIT.search(body[:first.start()]), head


def test_functions_are_found():
    names = {os.path.basename(p): [h for h, _ in functions(open(p).read()) if "__global__" in h]
             for p in glob.glob(os.path.join(B.CSRC, "*.cu*"))}
    assert sum(map(len, names.values())) >= 10
    assert any("linear_kernel" in h for h in names["kda_linear.cu"])
    assert any("kda_decode" in h for h in names["kda_decode_kernel.cuh"]), names["kda_decode_kernel.cuh"]

"""Properties that every kernel source of the library keeps, read from the text."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "nvfp4_w4a4_moe_permute_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))


def literals(path):
    """A file's string literals, neighbouring ones joined, comments left out."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r'"(?:[^"\\]|\\.)*"(?:\s*"(?:[^"\\]|\\.)*")*', text):
        yield m.group(0)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_is_multicast(path):
    """The library serves programs of several GPUs too, and a pointer argument may
    point anywhere: no TMA load of it may be a multicast one. (A commit of finished
    matrix products that arrives at two CTAs' barriers reads no memory.)"""
    for text in literals(path):
        assert "multicast" not in text or "tcgen05.commit" in text, text


def asm_statements(path):
    """(whether volatile, text) of every asm statement of a file."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"\basm\b\s*(volatile)?\s*\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield m.group(1) is not None, text[m.end():i - 1]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_loads_of_global_memory_stay_in_their_place(path):
    """A kernel may start before the one in front of it has ended and waits for it
    before its first access of global memory. A load written as asm has to be
    volatile and to clobber memory, or the compiler may move it ahead of that."""
    for volatile, text in asm_statements(path):
        if re.search(r"\bld\.(?!shared|param|const)\S*global", text):
            assert volatile and '"memory"' in text, text

"""Properties of the paged kernels that their source has to keep and that no run
shows."""

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rotate_then_quantize_b200", "csrc")

CHAIN = ["paged_attention.cuh", "prefix_mma.cuh", "prefix_pair.cuh"]
# what earlier launches of the chain write: the members of PrefixArgs, and the
# pointers taken from them
WORKSPACE = ["qrot", "q_image", "q_factor", "plan", "chunk_start", "chunk_of", "pre_ml", "pre_acc",
             "own_ml", "own_acc"]


def _source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def _arguments(text, call):
    """The argument text of every call of `call`."""
    for m in re.finditer(re.escape(call) + r"\s*\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield text[m.end():i - 1]


@pytest.mark.parametrize("name", CHAIN)
def test_workspace_is_not_read_through_the_read_only_path(name):
    """The launches of an attention call overlap (programmatic launches), so what
    one writes may change while the next is resident: a non-coherent load of it
    could return what the call before left there."""
    text = _source(name)
    taken = {m.group(1) for w in WORKSPACE
             for m in re.finditer(r"\*\s*(\w+)\s*=[^;]*\ba\." + w + r"\b[^;]*;", text)}
    names = WORKSPACE + sorted(taken)
    for arg in _arguments(text, "__ldg"):
        used = set(re.findall(r"\w+", arg))
        assert not used & set(names), arg


def _kernels(text):
    """Name and body of every kernel."""
    for m in re.finditer(r"__global__", text):
        start = text.index("{", text.index(")", re.compile(r"\w+_kernel\(").search(text, m.end()).start()))
        depth, i = 1, start + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield re.search(r"(\w+_kernel)\(", text[m.end():]).group(1), text[start:i]


@pytest.mark.parametrize("name", CHAIN + ["launch_block_tables.cu"])
def test_paged_kernels_check_their_indices(name):
    """In the debug build every kernel checks the global indices that it computes."""
    kernels = list(_kernels(_source(name)))
    assert kernels
    for kernel, body in kernels:
        assert re.search(r"\bdbg_\w+\(|\bpool_row\(", body), kernel


@pytest.mark.parametrize("name,calls", [("codec.cuh", 5), ("codec_split.cuh", 4)])
def test_paged_codec_checks_its_slots(name, calls):
    """The pool side of the paged codec: codes and scales, in and out."""
    assert len(list(_arguments(_source(name), "dbg_slot"))) >= calls

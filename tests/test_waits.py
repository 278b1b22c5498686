"""Every bounded wait of the kernels is acted upon.

A wait returns false when its limit has passed.  A kernel that went on would read tensor
memory or shared memory that is still being written and put results made from it into memory.
Only the waits of a kernel that is already leaving, which tell nobody (no status word), may
drop the result.  Running out of a wait on purpose would need a kernel broken on purpose, so
this is looked for in the sources.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_layer_backward_gb300", "csrc")
# the single-token kernel's copies in flight, awaited where it has already stopped
LEAVING = {"decode_persistent.cu": 1}
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def calls(text):
    """(position, what stands before the call, its arguments) of every mbar_wait call."""
    for m in re.finditer(r"\bmbar_wait\(", text):
        depth, end = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[end], 0)
            end += 1
        yield m.start(), text[:m.start()].rstrip(), text[m.end():end - 1]


def dropped(text):
    text = re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), text)
    for at, before, args in calls(text):
        if before.endswith("bool"):                            # its definition
            continue
        used = before.endswith(("!", "=", "&&", "||", "return", ",")) or re.search(r"\b(if|while|all_sync|or)\s*\($", before)
        if not used and not args.replace(" ", "").endswith("nullptr,0u"):
            yield text.count("\n", 0, at) + 1


def test_the_search_finds_what_it_looks_for():
    assert list(dropped("a;\nmbar_wait(&b, 1, p.status, 3u);")) == [2]
    assert list(dropped("if (x) mbar_wait(&b, f(1), p.status, 3u);")) == [1]
    assert not list(dropped("ok = mbar_wait(&b, 1, p.status, 3u); if (!mbar_wait(&b, 1, p.status, 3u)) {}\n"
                            "mbar_wait(&b, 0, nullptr, 0u); // mbar_wait(&b, 1, p.status, 3u);"))


@pytest.mark.parametrize("name", FILES)
def test_no_wait_is_dropped(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        assert len(list(dropped(f.read()))) == LEAVING.get(name, 0)

"""Waits of the attention's and the weights' persistent kernels (csrc/paged_attention.cu, csrc/paged_weights.cu) that can give
up, read from the source. One lane may run out of time, or see that another role gave up, where its neighbour sees the phase
complete, and what follows a wait takes the whole warp (tensor memory accesses, shuffles, votes): every such wait is
voted on, so that no lane leaves alone. The path itself is not run: nothing may hang a GPU."""
import os
import re

import pytest

from gated_linear_attention_gb300 import build

FILES = ("paged_attention.cu", "paged_weights.cu")


def _code(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", FILES)
def test_waits_are_voted_on(name):
    code = _code(name)
    assert code.count("wait_warp(") > 5
    for at in re.finditer(r"(tck::|tc::)?\b(wait_or_abort\w*|mbar_test_wait|mbar_try_wait)\(", code):
        assert code[:at.start()].endswith("__all_sync(0xffffffffu, "), code[at.start() - 60:at.end() + 40]
    # the product role notes its waits' results, and votes on them once a tile
    for line in code.splitlines():
        if "wait_at(" in line:
            assert "__all_sync(0xffffffffu, wait_at(" in line or "fine" in line or "scores(wait_at(" in line, line
    assert "__all_sync(0xffffffffu, fine)" in code


def test_the_wait_of_a_warp_votes():
    body = _code("paged_tiles.cuh").split("bool wait_warp(")[1].split("\n}\n")[0]
    assert body.count("__all_sync(0xffffffffu, ") == body.count("return") == 2


def _loops(code):
    """(header, body) of each loop with a braced body."""
    for at in re.finditer(r"\bfor \(", code):
        depth, i = 1, at.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(code[i], 0)
            i += 1
        if code[i:i + 2] != " {":
            continue
        end, depth = i + 2, 1
        while depth:
            depth += {"{": 1, "}": -1}.get(code[end], 0)
            end += 1
        yield code[at.end():i], code[i:end]


@pytest.mark.parametrize("name", FILES)
def test_a_loop_ends_with_a_wait_that_gave_up(name):
    """Either its header looks at the result, or each wait in it is followed by the way out."""
    seen = 0
    for header, body in _loops(_code(name)):
        for at in re.finditer(r"\bok = [^;]*(wait_warp|passed)\([^;]*;", body):
            seen += 1
            assert "&& ok" in header or body[at.end():].split()[:3] == ["if", "(!ok)", "break;"] or \
                body[at.end():].split()[:4] == ["if", "(!ok)", "return", "0.f;"], (header, at.group(0))
    assert seen > 3


@pytest.mark.parametrize("name", FILES)
def test_copies_and_products_in_flight_are_waited_for_whoever_gave_up(name):
    """A role that ends well may have copies or products in flight when another one gives up."""
    code = _code(name)
    assert "mbar_wait(&bar.drain" in code and "mbar_wait(&bar.q_full" in code
    assert not re.search(r"if \(!ok\)( \{)?\s*(drain|for|if \(q_issued\)|if \(tc::elect_one)", code)

"""The largest tables and budgets that the softmax layers' entry points take (no GPU needed): kernels count places in 32 bits
and step past the last one by a block's share, up to 8192 places, so that a request may have 2^30 places and no more."""
import os
import re

import pytest

from gated_linear_attention_gb300 import build
from test_abi_softmax_layers import CUDA, INVALID, _append, _attend, _evict, lib, no_gpu  # noqa: F401


@no_gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_places_of_a_request(lib, page):  # noqa: F811
    # arrays far apart: a table of 2^26 entries and three rows is 0.8 GB
    far = dict(page=page, table=0x100000000, lens=0x200000000, kp=0x300000000, vp=0x400000000, w=0x500000000)
    for width, want in (((1 << 30) // page, CUDA), ((1 << 30) // page + 1, INVALID), ((1 << 31) // page - 1, INVALID)):
        assert _append(lib, width=width, **far) == want
        assert _attend(lib, width=width, **far) == want
        assert _evict(lib, width=width, **far) == want


@no_gpu
@pytest.mark.parametrize("budget,kept,want", [(1 << 30, 0x700000000, CUDA), ((1 << 30) + 1, 0x700000000, INVALID),
                                              ((1 << 31) - 1, 0x700000000, INVALID), ((1 << 31) - 1, 0, CUDA), (1 << 31, 0, INVALID)])
def test_budget(lib, budget, kept, want):  # noqa: F811
    assert _evict(lib, budget=budget, kept=kept) == want


def test_steps_past_the_last_place_stay_in_32_bits():
    """The loops over places and kept entries of the eviction, with their steps, from the source."""
    with open(os.path.join(build.CSRC, "kv_evict.cu")) as f:
        code = f.read()
    const = {m[0]: int(m[1]) for m in re.findall(r"\b(k\w+) = (\d+)[;,]", code)}
    steps = {"kSelThreads": const["kSelThreads"], "kAtOnce * kSelThreads": const["kAtOnce"] * const["kSelThreads"],
             "rows * kEach": const["kMoveThreads"] * const["kEach"], "kMoveThreads * kEach": const["kMoveThreads"] * const["kEach"]}
    found = re.findall(r"for \(int [ib] = [^;]*; [^;]*; [ib] \+= ([^)]*)\)", code)
    assert len(found) >= 5 and set(found) <= set(steps)
    assert (1 << 30) + max(steps.values()) + const["kCached"] < 1 << 31

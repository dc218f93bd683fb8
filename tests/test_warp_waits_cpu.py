"""Lanes of a warp that wait side by side may find differently whether a bounded wait
has run out.  In the feed-forward kernels' whole-warp roles either nothing that needs
all lanes follows until the role's end, or all of them act on one answer: a lane that
broke out alone would otherwise leave the rest waiting for it at a vote or a
__syncwarp().  That cannot be provoked on a device without risking just that, so it
is read from the sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "async_copy_pipelined_gb300", "csrc")
MEETING = re.compile(r"__syncwarp\(|__(?:all|any|ballot|shfl|shfl_xor|reduce_\w+)_sync\(")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _braced(text, start):
    """From the first brace at or after `start` to the one that closes it."""
    at = text.index("{", start)
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError("unbalanced")


def _producers():
    pair, few = _source("pair_product.cuh"), _source("few_rows.cuh")
    return {"pair": _braced(pair, pair.index("void produce(")),
            "few": _braced(few, few.index("if (warp == 0) {\n        const uint32_t on"))}


def _multipliers():
    pair, few = _source("pair_product.cuh"), _source("few_rows.cuh")
    return {"pair": _braced(pair, pair.index("void multiply(")),
            "few": _braced(few, few.index("else if (warp == 1) {\n        const uint32_t on"))}


@pytest.mark.parametrize("which", ["pair", "few"])
def test_nothing_in_the_producers_loops_needs_all_lanes(which):
    body = _producers()[which]
    assert "producer_acquire(" in body
    assert not MEETING.search(body)


@pytest.mark.parametrize("which", ["pair", "few"])
def test_nothing_in_the_mma_warps_loops_needs_all_lanes(which):
    body = _multipliers()[which]
    assert "consumer_wait(" in body
    assert not MEETING.search(body)


def test_the_8_bit_epilogue_votes_on_both_waits():
    text = _source("gemm_fp8.cu")
    waits = [m.start() for m in re.finditer(r"mbar_wait_bounded\(scales\.full\(", text)]
    assert len(waits) == 1
    assert re.search(r"acquire\(p\.launch, b, acc,\s*$", text[:waits[0]])
    vote = _source("pair_product.cuh")
    vote = _braced(vote, vote.index("bool acquire("))
    assert re.search(r"ok = others && mbar_wait_bounded\(", vote) and "__all_sync(0xffffffffu, ok)" in vote
    # The warp that copies the scales: no lane waits for another there.
    loader = _braced(text, text.index("auto load_scales ="))
    assert "scales.empty(f)" in loader and "record_error(" in loader and not MEETING.search(loader)


@pytest.mark.parametrize("name", ["gated.cu", "gemm_fp8.cu", "pair_product.cuh"])
def test_epilogues_vote(name):
    """Waits for accumulators: the answer is voted on before it is acted upon."""
    text = _source(name)
    for m in re.finditer(r"mbar_wait_bounded\(\s*b\.acc_full", text):
        after = text[m.start():m.start() + 400]
        assert re.search(r"__all_sync\(0xffffffffu, ok\)", after), after

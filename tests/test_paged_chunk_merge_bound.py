"""The merge of the attention of a chunk (csrc/paged_chunk.cu) reads from the workspace how
many pieces a request was cut into.  The workspace needs no initialisation, so where the
attention gave up before it wrote the number, anything may stand there: it bounds a loop
and says which places are read.  No run shows that without a kernel that gives up, so the
check is read from the source (CPU)."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "sliding_window_gqa_ring_gb300", "csrc", "paged_chunk.cu")


def merge():
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    return text[text.index("paged_chunk_merge_kernel("):text.index("align256(")]


@pytest.mark.parametrize("splits", [2, 9, 76])
def test_a_number_of_pieces_that_nobody_wrote_is_not_used(splits):
    body = merge()
    guard = re.search(r"if \(!skip && \((.*)\)\) \{\s+if \(threadIdx.x == 0\) "
                      r"set_status\(p.dev_status, CARAT_DEV_TIMEOUT\);\s+skip = true;", body)
    assert guard, "the number of pieces is not checked"
    refused = guard[1].replace("||", "or").replace("plan.splits", "splits")
    for pieces in (-2 ** 31, -1, 0, 1, 2, splits - 1, splits, splits + 1, 77, 2 ** 28, 2 ** 31 - 1):
        assert eval(refused, {}, dict(pieces=pieces, splits=splits)) == (not 1 <= pieces <= splits)
    # in front of every use, and what is refused goes the way of rows without pieces
    used = [m.start() for m in re.finditer(r"\bpieces\b(?!\[)", body)]
    first = body.index("const int pieces = plan.pieces[b];")
    assert [u for u in used if u < guard.start()] == [first + len("const int ")]
    assert re.match(r"\s*\}\s+if \(skip \|\| pieces == 1\) \{", body[guard.end():])

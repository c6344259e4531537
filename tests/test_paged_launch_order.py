"""The order in which the paged operators' dependent launches wait, read memory and
let the next launch start.  No run shows a wrong order reliably, so it is read from
the sources (CPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sliding_window_gqa_ring_gb300", "csrc")
WAIT, TRIGGER = "wait_for_prior_launch();", "let_next_launch_start();"


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*", "", text)


def kernels(text):
    """name -> body of every __global__ function."""
    out = {}
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\s*\((?:[^()]|\([^()]*\))*\)\s*)?"
                         r"(\w+)\s*\(", text):
        at = text.index("{", m.end())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        out[m.group(1)] = text[at:end]
    return out


@pytest.mark.parametrize("name,want", [
    ("paged_rope.cu", {"rope_append_kernel", "rope_append_fp8_kernel"}),
    ("paged_fp8_attention.cu", {"paged_fp8_split_kernel", "paged_fp8_merge_kernel"})])
def test_a_kernel_waits_before_it_lets_the_next_one_start(name, want):
    """What comes after the next launch may start while this one runs; the launch
    before it is over by then only if this one has waited for it."""
    found = kernels(source(name))
    assert want <= set(found)
    for kernel in want:
        body = found[kernel]
        assert body.count(WAIT) == 1 and body.count(TRIGGER) == 1
        lead = body[1:body.index(WAIT)]
        assert TRIGGER not in lead, kernel
        # nothing but constants in front of the wait
        assert re.fullmatch(r"(\s*constexpr[^;]*;)*\s*", lead), (kernel, lead)


def test_the_attention_reads_through_l2_what_the_launches_before_it_wrote():
    """Its warps start while the queries' split runs and only the one that fetches the
    split queries waits: lengths, counts, page table and scales, which an append just
    before may have written, must not come from an SM's own cache."""
    text = source("paged_fp8_attention.cu")
    body = kernels(text)["paged_fp8_kernel"]
    assert body.count(WAIT) == 1
    for what in ("context_lengths", "new_counts"):
        uses = re.findall(r"\S*p\.%s\s*(?:\[|\+)" % what, text)
        assert uses and all("__ldcg(" in u for u in uses), (what, uses)
    uses = re.findall(r"\S*p\.page_table\s*(?:\[|\+)", body)
    assert len(uses) == 2 and all("__ldcg(" in u for u in uses), uses
    assert "src[(size_t)" not in body
    assert re.search(r"__ldcg\(src \+", body)


def test_the_attention_follows_its_split_launch():
    """The split launch goes first, so the attention's unwaited reads come after
    everything that the split has waited for."""
    text = source("paged_fp8_attention.cu")
    launch = text[text.index("cudaError_t launch(const PagedFp8Params"):]
    order = [launch.index(x) for x in ("launch_dependent(paged_fp8_split_kernel",
                                       "launch_dependent(kernel", "launch_dependent(merge")]
    assert order == sorted(order)

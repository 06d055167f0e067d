"""A kernel that lets the stream's next one go at its start may still be running, and so may the one before it, when that next one's
blocks begin.  What those read with non-coherent loads (__ldg) must not have been written since: an SM's
first-level cache may hold it from before.  The sources are read here, nothing runs."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_kv_cache_04_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels(text):
    """Bodies of the kernels of a source, by name."""
    found = {}
    for m in re.finditer(r"__global__[^;{]*?(\w+)\((?:[^()]|\([^()]*\))*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        found[m.group(1)] = text[m.end():i]
    return found


def test_kernels_that_change_tables_or_lengths_let_the_next_one_go_at_their_ends():
    pages = kernels(source("pages.cu"))
    assert {"release_kernel", "fork_kernel", "reserve_kernel", "reorder_kernel", "copy_pages_kernel"} <= set(pages)
    for name in ("release_kernel", "fork_kernel", "reserve_kernel", "reorder_kernel"):
        assert "grid_launch_dependents" not in pages[name], name
    body = pages["copy_pages_kernel"]  # with TABLE it writes the compacted table
    assert body.count("grid_launch_dependents") == body.count("if constexpr (!TABLE) grid_launch_dependents") == 1
    assert "grid_launch_dependents" not in kernels(source("append.cu"))["commit_lengths_kernel"]
    assert "grid_launch_dependents" not in kernels(source("prefix_attention.cu"))["prefix_plan_kernel"]


def non_coherent(name):
    """What a source reads with __ldg."""
    return re.findall(r"__ldg\(((?:[^()]|\((?:[^()]|\([^()]*\))*\))*)\)", source(name))


def test_norm_and_turn_reads_no_rows_that_kernels_write_with_non_coherent_loads():
    """In place it writes them itself."""
    assert non_coherent("qk_norm_rope.cu") == []


def test_chunk_attention_reads_only_tables_and_lengths_with_non_coherent_loads():
    """Those are written by kernels that let the next one go at their ends (above), or by the caller's; queries may come from
    any kernel of the stream."""
    got = non_coherent("chunk_kernel.cuh")
    allowed = ("a.cu_q", "a.seq_lens", "a.cp.block_table")
    assert got and all(x.startswith(allowed) for x in got), got

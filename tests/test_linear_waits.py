"""Rows that come into LDS by DMA are waited for by counts that the source
alone ensures: a count of younger loads would rest on the compiler emitting
one instruction for each of them, and it merges neighbours where it can."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "mixture_experts_prefill_amd", "csrc", "linear.hip")


def kernel(name):
    with open(SOURCE) as f:
        text = f.read()
    at = text.index(f") {name}(LinearArgs a) {{")
    return text[at:text.index("\n}\n", at)]


def test_no_wait_counts_loads():
    with open(SOURCE) as f:
        waits = re.findall(r"\bwait_\w+(?:<([^>]*)>)?\(", f.read())
    assert waits and all(w in ("", "0") for w in waits), waits


def test_long_chunks_rows_are_in_before_the_next_codes_go_out():
    """Step: barrier, next rows asked for, products; then the wait, then the codes after the next."""
    body = kernel("k_linear_many")
    loop = body[body.index("for (int kb = 0; kb < nkb; ++kb) {"):]
    order = [loop.index(s) for s in ("barrier_no_fence();", "load_rows(kb + 1)", "wait_vm<0>()", "expand(kb + 1)", "load_codes(")]
    assert order == sorted(order)
    before = body[:body.index("for (int kb = 0; kb < nkb; ++kb) {")]
    order = [before.index("load_rows(0)"), before.index("wait_vm<0>()"), before.rindex("load_codes(")]
    assert order == sorted(order)


def test_split_waits_for_its_reads_before_the_buffer_is_written_again():
    """A wave has no barrier between its reads of a buffer and the DMA that writes it two steps later."""
    body = kernel("k_linear_split")
    loop = body[body.index("while (true) {"):]
    loop = loop[:loop.index("\n    }\n")]
    assert re.findall(r"(wait_\w+|load|compute)(?:<0>)?\(", loop) == ["wait_rows_and_reads", "load", "compute"] * 2

"""Rules of the long-context kernels that no run can show reliably, read from the sources.

Kernels launched with programmatic stream serialisation begin while the kernel before them runs, up
to their griddepcontrol.wait.  Loads through the read-only path (ld.global.nc, __ldg) are allowed
only for data that no overlapping kernel writes: the compiler may move them above the wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "kv_cache_quantization_gb300", "csrc")


def source(name):
    """The file without comments."""
    s = open(os.path.join(CSRC, name), encoding="utf-8").read()
    s = re.sub(r"/\*.*?\*/", " ", s, flags=re.S)
    return re.sub(r"//[^\n]*", "", s)


def kernels(text):
    """(name, body) of each __global__ function."""
    for m in re.finditer(r"__global__.*?(\w+)\s*\(", text, re.S):
        name = m.group(1)
        if name == "__launch_bounds__":
            m = re.compile(r"__launch_bounds__\([^)]*\)\s*(\w+)\s*\(").search(text, m.start())
            name = m.group(1)
        begin = text.index("{", m.end())
        depth = 0
        for i in range(begin, len(text)):
            depth += (text[i] == "{") - (text[i] == "}")
            if not depth:
                break
        yield name, text[begin:i]


def test_the_row_operands_are_not_read_through_the_read_only_path():
    """rows_prep_kernel writes qop and qf while rows_attn_kernel may already run."""
    body = dict(kernels(source("rows_attn.cu")))["rows_attn_kernel"]
    wait = body.index("softmax_tiles")
    assert "a.qop" in body and "a.qf" in body
    assert "__ldg" not in body[:wait] and "load_early" not in body[:wait]


def test_the_preparation_starts_the_attention_after_its_own_wait():
    """rows_attn_kernel reads lengths, lists, tables and codes before it waits: that is right because
    it can start only once every CTA of rows_prep_kernel is past its wait for what came before."""
    body = dict(kernels(source("rows_attn.cu")))["rows_prep_kernel"]
    assert 0 < body.index("griddepcontrol.wait") < body.index("griddepcontrol.launch_dependents")


@pytest.mark.parametrize("kernel", ["block_score_kernel", "block_select_kernel"])
def test_bounds_and_tables_are_not_read_through_the_read_only_path(kernel):
    """The kernel before (tq_block_bounds, a caller's own) may have written bounds, queries, lengths
    and tables; block_bounds_kernel itself is an ordinary launch."""
    text = source("blocks.cu")
    assert "__ldg" not in dict(kernels(text))[kernel]
    helpers = text[:text.index("block_bounds_kernel")] + text[text.index("struct SelectArgs"):]
    assert "__ldg" not in helpers and ".nc" not in helpers
    internal = source("tq_internal.h")
    begin = internal.index("bool tq_map_slot")
    assert "__ldg" not in internal[begin:internal.index("return pg >= 0", begin)]


def test_inputs_of_waiting_kernels_are_not_read_through_the_read_only_path():
    """Queries of the decode's operand kernel and vectors of the appends, both read after the wait."""
    text = source("decode_tc.cu")
    begin = text.index("griddepcontrol.wait")
    prep = text[begin:text.index("query_prep_tc_kernel", begin)]
    assert "a.q)" in prep and "__ldg" not in prep
    text = source("append_small.h")
    begin = text.index("void append_load8")
    assert "__ldg" not in text[begin:text.index("__device__", begin)]

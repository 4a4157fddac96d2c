"""Kernels that may start under the one before them see its writes only after
griddepcontrol.wait: read in the sources, each runs it before it touches memory
and before it lets the next kernel's blocks in."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "paged_quantized_kv_append_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def _kernels():
    """(file, name, body) of every kernel."""
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        text = _source(name)
        for m in re.finditer(r"__global__\s", text):
            head = re.compile(r"(\w+)\((?:const\s)[^{;]*\)\s*\{").search(text, m.end())
            depth, at = 1, head.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            yield name, head.group(1), text[head.end():at]


def _pointers():
    """Members of the kernels' parameter structs that point to global memory."""
    found = set()
    for name in ("pqkv_internal.h", "shared_prefix.cuh"):
        found |= set(re.findall(r"^\s+(?:const\s+)?\w+\*\s+(\w+);", _source(name), flags=re.M))
    return found | {"plan"}


KERNELS = list(_kernels())


def test_the_kernels_are_found():
    names = {k[1] for k in KERNELS}
    assert {"paged_attention_kernel", "lse_merge_kernel", "shared_plan_kernel", "private_kernel",
            "shared_umma_kernel", "shared_merge_kernel", "extend_tables_kernel",
            "truncate_tables_kernel"} <= names
    assert {"q", "seq_lens", "pre_o", "suf_ml", "plan", "free_pages"} <= _pointers()


@pytest.mark.parametrize("file,name,body", KERNELS, ids=["%s-%s" % k[:2] for k in KERNELS])
def test_a_kernel_waits_before_it_touches_memory(file, name, body):
    wait = body.find("grid_dependency_wait()")
    assert wait >= 0, "no wait for the kernel before"
    start = body[:wait]
    assert "grid_dependents_launch" not in start
    touched = re.findall(r"\bp\.(%s)\b" % "|".join(sorted(_pointers())), start)
    assert not touched, "reads or writes %s before the wait" % touched
    # nor hands all its parameters to a function or an object
    assert not re.search(r"[({]\s*p\s*[,)}]", start)

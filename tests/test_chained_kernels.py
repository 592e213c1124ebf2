"""Kernels that a launch sets up while the kernel before them still runs
(``grid_wait`` in csrc) read global memory by ordinary loads: the read-only path
is for memory that nothing writes while the kernel lives, and a compiler may move
its loads above the wait."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ulysses_sequence_long_gb300", "csrc")


def _sources():
    """The files that launch or define such kernels, and the headers that they include."""
    text = {f: re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read()) for f in os.listdir(CSRC)}
    todo = [f for f, s in text.items() if re.search(r"\bgrid_wait\(\)", s) or "launch_chained(" in s]
    assert {"usp_bandwidth.cu", "usp_attn_fwd.cuh", "usp_attn_bwd.cuh", "usp_attn_mod_bwd.cu"} <= set(todo)
    out = {}
    while todo:
        f = todo.pop()
        if f in text and f not in out:
            out[f] = text[f]
            todo += re.findall(r'#include "([^"]+)"', text[f])
    return out


def test_no_read_only_loads():
    for f, s in _sources().items():
        assert "__ldg(" not in s, f
        assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", s), f


def test_every_chained_kernel_waits():
    """A kernel passed to launch_chained calls grid_wait before anything else touches global memory; one that did not
    would let the kernel after it start before the kernel before it has ended."""
    kernels = {}
    for f, s in _sources().items():
        for m in re.finditer(r"__global__[^;{]*?\b(\w+)\s*\(", s):
            if m.group(1) in ("__launch_bounds__",):
                m = re.compile(r"\b(\w+_kernel)\s*\(").search(s, m.end())
            body = s[m.end():]
            nxt = body.find("__global__")
            kernels[m.group(1)] = body if nxt < 0 else body[:nxt]
    chained = {"relayout_kernel", "relayout_reduce_kernel", "relayout_qkv_kernel", "scan_init_kernel", "scan_kernel",
               "scan_small_kernel", "rel_expand_kernel", "rel_sum_kernel", "rel_grad_kernel", "mod_dsink_kernel",
               "delta_kernel", "attn_fwd_kernel", "dkdv_kernel", "dq_kernel", "dq_ds_kernel", "preprocess_kernel"}
    assert chained <= set(kernels), chained - set(kernels)
    for name in chained:
        before, wait, _ = kernels[name].partition("grid_wait()")
        assert wait, name
        assert "gld(" not in before, name

"""Kernels that are launched while the one before them still runs (chained.cuh): all of them wait for it, and none tells the
compiler that nobody writes the memory that it reads (a restrict-qualified or read-only load may be taken from a cache that
does not follow other kernels' stores, or moved above the wait)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_scan_gb300", "csrc")
SOURCES = {os.path.basename(f): open(f).read() for f in glob.glob(os.path.join(CSRC, "*.cu"))}


def _kernels(text):
    """name -> text of every kernel, from its __global__ to the brace that ends it in the first column."""
    return {re.search(r"(\w+)\(\s*(const\b|\w)", re.sub(r"__\w+__\s*\([^()]*\)", "", part)).group(1): part
            for part in (m.group(0) for m in re.finditer(r"__global__ void.*?\n}\n", text, re.S))}


def test_chained_kernels():
    found = {}
    for name, text in SOURCES.items():
        kernels = _kernels(text)
        for k, body in kernels.items():
            if "wait_for_earlier()" in body:
                found[k] = body
        for call in re.finditer(r"launch_chained\((\w+)", text):
            at = call.group(1)
            if at in kernels:                              # (others are chosen among kernels by a variable)
                assert "wait_for_earlier()" in kernels[at], f"{name}: {at} does not wait"
    assert {"column_sum_kernel", "xent_gemm_kernel", "xent_gather_kernel", "xent_pack_kernel", "xent_join_kernel", "xent_scatter_kernel"} <= set(found)
    for k, body in found.items():
        assert "__restrict__" not in body and "__ldg(" not in body and "ld.global.nc" not in body, k

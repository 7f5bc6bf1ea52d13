"""The benchmark's record of DRAM traffic counts only while a kernel's sources are unchanged: the files
that it looks at have to hold the kernel, and whatever of this library's they include."""

import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "dynamic_causal_attention_gb300", "csrc")
KERNELS = {"hybrid_fwd": "hybrid_fwd_kernel", "static_dv": "hybrid_fwd_kernel",
           "bwd_dynamic": "bwd_dynamic_kernel", "param_grad": "param_grad_kernel"}


def read(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return f.read()


@pytest.mark.parametrize("name", sorted(bench.KERNEL_SOURCES))
def test_a_kernels_sources_hold_it(name):
    files = bench.KERNEL_SOURCES[name]
    code = "\n".join(read(f) for f in files)
    assert re.search(r"__launch_bounds__\([^)]*\)\s*" + KERNELS[name] + r"\(", code)


@pytest.mark.parametrize("name", sorted(bench.KERNEL_SOURCES))
def test_and_what_they_include(name):
    files = (*bench.KERNEL_SOURCES[name], "internal.h")   # (declarations of the host's side)
    for f in bench.KERNEL_SOURCES[name]:
        for other in re.findall(r'#include "([\w.]+)"', read(f)):
            assert other in files, (f, other)


def test_every_recorded_kernel_is_known():
    with open(os.path.join(bench.ROOT, "profiles", "dram_traffic.txt")) as f:
        rows = [line.split() for line in f if not line.startswith("#")]
    assert {r[1] for r in rows} == set(KERNELS)
    for workload, kernel, nbytes, digest in rows:
        assert workload in ("124m", "1b") and float(nbytes) > 0 and re.fullmatch(r"[0-9a-f]{16}", digest)
        if digest == bench.source_hash(kernel):
            assert bench.ncu_traffic(kernel, workload) == float(nbytes)

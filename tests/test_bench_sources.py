"""The sources that a stored traffic figure is tied to are all that its kernel is
made of: what its headers include, and what those include."""
import importlib.util
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "structured_sparse_quantized_b200", "csrc")


def included(name, seen):
    if name not in seen:
        seen.add(name)
        with open(os.path.join(CSRC, name)) as f:
            for other in re.findall(r'^#include "(\w+\.cuh)"', f.read(), re.M):
                included(other, seen)
    return seen


def test_gemm_sources_are_complete():
    spec = importlib.util.spec_from_file_location("bench_sources", os.path.join(ROOT, "bench.py"))
    bench = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bench)
    needed = included("ss_gemm_wide.cuh", included("ss_gemm.cuh", set()))
    assert needed <= set(bench.GEMM_SOURCES)
    for tr in bench.TRAFFIC.values():
        assert needed <= set(tr["sources"])

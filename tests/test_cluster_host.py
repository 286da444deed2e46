"""Kernels of a cluster write another CTA's shared memory only once every CTA has started
(no GPU needed: the sources are read)."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "paged_kv_cache_74_gb300", "csrc")


def text_of(name):
    text = open(os.path.join(CSRC, name), encoding="utf-8").read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", [n for n in sorted(os.listdir(CSRC)) if "map_shared_rank" in text_of(n)])
def test_remote_shared_memory_is_used_behind_a_barrier(name):
    """In every function that maps a peer's shared memory a cluster barrier comes first, and
    every kernel arrives on it before anything else it does with the cluster."""
    text = text_of(name)
    for use in re.finditer("map_shared_rank", text):
        start = text.rfind("\n__device__", 0, use.start())
        assert re.search(r"cluster_wait\(\)|cluster\.sync\(\)", text[start:use.start()]), name
    kernels = re.findall(r"__global__.*?\n}", text, re.S)
    assert kernels
    for body in kernels:
        if "exchange(" in body:
            assert body.index("cluster_started(") < body.index("griddep_wait(") < body.index("exchange(")

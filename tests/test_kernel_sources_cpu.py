"""What the kernels' sources must say for a launch to be safe, and what no run on one
GPU with one compiler could show: read from csrc/ as text."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_cache_179_gb300", "csrc")


def sources():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            yield name, re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_dynamic_shared_memory_states_its_alignment():
    """Kernels read and write it 16 bytes at a time (asynchronous copies want more); an
    array of int without a stated alignment may begin at any multiple of 4."""
    found = 0
    for name, text in sources():
        for decl in re.findall(r"extern\s+__shared__[^;]*;", text):
            found += 1
            stated = re.search(r"__align__\((\d+)\)", decl)
            assert stated and int(stated.group(1)) >= 16, f"{name}: {decl}"
    assert found >= 5


def test_cluster_barriers_follow_a_warp_barrier():
    """barrier.cluster's .aligned forms need all threads of a warp at the same instruction:
    each one stands right behind a __syncwarp(), which brings them there whatever loop or
    branch came before."""
    found = 0
    for name, text in sources():
        for m in re.finditer(r'asm volatile\(\s*"barrier\.cluster', text):
            found += 1
            before = text[:m.start()].rstrip()
            assert before.endswith("__syncwarp();"), f"{name}: {before[-60:]!r}"
    assert found >= 2

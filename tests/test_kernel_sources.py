"""Rules of the kernels' sources that no run shows: what orders shared memory between
ordinary accesses and those of the copy engine and the tensor cores."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_mxfp4_w4a4_gb300", "csrc")


def source(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "kv_attention*.cuh"))),
                         ids=os.path.basename)
def test_fenced_writes_meet_a_barrier_before_the_arrival(path):
    """Each lane fences its own writes; one lane's arrival on a barrier (or its copy) says
    that all are fenced, so a barrier of the lanes stands between the two."""
    text = source(path)
    for m in re.finditer(r"fence_proxy_async_smem\(\);", text):
        rest = text[m.end():]
        barrier = re.search(r"__syncwarp\(\);|__syncthreads\(\);|named_barrier_sync\(", rest)
        told = re.search(r"mbar_arrive|tma_store|bulk_store|bulk_commit", rest)
        assert barrier and (not told or barrier.start() < told.start()), text[:m.start()].count("\n") + 1


def test_scratch_of_prompt_attention_is_no_place_of_a_copy():
    """What finds a CTA's run writes shared memory as threads do; the copies that follow
    go elsewhere (a CTA barrier does not order the two)."""
    text = source(os.path.join(CSRC, "prompt_attention.cu"))
    scratch = re.search(r"= find_run\(p, (?:reinterpret_cast<Scan\*>\()?smem( \+ C::(\w+))?", text)
    copied = set(re.findall(r"tma_load_3d\(smem \+ (?:C::(OFF_\w+) \+)?", text))
    assert copied == {"", "OFF_K", "OFF_V"}       # queries, keys, values
    assert scratch and (scratch.group(2) or "") not in copied

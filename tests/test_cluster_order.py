"""Distributed shared memory may be touched only once every CTA of the cluster is known
to run, and a CTA may leave only once no other touches its memory: in every kernel
that reaches into another CTA, a cluster barrier is passed before the first such
access and after the last one.  A violation hardly ever shows in a run, so the order
is read from the source."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_layer_dual_b200", "csrc")
# what reaches another CTA of the cluster, or calls a helper that does
REMOTE = re.compile(r"\b(smem_in_rank|in_rank|arrive_cluster|mbar_arrive_cluster|add_tiles|add_rows|share_failed|"
                    r"warp_arrive_leader|tma_load_2d_pair)\s*[(<]|st\.shared::cluster|ld\.shared::cluster|mapa\.")
# prologue and teardown: the pair kernels' helpers, which hold their cluster_sync
PASSED = re.compile(r"\b(cluster_sync|cluster_wait|prologue|teardown)\s*\(")


def _body(text, at):
    """The brace-matched block that opens after `at`."""
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return text[start: i + 1]
    raise AssertionError("unbalanced braces")


def _strip(text):
    return re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", text), flags=re.S)


def _kernels():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu"):
            text = _strip(open(os.path.join(CSRC, name)).read())
            for m in re.finditer(r"__global__.*?\b(k_\w+)\s*\(", text, flags=re.S):
                yield f"{name}:{m.group(1)}", _body(text, m.end())


def _remote_kernels():
    return [(n, b) for n, b in _kernels() if REMOTE.search(b)]


def test_the_cluster_kernels_are_found():
    names = {n for n, _ in _remote_kernels()}
    assert {"balance.cu:k_balance_finish", "gemm_fp8_block.cu:k_product", "gemm_fp8_few.cu:k_product_few"} <= names


@pytest.mark.parametrize("name", [n for n, _ in _remote_kernels()])
def test_a_cluster_barrier_is_passed_before_and_after_remote_accesses(name):
    body = dict(_remote_kernels())[name]
    touched = [m.start() for m in REMOTE.finditer(body)]
    passed = [m.start() for m in PASSED.finditer(body)]
    assert passed and min(passed) < min(touched), f"{name}: another CTA is reached before the cluster has met"
    assert max(passed) > max(touched), f"{name}: a CTA may leave while another reaches it"


def test_the_pair_kernels_helpers_hold_the_barriers():
    text = _strip(open(os.path.join(CSRC, "gemm_bf16_2sm.cu")).read())
    for helper in ("prologue", "teardown"):
        body = _body(text, re.search(rf"\b{helper}\(", text).end())
        assert "cluster_sync()" in body
        assert not REMOTE.search(body), f"{helper} reaches the other CTA itself"

"""What no run can show: what the pairs of blocks behind a shared prefix order at the cluster's scope, read in the source."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_kv_csa_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, head):
    """From a head to the closing brace at the beginning of a line."""
    at = text.index(head)
    return text[at:text.index("\n}", at)]


def test_arrivals_across_blocks_release_and_their_waits_acquire_at_the_clusters_scope():
    """A block's queries and weights, written to its own shared memory, are read by products that the other block's threads issue: the
    arrival that says so has to release at the cluster's scope, a barrier operation of that scope carries it, and the wait acquires."""
    text = source("csa_tcgen05.cuh")
    arrive, wait = body(text, "void mbar_arrive_cluster("), body(text, "bool mbar_wait_cluster(").replace(
        "acquire_cluster();", "fence.acquire.cluster;" if "fence.acquire." in body(text, "void acquire_cluster()") else "")
    assert re.search(r"fence\.release\.[\w:.]*cluster;.*mbarrier\.arrive\.\w+\.cluster\.shared::cluster", arrive, re.S) or \
        "mbarrier.arrive.release.cluster" in arrive
    assert re.search(r"mbarrier\.try_wait\.parity\.\w+\.cluster", wait)
    assert re.search(r"mbarrier\.try_wait.*fence\.acquire\.[\w:.]*cluster;", wait, re.S) or "try_wait.parity.acquire.cluster" in wait


def test_the_warps_of_products_wait_so_for_both_blocks_arrivals():
    kernel = source("csa_shared.cu")
    kernel = kernel[kernel.index("latent_pair_kernel(const AttnParams"):kernel.index("shared_plan_kernel(")]
    issue = kernel[kernel.index("kQueryStep = kQueryChunk"):kernel.index("mma_commit_pair(smem_addr(&sh.drained))")]
    assert re.search(r"wait_both = .*mbar_wait_cluster", issue)
    for bar in ("p_full", "q_full"):
        waits = re.findall(r"(\w+)\(&sh\.%s\b" % bar, issue)
        assert waits and set(waits) == {"wait_both"}, (bar, waits)
    # the arrivals at them come from both blocks, behind the writes' proxy fence
    for bar in ("p_full", "q_full"):
        for at in [m.start() for m in re.finditer(r"mbar_arrive_cluster\(%s" % bar, kernel)]:
            before = kernel[:at]
            assert before.rindex("fence_async_smem();") > max(before.rindex("copy_async_16(") if bar == "q_full" else before.rindex("make_uint4("), 0)
        assert "mbar_arrive_cluster(%s" % bar in kernel


def test_and_for_the_other_blocks_copies():
    kernel = source("csa_shared.cu")
    issue = kernel[kernel.index("kQueryStep = kQueryChunk"):kernel.index("mma_commit_pair(smem_addr(&sh.drained))")]
    here = issue[issue.index("auto arrived ="):issue.index("PairWalk w(")]
    assert "mbar_test_cluster(" in issue[issue.index("auto ready ="):issue.index("auto arrived =")]
    assert "acquire_cluster();" in here and "wait_both(&sh.kv_full[" in here and " wait(" not in issue

"""How the kernels hand shared memory from one CTA of a cluster to another:
an arrival on another CTA's barrier must release at the cluster's scope, itself
or by a fence before it (the default scope is the CTA, which orders nothing for
the other one), and a kernel that sends such arrivals must wait for them with an
acquire at that scope.
Read from the sources: a missing order shows in no result that can be relied
on."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(__file__), "..", "blockwise_attention_ffn_gb300", "csrc")


def sources():
    paths = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))
    assert paths
    return {os.path.basename(p): open(p).read() for p in paths}


def test_arrivals_on_other_ctas_release_at_cluster_scope():
    found = 0
    for name, text in sources().items():
        code = re.sub(r"//[^\n]*", "", text)
        for asm in re.findall(r"\basm volatile\((.*?)\);", code, re.S):
            for op in re.findall(r"\bmbarrier\.arrive[\w.:]*", asm):
                if "shared::cluster" in op and not op.startswith("mbarrier.arrive.expect_tx"):
                    found += 1
                    fenced = re.search(r"fence\.release\.[\w.:]*\.cluster;.*mbarrier\.arrive\.relaxed\.cluster", asm, re.S)
                    assert ".release.cluster" in op or fenced, f"{name}: {op}"
    assert found


def test_kernels_that_arrive_across_wait_at_cluster_scope():
    """Every barrier that mbar_arrive_cluster is given the address of (cluster_addr(smem_u32(<barrier>), 0)) is
    waited for by a cluster-scope wait in the same file."""
    found = 0
    for name, text in sources().items():
        if name == "ptx.cuh":
            continue
        code = re.sub(r"//[^\n]*", "", text)
        bars = dict(re.findall(r"(\w+) = (?:PAIR \? )?cluster_addr\(smem_u32\((\w+)\), 0\)", code))
        for var in set(re.findall(r"mbar_arrive_cluster(?:_smem)?\((\w+)", code)):
            if var in bars:
                found += 1
                assert re.search(r"bounded_wait_cluster_w\(&%s\[" % bars[var], code), f"{name}: {bars[var]}"
    assert found >= 3  # the accumulators of both products, and the grouped product's copies

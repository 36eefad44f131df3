"""Arrivals on the barrier of another CTA of the cluster that hand memory over are ordered at
cluster scope: a release at CTA scope orders nothing for a waiter in the other CTA. Read
from the sources: such a race has no run that shows it for certain."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def sources():
    for d in ("csrc", "csrc_experts"):
        for f in sorted(glob.glob(os.path.join(ROOT, "dense_gemm_persistent_gb300", d, "*.cu*"))):
            yield os.path.basename(f), open(f).read()


def test_no_arrival_on_a_cluster_address_is_ordered_at_cta_scope():
    seen = 0
    for name, text in sources():
        for form in re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*", text):
            seen += 1
            assert ".cluster." in form.replace("shared::cluster", ""), (name, form)
    assert seen > 0


def test_what_is_handed_over_is_released_first():
    text = dict(sources())
    arrive = text["experts_ptx.cuh"].split("void mbar_arrive_peer(")[1].split("}")[0]
    assert arrive.index("fence.release.sync_restrict::shared::cta.cluster;") < arrive.index("mbar_arrive_cluster_relaxed(")
    for name in ("experts_mma.cuh", "experts_int8.cuh"):
        assert text[name].count("mbar_arrive_peer(mapa_shared(") == 1


def test_waits_for_the_other_cta_acquire_at_cluster_scope():
    """The MMA issuers of kernels whose rows the peer CTA writes with ordinary stores or cp.async."""
    text = dict(sources())
    assert "mbar_wait_warp_at<CF::PAIR && CF::GATHER>(&full[stage]" in text["experts_mma.cuh"]
    assert "mbar_wait_warp_at<CF::PAIR>(&full[two]" in text["experts_int8.cuh"]

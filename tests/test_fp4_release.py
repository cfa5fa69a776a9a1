"""The FP4 stream kernel's exchange of partial sums between the CTAs of a cluster, read from its source.

A buffer of sums is handed to other CTAs (full) and back (free) by arrivals on their barriers.  What an
arrival orders are plain accesses to shared memory of one CTA before accesses of another, so it has to release
at cluster scope, and the wait for it to acquire at cluster scope; tcgen05 and async-proxy fences, which let
other arrivals do with CTA scope, have no part in it.  (Sums that are sent by st.async complete their barrier
themselves.)
"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_precision_quantized_mx_b200", "csrc")


def source(name):
    return open(os.path.join(CSRC, name)).read()


def test_arrivals_on_other_ctas_buffers_release_at_cluster_scope():
    text = source("fp4_stream.cu")
    remote = re.findall(r"(\w+)\(mapa_shared\(&S\.(red_\w+)\[\w+\], lane\)\)", text)
    assert sorted(b for _, b in remote) == ["red_free", "red_free", "red_full"]
    assert {f for f, _ in remote} == {"arrive_release_cluster"}
    assert re.search(r"arrive_release_cluster\(uint32_t bar\) \{\s*asm volatile\(\"mbarrier\.arrive\.release\.cluster\.",
                     source("fp4_mma.cuh"))


def test_their_waits_acquire_at_cluster_scope():
    waits = re.findall(r"(\w+)\(&S\.red_\w+\[\w+\], [^;]*?abort", source("fp4_stream.cu"))
    assert len(waits) == 4 and set(waits) == {"wait_cluster"}
    assert "mbarrier.try_wait.parity.acquire.cluster." in source("fp4_mma.cuh")

"""The order between the two CTAs of a pair, read from the source: an arrival on the other CTA's barrier releases at
cluster scope what its instructions for the pair are to read, and the waits of the kernels that use pairs acquire there.
(CTA scope, the default, gives no order between two CTAs; a test on the GPU cannot show that it is missing.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int8_expert_weight_b200", "csrc")


def sources():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            with open(os.path.join(CSRC, name)) as f:
                yield name, re.sub(r"//[^\n]*", "", f.read())


def functions(text):
    """Bodies that hold inline PTX, each from its __device__ to the next one."""
    return re.split(r"(?=__device__)", text)


def test_remote_arrivals_release_at_cluster_scope():
    found = 0
    for name, text in sources():
        for body in functions(text):
            if re.search(r"mbarrier\.arrive[a-z._]*\.shared::cluster", body):
                found += 1
                assert re.search(r"mbarrier\.arrive\.release\.cluster|fence\.release\.[a-z_:]*\.?cluster;|"
                                 r"fence\.release\.sync_restrict::shared::cta\.cluster", body), name
    assert found == 1


def test_waits_of_pairs_acquire_at_cluster_scope():
    texts = dict(sources())
    wait = next(b for b in functions(texts["tc.cuh"]) if re.search(r"bool mbar_wait_bounded\(", b))
    assert re.search(r"if constexpr \(kCluster\)[^;]*fence\.acquire\.sync_restrict::shared::cluster\.cluster", wait)
    assert re.search(r"mbarrier\.try_wait\.parity\.(acquire|relaxed)\.cluster", texts["tc.cuh"])
    users = [n for n, t in texts.items() if "mbar_arrive_cluster(" in t and n != "tc.cuh"]
    assert users == ["gemm_mx4.cu"]
    for name in users:
        assert re.findall(r"mbar_wait_bounded(<\w+>)?\(", texts[name]) == ["<kPair>"], name

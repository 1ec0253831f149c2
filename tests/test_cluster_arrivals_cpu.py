"""What the kernels' sources say of barriers that another CTA of a cluster waits on. Such an ordering can be left out for a long time before a
wrong result shows, so it is looked for in the text: an arrival that names no scope has that of its own CTA."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_ffn_topk_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return "\n".join(line.split("//")[0] for line in f)


def function(text, name):
    """The text of a __device__ function of that name."""
    start = re.search(r"__device__[^;{]*\b%s\(" % name, text).start()
    return text[start:text.index("\n}", start)]


def test_arrivals_on_a_cluster_address_have_the_cluster_scope():
    found = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        for arrive in re.findall(r"mbarrier\.arrive[\w.:]*", source(os.path.basename(path))):
            if ".shared::cluster" in arrive:
                found += 1
                assert ".release.cluster." in arrive or ".relaxed.cluster." in arrive, (path, arrive)
    assert found >= 3


def test_int8_operands_are_released_to_the_pair():
    """The other CTA's converters write shared memory that the even CTA's MMAs read: a release of cluster scope before the arrival (a relaxed one
    is enough for tensor memory alone, with tcgen05's own fences), and waits of that scope at the other end."""
    text = source("int8_matmul.cu")
    body = function(text, "mbar_arrive_remote")
    assert re.search(r"fence\.release\S*\.cluster|fence\.acq_rel\.cluster|arrive\.release\.cluster", body)
    assert re.search(r"mbar_arrive_remote\(mapa_shared\(op_full\(", text) and not re.search(r"mbar_arrive_relaxed\(mapa_shared\(op_full\(", text)
    for barrier in ("op_full", "op_free", "acc_full", "acc_free"):
        waits = re.findall(r"(?:wait_for|completed)(<\w+>)?\(%s\(" % barrier, text)
        assert waits and all(w == "<kPair>" for w in waits), barrier

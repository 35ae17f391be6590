"""What can be seen only in the kernels' source: an order that a fault would
need luck (of when blocks start) to show."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_exact_xor_gb300", "csrc")


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_no_block_reaches_into_another_before_the_cluster_runs():
    # every access to a cluster's shared memory comes behind a wait of the cluster's barrier in the same kernel
    body = _code("policy_loss.cu").split("loss_kernel(LossArgs A, uint32_t cluster)", 1)[1]
    remote = body.index("st.shared::cluster")
    assert "barrier.cluster.arrive" in body[:remote] and "barrier.cluster.wait" in body[:remote]
    kernel = _code("nvfp4_matmul.cu").split("\nmatmul_kernel(", 1)[1]
    assert "cluster_sync();" in kernel[:kernel.index("load_cluster(")]

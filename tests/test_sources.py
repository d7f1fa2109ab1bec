"""What the library's sources must not hold (no GPU needed)."""
import glob
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_kernel_uses_cluster_multicast():
    """One library serves every replica of a job on several GPUs, where multicast into a cluster is not to be used."""
    files = [f for d in ("gqa_decode_attention_paged_gb300/csrc", "include") for f in glob.glob(os.path.join(ROOT, d, "*"))]
    assert len(files) > 10
    for f in files:
        with open(f) as src:
            assert "multicast" not in src.read().lower(), os.path.basename(f)

"""What the library's sources must not contain, checked on the text without a GPU."""
import glob
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _sources():
    names = glob.glob(os.path.join(ROOT, "dtensor_reshard_gb300", "csrc", "*"))
    names += glob.glob(os.path.join(ROOT, "include", "*"))
    assert len(names) > 15
    return {n: open(n, encoding="utf-8").read() for n in names}


def test_no_multicast_over_a_cluster():
    """The library is loaded by every rank of a run on several GPUs, and an operand may be
    memory of another GPU: every CTA loads its own tiles."""
    for name, text in _sources().items():
        assert ".multicast" not in text, name

"""What the sources may hold.  The library serves as one of several replicas of
a job, one process per GPU: every CTA fetches its own tiles, and no kernel uses
a multicast load or commit."""
import os

from protein_folding_attention_gb300 import build_lib


def sources():
    for folder in (build_lib.CSRC, build_lib.INCLUDE):
        for name in sorted(os.listdir(folder)):
            yield os.path.join(folder, name)


def test_no_multicast():
    named = []
    for path in sources():
        with open(path) as f:
            named += [path] if "multicast" in f.read() else []
    assert not named

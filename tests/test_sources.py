"""What the library's sources must not hold, checked on their text."""
import os

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mxfp4_routed_expert_route_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(os.listdir(CSRC)))
def test_no_copy_or_arrival_leaves_its_cta(name):
    """The library is loaded by every rank of a job on several GPUs and takes
    whatever device pointers it is given, so no copy is sent to several CTAs at
    once, and no CTA waits on another, whose arrivals could outlive it."""
    text = open(os.path.join(CSRC, name)).read()
    for word in (".multicast", "barrier.cluster", "cudaLaunchAttributeClusterDimension", "mapa."):
        assert word not in text, f"{name}: {word}"

"""What no run can show of the layer operators' kernels, read from their source.

A wait for what other CTAs of a cluster have sent has to acquire at cluster scope: at
CTA scope the reads after it are not ordered behind those stores, whatever a run gives.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "state_space_model_03_gb300", "csrc")


def _text(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def _function(text, name):
    """From a function's name to the closing brace at the start of a line."""
    return re.search(rf"\b{name}\([^;{{]*\{{.*?\n\}}", text, re.S).group(0)


@pytest.mark.parametrize("source", ["ss_gated_scan.cu", "ss_gated_bwd.cu"])
def test_the_exchange_is_acquired_at_cluster_scope(source):
    waits = re.findall(r"\b(\w*wait\w*)\(&here\[", _text(source))
    assert waits == ["mbar_wait_cluster"]
    assert re.findall(r"try_wait\S*?(acquire\.\w+)", _function(_text("ss_gated.cuh"), "mbar_wait_cluster")) == ["acquire.cluster"]

"""A kernel's source fingerprint covers every file of csrc/ that it is compiled
from: an edit to any of them outdates a stored profile of that kernel (no GPU)."""
import os
import re

import pytest

from top_routing_grouped_moe_gb300 import build


def _text(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return f.read()


def _included(name):
    """The csrc/ files that `name` includes, directly or not."""
    found = set()
    for inc in re.findall(r'^#include "([^"/]+)"', _text(name), flags=re.M):
        if os.path.exists(os.path.join(build.CSRC, inc)):  # not the public header
            found |= {inc} | _included(inc)
    return found


def _launch_names():
    """Every launch name given in the sources: (file, name)."""
    for src in sorted(f for f in os.listdir(build.CSRC) if f.endswith(".cu") and f != "moe_abi.cu"):
        text = _text(src)
        names = set(re.findall(r'timing_mark\(s, "(\w+)"\)', text)) | set(re.findall(r'"((?:gemm|vocab)_\w+)"', text))
        for name in sorted(names):
            yield src, name


@pytest.mark.parametrize("src,name", list(_launch_names()))
def test_fingerprint_covers_the_sources(src, name):
    listed = {os.path.basename(p) for p in build._kernel_sources(name)}
    assert src in listed
    for f in listed:
        missing = _included(f) - listed
        assert not missing, f"{name}: {f} includes {sorted(missing)}"

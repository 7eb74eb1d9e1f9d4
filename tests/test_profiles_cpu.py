"""The recorded measurements under profiles/ name the sources that they were taken on.
Where that is what the sources are now, the kernels that they name are kernels of the
library built from them: figures of other kernels cannot pass as theirs."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import bench  # noqa: E402
import microscaling_quantized_linear_amd as mx  # noqa: E402

PROFILES = sorted(f for f in os.listdir(os.path.join(ROOT, "profiles")) if f.endswith(".md"))


@pytest.fixture(scope="module")
def kernels():
    if not os.path.exists(mx.LIB_PATH):
        pytest.skip("the library is not built")
    r = subprocess.run(["nm", "-C", mx.LIB_PATH], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return {m[1] for m in re.finditer(r"(mx::\w+kernel(?:<[^()]*>)?)\(", r.stdout)}


@pytest.mark.parametrize("name", PROFILES)
def test_recorded_kernels_are_the_sources(kernels, name):
    text = open(os.path.join(ROOT, "profiles", name)).read()
    start = 0
    for m in re.finditer(r"Kernel sources: `([^`]+)`, sha256 prefix (\w+)\.", text):
        section, start = text[start:m.start()], m.end()
        named = set(re.findall(r"`(?:void )?(mx::\w+kernel(?:<[^()`]*>)?)\([^`.]*\)`", section))
        assert named, f"{name}: no kernel named"
        if bench.source_sha(*m[1].split(", ")) == m[2]:
            assert named <= kernels, (name, named - kernels)
    for m in re.finditer(r'"source_sha": "(\w+)"', text):
        assert f"sha256 prefix {m[1]}." in text, (name, m[1])

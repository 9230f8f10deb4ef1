"""Tests that make valid calls with made-up addresses run only where no device could take them."""
import os
import re
import subprocess
import sys

import pytest

from tests.conftest import NO_DEVICE_TESTS, ROOT

# pytest as on a host with so many devices; the library itself sees none.
RUN = """
import sys, pytest, torch
torch.cuda.device_count = lambda: %d
sys.exit(pytest.main(["-q", "-rs", "-p", "no:cacheprovider"] + sys.argv[1:]))
"""


@pytest.mark.parametrize("devices", [0, 1])
def test_calls_with_made_up_addresses_are_skipped_beside_a_device(devices):
    names = sorted("tests/" + n for n in NO_DEVICE_TESTS)
    out = subprocess.run([sys.executable, "-c", RUN % devices, *names], cwd=ROOT, capture_output=True, text=True,
                         env={**os.environ, "HIP_VISIBLE_DEVICES": "-1"}, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr
    assert re.search(r"\b%d %s" % (len(names), "skipped" if devices else "passed"), out.stdout), out.stdout

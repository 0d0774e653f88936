"""Every copy into shared memory is the copying CTA's own (CPU).

One library serves jobs on one GPU and every rank of a job on several, where a copy that fans out to
the CTAs of a cluster must not run; so no source of the library has the instruction's modifier.
"""

import glob
import os

import pytest

from paged_mla_decode_gb300 import build as mbuild

SOURCES = sorted(p for kind in ("*.cu", "*.cuh", "*.h") for p in glob.glob(os.path.join(mbuild.CSRC, kind)))


def test_sources_are_found():
    assert any(p.endswith("tc_ptx.cuh") for p in SOURCES)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_copy_fans_out(path):
    with open(path) as f:
        found = [n for n, line in enumerate(f, 1) if "multi" + "cast" in line.lower()]
    assert not found

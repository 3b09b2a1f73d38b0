"""The words that the recurrence's segments pass to each other (gdn_glr.hip), in the compiled
code: accesses of device scope are of 8 bytes, the widest that arrive whole, and none were
merged."""
import os
import re
import shutil
import subprocess

import pytest

from gated_deltanet_chunked_gdn_amd import build


@pytest.mark.skipif(shutil.which(build.HIPCC) is None, reason="needs hipcc")
def test_words_are_single_accesses(tmp_path):
    out = str(tmp_path / "glr.s")
    r = subprocess.run([build.HIPCC, *build.COMMON, "--cuda-device-only", "-S", os.path.join(build.CSRC, "gdn_glr.hip"), "-o", out],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    found = {"load": set(), "store": set()}
    for line in open(out):
        m = re.match(r"\s+(?:buffer|global|flat)_(load|store)_(\S+) .*\bsc1\b", line)
        if m:
            found[m[1]].add(m[2])
    assert found == {"load": {"dwordx2"}, "store": {"dwordx2"}}

"""The matrix product's and the RMS norm's kernels are compiled in one piece too: split over the
compiler's threads, two builds of one source on one machine differed, and ran 134.9 or 119.5 us
(bf16 8192 x 1024 x 4096 with GELU and the pre-activation kept)."""
import os

import pytest

from transformer_epilogue_gb300 import build


@pytest.mark.parametrize("source", ["matmul.cu", "rms_norm_mx8.cu"])
def test_compiled_in_one_piece(monkeypatch, tmp_path, source):
    ran = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: ran.append(cmd) or Done())
    for cores in (2, 16, 96):
        monkeypatch.setattr(build.os, "cpu_count", lambda: cores)
        build._compile(source, True, False, [], str(tmp_path))
    assert all(os.path.basename(c[2]) == source and c == ran[0] for c in ran)
    assert not any("split" in x for x in ran[0])

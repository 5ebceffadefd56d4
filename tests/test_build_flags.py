"""GroupNorm's kernels are compiled in one piece: split over the compiler's threads, their
code depended on the number of cores and on what else the file held."""
import os

from transformer_epilogue_gb300 import build


def test_group_norm_is_compiled_in_one_piece(monkeypatch, tmp_path):
    ran = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: ran.append(cmd) or Done())
    for src in build.SOURCES:
        for cores in (4, 96):
            monkeypatch.setattr(build.os, "cpu_count", lambda: cores)
            build._compile(src, True, False, [], str(tmp_path))
    assert len(ran) == 2 * len(build.SOURCES)
    for a, b in zip(ran[::2], ran[1::2]):
        source = os.path.basename(a[2])
        if source in ("group_norm.cu", "group_norm_fused.cu"):
            assert a == b and not any("split" in x for x in a)

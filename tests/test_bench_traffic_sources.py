"""bench.py's traffic guard hashes everything the captured kernels are compiled from:
the files that the compiler itself names, and no others."""
import os
import subprocess

import pytest

import bench
from transformer_epilogue_gb300 import build


@pytest.mark.parametrize("source", bench.TRAFFIC_KERNELS)
def test_sources_hold_what_the_compiler_reads(source):
    p = subprocess.run([build.nvcc(), "-M", os.path.join(bench.CSRC, source), "-std=c++17", "-I", build.INCLUDE, "-I",
                        bench.CSRC] + build.ARCH, capture_output=True, text=True, check=True, timeout=300)
    read = {os.path.basename(f) for f in p.stdout.replace("\\\n", " ").split()[1:]
            if os.path.dirname(os.path.realpath(f)) == os.path.realpath(bench.CSRC)}
    assert source in read and read <= set(bench.traffic_sources())


def test_sources_are_the_kernels_and_their_headers():
    got = bench.traffic_sources()
    assert set(bench.TRAFFIC_KERNELS) < set(got) and "ep_internal.h" in got
    assert not {"group_norm.cu", "bias_dropout.cu", "ep_api.cpp"} & set(got)


def test_a_change_to_a_header_changes_the_hash(tmp_path, monkeypatch):
    for f in bench.traffic_sources():
        with open(os.path.join(bench.CSRC, f), encoding="utf-8") as src:
            (tmp_path / f).write_text(src.read())
    monkeypatch.setattr(bench, "CSRC", str(tmp_path))
    before = bench.kernel_source_hash()
    (tmp_path / "ep_internal.h").write_text((tmp_path / "ep_internal.h").read_text() + "\nextern int another;\n")
    assert bench.kernel_source_hash() != before

"""The benchmark's measured traffic figures and the sources that they belong to."""
import os
import shutil

import bench


def test_traffic_figures_belong_to_the_sources_of_the_measured_kernels(tmp_path, monkeypatch):
    """Sources of kernels that the benchmark does not launch leave the figures valid, any other
    source does not."""
    csrc = os.path.join("bit_groupwise_weight_amd", "csrc")
    shutil.copytree(os.path.join(bench.ROOT, csrc), tmp_path / csrc)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    before = bench.kernel_source_hash()
    for name in sorted(os.listdir(tmp_path / csrc)):
        path = tmp_path / csrc / name
        text = path.read_bytes()
        path.write_bytes(text + b"\n// a comment\n")
        measured = name not in ("f8_common.h", "linear_f8.hip", "norm_q8.hip", "probe.hip")
        assert (bench.kernel_source_hash() != before) == measured, name
        path.write_bytes(text)
    assert bench.kernel_source_hash() == before

"""CPU checks of what ties the committed HBM traffic summary to the sources."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bench  # noqa: E402


def test_traffic_hash_covers_the_counted_kernels_only(monkeypatch, tmp_path):
    """An operator that the benchmark does not launch leaves the summary valid;
    the counted kernels, their launches and every header do not."""
    names = {os.path.basename(f) for f in bench._counted_sources()}
    assert {"lp_api.hip", "lp_device.hpp", "lp_gemm.hpp", "lp_internal.hpp", "lp_lmhead.hip", "lp_rows.hip"} <= names
    assert not names & set(bench.UNCOUNTED_SOURCES)
    csrc = tmp_path / "entropy_chunked_row_amd" / "csrc"
    csrc.mkdir(parents=True)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    (csrc / "lp_rows.hip").write_text("int a;")
    (csrc / "lp_w4.hip").write_text("int b;")
    first = bench._csrc_sha256()
    (csrc / "lp_w4.hip").write_text("int c;")
    (csrc / "lp_rows.hip").write_text("int a;  // a comment")
    assert bench._csrc_sha256() == first
    (csrc / "lp_rows.hip").write_text("int d;")
    assert bench._csrc_sha256() != first


def test_stale_traffic_summary_is_reported(monkeypatch, tmp_path, capsys):
    (tmp_path / "profiles").mkdir()
    (tmp_path / "entropy_chunked_row_amd" / "csrc").mkdir(parents=True)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    doc = '```json\n{"source_sha256": "%s", "kernels": {"k": {"bytes_per_launch": 5}}}\n```\n'
    (tmp_path / "profiles" / "hbm_traffic.md").write_text(doc % bench._csrc_sha256())
    assert bench.measured_traffic("k") == 5 and "retaken" not in capsys.readouterr().err
    (tmp_path / "profiles" / "hbm_traffic.md").write_text(doc % "0")
    assert bench.measured_traffic("k") is None and "retaken" in capsys.readouterr().err

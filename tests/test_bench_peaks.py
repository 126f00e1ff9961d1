"""bench.py's rates with and without the measured ones."""

import json

import bench


def test_peaks_without_the_measured_file(tmp_path, monkeypatch):
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.peaks() == {"hbm_gbs": 6800.0, "bf16_tflops": 1900.0, "source": "fallback"}


def test_peaks_measured(tmp_path, monkeypatch):
    (tmp_path / "MEASURED_PEAKS.json").write_text(
        json.dumps({"hbm_gbs": 6782.8, "bf16_tflops": 1923.8, "bf16_tflops_sustained": 1714.2}))
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.peaks() == {"hbm_gbs": 6782.8, "bf16_tflops": 1923.8, "source": "measured"}

"""What the benchmark says of its kernels, on the host."""
import os
import shutil

import bench
from conftest import ROOT


def test_the_traffic_record_is_of_the_kernels_source(monkeypatch, tmp_path):
    """The record counts for the files that hold the timed kernels, and for no other version of any of them."""
    csrc = tmp_path / "rotated_kv_cache_gb300" / "csrc"
    csrc.mkdir(parents=True)
    names = ("tq_attention.cuh", "tq_attention.cu")
    for n in names:
        shutil.copy(os.path.join(ROOT, "rotated_kv_cache_gb300", "csrc", n), csrc / n)
    text = "".join((csrc / n).read_text() for n in names)
    assert "attn_split_kernel(" in text and "attn_combine_kernel(" in text
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    now = bench.kernel_source_hash()
    (tmp_path / "profiles").mkdir()
    record = tmp_path / "profiles" / "attention_decode_traffic.txt"
    record.write_text(f"kernel_source_sha256 = {now}\ndram_bytes_per_launch_full_workload = 1.5e9\n")
    assert bench.attention_traffic(now) == 1.5e9
    for n in names:
        kept = (csrc / n).read_text()
        (csrc / n).write_text(kept + "\n")
        assert bench.kernel_source_hash() != now
        assert bench.attention_traffic(bench.kernel_source_hash()) is None
        (csrc / n).write_text(kept)

"""A recorded DRAM traffic figure counts only for the source it was taken on: the
kernel's file and every header of its own that decides what it reads."""
import json
import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


@pytest.fixture
def tree(tmp_path):
    for d in ("paged_kv_gqa_row_gb300/csrc", "include", "profiles"):
        shutil.copytree(os.path.join(ROOT, d), tmp_path / d)
    for kernel in ("decode.cu", "chunk.cu"):
        entry = {"source_sha256": bench.kernel_source_hash(kernel, str(tmp_path)), "dram_bytes_per_launch": 1234.0}
        records = json.loads((tmp_path / "profiles/traffic.json").read_text())
        records[kernel] = entry
        (tmp_path / "profiles/traffic.json").write_text(json.dumps(records))
    return tmp_path


def test_a_record_of_the_present_source_counts(tree):
    assert bench.recorded_traffic("decode.cu", "decode.cu", str(tree)) == 1234.0
    assert bench.recorded_traffic("chunk.cu", "chunk.cu", str(tree)) == 1234.0
    assert bench.recorded_traffic("chunk.cu", "decode.cu", str(tree)) is None
    assert bench.recorded_traffic("decode.cu", "no such line", str(tree)) is None


@pytest.mark.parametrize("name,stale", [("decode.cu", {"decode.cu"}), ("decode_plan.cuh", {"decode.cu"}),
                                        ("rope_math.cuh", {"decode.cu"}), ("common.cuh", {"decode.cu", "chunk.cu"}),
                                        ("ptx.cuh", {"decode.cu", "chunk.cu"}), ("append4.cu", set())])
def test_a_record_is_stale_when_a_file_that_decides_its_work_changes(tree, name, stale):
    path = tree / "paged_kv_gqa_row_gb300/csrc" / name
    src = path.read_text()
    path.write_text("/* a comment\n * of two lines */\n" + src.replace("\n", "  // and more\n", 1))
    for kernel in ("decode.cu", "chunk.cu"):  # (comments change nothing)
        assert bench.recorded_traffic(kernel, kernel, str(tree)) == 1234.0
    path.write_text(src + "\nstatic int one_more_line;\n")
    for kernel in ("decode.cu", "chunk.cu"):
        assert (bench.recorded_traffic(kernel, kernel, str(tree)) is None) == (kernel in stale)

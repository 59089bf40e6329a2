"""Calls that are given addresses and a stream as integers need no torch."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
sys.modules["torch"] = None  # any import of it fails
import paged_kv_gqa_row_gb300 as lnk
desc = lnk.attn_desc(8, 2, 128, 4, 1, 4, kv_dtype=lnk.KV_E2M1)
lnk.lnk_paged_copy_pages(desc, 4096, 8192, 64, 128, 0, None, 0)
lnk.lnk_paged_copy_pages_layers(desc, [4096, 4096], [8192, None], 64, 128, 0, None, 0)
lnk.lnk_paged_copy_pages_layers(desc, [], [], 64, 128, 3, None, 0)
try:
    lnk.lnk_paged_copy_pages_layers(desc, [4096, 4096], [8192, None], 64, 128, 1, None, 0)
except lnk.LnkError as e:
    assert e.status == 1  # (a layer without a pool)
else:
    raise AssertionError("accepted")
"""


def test_page_copies_of_integer_addresses():
    subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, check=True, timeout=120)

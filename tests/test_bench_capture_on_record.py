"""The decode traffic that bench.py reports was captured on the source it is tagged with: the
profile page records the tag beside the capture's bytes."""
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bench  # noqa: E402


def test_decode_tags_are_on_record_with_their_bytes():
    with open(os.path.join(ROOT, "profiles", "decode_stream_decode_32k.md")) as f:
        page = f.read()
    for kernel in ("decode_main", "decode_planted"):
        nbytes, files = bench.NCU_TRAFFIC[kernel]
        row = [x for x in page.splitlines() if x.startswith(f"| {kernel} |")]
        assert len(row) == 1, kernel
        assert files["decode_stream.cu"] in row[0] and files["tc_common.cuh"] in row[0], kernel
        gb = float(re.search(r"([0-9.]+) GB", row[0]).group(1))
        assert abs(gb * 1e9 - nbytes) <= 1e-3 * nbytes, kernel

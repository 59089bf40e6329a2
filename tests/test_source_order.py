"""Orders that no run can show to be missing, shown on the source: memory written by some threads and read
or written again by others, with what has to stand between."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_gqa_row_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


@pytest.mark.parametrize("name,call", [("latent_attn.cu", "attend_again<"), ("latent_pair.cu", "attend_again<"),
                                       ("latent_prompt.cu", "attend_row<D>(p,")])
def test_rows_that_are_stored_again_wait_for_the_lanes_that_stored_them_first(name, call):
    src = source(name)
    calls = [m.start() for m in re.finditer(re.escape(call), src)]
    assert calls
    for at in calls:
        assert "__syncwarp();" in src[at - 160:at], src[at - 160:at]

"""What the 4-bit product with few rows does once a wait has run out, by its source: no call
makes one run out, and no kernel is broken on a GPU to see it."""
import os
import re

import routing_permute_grouped_gb300 as moe

CSRC = os.path.join(os.path.dirname(moe.__file__), "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_a_wait_that_ran_out_stops_the_others_and_the_stores():
    text = _source("int4_gemm.cu")
    # every wait that runs out raises the flag that the other warps' waits look at, before
    # anything else is done
    waits = re.findall(r"timed_out = timed_out \|\| !warp_wait\([^;]*&sh\.abort\);\s*if \(timed_out\) \*abort_flag = 1;", text)
    assert len(waits) == text.count("warp_wait(") == 2
    assert "volatile uint32_t* abort_flag = &sh.abort;" in text
    # and nothing is stored once it is up
    before, after = text.split("if (!live || *abort_flag) return;")
    store = r"\by\[[^\]]*\] = "
    assert not re.search(store, before) and len(re.findall(store, after)) == 2

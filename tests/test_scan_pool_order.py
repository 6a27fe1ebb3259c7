"""Where the selective scan's kernels touch the state pool, read from their source: workgroups of one launch are in no
order, so that a launch may not read a slot that another of its workgroups writes."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "replayssm_persistent_rssm_amd", "csrc")


def body(name):
    text = open(os.path.join(CSRC, "scan_kernel.h")).read()
    start = text.index(f"void {name}(ScanArgs a)")
    return text[start:text.index("\n}\n", start)]


def test_stretches_read_the_pool_in_one_launch_and_write_it_in_the_next():
    code = re.sub(r"//.*", "", body("scan_kernel"))
    loads = [m.start() for m in re.finditer(r"scan_state_load\(", code)]
    stores = [m.start() for m in re.finditer(r"scan_state_store\(", code)]
    assert len(loads) == 1 and len(stores) == 1
    # the fold's first stretch; the main kernel only where the sequence has one stretch, whose workgroup reads and writes
    guard = code.rindex("if (", 0, loads[0])
    assert "(FOLD ? seg == 0 : last == 0)" in code[guard:loads[0]]
    # the main kernel alone writes, from the last stretch
    main = code.rindex("if constexpr (FOLD)", 0, stores[0])
    assert "else if (seg == last && has_j)" in code[main:stores[0]]

"""What the header says of the status word: an operator whose kernels wait for copies or products can report that a wait ran out."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "mk.h")).read()
CSRC = os.path.join(ROOT, "persistent_megakernel_decode_sm_gb300", "csrc")


@pytest.mark.parametrize("entry,args,source", [("mk_linear", "mk_linear_args", "mk_linear.cuh"), ("mk_attend", "mk_attend_args", "mk_attend.cu"),
                                               ("mk_linear_adapted", "mk_adapters", "mk_linear.cuh"), ("mk_rope_append", "mk_rope_args", "mk_rope.cu")])
def test_waits_that_run_out_are_documented(entry, args, source):
    assert re.search(r"bar_wait\w*\([^;]*p\.status\)", open(os.path.join(CSRC, source)).read())
    at = HEADER.index("} %s;" % args)   # the comment in front of the arguments' struct
    comment = HEADER[HEADER.rindex("/*", 0, HEADER.rindex("typedef struct", 0, at)):at]
    assert "MK_ERR_TIMEOUT" in comment, entry

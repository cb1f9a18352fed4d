"""M0 and the direct-to-LDS loads in the built code object (no GPU): such a
load takes its LDS address from M0, and between a scalar write of M0 and the
load one wait state has to pass.  The compiler puts it after its own writes;
inside an asm statement the statement itself has to."""

import os
import re
import tempfile

import pytest

from implicit_gemm_conv_dp_amd import _lib
from test_host_library import code_objects, instrs, kernels

WRITES_M0 = re.compile(r"^\w+ m0[, ]")


def test_a_wait_state_between_m0_and_the_load():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built")
    with tempfile.TemporaryDirectory() as tmp:
        objs = code_objects(tmp)
    loads, bad = 0, {}
    for dis in objs:
        for name, body in kernels(dis).items():
            ins = instrs(body)
            for before, x in zip(ins, ins[1:]):
                if x.startswith("buffer_load") and x.endswith(" lds"):
                    loads += 1
                    if WRITES_M0.match(before):
                        bad[name] = bad.get(name, 0) + 1
    assert loads, "no direct-to-LDS load in the library"
    assert not bad, "%d of %d loads right after a write of M0, in %d kernels, such as %s" % (
        sum(bad.values()), loads, len(bad), sorted(bad)[0])

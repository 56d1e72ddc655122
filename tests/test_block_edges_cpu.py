"""Block operators without a GPU: rules of the sources, refusals at the edges
of the ranges, the cache's and the autograd functions' bookkeeping. Pointers
are made up; every call comes back before it would use them."""
import glob
import os
import re

from test_block_cpu import CSRC


def test_every_asm_statement_that_writes_m0_names_it():
    """The compiler keeps values of its own in m0."""
    found = 0
    for path in glob.glob(os.path.join(CSRC, "*.h*")):
        for asm in re.findall(r"asm(?: volatile)?\s*\((.*?)\);", open(path).read(), flags=re.S):
            if re.search(r"s_mov_b32 m0", asm):
                found += 1
                assert '"m0"' in asm.rsplit(":", 1)[1], (path, asm)
    assert found == 2

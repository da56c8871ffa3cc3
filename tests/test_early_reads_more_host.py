"""The kernels of the cache held in 8 bits and of page assignment start early as those of test_early_reads_host.py do, and
read what the one ahead of them writes by ordinary loads too. The list is complete: every source of a kernel that waits for the one
ahead is in one of the two tests or among the dense ones."""
import glob
import os
import re

import pytest

from attention_fa_fwd_03_gb300 import build_lib
from test_early_reads_host import SOURCES

MORE = ["fa_paged8.cuh", "fa_kv_append8.cu", "fa_append.cuh", "fa_page_assign.cu"]
# dense kernels, whose pointers are __restrict__; two read Q by the read-only path, which was there before fa_bwd's first pass
DENSE = {"fa_fwd.cuh", "fa_bwd_pipelined.cuh", "fa_bwd_d256.cuh", "fa_decode.cuh"}


def code_of(name):
    with open(os.path.join(build_lib.CSRC, name), encoding="utf-8") as fh:
        return re.sub(r"//[^\n]*", "", fh.read())


@pytest.mark.parametrize("name", MORE)
def test_no_read_only_loads(name):
    assert not re.search(r"__ldg|ld\.global\S*\.nc|__restrict__", code_of(name))


def test_every_early_kernel_is_looked_at():
    early = {os.path.basename(p) for p in glob.glob(os.path.join(build_lib.CSRC, "*.cu*"))
             if "grid_wait_prior()" in code_of(os.path.basename(p))}
    early -= {"sm103_ptx.cuh"}  # where it is defined
    assert early <= set(SOURCES) | set(MORE) | DENSE

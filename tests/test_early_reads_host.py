"""Kernels that start before the one ahead of them has ended read what it writes (lengths, rotated queries, selections,
bounds, O) by ordinary loads: the read-only path is for memory that nobody writes while the kernel runs, and its loads may
be moved above the wait for the earlier kernel."""
import os
import re

import pytest

from attention_fa_fwd_03_gb300 import build_lib

SOURCES = ["fa_paged.cuh", "fa_paged_walk.h", "fa_paged_fwd.cuh", "fa_paged_tc.cuh", "fa_kv_append.cu", "fa_page_select.cu",
           "fa_bwd.cuh"]


@pytest.mark.parametrize("name", SOURCES)
def test_no_read_only_loads(name):
    with open(os.path.join(build_lib.CSRC, name), encoding="utf-8") as fh:
        code = re.sub(r"//[^\n]*", "", fh.read())
    assert not re.search(r"__ldg|ld\.global\S*\.nc|__restrict__", code)

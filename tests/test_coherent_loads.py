"""Kernels that are in place before the work ahead of them has finished read nothing through
the non-coherent path (CPU only: the sources)."""
import os
import re

import pytest

from long_context_serving_gb300 import build as Bd

# The sources of the fused step's kernels, the 8-bit attention's, the append's and the page calls'.
FILES = ["bs_step.cu", "bs_summaries_impl.cuh", "bs_score_impl.cuh", "bs_select_impl.cuh", "bs_attn_impl.cuh",
         "bs_attn_bf16.cu", "bs_attn_f32.cu", "bs_attn_quant.cu", "bs_append.cu", "bs_pages.cu", "bs_quant.cuh",
         "bs_internal.cuh"]


@pytest.mark.parametrize("name", FILES)
def test_no_non_coherent_loads(name):
    """ld.global.nc takes memory for constant over the kernel's life; a page table, lengths, codes or
    scales that the call ahead writes are not. The compiler makes such loads of const __restrict__
    parameters too."""
    text = open(os.path.join(Bd.CSRC, name), encoding="utf-8").read()
    text = re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))
    assert not re.search(r"\b__ldg\s*\(|\.nc\b|__restrict__", text)

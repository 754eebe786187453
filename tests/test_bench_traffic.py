"""The DRAM traffic that bench.py reports comes from ncu summaries, and only while the
kernels' sources are the ones they were taken on."""
import pytest

import bench

SHARED = ["ptx.cuh", "exp2_poly.cuh", "fa_internal.h"]


@pytest.mark.parametrize("source,summary", [("fa_bwd.cu", "bwd_dkdv_pair_kernel_headline.md"),
                                            ("fa_fwd.cu", "fa_fwd_kernel_gqa.md")])
def test_summaries_belong_to_the_sources(source, summary):
    assert bench.profiled_traffic(summary, bench.kernel_source_hash([source] + SHARED))

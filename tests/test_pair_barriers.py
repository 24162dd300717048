"""Arrivals on a barrier of another CTA, read in the kernels' source (CPU).  Without an order and a scope such an arrival
is a release to the arriving thread's own CTA: nothing that it wrote is then ordered before the other CTA's wait, however
seldom that shows in a run."""
import glob
import os
import re

import mixture_experts_ffn_planner_b200._build as build


def _sources():
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu*"))):
        yield os.path.basename(path), open(path).read()


def test_remote_arrivals_name_their_order_and_scope():
    found = 0
    for name, text in _sources():
        for form in re.findall(r"mbarrier\.arrive[\w.:]*\.shared::cluster[\w.:]*", text):
            found += 1
            assert re.search(r"\.(release|relaxed)\.cluster\.", form), f"{name}: {form}"
    assert found


def test_cleared_rows_are_released_to_the_pair():
    """The warp that clears rows behind an expert's last writes shared memory that the pair's MMA reads: fenced for the
    async proxy, then released at cluster scope; and the issuer of the MMA acquires at that scope."""
    text = dict(_sources())["tile_gemm.cuh"]
    patch = text[text.index("warp == kGPatchWarp"):]
    patch = patch[:patch.index("epilogue")]
    arrive = re.search(r"(\w+)\(cluster_addr\(&full\[s\], 0\)\)", patch)
    assert "fence_proxy_async_smem();" in patch[:arrive.start()]
    helper = dict(_sources())["ptx.cuh"]
    body = helper[helper.index(f"void {arrive.group(1)}("):]
    assert ".release.cluster." in body[:body.index("\n}")]
    assert "cut ? wait_cluster(&full[s], ph)" in text

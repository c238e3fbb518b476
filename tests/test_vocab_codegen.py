"""The embedding's and the head's kernels compile without register spills: a
spill in a product's loop costs it a multiple of its time."""
import os

import pytest

import test_codegen


@pytest.mark.skipif(not os.path.exists(f"{test_codegen.ROCM}/bin/hipcc"), reason="no hipcc")
@pytest.mark.parametrize("src,kernels", [("head_kernel.hip", 25), ("embed_kernel.hip", 15)])
def test_no_scratch(tmp_path, src, kernels):
    sizes = test_codegen._private_sizes(src, str(tmp_path))
    assert len(sizes) >= kernels, sorted(sizes)
    assert not {k: v for k, v in sizes.items() if v}, "kernels with register spills"

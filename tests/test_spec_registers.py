"""Register budgets of the kernels of a speculative decoding step on the compiled
gfx950 code (host-only), as those of the attention kernels that they stand beside."""
import os

import pytest

from test_register_bounds import _kernel_metadata
from w4a16_bit_matmul_amd import _build


@pytest.mark.skipif(not os.path.exists(_build.HIPCC), reason="hipcc is not installed")
def test_tree_kernels_keep_to_their_registers():
    meta = _kernel_metadata("wq_kv_tree.hip")
    for kernel, instances, most in (("14kv_attn_kernel", 20, 256), ("19kv_attn_join_kernel", 14, 128), ("14kv_tree_kernel", 4, 256), ("19kv_tree_join_kernel", 8, 128)):
        found = {n: v for n, v in meta.items() if kernel in n}
        assert len(found) == instances, sorted(found)
        for name, (vgpr, scratch) in found.items():
            assert scratch == 0 and vgpr <= most, (name, vgpr, scratch)


@pytest.mark.skipif(not os.path.exists(_build.HIPCC), reason="hipcc is not installed")
@pytest.mark.parametrize("src", ["wq_kv_append.hip", "wq_verify.hip"])
def test_the_other_kernels_do_not_spill(src):
    for name, (vgpr, scratch) in _kernel_metadata(src).items():
        assert scratch == 0 and vgpr <= (64 if "kv_append_kernel" in name else 256), (name, vgpr, scratch)

"""Register budgets of the attention kernels on the compiled gfx950 code
(host-only): a spill inside a walk over keys costs a memory round trip a tile,
and past 256 registers one workgroup a CU runs instead of two."""
import os

import pytest

from test_register_bounds import _kernel_metadata
from w4a16_bit_matmul_amd import _build


@pytest.mark.skipif(not os.path.exists(_build.HIPCC), reason="hipcc is not installed")
@pytest.mark.parametrize("src,kernel,instances", [("wq_kv_attn.hip", "14kv_attn_kernel", 20), ("wq_kv_chunk.hip", "15kv_chunk_kernel", 2),
                                                  ("wq_prompt_attn.hip", "18prompt_attn_kernel", 8), ("wq_prompt_attn.hip", "19prompt_split_kernel", 4), ("wq_rope.hip", "qk_norm_rope_kernel", 24)])
def test_attention_kernels_keep_to_their_registers(src, kernel, instances):
    meta = {n: v for n, v in _kernel_metadata(src).items() if kernel in n}
    assert len(meta) == instances, sorted(meta)
    for name, (vgpr, scratch) in meta.items():
        one_a_cu = "prompt_attn_kernelILi256" in name
        assert scratch == 0 and vgpr <= (512 if one_a_cu else 256), (name, vgpr, scratch)
        if src == "wq_rope.hip":
            assert vgpr <= 64, (name, vgpr)  # eight waves a SIMD hide a row's latency


@pytest.mark.skipif(not os.path.exists(_build.HIPCC), reason="hipcc is not installed")
def test_the_joining_kernel_keeps_its_pieces_in_registers():
    """Up to 16 pieces of a row a lane are in flight together, four waves to a SIMD."""
    meta = {n: v for n, v in _kernel_metadata("wq_kv_attn.hip").items() if "19kv_attn_join_kernel" in n}
    assert len(meta) == 14, sorted(meta)
    for name, (vgpr, scratch) in meta.items():
        assert scratch == 0 and vgpr <= 128, (name, vgpr, scratch)

"""Host-side refusals of the serving entry points that depend on more than one
argument.  Nothing here reaches a GPU."""
import os
import re

import pytest
import torch

from mass_adaptive_sparse_gb300 import api

BF16, FP32 = torch.bfloat16, torch.float32


def test_cache_read_refuses_outputs_of_another_length_or_type():
    """`out` is of the T and the dtype that the call names, or the call is refused; nothing of it is ignored."""
    cache = api.quant_cache(2, 10, 2, 64, device="cpu")
    out = tuple(torch.zeros((2, 5, 2, 64), dtype=FP32) for _ in range(2))
    for T, dtype in ((10, FP32), (4, None), (0, None), (5, BF16)):
        with pytest.raises(ValueError, match="k must be"):
            api.cache_read(cache, T, dtype=dtype, out=out)
    for T in (-1, -5):
        with pytest.raises(ValueError, match="negative"):
            api.cache_read(cache, T, out=out)
        with pytest.raises(ValueError, match="negative"):
            api.cache_read(cache, T)
    with pytest.raises(ValueError, match="v must be"):
        api.cache_read(cache, 5, out=(out[0], out[1][:, :4].contiguous()))
    # the right ones go on to the check of their device, with or without the type
    for dtype in (FP32, None):
        with pytest.raises(ValueError, match="CUDA"):
            api.cache_read(cache, 5, dtype=dtype, out=out)


@pytest.mark.parametrize("splits", [257, 10 ** 6, 2 ** 29, 2 ** 31 - 1, -2 ** 31])
def test_workspace_sizes_are_zero_for_splits_that_the_calls_refuse(splits):
    """Nothing is allocated for them (and nothing overflows on the way)."""
    lib = api.lib()
    assert lib.mala_decode_quant_workspace_size(4, 8, 128, splits) == 0
    assert lib.mala_decode_shared_workspace_size(4, 8, 128, splits, 2) == 0
    assert lib.mala_decode_shared_workspace_size(4, 8, 128, 3, splits) == 0
    assert lib.mala_decode_quant_workspace_size(4, 8, 128, 256) >= 1025 * 4 * 8 * 132 * 4
    assert lib.mala_decode_shared_workspace_size(4, 8, 128, 256, 256) >= 1281 * 4 * 8 * 132 * 4


def test_prefix_softmax_warps_stay_together_after_an_expired_wait():
    """A wait that expires or is aborted can end differently for the lanes of a warp, and the loads from tensor memory
    behind it need every lane.  No call can bring this about at will, so the source is read: nothing in the softmax
    role's loop leaves it."""
    src = open(os.path.join(os.path.dirname(api.__file__), "csrc", "prefix_tc.cu")).read()
    role = src[src.index("softmax: thread r of slot s"):]
    loop = role[role.index("for (int u = 0; u < steps; ++u)"):role.index("if (steps > 0)")]
    assert "tmem_ld64_sync" in loop and "mbar_arrive(smem_u32(&bars.p_ready[s]))" in loop
    assert not re.search(r"\b(break|continue|return|goto)\b", loop)


def test_cache_read_refuses_outputs_that_are_missing():
    """None inside `out` is not a wish for new tensors (whose rows behind the lengths nothing would write)."""
    cache = api.quant_cache(2, 10, 2, 64, device="cpu")
    x = torch.zeros((2, 5, 2, 64), dtype=BF16)
    for out in ((None, x), (x, None), (None, None)):
        with pytest.raises(ValueError, match="two tensors"):
            api.cache_read(cache, 5, out=out)

"""The operators together: a served attention layer (tables, fused append,
attention, release) between two 4-bit linears."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("fmt", [0, 1])
def test_single_tokens_agree_with_whole_prompts_and_pages_come_back(fmt):
    import serve_attention
    off, back, held = serve_attention.serve(requests=5, steps=6, fmt=fmt, report=lambda s: None)
    # Both runs read the same cache and differ by two 16-bit roundings of the
    # attention (2^-8 each, of the sum of |p v|), which the output projection's
    # own 4-bit quantizer can turn into steps of its codes: a step is at most a
    # sixth of a group's largest value, and a relative change of 2^-7 moves about
    # one code in 16 by one.
    assert off <= 0.08
    assert back == held


def test_layer_refuses_wrong_shapes():
    import numpy as np
    from diffusion_smooth_group_amd import kv
    from diffusion_smooth_group_amd import svdq as S
    from diffusion_smooth_group_amd.attention_layer import SVDQAttention
    w = np.zeros((128, 256), np.uint16)
    lin = S.SVDQLinear.pack(w, S.BF16, None, 0, S.FMT_MXFP4_G32)
    cache = kv.KVCache(1, 16, 1, 64, S.FMT_MXFP4_G32)
    SVDQAttention(lin, lin, 2, cache, None, None)            # 4 rows of heads of 64, and 2 x 64 back
    with pytest.raises(ValueError):
        SVDQAttention(lin, lin, 3, cache, None, None)

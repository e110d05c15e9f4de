"""A call's options hold addresses: a tensor that only they name has to live as long as they do."""
import gc
import weakref

import pytest
import torch

import attention_tensor_cores_gb300 as F


@pytest.mark.parametrize("name", ["workspace", "seqlens_k", "out_scales", "out_tensor_scale", "out_f32", "nvfp4_scale_in", "out_amax"])
def test_tensors_live_with_their_options(name):
    t = torch.zeros(16)
    seen, opts = weakref.ref(t), F.make_opts(**{name: t})
    del t
    gc.collect()
    assert seen() is not None
    del opts
    gc.collect()
    assert seen() is None

"""An atten_mask beside ALiBi slopes is not dropped silently: the binding refuses
it in sparse mode 0, where a call without slopes would read it, in the forward
and in the backward (before any tensor is looked at, so without a GPU). The other
modes ignore atten_mask with slopes as without."""
import pytest
import torch

import masked_attention_fa_b200 as fa


def attention(mode):
    return fa.MaskedAttention("BNSD", 1, 2, 130, 130, 64, mode, alibi="right")


def tensors():
    x = torch.zeros(1, 2, 130, 64, dtype=torch.bfloat16)
    return x, torch.zeros(1, 2, 130), torch.zeros(2), torch.zeros(130, 130, dtype=torch.uint8)


def test_refused_in_mode_0():
    x, lse, slopes, mask = tensors()
    attn = attention(0)
    with pytest.raises(ValueError, match="atten_mask"):
        attn(x, x, x, slopes=slopes, atten_mask=mask)
    with pytest.raises(ValueError, match="atten_mask"):
        attn.backward(x, x, x, x, x, lse, slopes=slopes, atten_mask=mask)
    with pytest.raises(ValueError, match="ranges"):
        attn(x, x, x, slopes=slopes, ranges=torch.zeros(1, 2, 4, dtype=torch.int32))
    attn.close()


def test_ignored_in_the_modes_that_ignore_masks():
    x, lse, slopes, mask = tensors()
    attn = attention(2)
    with pytest.raises(ValueError, match="CUDA"):  # as far as the tensors' own check
        attn(x, x, x, slopes=slopes, atten_mask=mask)
    with pytest.raises(ValueError, match="CUDA"):
        attn.backward(x, x, x, x, x, lse, slopes=slopes, atten_mask=mask)
    attn.close()

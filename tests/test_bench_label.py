"""The kernel instance that the bench line names: the arguments of the kernel's
template, in its order and of its types."""
import os
import re
import types

import pytest
import torch

import bench
from masked_attention_fa_b200.workloads import named_workloads

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "masked_attention_fa_b200", "csrc", "fa_kernel_sm100.cu")


@pytest.mark.parametrize("name,dense,want", [
    ("prefix_8k", False, "fa_fwd_sm100<128, true, false, true, 0>"),
    ("leftup_causal_4k", False, "fa_fwd_sm100<128, true, false, false, 0>"),
    ("alibi_causal_4k", False, "fa_fwd_sm100<128, true, false, false, 1>"),
    ("allmask_causal_4k", True, "fa_fwd_sm100<128, true, true, false, 0>"),
])
def test_label(name, dense, want, monkeypatch):
    monkeypatch.setattr(torch.cuda, "get_device_properties",
                        lambda dev: types.SimpleNamespace(multi_processor_count=148))
    assert bench.kernel_label(named_workloads()[name], dense, 0) == want


def test_the_template_it_names():
    src = open(SRC).read()
    args = re.search(r"template <([^>]*)>\s*__global__ void [^{]*fa_fwd_sm100\(", src).group(1)
    assert [a.split()[0] for a in args.split(",")] == ["int", "bool", "bool", "bool", "int"]
    assert re.search(r"kBiasNone = 0, kBiasAlibi = 1,", src)

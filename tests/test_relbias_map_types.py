"""Bucket maps of other types than int32: whole numbers are taken as they are,
fractions and numbers that do not fit are refused and not cut or wrapped."""
import numpy as np
import pytest
import torch

from masked_attention_fa_b200 import _relbias, relative_buckets

M = relative_buckets(8, 20)
TABLE = torch.zeros(8, 2)


@pytest.mark.parametrize("m", [M, M.astype(np.int64), M.astype(np.uint8), M.tolist(),
                               M.astype(np.float32), torch.from_numpy(M).long(),
                               torch.from_numpy(M)],
                         ids=["int32", "int64", "uint8", "list", "float", "torch64", "torch32"])
def test_whole_numbers(m):
    b, keep = _relbias(TABLE, m)
    assert keep.dtype == np.int32 and np.array_equal(keep, M)
    assert (b.num_buckets, b.reach) == (8, 20)


def wrapped(to):
    m = M.astype(np.int64)
    m[3] = to
    return m


@pytest.mark.parametrize("m", [M + 0.5, torch.from_numpy(M) + 0.25, wrapped(2 ** 32), wrapped(2 ** 31),
                               wrapped(-2 ** 32 + 1), np.where(M == 3, np.nan, M)],
                         ids=["half", "torch", "2^32", "2^31", "negative", "nan"])
def test_refused(m):
    with pytest.raises(ValueError):
        _relbias(TABLE, m)

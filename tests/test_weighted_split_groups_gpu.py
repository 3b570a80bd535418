"""Prompt weights of few queries where a kv head's group takes several row tiles: all of them are
held while the keys stream by."""
import math

import pytest
import torch

from tests.test_weighted_gpu import DT, _built, _chunk  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,n", [(256, 1, 1), (256, 1, 2), (130, 1, 1), (130, 1, 2),
                                      (512, 1, 1), (260, 2, 2), (384, 1, 1)])
def test_few_queries_of_large_groups(hq, hkv, n, d, dtype):
    _chunk([0, 100, 257], n, hq, hkv, d, DT[dtype], hq + n, 1 / math.sqrt(d), None)


@pytest.mark.parametrize("hq,n", [(256, 2), (130, 2), (512, 1)])
def test_few_queries_of_large_groups_over_many_keys(hq, n):
    _chunk([6000, 5, 1500], n, hq, 1, 128, torch.bfloat16, 3, 0.1, 0)

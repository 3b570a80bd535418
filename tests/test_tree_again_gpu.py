"""Tree attention called again and again: each form of its CTAs (few rows, up to 128, more; one
range of keys and many; CTAs without keys) beside the others, without a wait in between."""
import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests import evict_reference as ref
from tests.test_tree_gpu import _built, _case, _parents, _seen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dt", [(64, torch.bfloat16), (128, torch.float16)])
def test_the_same_bits_in_every_run(d, dt):
    forms = []
    for lens, n, hq in (([3000, 40], 7, 8), ([900, 1], 16, 8), ([2000, 300, 0], 40, 8),
                        ([700] * 80, 5, 8), ([10], 1, 1), ([5000, 0], 33, 24)):
        q, k, v, bt, ctx = _case(lens, n, hq, 1, d, dt, n)
        seen, _ = _seen(_parents(len(lens), n, n))
        want, bound = ref.tree(q, k, v, bt, ctx, seen, 0.1)
        args = [x.cuda() for x in (q, k, v, bt, ctx, ref.bits(seen))]
        forms.append((args, want, bound))
    runs = [[pa.prefill_tree(*args, 0.1) for args, _, _ in forms] for _ in range(30)]
    assert pa.pa_last_device_error() == 0
    for i, (_, want, bound) in enumerate(forms):
        assert ((runs[0][i].cpu().double() - want).abs() <= bound).all(), i
        for r in runs[1:]:
            assert torch.equal(r[i], runs[0][i]), i

"""The rotated append at positions of its own: which entry point an error names."""
import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests.test_evict_flow_gpu import _built, _i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rope_pos,name", [(None, "pa_append_kv_rope"), ([1], "pa_append_kv_rope_at")])
def test_errors_name_the_call(rope_pos, name):
    kc = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    cs = torch.zeros((10, 24), device="cuda")  # 24 is no rotated dimension
    with pytest.raises(pa.PAError) as e:
        pa.append_kv_rope(w, w, kc, kc.clone(), _i32([[0, 1]]), _i32([0]), _i32([3]), cs,
                          rope_pos=None if rope_pos is None else _i32(rope_pos))
    assert str(e.value).split(":")[0].split()[0] == name

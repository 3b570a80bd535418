"""Two serving loops at once, each on a stream of its own with its own pools and workspace."""
import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests.test_evict_flow_gpu import WRITTEN, _built, _loop, _results  # noqa: F401

pytestmark = pytest.mark.gpu


def test_two_loops_at_once():
    want = []
    for seed in (41, 42):
        s, step = _loop(seed)
        start = {x: s[x].clone() for x in WRITTEN}
        step()
        want.append(_results(s))
        for x, y in start.items():
            s[x].copy_(y)
        want[-1] = (s, step, start, want[-1])
    streams = [torch.cuda.Stream() for _ in want]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(25):
        for i, (s, step, start, _) in enumerate(want):
            with torch.cuda.stream(streams[i]):
                for x, y in start.items():
                    s[x].copy_(y)
                step()
                got[i].append(_results(s))
    torch.cuda.synchronize()
    assert pa.pa_last_device_error() == 0
    for i, (_, _, _, w) in enumerate(want):
        for run in got[i]:
            for a, b, name in zip(run, w, WRITTEN):
                assert torch.equal(a, b), (i, name)

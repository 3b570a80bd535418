"""The 4-bit cache's calls one behind the other, as a program makes them."""
import pytest
import torch

import paged_kv_cache_171_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_171_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert pa.pa_last_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv,d,n", [(8, 2, 128, 600), (4, 4, 64, 37), (16, 16, 128, 3000)])
def test_a_kernel_sees_what_the_one_before_it_wrote(hq, hkv, d, n, dtype):
    """Angles, places and rows rewritten, stored over the same tokens and read back, in many
    rounds without a wait between the launches: each round gives its own rows."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    blocks = -(-n // 16)
    kv = pa.kv4_cache(2 * blocks, hkv, d)
    perm = [torch.randperm(2 * blocks, generator=gen, device="cuda")[:blocks].to(torch.int32)[None]
            for _ in range(2)]
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    tables = [pa.rope_table(n, d, base=b) for b in (10000.0, 77.0)]
    rounds = [torch.randn((n, hq + 2 * hkv, d), generator=gen, device="cuda").to(dtype)
              for _ in range(4)]
    bt, cs, ctx = perm[0].clone(), tables[0].clone(), pos[n - 1:].clone()

    def step(i):
        bt.copy_(perm[i % 2])
        cs.copy_(tables[i // 2 % 2])
        ctx.copy_(pos[n - 1 - i:n - i])
        w = rounds[i % 4]
        q = pa.append_kv4(w[:, hq:hq + hkv], w[:, hq + hkv:], kv, bt, seq, pos, cos_sin=cs,
                          q=w[:, :hq])
        k, v = pa.read_kv4(kv, bt, seq, pos, dtype=dtype)
        return (q, k, v, pa.decode_kv4(q[n - 1:], kv, bt, ctx, 0.1),
                pa.prefill_kv4(q[None, n - 1:], kv, bt, ctx, 0.1))

    want = []
    for i in range(4):
        want.append(step(i))
        torch.cuda.synchronize()
    got = [step(i % 4) for i in range(60)]
    torch.cuda.synchronize()
    assert pa.pa_last_device_error() == 0
    for i, g in enumerate(got):
        for a, b in zip(g, want[i % 4]):
            assert torch.equal(a, b), i

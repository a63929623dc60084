"""A windowed prefill gives the same bits every time: its warps hand tiles to one another by
barriers alone, and a copy that overtook its readers would change a few values now and then."""
import math

import pytest
import torch

from paged_kv_cache_253_gb300.api import KVPool

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp8b"])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,T,G,hkv", [(8000, 70, 4, 2), (8000, 256, 4, 8), (1500, 512, 4, 8), (20000, 300, 1, 8)])
def test_the_same_bits_every_time(kind, out_dtype, n, T, G, hkv):
    g = torch.Generator(device=DEV).manual_seed(n)
    nb = -(-n // 16)
    pool = KVPool(nb, 16, hkv, 128, kind, DEV)
    if kind == "fp8":
        pool.set_kv_scales(2.0 ** -6, 2.0 ** -6)
    k, v = (torch.randn(n, hkv, 128, generator=g, device=DEV).bfloat16() for _ in range(2))
    pool.append_kv(k, v, torch.arange(n, device=DEV))
    q = torch.randn(T, hkv * G, 128, generator=g, device=DEV).bfloat16()
    i32 = dict(dtype=torch.int32, device=DEV)
    t, cu, lens = torch.arange(nb, **i32)[None], torch.tensor([0, T], **i32), torch.tensor([n], **i32)
    run = lambda: pool.prefill(q, cu, t, lens, 1 / math.sqrt(128), max_q_len=T, out_dtype=out_dtype,  # noqa: E731
                               window=1 << 30)
    first = run()
    differ = sum(not torch.equal(first, run()) for _ in range(100))
    assert differ == 0 and pool.get_error() == 0

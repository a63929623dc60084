"""Block-scaled, windowed and rotary operators at the limits of what they are given: the
largest scales, reserved workspaces, scratch, and calls that are refused before they have
done anything."""
import pytest
import torch

from paged_kv_cache_253_gb300 import _lib as L
from paged_kv_cache_253_gb300.api import KVPool
from test_gpu_block_scaled import Model, pool_values

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("B,D,T", [(16, 128, 3), (16, 128, 600), (32, 128, 5), (16, 64, 4)])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("exponent", [254, 253, 250])
def test_appends_to_blocks_of_the_largest_scales(B, D, T, rotate, exponent):
    """A started block whose imported scale is 2^127 (or a little less): values above 2^117 leave
    codes, infinities become +-448 of the scale, small values zero.  (Angles of zero turn nothing.)"""
    H = 2
    nb = T // (B - 1) + 2
    pool, m = KVPool(nb, B, H, D, "fp8b", DEV), Model(nb, B, H, D)
    pool.import_scales(torch.full((nb, H, 2), exponent, dtype=torch.uint8, device=DEV))
    m.ek += exponent
    m.ev += exponent
    g = torch.Generator().manual_seed(T)
    k, v = ((torch.randn(T, H, D, generator=g) * 2.0 ** 122).bfloat16() for _ in range(2))
    k[0, 0, :4] = torch.tensor([2.0 ** 120, -(2.0 ** 118), 2.0 ** 100, 1.0])
    v[0, 1, :3] = torch.tensor([float("inf"), float("-inf"), 2.0 ** 127])
    if not rotate:
        k[1, 1, 5] = float("-inf")
    slots = [1 + i + i // (B - 1) for i in range(T)]                 # every offset but 0
    at = torch.tensor(slots, device=DEV)
    if rotate:
        pool.append_rope(None, k.to(DEV), v.to(DEV), at, torch.zeros(T, dtype=torch.int32, device=DEV),
                         torch.ones(D // 2, device=DEV))
    else:
        pool.append_kv(k.to(DEV), v.to(DEV), at)
    m.append(k, v, slots)
    assert pool.get_error() == 0
    m.same(pool)
    assert (pool_values(pool)[1].abs() == 448 * 2.0 ** (exponent - 127)).sum() >= 2


@pytest.mark.parametrize("kind,window", [("bf16", True), ("fp8b", False), ("fp8b", True)])
def test_a_reserve_takes_what_a_call_uses(kind, window):
    """The windowed decodes' workspace: partials by the GPU's size (some 5 MB for each of the two
    kernels, with 16 heads a group) and four bytes per sequence and KV head; a batch of that many
    sequences then runs without more."""
    pool = KVPool(64, 16, 8, 128, kind, DEV)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    pool.reserve(16384, 128, window=window)
    assert free - torch.cuda.mem_get_info()[0] <= 64 << 20
    S = 2048
    q = torch.randn(S, 128, 128, device=DEV).bfloat16()
    t = torch.zeros(S, 1, dtype=torch.int32, device=DEV)
    lens = torch.full((S,), 5, dtype=torch.int32, device=DEV)
    out = torch.empty(S, 128, 128, device=DEV)
    free = torch.cuda.mem_get_info()[0]
    for o in (out, torch.empty(out.numel() + 1, device=DEV)[1:].view(out.shape)):        # (the plain kernel: unaligned)
        free = torch.cuda.mem_get_info()[0]
        pool.decode(q, t, lens, 0.1, out=o, window=9)
        assert torch.cuda.mem_get_info()[0] == free and pool.get_error() == 0
        assert not o.any()                                                               # an empty cache

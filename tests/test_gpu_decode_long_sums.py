"""Windowed decode on code pools with fp32 results, where one range holds many steps of a
sequence: sums that the tensor cores cut to fp32 must not shrink with the range's length, and
the chunks that a range is walked in join to the same result."""
import math

import pytest
import torch

import plain64
from paged_kv_cache_253_gb300.api import KVPool

pytestmark = pytest.mark.gpu
DEV = "cuda"
D, B = 128, 16


def cache(kind, n, hkv, seed, ramp=0.0):
    """One sequence of n tokens whose values share a sign; scores of a query of ones rise by
    `ramp` along it."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    pool = KVPool(-(-n // B), B, hkv, D, kind, DEV)
    if kind == "fp8":
        pool.set_kv_scales(2.0 ** -6, 2.0 ** -6)
    slots = torch.arange(n, device=DEV)
    k = torch.randn(n, hkv, D, generator=g, device=DEV)
    if ramp:
        k = torch.linspace(0, ramp / math.sqrt(D), n, device=DEV)[:, None, None] + 0.02 * k
    v = 1 + 0.25 * torch.randn(n, hkv, D, generator=g, device=DEV)
    pool.append_kv(k.bfloat16(), v.bfloat16(), slots)
    k, v = pool.read_kv(slots)
    return pool, k.double(), v.double(), torch.arange(-(-n // B), dtype=torch.int32, device=DEV)[None], g


def decode(pool, q, t, n, S, **kw):
    lens = torch.full((S,), n, dtype=torch.int32, device=DEV)
    got = pool.decode(q.expand(S, -1, -1).contiguous(), t.expand(S, -1).contiguous(), lens, 1 / math.sqrt(D), **kw)
    assert pool.get_error() == 0
    return got


# a chunk is 8192 keys, 256 products of 32, each of which cuts the sum by less than 2^-23 of itself:
# 2^-15; as a rule a cut is half of 2^-23 to 2^-24, of a sum that is half complete: 2^-17.5
@pytest.mark.parametrize("kind", ["fp8", "fp8b"])
@pytest.mark.parametrize("n,S,G,hkv,window,sinks,size", [(131072, 304, 4, 1, 1 << 30, 0, 2.0), (131072, 304, 4, 1, 1 << 30, 0, 0.3),
                                                         (100001, 3, 8, 8, 1 << 30, 0, 2.0), (70000, 100, 16, 2, 65000, 40, 1.0),
                                                         (30000, 304, 5, 1, 20000, 4, 1.0), (8193, 304, 1, 1, 1 << 30, 0, 1.0)])
def test_fp32_results_do_not_shrink_with_the_length(kind, n, S, G, hkv, window, sinks, size):
    pool, k, v, t, g = cache(kind, n, hkv, n)
    q = (size * torch.randn(1, hkv * G, D, generator=g, device=DEV)).bfloat16()
    got = decode(pool, q, t, n, S, window=window, sinks=sinks)
    j = torch.arange(n, device=DEV)[None]
    want, mag, top = plain64.attend(q, k, v, 1 / math.sqrt(D), (j < sinks) | (n - 1 - j < window))
    err = got.double() - want
    tol = 2.0 ** -15 * mag + plain64.tolerance(want, mag, top, float(v.abs().max()), torch.float32)
    assert (err.abs() <= tol).all(), f"{float((err.abs() / tol).max()):.3g} times the bound"
    assert float(err.mean().abs()) <= 2.0 ** -17 * float(want.abs().mean())


@pytest.mark.parametrize("kind", ["fp8", "fp8b"])
@pytest.mark.parametrize("ramp", [40.0, -40.0])
def test_chunks_join_by_their_references(kind, ramp):
    """Scores that rise (fall) by 40 nats along the context: every chunk's reference is another
    one; a head whose query is not a number stays so, alone."""
    n = 40000
    pool, k, v, t, _ = cache(kind, n, 1, 3, ramp)
    q = torch.ones(1, 4, D, device=DEV).bfloat16()
    q[0, 2, 7] = float("nan")
    for S in (1, 304):
        got = decode(pool, q, t, n, S, window=1 << 30)
        want, mag, top = plain64.attend(q.nan_to_num(1.0), k, v, 1 / math.sqrt(D), torch.ones(1, n, dtype=torch.bool, device=DEV))
        tol = 2.0 ** -15 * mag + plain64.tolerance(want, mag, top, float(v.abs().max()), torch.float32) + n * 2.0 ** -32 * 2
        bad = torch.tensor([False, False, True, False], device=DEV)
        assert got[:, bad].isnan().all()
        assert ((got.double() - want).abs() <= tol)[:, ~bad].all()
        again = decode(pool, q, t, n, S, window=1 << 30)
        assert torch.equal(again[:, ~bad], got[:, ~bad])

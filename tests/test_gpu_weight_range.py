"""Attention in which one key outweighs all others by many binary orders, over long
contexts: the small weights together still count, and where the heavy key's value is
zero (a first token that only soaks up weight) they are the whole result.

The heavy key's score is `gap` nats above the middle of the others'.  Keys and values are
what the pool holds, read back exactly (powers of two scale the codes)."""
import math

import pytest
import torch

import plain64
from paged_kv_cache_253_gb300.api import KVPool

pytestmark = pytest.mark.gpu
DEV = "cuda"
D, B = 128, 16
HEADS = torch.tensor([0.5625, 0.75, 0.875, 1.0])        # each head's share of the gap


def heavy(kind, n, at, gap, spread, seed):
    """A pool with one sequence of n tokens whose token `at` is the heavy one."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    pool = KVPool(n // B, B, 1, D, kind, DEV)
    if kind == "fp8":
        pool.set_kv_scales(2.0 ** -6, 2.0 ** -6)
    k = spread * torch.randn(n, 1, D, generator=g, device=DEV)
    v = 1 + 0.25 * torch.randn(n, 1, D, generator=g, device=DEV)
    k[at], v[at] = gap / math.sqrt(D), 0.0
    slots = torch.arange(n, device=DEV)
    pool.append_kv(k.bfloat16(), v.bfloat16(), slots)
    kk, vv = pool.read_kv(slots)
    tables = torch.arange(n // B, dtype=torch.int32, device=DEV)[None]
    return pool, kk.double(), vv.double(), tables


def bound(q, k, v, mask, out_dtype, floor, cut=0.0):
    """(out, tolerance): plain64's, and what the kernel's weights add: `floor` of the largest
    weight for each key (half the last place of the smallest weights), and `cut` of the sum."""
    out, mag, top = plain64.attend(q, k, v, 1 / math.sqrt(D), mask)
    vmax = float(v.abs().max())
    tol = plain64.tolerance(out, mag, top, vmax, out_dtype) + k.shape[0] * floor * vmax + cut * mag
    return out, tol


# half the last place of a weight, of the largest: bf16 results 2^-26 of 2^12 at least, fp32
# results 2^-26 of 2^6
@pytest.mark.parametrize("kind", ["fp8", "fp8b", "bf16"])
@pytest.mark.parametrize("out_dtype,floor", [(torch.bfloat16, 2.0 ** -38), (torch.float32, 2.0 ** -32)])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("at,gap,spread", [(0, 15.5, 0.3), (0, 17.0, 0.3), (131071, 15.5, 0.3), (0, 15.5, 0.0)])
def test_decode_keeps_small_weights(kind, out_dtype, floor, many, at, gap, spread):
    """One sequence (cut into many ranges), and as many as there are ranges (each a whole
    sequence: all its keys share one reference)."""
    n = 131072
    pool, k, v, t = heavy(kind, n, at, gap, spread, seed=int(gap * 2))
    S = 2 * torch.cuda.get_device_properties(0).multi_processor_count if many else 1
    q = HEADS.to(DEV)[None, :, None].expand(1, 4, D).bfloat16().contiguous()
    lens = torch.full((S,), n, dtype=torch.int32, device=DEV)
    got = pool.decode(q.expand(S, 4, D).contiguous(), t.expand(S, -1).contiguous(), lens, 1 / math.sqrt(D),
                      out_dtype=out_dtype, window=1 << 30)
    assert pool.get_error() == 0
    out, tol = bound(q, k, v, torch.ones(1, n, dtype=torch.bool, device=DEV), out_dtype, floor)
    worst = ((got.double() - out).abs() / tol).amax((0, 2))
    assert (worst <= 1).all(), f"{worst.tolist()} times the bound (by head)"


# 2^-25 of 2^9 at least; each product of 16 keys cuts the sum by less than 2^-23 of itself, and
# fp32 results take two (a rounded part and a remainder)
@pytest.mark.parametrize("kind", ["fp8", "fp8b", "bf16"])
@pytest.mark.parametrize("out_dtype,cut", [(torch.bfloat16, 2.0 ** -27), (torch.float32, 2.0 ** -26)])
@pytest.mark.parametrize("at,gap,spread", [(0, 17.0, 0.3), (0, 17.6, 0.1), (131068, 17.0, 0.3)])
def test_prefill_keeps_small_weights(kind, out_dtype, cut, at, gap, spread):
    n, T = 131072, 3
    pool, k, v, t = heavy(kind, n, at, gap, spread, seed=int(gap * 2))
    q = HEADS.to(DEV)[None, :, None].expand(T, 4, D).bfloat16().contiguous()
    i32 = dict(dtype=torch.int32, device=DEV)
    got = pool.prefill(q, torch.tensor([0, T], **i32), t, torch.tensor([n], **i32), 1 / math.sqrt(D), max_q_len=T,
                       out_dtype=out_dtype, window=1 << 30)
    assert pool.get_error() == 0
    j, p = torch.arange(n, device=DEV)[None], torch.arange(n - T, n, device=DEV)[:, None]
    out, tol = bound(q, k, v, j <= p, out_dtype, 2.0 ** -34, n * cut)
    worst = ((got.double() - out).abs() / tol).amax((0, 2))
    assert (worst <= 1).all(), f"{worst.tolist()} times the bound (by head)"

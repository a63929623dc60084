"""Windowed prefill with fp32 results over long contexts: sums that are cut to fp32 instead
of rounded shrink with every addition, so a result's error must not grow with its length."""
import math

import pytest
import torch

import plain64
from paged_kv_cache_253_gb300.api import KVPool

pytestmark = pytest.mark.gpu
DEV = "cuda"
D, B = 128, 16


def cache(kind, n, hkv, seed):
    """One sequence of n tokens whose values share a sign, so that nothing cancels."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    pool = KVPool(-(-n // B) + 1, B, hkv, D, kind, DEV)
    if kind == "fp8":
        pool.set_kv_scales(2.0 ** -6, 2.0 ** -6)
    slots = torch.arange(B, n + B, device=DEV)
    k = torch.randn(n, hkv, D, generator=g, device=DEV).bfloat16()
    v = (1 + 0.25 * torch.randn(n, hkv, D, generator=g, device=DEV)).bfloat16()
    pool.append_kv(k, v, slots)
    k, v = pool.read_kv(slots)
    return pool, k.double(), v.double(), torch.arange(1, -(-n // B) + 1, dtype=torch.int32, device=DEV)[None], g


# Each product of 16 keys cuts a sum by less than 2^-23 of itself; two of them per 16 keys over
# 4096 keys, then a rounded addition (2^-24 each): 2^-14 of sum w |v| and a little.  As a rule a
# cut is half of 2^-23 to 2^-24, of a sum that is half complete: 2^-16.5 of the result
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp8b"])
@pytest.mark.parametrize("n,T,G,window,sinks", [(131072, 70, 4, 1 << 30, 0), (40000, 33, 1, 1 << 30, 0),
                                                (30001, 200, 5, 9000, 100), (6000, 6000, 2, 1 << 30, 0),
                                                (5000, 64, 2, 4096, 0), (2300, 9, 2, 1 << 30, 0), (4097, 1, 16, 4096, 4)])
def test_fp32_results_of_long_contexts(kind, n, T, G, window, sinks):
    pool, k, v, t, g = cache(kind, n, 2, n)
    q = (0.3 * torch.randn(T, 2 * G, D, generator=g, device=DEV)).bfloat16()
    out = torch.full((T + 8, 2 * G, D), float("nan"), device=DEV)      # what was there is not a number
    i32 = dict(dtype=torch.int32, device=DEV)
    pool.prefill(q, torch.tensor([0, T], **i32), t, torch.tensor([n], **i32), 1 / math.sqrt(D), max_q_len=T,
                 out=out[:T], window=window, sinks=sinks)
    assert pool.get_error() == 0 and out[T:].isnan().all()
    rows = torch.tensor(sorted({0, 1, T // 3, T // 2, T - 1} & set(range(T))), device=DEV)
    j, p = torch.arange(n, device=DEV)[None], (n - T + rows)[:, None]
    mask = (j <= p) & ((j < sinks) | (p - j < window))
    want, mag, top = plain64.attend(q[rows], k, v, 1 / math.sqrt(D), mask)
    tol = 2.0 ** -14 * mag + 2.0 ** -24 * (n / 4096) * mag + plain64.tolerance(want, mag, top, float(v.abs().max()),
                                                                              torch.float32)
    err = (out[rows].double() - want).abs()
    assert (err <= tol).all(), f"{float((err / tol).max()):.3g} times the bound"
    # the errors' mean (values share a sign)
    assert float((out[rows].double() - want).mean().abs()) <= 2.0 ** -16 * float(want.abs().mean())


@pytest.mark.parametrize("kind", ["bf16", "fp8b"])
def test_totals_follow_their_references(kind):
    """Scores that rise by 40 nats along the context: every total is scaled down again and again;
    a row that is not a number stays one and leaves the others alone."""
    n, T = 9000, 3
    pool, k, v, t, g = cache(kind, n, 1, 7)
    slots = torch.arange(B, n + B, device=DEV)
    ramp = torch.linspace(0, 40.0 / math.sqrt(D), n, device=DEV)[:, None, None] + 0.05 * k.float()
    pool.append_kv(ramp.bfloat16(), v.bfloat16(), slots)
    k, v = (x.double() for x in pool.read_kv(slots))
    q = torch.ones(T, 4, D, device=DEV).bfloat16()
    q[1, 2, 5] = float("nan")
    i32 = dict(dtype=torch.int32, device=DEV)
    got = pool.prefill(q, torch.tensor([0, T], **i32), t, torch.tensor([n], **i32), 1 / math.sqrt(D), max_q_len=T,
                       window=1 << 30)
    bad = torch.zeros(T, 4, dtype=torch.bool, device=DEV)
    bad[1, 2] = True
    assert got[bad].isnan().all()
    j, p = torch.arange(n, device=DEV)[None], torch.arange(n - T, n, device=DEV)[:, None]
    want, mag, top = plain64.attend(q.nan_to_num(1.0), k, v, 1 / math.sqrt(D), j <= p)
    tol = 2.0 ** -14 * mag + plain64.tolerance(want, mag, top, float(v.abs().max()), torch.float32)
    assert ((got.double() - want).abs() <= tol)[~bad].all() and pool.get_error() == 0

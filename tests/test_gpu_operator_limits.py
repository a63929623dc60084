"""Block-scaled, windowed and rotary operators at the limits of what they are given: the
largest scales, reserved workspaces, scratch, and calls that are refused before they have
done anything."""
import gc

import pytest
import torch

import plain64
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


@pytest.mark.parametrize("kind,es", [("bf16", 2), ("fp8", 1)])
def test_pools_without_block_scales_hold_no_scratch(kind, es):
    """Keys and values alone, up to the allocator's pages."""
    nb, D = 1 << 20, 4
    gc.collect()
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    pool = KVPool(nb, 16, 1, D, kind, DEV)
    assert free - torch.cuda.mem_get_info()[0] <= 2 * nb * 16 * D * es + (16 << 20)
    pool.close()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_a_first_rotary_append_inside_a_capture(kind):
    """More tokens than a call searches by itself, first captured and replayed, then called: the
    rows are the formula's either way."""
    g = torch.Generator().manual_seed(5)
    T, H, Hq, D = 700, 2, 4, 128
    pool = KVPool(60, 16, H, D, kind, DEV)
    if kind == "fp8":
        pool.set_kv_scales(2.0 ** -5, 2.0 ** -5)
    q, k, v = (torch.randn(T, h, D, generator=g).bfloat16().to(DEV) for h in (Hq, H, H))
    slots = torch.randperm(60 * 16, generator=g)[:T].to(DEV)
    pos = torch.randint(0, 100000, (T,), generator=g, dtype=torch.int32).to(DEV)
    inv = (1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().to(DEV)
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.append_rope(q, k, v, slots, pos, inv, q_out=out)
    want_q, want_k = (plain64.rotate(x.cpu(), pos[None].cpu(), inv.cpu(), torch.zeros(64), False) for x in (q, k))
    for call in (graph.replay, lambda: pool.append_rope(q, k, v, slots, pos, inv, q_out=out), graph.replay):
        out.zero_()
        pool.import_(*(torch.zeros_like(x) for x in pool.export()))
        call()
        kk, vv = (x.cpu().double() for x in pool.read_kv(slots))
        # one rounding to bf16, and 2^-20 of the pair's length for the rotation in 32 bits; codes:
        # half a step of e4m3, 2^-4 of the value or 2^-10 of the scale
        r = 2.0 ** -20 * 8
        assert ((out.cpu().double() - want_q).abs() <= 2.0 ** -8 * want_q.abs() + r).all()
        if kind == "bf16":
            assert ((kk - want_k).abs() <= 2.0 ** -8 * want_k.abs() + r).all() and torch.equal(vv, v.cpu().double())
        else:
            assert ((kk - want_k).abs() <= 2.0 ** -4 * want_k.abs() + 2.0 ** -15 + 2 * r).all()
            assert ((vv - v.cpu().double()).abs() <= 2.0 ** -4 * v.cpu().double().abs() + 2.0 ** -15).all()
    assert pool.get_error() == 0


@pytest.mark.parametrize("B", [16, 32])
def test_a_refused_append_decode_appends_nothing(B):
    """Block-scaled pools append, then decode: an output that the decode refuses is refused before."""
    pool = KVPool(4, B, 2, 128, "fp8b", DEV)
    k, q = torch.randn(1, 2, 128, device=DEV).bfloat16(), torch.randn(1, 8, 128, device=DEV).bfloat16()
    slot, out = torch.zeros(1, dtype=torch.int64, device=DEV), torch.full((1100,), 7.0, device=DEV)
    t, lens = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    args = (pool.handle, k.data_ptr(), k.data_ptr(), slot.data_ptr(), q.data_ptr(), 1, 8, t.data_ptr(), 1, lens.data_ptr(), 0.1)
    assert L.pa_append_decode(*args, out.data_ptr() + 2, L.PA_F32, None) == L.PA_ERR_INVALID_ARG
    assert L.pa_append_decode(*args, out.data_ptr() + 1, L.PA_BF16, None) == L.PA_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert not pool.export()[0].any() and not pool.export_scales().any() and (out == 7).all()
    assert L.pa_append_decode(*args, out.data_ptr(), L.PA_F32, None) == 0 and pool.get_error() == 0
    assert pool.export()[0].any() and (out[:1024] != 7).all() and (out[1024:] == 7).all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8", "fp8b"])
def test_pointers_that_are_not_aligned_to_their_elements_are_refused(kind):
    """By the host, before anything is launched; k, v and outputs at half an element, tables and
    lengths at half an int."""
    pool = KVPool(4, 16, 2, 128, kind, DEV)
    buf = torch.zeros(64 * 1024, dtype=torch.uint8, device=DEV)
    a, half = buf.data_ptr(), 2 if kind == "f32" else 1
    for k, v, s in ((a + half, a, a), (a, a + half, a), (a, a, a + 4)):
        assert L.pa_append_kv(pool.handle, k, v, s, 1, None) == L.PA_ERR_INVALID_ARG
        assert L.pa_append_rope(pool.handle, None, 0, 0, k, 256, v, 256, s, 1, a, 1, a, None, 128, 0, None, None) \
            == L.PA_ERR_INVALID_ARG
        assert L.pa_read_kv(pool.handle, s, 1, k, v, None) == L.PA_ERR_INVALID_ARG
    for t, n, o, dt in ((a + 2, a, a, L.PA_F32), (a, a + 2, a, L.PA_F32), (a, a, a + 2, L.PA_F32), (a, a, a + 1, L.PA_BF16)):
        assert L.pa_decode_window(pool.handle, a, 1, 8, t, 1, n, 9, 0, 0.1, o, dt, None) == L.PA_ERR_INVALID_ARG
        assert L.pa_decode(pool.handle, a, 1, 8, t, 1, n, 0.1, o, dt, None) == L.PA_ERR_INVALID_ARG
        assert L.pa_prefill_window(pool.handle, a, 1, 8, a, 1, 1, t, 1, n, 9, 0, 0.1, o, dt, None) == L.PA_ERR_INVALID_ARG
        if kind in ("bf16", "fp8", "fp8b"):
            assert L.pa_prefill(pool.handle, a, 1, 8, a, 1, 1, t, 1, n, 0.1, o, dt, None) == L.PA_ERR_INVALID_ARG
    assert L.pa_prefill_window(pool.handle, a, 1, 8, a + 2, 1, 1, a, 1, a, 9, 0, 0.1, a, L.PA_F32, None) == L.PA_ERR_INVALID_ARG
    assert pool.get_error() == 0 and not pool.export()[0].any()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_a_first_call_inside_a_capture_is_the_call(kind):
    """The scratch of a long rotary append is made beside the capture: replays run the kernels that
    an ordinary call runs, bit for bit, and an ordinary call may come before the first replay."""
    g = torch.Generator().manual_seed(6)
    T, H, Hq, D = 5000, 2, 4, 128
    q, k, v = (torch.randn(T, h, D, generator=g).bfloat16().to(DEV) for h in (Hq, H, H))
    slots = torch.randperm(400 * 16, generator=g)[:T].to(DEV)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32).to(DEV)
    inv = (1e6 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().to(DEV)
    plain, pool = KVPool(400, 16, H, D, kind, DEV), KVPool(400, 16, H, D, kind, DEV)
    want = plain.append_rope(q, k, v, slots, pos, inv), *plain.export()
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.append_rope(q, k, v, slots, pos, inv, q_out=out)
    for call in (lambda: pool.append_rope(q, k, v, slots, pos, inv, q_out=out), graph.replay, graph.replay):
        out.zero_()
        pool.import_(*(torch.zeros_like(x) for x in pool.export()))
        call()
        assert all(torch.equal(a, b) for a, b in zip(want, (out, *pool.export())))
    assert pool.get_error() == 0

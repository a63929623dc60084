"""Arguments that the Python calls turn into C ones: none becomes another value on the way,
none of the wrong shape is taken for a part of itself.  No GPU is needed."""
import pytest
import torch

from paged_kv_cache_253_gb300 import api

NO_GPU = torch.device("cpu")


def bare_pool():
    pool = api.KVPool.__new__(api.KVPool)
    pool.device, pool.dtype, pool.handle = NO_GPU, torch.bfloat16, None
    pool.kv_heads, pool.head_dim = 2, 128
    return pool


@pytest.mark.parametrize("x", [-1, -(1 << 31), -(1 << 31) - 1, -(1 << 32) + 5, -(1 << 40), -(1 << 64) + 9])
def test_negative_counts_stay_negative_as_c_ints(x):
    import ctypes
    assert ctypes.c_int(api._span(x)).value < 0


def test_slots_are_one_list():
    """A table of slots is not read as its first row's worth."""
    pool, k = bare_pool(), torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    pos, inv = torch.zeros(3, dtype=torch.int32), torch.ones(64)
    for slots in (torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 1, dtype=torch.int64), torch.tensor(3)):
        with pytest.raises(ValueError):
            pool.read_kv(slots)
        with pytest.raises(ValueError):
            pool.append_rope(None, k, k, slots, pos, inv)


def test_the_front_end_does_without_private_torch_names():
    """A torch whose private stream query is gone (or a build without CUDA, which has none) still
    imports the front end, which then asks for streams the public way."""
    import subprocess
    import sys
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getCurrentStream'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import paged_kv_cache_253_gb300.api as a\n"
            "print(a.fnv1a64(b''))\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.gpu
def test_streams_are_the_same_either_way(monkeypatch):
    dev, st = torch.device("cuda", torch.cuda.current_device()), torch.cuda.Stream()
    for use in (torch.cuda.current_stream(), st):
        with torch.cuda.stream(use):
            fast = api._stream(dev)
            monkeypatch.setattr(api, "_raw_stream", None)
            assert api._stream(dev) == fast == use.cuda_stream
            monkeypatch.undo()

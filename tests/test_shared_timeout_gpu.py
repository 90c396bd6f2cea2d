"""Bounded waits of the shared-latent kernels: a wait that runs out is reported, the kernel
returns, and the next call on the same buffers is right.

As for the older kernels this uses libstief_testhooks.so (50 ms waits; stief_test_set_stall makes
the first copy's barrier expect bytes that no copy delivers).  The decode needs nothing put back:
its workspace's contents do not matter.
"""
import ctypes

import pytest
import torch

import decode_attention_stief_b200 as stief
from decode_attention_stief_b200 import _binding
from decode_attention_stief_b200 import build as stief_build
from shared_util import bf, pool_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module")
def hooks():
    lib = ctypes.CDLL(stief_build.library_file("testhooks"))
    for name in ("stief_decode_shared_paged", "stief_expand_shared_paged", "stief_prefill_attention"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_int, getattr(stief.library(), name).argtypes
    lib.stief_test_set_stall.restype = None
    lib.stief_test_set_stall.argtypes = [ctypes.c_uint32]
    yield lib
    lib.stief_test_set_stall(0)


def _stalled_then_right(hooks, fn, args, status, outs, **kw):
    """fn(*args) through the test library, stalled (the timeout is reported), then not: its outputs
    equal those of the library itself."""
    prepared = stief.prepare(fn, *args, dev_status=status, **kw)
    call = lambda: getattr(hooks, prepared.name)(*prepared._cargs)  # noqa: E731
    hooks.stief_test_set_stall(16)
    try:
        assert call() == 0
        torch.cuda.synchronize()  # the context is still usable
        assert int(status.item()) & stief.DEV_WAIT_TIMEOUT
    finally:
        hooks.stief_test_set_stall(0)
    status.zero_()
    assert call() == 0
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = [x.clone() for x in outs]
    fn(*args, dev_status=status, **kw)
    assert all(torch.equal(x, y) for x, y in zip(got, outs)) and int(status.item()) == 0


@pytest.mark.parametrize("lens,Hq,most", [([3000, 10, 0, 700], 100, 3000), ([200, 64, 1], 16, 200)])
def test_decode(hooks, lens, Hq, most):
    """Split sequences with the joining kernel, and short ones without."""
    gen = torch.Generator().manual_seed(1)
    pool, table = pool_of(lens, 64, 256 + 64, gen)
    q, out = bf(len(lens), Hq, 320, gen=gen).to(DEV), torch.zeros((len(lens), Hq, 256), dtype=torch.bfloat16, device=DEV)
    ws = stief.shared_workspace_for(len(lens), Hq, 256)
    _stalled_then_right(hooks, stief.stief_decode_shared_paged,
                        (q, pool.to(DEV), table.to(DEV), _i(lens), out, ws, most, 0.08), _i([0]), [out])


def test_expand(hooks):
    gen = torch.Generator().manual_seed(2)
    pool, table = pool_of([700, 130], 64, 512 + 64, gen)
    W = bf(8, 128, 512, gen=gen, scale=0.05).to(DEV)
    k, v = (torch.zeros((830, 8, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pe = torch.zeros((830, 64), dtype=torch.bfloat16, device=DEV)
    _stalled_then_right(hooks, stief.stief_expand_shared_paged,
                        (pool.to(DEV), table.to(DEV), _i([0, 700, 830]), W, W, k, v, pe), _i([0]), [k, v, pe])


@pytest.mark.parametrize("dr", [0, 64])
def test_prefill(hooks, dr):
    gen = torch.Generator().manual_seed(3)
    q, k, v = (bf(*s, gen=gen).to(DEV) for s in ((600, 4, 128 + dr), (700, 2, 128), (700, 2, 128)))
    pe = bf(700, dr, gen=gen).to(DEV) if dr else None
    out = torch.zeros((600, 4, 128), dtype=torch.bfloat16, device=DEV)
    _stalled_then_right(hooks, stief.stief_prefill_attention, (q, k, v, _i([0, 600]), _i([0, 700]), out, 600, 0.1),
                        _i([0]), [out], k_pe=pe)


def test_prefill_over_a_long_walk(hooks):
    gen = torch.Generator().manual_seed(4)
    q, k, v = (bf(*s, gen=gen).to(DEV) for s in ((600, 4, 192), (1400, 2, 128), (1400, 2, 128)))
    pe, out = bf(1400, 64, gen=gen).to(DEV), torch.zeros((600, 4, 128), dtype=torch.bfloat16, device=DEV)
    _stalled_then_right(hooks, stief.stief_prefill_attention, (q, k, v, _i([0, 600]), _i([0, 1400]), out, 600, 0.1),
                        _i([0]), [out], k_pe=pe)


def test_prefill_pairs(hooks):
    gen = torch.Generator().manual_seed(6)
    q, k, v = (bf(*s, gen=gen).to(DEV) for s in ((600, 40, 192), (1400, 40, 128), (1400, 40, 128)))
    pe, out = bf(1400, 64, gen=gen).to(DEV), torch.zeros((600, 40, 128), dtype=torch.bfloat16, device=DEV)
    _stalled_then_right(hooks, stief.stief_prefill_attention, (q, k, v, _i([0, 600]), _i([0, 1400]), out, 600, 0.1),
                        _i([0]), [out], k_pe=pe)


def test_library_is_the_one_of_the_binding():
    assert _binding.library_path() != stief_build.library_file("testhooks")

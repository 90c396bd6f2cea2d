"""Paired prompt CTAs whose tensor memory does not match: reported as such, no row written, and the
next call is right.  (libstief_testhooks.so, whose stief_test_set_tmem_apart makes the comparison
fail; nothing is computed then.)"""
import ctypes

import pytest
import torch

import decode_attention_stief_b200 as stief
from decode_attention_stief_b200 import build as stief_build
from shared_util import bf

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def test_rows_are_left_as_they_were():
    hooks = ctypes.CDLL(stief_build.library_file("testhooks"))
    fn = hooks.stief_prefill_attention
    fn.restype, fn.argtypes = ctypes.c_int, stief.library().stief_prefill_attention.argtypes
    hooks.stief_test_set_tmem_apart.restype, hooks.stief_test_set_tmem_apart.argtypes = None, [ctypes.c_uint32]
    gen = torch.Generator().manual_seed(7)
    q, k, v, pe = (bf(*s, gen=gen).to(DEV) for s in ((600, 40, 192), (1400, 40, 128), (1400, 40, 128), (1400, 64)))
    out = torch.full((600, 40, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    qs, ks, status = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 600], [0, 1400], [0]))
    call = stief.prepare(stief.stief_prefill_attention, q, k, v, qs, ks, out, 600, 0.1, k_pe=pe, dev_status=status)
    hooks.stief_test_set_tmem_apart(128)
    try:
        assert fn(*call._cargs) == 0
        torch.cuda.synchronize()
    finally:
        hooks.stief_test_set_tmem_apart(0)
    assert int(status.item()) == stief.DEV_TMEM_PAIR
    assert torch.all(out == 7.0)
    status.zero_()
    assert fn(*call._cargs) == 0
    torch.cuda.synchronize()
    got = out.clone()
    call()
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(got, out) and not torch.any(out == 7.0)

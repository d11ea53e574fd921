"""The choice's lengths: new_lens is written while other rows still read
context_lens, so the two may not share a word."""
import ctypes

import pytest

from paged_kv_cache_309_gb300 import build as pabuild
from paged_kv_cache_309_gb300 import pa

P = ctypes.c_void_p
AT = 0x200000  # never dereferenced


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("offset", [0, 4, -4, 12, -12])
def test_overlapping_lengths_are_refused(paged, offset):
    pabuild.build()
    lib = pa.library()
    args = [P(0x100000), P(AT + offset), None, P(0x300000), P(AT)]
    args += [P(0x400000)] if paged else []
    args += [4, 8, 128, 64, 4, 16] + ([16, 8, 64] if paged else []) + [None]
    fn = lib.pa_evict_select_paged if paged else lib.pa_evict_select
    assert fn(*args) == pa.PA_ERR_INVALID

"""The serving step over a paged cache at its edges: sequences and pages that do
not fit, values that are not finite, packed rows and lengths that other kernels
or other paths of them take.  Plain 64-bit forms are in paged_ref.py."""
import ctypes
import math

import pytest
import torch

import query_group_top_b200 as qg
from tests import paged_ref as ref
from tests.test_paged_step import attend, check_attention, check_index_rows, normal, same_bits

gpu = pytest.mark.gpu


def status():
    """The kernels' status bits, which sync_status() turns into an exception, and its message."""
    lib = qg.load_library()
    flags = ctypes.c_int(0)
    rc = lib.pivot_sync_status(torch.cuda.current_stream().cuda_stream, ctypes.byref(flags))
    return flags.value, (lib.pivot_last_error().decode() if rc else "")


# ------------------------------------------------------------------ sequences that do not fit
@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("top_k", [5, 900])
def test_index_rows_of_a_sequence_that_does_not_fit(top_k, d):
    """The rule of all calls over the cache: lengths past the table, or below the sequence's own new tokens, skip the
    sequence (zeros) and are told, whatever its index rows hold; the others are as without it (one CTA a row, and a
    cluster)."""
    g, H = 3, 2
    c = ref.Cache([1000, 970, 990], [g] * 3, H, d, 16, seed=40)
    q = normal((3, g, H, d), 41)
    idx = torch.arange(top_k, dtype=torch.int32, device="cuda").expand(3, g, H, top_k).contiguous()
    good = qg.sparse_attention_paged(q, c.kpages, c.vpages, c.table, c.seqlens, idx)
    assert status()[0] == 0
    for wrong in (c.table.shape[1] * c.page + 1, 2**31 - 1, g - 1, 0, -5):
        lens = c.seqlens.clone()
        lens[1] = wrong
        out = torch.full_like(good, 9.0)
        qg.sparse_attention_paged(q, c.kpages, c.vpages, c.table, lens, idx, out=out)
        assert status()[0] == qg.FLAG_BADLEN, wrong
        assert bool((out[1] == 0).all()), wrong
        assert same_bits(out[0], good[0]) and same_bits(out[2], good[2])

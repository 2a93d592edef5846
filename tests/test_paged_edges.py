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


# ------------------------------------------------------------------ without a GPU
def test_index_rows_longer_than_their_places_count_are_refused():
    """Near 2^31 places a walk in 32 bits would pass its end: refused before any device is asked for."""
    from query_group_top_b200 import build
    build.build()
    lib = qg.load_library()
    buf = ctypes.create_string_buffer(64)
    p = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16
    for top_k in ((1 << 30) + 1, 2**31 - 200, 2**31 - 1):
        assert lib.pivot_sparse_attention_paged(p, p, p, p, p, p, 1, 1, 64, 1, 1, 16, 1, top_k, p, None) == 1
        assert b"top_k" in lib.pivot_last_error()


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


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_append_gives_zeros_for_the_queries_of_tokens_left_out(d, dtype):
    """Queries that the call allocates hold a result or zeros, never what the memory held: a page outside the cache, a
    length that does not fit, tokens behind the last sequence, no sequence at all."""
    H, Hq, page = 2, 5, 16
    c = ref.Cache([20, 3, 40, 9], [4] * 4, H, d, page, seed=42)
    k, v, q = normal((19, H, d), 43, dtype), normal((19, H, d), 44, dtype), normal((19, Hq, d), 45, dtype)
    f, _ = qg.rope_frequencies(d)
    good = qg.paged_append(k, v, c.kpages.clone(), c.vpages.clone(), c.table, c.seqlens, cu_new=c.cu, freqs=f, q=q)
    assert status()[0] == 0 and bool((good[16:] == 0).all()) and bool(good[:16].any(-1).all())
    table, lens = c.table.clone(), c.seqlens.clone()
    table[0, 1] = c.kpages.shape[0]          # rows 16.. of sequence 0
    lens[2] = 3                              # fewer rows than new tokens
    for ragged in (True, False):
        n = 19 if ragged else 16
        shape = (lambda x: x) if ragged else (lambda x: x[:16].view(4, 4, *x.shape[1:]))  # noqa: E731
        junk = torch.full((n, Hq, d), math.nan, dtype=torch.bfloat16, device="cuda")
        del junk                             # the allocator hands this memory out again
        out = qg.paged_append(shape(k), shape(v), c.kpages.clone(), c.vpages.clone(), table, lens,
                              cu_new=c.cu if ragged else None, freqs=f, q=shape(q)).view(n, Hq, d)
        assert status()[0] == qg.FLAG_BADLEN | qg.FLAG_BADPAGE
        want = good[:n].clone()
        want[0:4], want[8:12] = 0, 0
        assert same_bits(out, want)
        mine = torch.full((n, Hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
        qg.paged_append(shape(k), shape(v), c.kpages.clone(), c.vpages.clone(), table, lens,
                        cu_new=c.cu if ragged else None, freqs=f, q=shape(q), out_q=mine.view(shape(q).shape))
        status()
        want[0:4], want[8:12], want[16:] = 9, 9, 9
        assert same_bits(mine, want)
    junk = torch.full((19, Hq, d), math.nan, dtype=torch.bfloat16, device="cuda")
    del junk
    none = qg.paged_append(k, v, c.kpages.clone(), c.vpages.clone(), c.table[:0], c.seqlens[:0], cu_new=c.cu[:1], freqs=f, q=q)
    assert bool((none == 0).all())


@gpu
@pytest.mark.parametrize("where", [0, 1, 150, 599])
def test_append_tells_of_lengths_that_do_not_fit_in_sequences_without_new_tokens(where):
    """As the attention does over the same arrays; the tokens of the others are written all the same."""
    new = [0] * 600
    new[3], new[400] = 5, 1                  # six tokens, so the launch has far fewer blocks than the batch sequences
    held = [i % 30 for i in range(600)]
    c = ref.Cache(held, new, 1, 64, 16, seed=46)
    k = normal((6, 1, 64), 47)
    q = normal((6, 1, 64), 48)
    want = c.kpages.clone(), c.vpages.clone()
    qg.paged_append(k, k, *want, c.table, c.seqlens, cu_new=c.cu)
    assert status()[0] == 0
    for wrong in (-1, c.table.shape[1] * c.page + 1):
        lens = c.seqlens.clone()
        lens[where] = wrong
        got = c.kpages.clone(), c.vpages.clone()
        qg.paged_append(k, k, *got, c.table, lens, cu_new=c.cu)
        assert status()[0] == qg.FLAG_BADLEN
        assert same_bits(got[0], want[0]) and same_bits(got[1], want[1])
        qg.paged_attention(q, *got, c.table, lens, 4096, cu_q=c.cu)
        assert status()[0] == qg.FLAG_BADLEN

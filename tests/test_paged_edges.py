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


def test_a_binding_built_for_another_torch_is_told_and_built_anew(monkeypatch, tmp_path):
    """The compiled half of the binding calls one torch's C++ classes: another torch's is neither loaded nor left."""
    from query_group_top_b200 import build
    build.build()
    assert not build.stale(build.BINDING) and build.built_for() == torch.__version__
    assert qg._load_step().built_for == torch.__version__
    monkeypatch.setattr(build, "torch_version", lambda: "9.9.9")
    assert build.stale(build.BINDING) and not build.stale(build.LIB)
    monkeypatch.undo()
    monkeypatch.setattr(build, "BUILT_FOR", str(tmp_path / "none.txt"))
    assert build.stale(build.BINDING)                      # built when nobody wrote it down
    monkeypatch.undo()
    monkeypatch.setattr(qg.torch, "__version__", "9.9.9")
    with pytest.raises(qg.PivotError, match="not built for this torch"):
        qg._load_step()


def test_the_library_is_built_without_the_binding(monkeypatch):
    """A user of the C library alone needs neither torch nor Python's headers."""
    from query_group_top_b200 import build

    def no(*_):
        raise AssertionError("the binding was asked for")

    monkeypatch.setattr(build, "build_binding", no)
    monkeypatch.setattr(build, "torch_version", no)
    assert build.build(binding=False) == build.LIB


def test_no_workspace_where_the_rows_fill_the_device():
    """Parts of the key axis are for few rows: a prefill whose row tiles are several rounds of the device's has none."""
    from query_group_top_b200 import build
    build.build()
    size = qg.load_library().pivot_paged_attention_workspace_size
    assert size(8192, 1, 16, 16, 128, 8192) == 0
    assert size(2048, 64, 32, 8, 128, 2048) == 0
    assert size(64, 1, 16, 16, 128, 8192) > 0


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


# ------------------------------------------------------------------ packed rows and lengths of every path
SIXTEEN = [  # held, new, Hq, Hk, d, page, itself, ragged, longest: 9 to 16 packed rows a sequence
    ([300, 17, 0], [1] * 3, 16, 1, 128, 16, True, False, None),
    ([200], [3], 12, 3, 128, 32, True, False, None),              # 12 rows
    ([90, 500], [4, 4], 8, 2, 128, 8, False, False, None),
    ([5000, 3], [1, 1], 32, 2, 128, 64, True, False, 1 << 20),    # many parts
    ([1500] * 30, [2] * 30, 10, 2, 128, 16, True, False, None),   # 10 rows, two or more a scheduler
    ([40, 700, 0, 9], [4, 1, 3, 2], 8, 2, 128, 1, True, True, None),
    ([4000, 60], [3, 3], 5, 1, 64, 16, True, False, None),        # 15 rows of 64 channels
]


@gpu
@pytest.mark.parametrize("case", SIXTEEN, ids=str)
def test_attention_of_nine_to_sixteen_packed_rows(case):
    held, new, Hq, Hk, d, page, itself, ragged, longest = case
    c = ref.Cache(held, new, Hk, d, page, seed=60)
    q = normal((sum(new), Hq, d), 61)
    kw = {} if longest is None else {"longest": longest}
    out, lse = attend(c, q, itself, ragged, **kw)
    assert status()[0] == 0
    check_attention(c, q, out, lse, itself, d ** -0.5)
    again, lse2 = attend(c, q, itself, ragged, **kw)
    assert same_bits(out, again) and same_bits(lse, lse2)


LONG = [  # held, new, Hq, Hk, d, page
    ([0], [4096], 16, 16, 128, 128),        # 256 row tiles: more than the device takes at a time
    ([40000], [300], 8, 2, 64, 64),         # a chunk behind a long context, in parts
    ([60000], [2], 16, 1, 128, 16),         # 32 packed rows: matrix tiles in many parts
    ([60000, 20000], [1, 1], 32, 2, 128, 16),   # 16 packed rows
    ([100000], [1], 4, 4, 64, 4),
    ([30000], [40], 4, 1, 128, 2),
]


@gpu
@pytest.mark.parametrize("case", LONG, ids=str)
def test_attention_over_long_contexts_within_a_narrow_bound(case):
    """Where thousands of keys share the weight, the roundings' worst case is a tenth of a typical output and more.  They
    are independent: a weight's is at most HALF of it, anywhere between, so its deviation at most HALF / sqrt(3), and their
    sum's HALF / sqrt(3) sqrt(sum p^2 v^2); 7 of those (one value in 10^11) are allowed, HALF of the output twice (its own
    rounding, and the sum's correction by the heaviest weights' roundings), and fp32's part as in paged_ref."""
    held, new, Hq, Hk, d, page = case
    c = ref.Cache(held, new, Hk, d, page, seed=62)
    q = normal((sum(new), Hq, d), 63)
    out, lse = attend(c, q, True, True)
    assert status()[0] == 0
    t = 0
    for b, n in enumerate(new):
        for h in sorted({0, Hq // 2, Hq - 1}):
            k, v = c.k[b][:, h // (Hq // Hk)].double(), c.v[b][:, h // (Hq // Hk)].double()
            x = q[t:t + n, h].double() @ k.T * d ** -0.5
            ds = float((q[t:t + n, h].double().abs() @ k.abs().T).max()) * d ** -0.5 * (d + 4) * ref.FP32
            x = x.masked_fill(torch.arange(c.lens[b], device="cuda") > torch.arange(held[b], held[b] + n, device="cuda")[:, None],
                              -math.inf)
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - z[:, None])
            y, far, dev = p @ v, p @ v.abs(), (p * p @ (v * v)).sqrt()
            soft = 2 * ds + 2.0 ** -20 + (math.sqrt(c.lens[b]) + 16) * ref.FP32
            bound = ref.HALF * (2 * y.abs() + 7 / math.sqrt(3) * dev) + soft * far
            ref.close(out[t:t + n, h], y, bound, f"head {h} of sequence {b}")
            ref.close(lse[t:t + n, h], z, ds + 2.0 ** -20 + 4 * ref.FP32 * (z.abs() + x.amax(1).abs()), "lse")
            if held[b]:
                assert float(bound.mean()) < 0.05 * float(y.square().mean().sqrt())       # narrow indeed
        t += n


# ------------------------------------------------------------------ values that are not finite
NONFINITE = [  # held, new, Hq, Hk, d, page, longest
    ([70, 9], [1, 2], 4, 2, 64, 16, None),          # few rows, one part
    ([300], [2], 14, 1, 128, 16, None),             # 28 packed rows: matrix tiles
    ([300], [2], 7, 1, 128, 16, None),              # 14: few rows, two tiles of them
    ([900], [2], 2, 2, 128, 16, 1 << 20),           # few rows, many parts
    ([0], [150], 2, 1, 64, 64, None),               # matrix tiles from nothing
    ([500, 40], [60, 30], 4, 2, 128, 32, 1 << 20),  # ... in parts
    ([200], [90], 3, 1, 64, 2, None),               # ... over pages that are copied row by row
    ([200], [90], 3, 1, 128, 4, None),
    ([30] * 60 + [300], [1] * 60 + [90], 4, 1, 64, 16, None),   # a chunk among single tokens: both kernels
]


def check_not_finite(out, want, bound, what):
    assert torch.equal(torch.isnan(out), torch.isnan(want)), what
    inf = torch.isinf(want)
    assert torch.equal(out[inf].double(), want[inf]), what
    whole = torch.isfinite(want)
    ref.close(out[whole], want[whole], bound[whole], what)


@gpu
@pytest.mark.parametrize("case", NONFINITE, ids=str)
def test_attention_over_values_that_are_not_finite(case):
    """Channel by channel the definition's: an infinity or NaN that a query sees makes its channel so, whatever its
    weight; one that it does not see leaves it alone, in its own tile too."""
    held, new, Hq, Hk, d, page, longest = case
    c = ref.Cache(held, new, Hk, d, page, seed=50)
    q = normal((sum(new), Hq, d), 51)
    t = 0
    rng = torch.Generator().manual_seed(52)
    for b, n in enumerate(new):
        S = c.lens[b]
        put = [(0, 0, math.inf), (min(3, S - 1), 1, -math.inf), (S // 2, 2, math.nan), (S // 3, 3, math.inf),
               (S // 2, 3, -math.inf)]
        put += [(S - 1 - i, 8 + i % 8, (math.inf, math.nan, -math.inf)[i % 3]) for i in range(n)]          # new tokens' own
        put += [(int(torch.randint(S, (1,), generator=rng)), 20 + i, math.inf) for i in range(12)]
        for row, ch, x in put:
            c.v[b][row, 0, ch] = x
            c.vpages[int(c.table[b, row // page]), row % page, 0, ch] = x
    out, lse = attend(c, q, True, True, **({} if longest is None else {"longest": longest}))
    assert status()[0] == 0
    for b, n in enumerate(new):
        lim = [held[b] + i + 1 for i in range(n)]
        y, z, yb, zb = ref.attention(q[t:t + n], c.k[b], c.v[b], lim, d ** -0.5)
        check_not_finite(out[t:t + n], y, yb, f"sequence {b}")
        ref.close(lse[t:t + n], z, zb, f"lse of sequence {b}")
        t += n


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("held,new,longest", [(100, 1, None), (3000, 1, 1 << 20), (100, 40, None), (3000, 40, 1 << 20)])
def test_attention_over_an_infinite_value_whose_weight_rounds_to_zero(held, new, longest, d):
    """150 below the others in the exponent: positive by definition, zero in fp32."""
    c = ref.Cache([held], [new], 1, d, 16, seed=53)
    q = torch.ones((new, 1, d), dtype=torch.bfloat16, device="cuda")
    row, low = 20, -152.0 / math.sqrt(d)
    for pages, x in ((c.kpages, low), (c.vpages, torch.where(torch.arange(d, device="cuda") == 7, math.inf, 1.0))):
        pages[int(c.table[0, row // 16]), row % 16, 0] = x
    c.k[0][row, 0] = low
    c.v[0][row, 0] = 1.0
    c.v[0][row, 0, 7] = math.inf
    out, _ = attend(c, q, True, True, **({} if longest is None else {"longest": longest}))
    y, _, yb, _ = ref.attention(q, c.k[0], c.v[0], [held + i + 1 for i in range(new)], d ** -0.5)
    check_not_finite(out, y, yb, "dense")
    if new == 1:
        idx = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 1, 1, 64)
        out = qg.sparse_attention_paged(q.view(1, 1, 1, d), c.kpages, c.vpages, c.table, c.seqlens, idx)
        y, _, yb, _ = ref.attention(q, c.k[0][:64], c.v[0][:64], [64], d ** -0.5)
        check_not_finite(out[0], y, yb, "index rows")


@gpu
@pytest.mark.parametrize("case", NONFINITE, ids=str)
def test_attention_over_values_near_the_types_end(case):
    """Every value of a channel 3e38 (another's -3e38, a third's in turn): a mean of them is finite, a sum is not."""
    held, new, Hq, Hk, d, page, longest = case
    c = ref.Cache(held, new, Hk, d, page, seed=56)
    q = normal((sum(new), Hq, d), 57)
    for b, n in enumerate(new):
        for row in range(c.lens[b]):
            big = torch.tensor([3e38, -3e38, 3e38 if row % 2 else -3e38], device="cuda").to(torch.bfloat16)
            c.v[b][row, 0, 4:7] = big
            c.vpages[int(c.table[b, row // page]), row % page, 0, 4:7] = big
    out, _ = attend(c, q, True, True, **({} if longest is None else {"longest": longest}))
    assert status()[0] == 0
    t = 0
    for b, n in enumerate(new):
        y, _, yb, _ = ref.attention(q[t:t + n], c.k[b], c.v[b], [held[b] + i + 1 for i in range(n)], d ** -0.5)
        ref.close(out[t:t + n], y, yb, f"sequence {b}")
        t += n
    if len(held) == 1 and new[0] == 2 and Hq == Hk:
        idx = torch.arange(held[0], dtype=torch.int32, device="cuda").expand(1, 2, Hq, held[0]).contiguous()
        out = qg.sparse_attention_paged(q.view(1, 2, Hq, d), c.kpages, c.vpages, c.table, c.seqlens, idx)
        y, _, yb, _ = ref.attention(q, c.k[0][:held[0]], c.v[0][:held[0]], [held[0]] * 2, d ** -0.5)
        ref.close(out[0], y, yb, "index rows")


def microseconds(f):
    f()
    torch.cuda.synchronize()
    best = math.inf
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, 1000 * a.elapsed_time(b))
    return best


@gpu
@pytest.mark.parametrize("what", ["prefill", "chunk", "decode", "index rows"])
def test_a_value_that_is_not_finite_costs_a_few_calls_not_hundreds(what):
    """An overflowed value at a sequence's start stands in every later row.  The bound of 20 calls' time is far from
    both sides: 2 to 4 with the values looked at once, 60 to 900 with every row walked key by key."""
    held, new, Hq, Hk, d, page = {"prefill": ([0], [3000], 8, 8, 64, 64), "chunk": ([6000], [300], 16, 4, 128, 64),
                                  "decode": ([8000] * 16, [1] * 16, 32, 8, 128, 16),
                                  "index rows": ([2500] * 16, [2] * 16, 16, 16, 128, 16)}[what]
    c = ref.Cache(held, new, Hk, d, page, seed=54)
    q = normal((sum(new), Hq, d), 55)
    if what == "index rows":
        idx = torch.arange(2048, dtype=torch.int32, device="cuda").expand(16, 2, 16, 2048).contiguous()
        call = lambda: qg.sparse_attention_paged(q.view(16, 2, 16, 128), c.kpages, c.vpages, c.table, c.seqlens, idx)  # noqa: E731
    else:
        call = lambda: qg.paged_attention(q, c.kpages, c.vpages, c.table, c.seqlens, c.longest, cu_q=c.cu)  # noqa: E731
    plain = microseconds(call)
    for row in (0, max(new) - 1):                    # seen by all, or by some after it
        for b in range(len(held)):
            c.vpages[int(c.table[b, row // page]), row % page, :, 5 + row % 7] = (math.inf, math.nan)[row % 2]
        assert not bool(torch.isfinite(call()).all())
        took = microseconds(call)
        print(f"{what}: {plain:.0f} us, {took:.0f} with row {row} not finite")
        assert took < 20 * plain, (plain, took)


# ------------------------------------------------------------------ waits that run out
@gpu
@pytest.mark.parametrize("page", [2, 16])        # rows copied one by one, and by TMA
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [1, 90])           # parts of two key tiles; rings that are filled more than once
def test_attention_gives_up_under_a_limit_of_a_nanosecond(B, d, page):
    """Under a limit that no wait for memory or for the products keeps, a call gives up and says so, and leaves the device
    as it was: the next call is exact."""
    c = ref.Cache([9000 if B == 1 else 1500] * B, [64] * B, 2, d, page, seed=58)
    q = normal((64 * B, 4, d), 59)
    want, lse = attend(c, q, True, True)
    assert status()[0] == 0
    lib = qg.load_library()
    told = 0
    try:
        lib.pivot_set_wait_limit(1)
        for _ in range(20):
            attend(c, q, True, True)
            flags, message = status()
            assert flags in (0, qg.FLAG_TIMEOUT) and ("timed out" in message) == (flags != 0)
            told += flags != 0
    finally:
        lib.pivot_set_wait_limit(0)
    print(f"{told} of 20 calls gave up")
    assert told > 0
    again, lse2 = attend(c, q, True, True)
    assert status()[0] == 0
    assert same_bits(again, want) and same_bits(lse, lse2)

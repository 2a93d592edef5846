"""The serving step over a paged cache: norm and rotation of heads, the append
into pages, dense attention of new tokens, attention over index rows, and the
run of them around the indexer.  Plain 64-bit forms and the bounds that the
roundings allow are in paged_ref.py."""
import ctypes
import math
import os
import struct
import subprocess

import numpy as np
import pytest
import torch

import query_group_top_b200 as qg
from tests import paged_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# The C ABI's option structs, packed: pivot_heads_t (data, weight, token_stride, head_stride, heads), pivot_rope_t
# (freqs, amplitude, eps, rot_dim, layout), pivot_attend_t (scale, include_self).
PACK_HEADS = struct.Struct("@PPqqi4x").pack
PACK_ROPE = struct.Struct("@Pddii").pack
PACK_ATTEND = struct.Struct("@di4x").pack


# ------------------------------------------------------------------ without a GPU
@pytest.fixture(scope="module")
def lib():
    from query_group_top_b200 import build
    build.build()
    return qg.load_library()


def heads(p, n=2, ts=256, hs=128, w=None):
    return PACK_HEADS(p, w or 0, ts, hs, n)


@pytest.fixture()
def ptr():
    buf = ctypes.create_string_buffer(256)
    p = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16
    yield p
    del buf


def test_rope_arguments_are_refused_on_the_host(lib, ptr):
    rope = PACK_ROPE(ptr, 1.0, 1e-6, 128, 0)

    def call(q=heads(ptr), k=None, dtype=0, pos=ptr, rope=rope, T=4, d=128, oq=ptr, ok=None):
        return lib.pivot_qk_rope(q, k, dtype, pos,
                                 rope, T, d, oq, ok, None)

    assert call(q=None) == 1                                            # neither q nor k
    assert call(oq=None) == 1                                           # no output
    assert call(k=heads(ptr)) == 1                                      # k without an output
    assert call(dtype=3) == 1
    assert call(T=0) == 1
    assert call(d=96) == 2
    assert call(pos=None) == 1                                          # a rotation without positions
    assert call(q=heads(ptr, n=0)) == 1
    assert call(q=heads(ptr + 2)) == 1                                  # misaligned rows
    assert call(q=heads(ptr, ts=260)) == 1
    assert call(q=heads(ptr, hs=4)) == 1
    assert call(oq=ptr + 8) == 1
    for rot in (8, 24, 144, 0, -16):
        assert call(rope=PACK_ROPE(ptr, 1.0, 1e-6, rot, 0)) == 1, rot
    assert call(rope=PACK_ROPE(ptr, 1.0, 1e-6, 64, 2)) == 1              # no such layout
    assert b"layout" in lib.pivot_last_error()


def test_append_and_attention_arguments_are_refused_on_the_host(lib, ptr):
    rope = PACK_ROPE(ptr, 1.0, 1e-6, 128, 0)

    def append(k=heads(ptr), v=heads(ptr), q=None, T=4, B=2, d=128, g=2, n=8, page=16, mp=4, kp=ptr, vp=ptr, bt=ptr,
               sl=ptr, cu=None, oq=None):
        return lib.pivot_paged_append(k, v,
                                      q, 0, rope, bt, sl, cu, T, B, d, g, n, page, mp,
                                      kp, vp, oq, None)

    assert append(k=None) == 1
    assert append(kp=None) == 1 and append(vp=None) == 1
    assert append(v=heads(ptr, n=3)) == 1                               # other heads than k
    assert append(v=heads(ptr, w=ptr)) == 1                             # a weight for the values
    assert append(q=heads(ptr)) == 1                                    # queries without an output
    assert append(T=5) == 1                                             # T is not B * g
    assert append(page=24) == 1 and append(page=0) == 1
    assert append(n=0) == 1 and append(mp=0) == 1 and append(bt=None) == 1 and append(sl=None) == 1
    assert append(d=96) == 2

    def attend(q=ptr, kp=ptr, vp=ptr, bt=ptr, sl=ptr, cu=None, opt=None, T=4, B=2, Hq=4, Hk=2, d=128, g=2, n=8, page=16,
               mp=4, ms=64, out=None, ws=None, nb=0):
        out = ptr + 32 if out is None else out
        return lib.pivot_paged_attention(q, kp, vp, bt, sl, cu, opt, T, B, Hq, Hk, d, g,
                                         n, page, mp, ms, out, None, ws, nb, None)

    assert attend(q=None) == 1 and attend(out=0) == 1 and attend(kp=None) == 1 and attend(vp=None) == 1
    assert attend(q=ptr + 4) == 1
    assert attend(out=ptr + 32) == 2 if not torch.cuda.is_available() else True    # right otherwise: no device
    assert attend(out=ptr) == 1 and b"out must not be q" in lib.pivot_last_error()
    assert attend(Hq=3) == 1 and attend(Hk=0) == 1 and attend(Hq=1) == 1
    assert attend(d=80) == 2
    assert attend(T=3) == 1 and attend(g=0) == 1
    assert attend(ms=0) == 1 and attend(ms=1 << 30) == 1
    for s in (0.0, -1.0, math.nan, math.inf):
        assert attend(opt=PACK_ATTEND(s, 1)) == 1, s
    assert lib.pivot_sparse_attention_paged(ptr, ptr, ptr, ptr, ptr, None, 1, 1, 64, 1, 1, 1, 1, 1, ptr, None) == 1
    assert lib.pivot_sparse_attention_paged(ptr, ptr, ptr, ptr, ptr, ptr, 1, 1, 64, 1, 1, 1, 1, 0, ptr, None) == 1
    assert lib.pivot_sparse_attention_paged(ptr, ptr, ptr, ptr, ptr, ptr, 1, 1, 32, 1, 1, 1, 1, 1, ptr, None) == 2
    # the workspace is host arithmetic: parts of a long axis for few rows, none where the rows fill the device
    assert lib.pivot_paged_attention_workspace_size(2, 1, 16, 16, 128, 131072) >= 2 * 2 * 16 * 129 * 4
    assert lib.pivot_paged_attention_workspace_size(0, 1, 16, 16, 128, 131072) == 0


@pytest.fixture(scope="module")
def rows_lib(tmp_path_factory):
    """paged_rows.cuh, whose arithmetic is plain C++, compiled for the host."""
    d = tmp_path_factory.mktemp("rows")
    src = d / "rows.cpp"
    src.write_text('#include "paged_rows.cuh"\n#include <cstddef>\nusing namespace pivot;\n'
                   'extern "C" void span(const int* t, const int* sl, const int* cu, int B, int T, int g, int mp, int np, '
                   'int lg, int ml, int b, int* out) {\n'
                   '  PagedRows p{t, sl, cu, B, T, g, mp, np, lg, paged_max_len(mp, lg, ml)};\n'
                   '  NewSpan s = p.span(b); out[0] = s.tok0; out[1] = s.n; out[2] = s.len; out[3] = s.ok;\n'
                   '  out[4] = p.new_tokens(b);\n}\n'
                   'extern "C" long long row(const int* t, int mp, int np, int lg, int b, int r) {\n'
                   '  PagedRows p{t, nullptr, nullptr, 1, 1, 1, mp, np, lg, 1 << 30}; return p.row(b, r);\n}\n'
                   'extern "C" int seq_row(const int* t, int mp, int np, int lg, int b, int r) {\n'
                   '  PagedRows p{t, nullptr, nullptr, 1, 1, 1, mp, np, lg, 1 << 30}; return SequenceRows(p, b).row(r);\n}\n')
    so = d / "rows.so"
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I",
                           os.path.join(ROOT, "query_group_top_b200", "csrc"), "-o", str(so), str(src)])
    lib = ctypes.CDLL(str(so))
    lib.row.restype = ctypes.c_longlong
    return lib


def test_spans_and_pages_that_do_not_fit_are_refused(rows_lib):
    def span(sl, cu, T, g, mp, lg, ml, b):
        sl = (ctypes.c_int * len(sl))(*sl)
        c = None if cu is None else (ctypes.c_int * len(cu))(*cu)
        out = (ctypes.c_int * 5)()
        rows_lib.span(None, sl, c, len(sl), T, g, mp, 9, lg, ml, b, out)
        assert out[4] == out[1]
        return list(out)[:4]

    assert span([5, 7], None, 4, 2, 1, 4, 100, 1) == [2, 2, 7, 1]
    assert span([5, 1], None, 4, 2, 1, 4, 100, 1)[3] == 0                # fewer rows than new ones
    assert span([5, 17], None, 4, 2, 1, 4, 100, 1)[3] == 0               # more than the table covers
    assert span([5, 16], None, 4, 2, 1, 4, 100, 1)[3] == 1
    assert span([5, 16], None, 4, 2, 9, 4, 15, 1)[3] == 0                # more than max_seqlen
    assert span([5, -1], None, 4, 2, 1, 4, 100, 1)[3] == 0
    assert span([5, 9], [0, 3, 7], 7, 0, 1, 4, 100, 1) == [3, 4, 9, 1]
    assert span([5, 9], [0, 3, 8], 7, 0, 1, 4, 100, 1)[1::2] == [0, 0]   # offsets behind the tokens
    assert span([5, 9], [0, 3, 2], 7, 0, 1, 4, 100, 1)[1::2] == [0, 0]   # falling offsets
    assert span([5, 9], [0, -3, 2], 7, 0, 1, 4, 100, 1)[1::2] == [0, 0]
    assert span([5, 0], [0, 3, 3], 7, 0, 1, 4, 100, 1) == [3, 0, 0, 1]   # an empty sequence
    assert span([5, 9], [0, 2147483647, -2147483648], 7, 0, 1, 4, 100, 1)[1::2] == [0, 0]

    table = (ctypes.c_int * 6)(3, 8, -1, 9, 2147483647, 0)
    assert rows_lib.row(table, 3, 9, 4, 0, 0) == 48 and rows_lib.row(table, 3, 9, 4, 0, 31) == 8 * 16 + 15
    assert rows_lib.row(table, 3, 9, 4, 0, 32) == -1                     # page -1
    assert rows_lib.row(table, 3, 9, 4, 1, 0) == -1 and rows_lib.row(table, 3, 9, 4, 1, 16) == -1   # pages past the cache
    assert rows_lib.row(table, 3, 9, 4, 1, 47) == 15
    for b in range(2):
        for r in range(48):
            assert rows_lib.seq_row(table, 3, 9, 4, b, r) == rows_lib.row(table, 3, 9, 4, b, r)
    # a cache row behind 32 bits
    far = (ctypes.c_int * 1)(2000000000)
    assert rows_lib.row(far, 1, 2147483647, 8, 0, 255) == 2000000000 * 256 + 255


def test_option_structs_are_packed_as_the_header_lays_them_out(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include "pivot.h"\n#include <stdio.h>\n#include <string.h>\nint main(void) {\n'
                   '  pivot_heads_t h; pivot_rope_t r; pivot_attend_t a;\n'
                   '  memset(&h, 0, sizeof h); memset(&r, 0, sizeof r); memset(&a, 0, sizeof a);\n'
                   '  h.data = (void*)1; h.weight = (void*)2; h.token_stride = 3; h.head_stride = -4; h.heads = 5;\n'
                   '  r.freqs = (double*)6; r.amplitude = 0.5; r.eps = 0.25; r.rot_dim = 7; r.layout = 8;\n'
                   '  a.scale = 0.125; a.include_self = 9;\n'
                   '  fwrite(&h, sizeof h, 1, stdout); fwrite(&r, sizeof r, 1, stdout); fwrite(&a, sizeof a, 1, stdout);\n'
                   '  return 0;\n}\n')
    exe = tmp_path / "sizes"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)])
    want = PACK_HEADS(1, 2, 3, -4, 5) + PACK_ROPE(6, 0.5, 0.25, 7, 8) + PACK_ATTEND(0.125, 9)
    assert subprocess.check_output([str(exe)]) == want


def test_the_binding_refuses_what_is_no_cuda_tensor(lib):
    """Without a GPU: the compiled half of the binding loads, and tells by the package's own exception."""
    q = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    t, n = torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    pages = torch.zeros((1, 16, 4, 64), dtype=torch.bfloat16)
    for call in (lambda: qg.paged_attention(q, pages, pages, t, n, 16), lambda: qg.qk_rope(q, None, n, None),
                 lambda: qg.qk_rope(None, None, None, None), lambda: qg.paged_append(q, q, pages, pages, t, n),
                 lambda: qg.sparse_attention_paged(q, pages, pages, t, n, t), lambda: qg.paged_append(None, q, pages, pages, t, n),
                 lambda: qg.qk_rope(7, None, n, None), lambda: qg.paged_attention(q, pages, "pages", t, n, 16),
                 lambda: qg.paged_attention(q, pages, pages, t, n, "many")):
        with pytest.raises(qg.PivotError):
            call()


def test_rope_frequencies():
    rot, base = 64, 10000.0
    i = np.arange(rot // 2)
    plain = base ** (-2.0 * i / rot)
    f, a = qg.rope_frequencies(rot, base, device="cpu")
    assert f.dtype == torch.float64 and a == 1.0
    np.testing.assert_allclose(f.numpy(), plain, rtol=1e-15)
    np.testing.assert_allclose(qg.rope_frequencies(rot, base, "linear", 4.0, device="cpu")[0].numpy(), plain / 4, rtol=1e-15)
    f, a = qg.rope_frequencies(rot, base, "ntk", 8.0, device="cpu")
    assert f[0] == 1.0 and a == 1.0
    np.testing.assert_allclose(float(f[-1]), plain[-1] / 8, rtol=1e-12)
    f, a = qg.rope_frequencies(rot, base, "yarn", 8.0, original_length=4096, device="cpu")
    turns = 4096 * plain / (2 * math.pi)
    np.testing.assert_allclose(a, 0.1 * math.log(8) + 1)
    fast, slow = turns > 40, turns < 0.8        # a pair's width away from the ramp's ends
    assert fast.any() and slow.any()
    np.testing.assert_allclose(f.numpy()[fast], plain[fast], rtol=1e-15)
    np.testing.assert_allclose(f.numpy()[slow], plain[slow] / 8, rtol=1e-15)
    assert bool((f.diff() < 0).all()) and bool((f <= torch.tensor(plain) * (1 + 1e-15)).all())
    for bad in (dict(rot_dim=24), dict(rot_dim=0), dict(scaling="other"), dict(scaling="yarn"), dict(factor=0.5),
                dict(base=1.0)):
        with pytest.raises(qg.PivotError):
            qg.rope_frequencies(**{"rot_dim": 64, "device": "cpu", **bad})


# ------------------------------------------------------------------ norm and rotation
gpu = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def normal(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def same_bits(a, b):
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(a.contiguous().view(torch.int16 if a.element_size() == 2 else torch.int32),
                                                                     b.contiguous().view(torch.int16 if b.element_size() == 2 else torch.int32))


ROPE = [(T, Hq, Hk, d, rot, layout, norm, dtype)
        for T, Hq, Hk, d, rot, layout, norm, dtype in [
            (1, 1, 1, 128, 128, "half", False, "bf16"), (2, 16, 16, 128, 128, "half", True, "bf16"),
            (7, 3, 2, 64, 16, "interleaved", True, "fp32"), (33, 5, 1, 64, 48, "half", False, "fp16"),
            (129, 32, 8, 128, 64, "interleaved", True, "fp16"), (1000, 40, 8, 128, 96, "half", True, "fp32"),
            (4097, 1, 1, 64, 64, "half", True, "bf16"), (517, 7, 3, 128, 112, "interleaved", False, "bf16")]]


@gpu
@pytest.mark.parametrize("case", ROPE, ids=str)
def test_qk_rope(case):
    T, Hq, Hk, d, rot, layout, norm, dtype = case
    t = TYPES[dtype]
    q, k = normal((T, Hq, d), 1, t), normal((T, Hk, d), 2, t)
    qw, kw = ((1 + normal((d,), 3, torch.float32) * 0.3).to(t), (1 + normal((d,), 4, torch.float32) * 0.3).to(t)) if norm else (None, None)
    f, amp = qg.rope_frequencies(rot, scaling="yarn", factor=4.0, original_length=2048)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 77
    oq, ok = qg.qk_rope(q, k, pos, f, layout, amp, qw, kw, eps=1e-5)
    ref.close(oq, *ref.rope(q, qw, pos, f, layout, amp, 1e-5), "q")
    ref.close(ok, *ref.rope(k, kw, pos, f, layout, amp, 1e-5), "k")
    # one of the two alone, and with only one of the norms
    assert same_bits(qg.qk_rope(q, None, pos, f, layout, amp, qw, eps=1e-5)[0], oq)
    assert same_bits(qg.qk_rope(None, k, pos, f, layout, amp, None, kw, eps=1e-5)[1], ok)
    mixed = qg.qk_rope(q, k, pos, f, layout, amp, None, kw, eps=1e-5)
    ref.close(mixed[0], *ref.rope(q, None, pos, f, layout, amp, 1e-5), "q without a norm")
    assert same_bits(mixed[1], ok)


@gpu
def test_qk_rope_far_positions_and_negative_ones():
    """Angles of positions up to the type's ends: an fp32 product would be off by whole turns."""
    pos = torch.tensor([0, 1, 131071, 1000003, 16777217, 2**31 - 1, -1, -5000001], dtype=torch.int32, device="cuda")
    q = normal((8, 2, 128), 5)
    f, _ = qg.rope_frequencies(128)
    # one more error here than paged_ref counts: the fp64 angle in radians, |pos| f 2^-52 a side, below 2^-20
    for layout in ("half", "interleaved"):
        y, b = ref.rope(q, None, pos, f, layout, 1.0, 0.0)
        ref.close(qg.qk_rope(q, None, pos, f, layout)[0], y, b + 2.0 ** -20 * q.double().abs().amax(), layout)


@gpu
def test_qk_rope_views_and_in_place():
    """Slices of a fused projection are read where they are; bf16 inputs may take the result."""
    T, Hq, Hk, d = 37, 6, 2, 128
    fused = normal((T, (Hq + 2 * Hk) * d), 6)
    q, k = fused[:, :Hq * d].view(T, Hq, d), fused[:, Hq * d:(Hq + Hk) * d].view(T, Hk, d)
    f, _ = qg.rope_frequencies(128)
    pos = torch.randperm(T, device="cuda").to(torch.int32)
    oq, ok = qg.qk_rope(q, k, pos, f)
    wq, wk = qg.qk_rope(q.contiguous(), k.contiguous(), pos, f)
    assert same_bits(oq, wq) and same_bits(ok, wk)
    # heads outermost, and one token for all (stride 0)
    ht = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert same_bits(qg.qk_rope(ht, None, pos, f)[0], wq)
    one = q[:1].expand(T, Hq, d)
    assert same_bits(qg.qk_rope(one, None, pos, f)[0], qg.qk_rope(one.contiguous(), None, pos, f)[0])
    x = q.contiguous()
    got, _ = qg.qk_rope(x, None, pos, f, out_q=x)
    assert got is x and same_bits(x, wq)
    # [B, g, H, d] with one position a token
    q4 = normal((5, 3, 4, 64), 7)
    p4 = torch.arange(15, dtype=torch.int32, device="cuda").view(5, 3)
    f4, _ = qg.rope_frequencies(64)
    got = qg.qk_rope(q4, None, p4, f4)[0]
    assert same_bits(got.view(15, 4, 64), qg.qk_rope(q4.view(15, 4, 64), None, p4.view(-1), f4)[0])


@gpu
def test_qk_norm_alone_zero_rows_and_no_tokens():
    q = normal((9, 3, 64), 8)
    q[4] = 0
    w = (1 + normal((64,), 9, torch.float32)).to(torch.bfloat16)
    got = qg.qk_rope(q, None, None, None, q_weight=w, eps=1e-6)[0]
    ref.close(got, *ref.rope(q, w, None, None, "half", 1.0, 1e-6), "norm")
    assert bool((got[4] == 0).all())
    f, _ = qg.rope_frequencies(64)
    none = qg.qk_rope(q[:0], q[:0], torch.empty(0, dtype=torch.int32, device="cuda"), f)
    assert none[0].shape == none[1].shape == (0, 3, 64)
    # a NaN stays in its head
    q[2, 1, 5] = float("nan")
    got = qg.qk_rope(q, None, torch.arange(9, dtype=torch.int32, device="cuda"), f, q_weight=w)[0]
    assert bool(torch.isnan(got[2, 1]).all()) and int(torch.isnan(got).any(-1).sum()) == 1


# ------------------------------------------------------------------ append
APPEND = [  # held, new, H, Hq, d, page, rot, layout, norm, dtype, ragged
    ([5, 0, 31], [2, 2, 2], 2, 4, 128, 16, 128, "half", True, "bf16", False),
    ([0], [1], 1, 0, 64, 1, 64, "interleaved", False, "bf16", False),
    ([0, 100, 7, 15], [130, 1, 0, 17], 3, 6, 64, 8, 32, "half", False, "fp32", True),
    ([500, 3], [77, 300], 8, 8, 128, 256, 64, "interleaved", True, "fp16", True),
    (list(range(70)), [1 + i % 3 for i in range(70)], 2, 2, 64, 16, 64, "half", True, "bf16", True),
]


def appended(case, with_values=True):
    held, new, H, Hq, d, page, rot, layout, norm, dtype, ragged = case
    c = ref.Cache(held, new, H, d, page, seed=len(held) + page)
    t, T = TYPES[dtype], sum(new)
    k, v = normal((T, H, d), 11, t), normal((T, H, d), 12, t)
    q = normal((T, Hq, d), 13, t) if Hq else None
    kw, qw = ((1 + 0.3 * normal((d,), 14, torch.float32)).to(t), (1 + 0.3 * normal((d,), 15, torch.float32)).to(t)) if norm else (None, None)
    f, amp = qg.rope_frequencies(rot, scaling="linear", factor=2.0)
    shape = (lambda x: x) if ragged else (lambda x: None if x is None else x.view(len(held), new[0], *x.shape[1:]))
    kp, vp = c.kpages.clone(), c.vpages.clone() if with_values else None
    out = qg.paged_append(shape(k), shape(v) if with_values else None, kp, vp, c.table, c.seqlens,
                          cu_new=c.cu if ragged else None, freqs=f, layout=layout, amplitude=amp, k_weight=kw,
                          q=shape(q), q_weight=qw if Hq else None)
    assert qg.sync_status() == 0
    return c, k, v, q, kw, qw, f, amp, kp, vp, out


@gpu
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"B{len(c[0])}-page{c[5]}-{c[7]}-{c[9]}")
def test_paged_append(case):
    layout, Hq = case[7], case[3]
    c, k, v, q, kw, qw, f, amp, kp, vp, out = appended(case)
    pos = torch.cat([torch.arange(h, h + n) for h, n in zip(c.held, c.new)]).to(torch.int32).cuda()
    y, b = ref.rope(k, kw, pos, f, layout, amp, 1e-6)
    written = torch.zeros(kp.shape[:2], dtype=torch.bool, device="cuda")
    t = 0
    for s, (h, n) in enumerate(zip(c.held, c.new)):
        rows = torch.arange(h, h + n, device="cuda")
        pg, sl = c.table[s, rows // c.page].long(), rows % c.page
        ref.close(kp[pg, sl], y[t:t + n], b[t:t + n], f"keys of sequence {s}")
        assert torch.equal(vp[pg, sl], v[t:t + n].to(torch.bfloat16)), s
        written[pg, sl] = True
        t += n
    # every other row of the cache keeps its bits
    assert same_bits(kp[~written], c.kpages[~written]) and same_bits(vp[~written], c.vpages[~written])
    # the same rows as the pass without a cache gives, queries included
    f_ = dict(layout=layout, amplitude=amp)
    want = qg.qk_rope(q, k, pos, f, q_weight=qw if Hq else None, k_weight=kw, **f_)
    if Hq:
        assert same_bits(out.view(want[0].shape), want[0])
    got = torch.cat([kp[c.table[s, torch.arange(h, h + n, device="cuda") // c.page].long(),
                        torch.arange(h, h + n, device="cuda") % c.page] for s, (h, n) in enumerate(zip(c.held, c.new))])
    assert same_bits(got, want[1])
    # a cache of keys alone
    assert same_bits(appended(case, with_values=False)[8], kp)


@gpu
def test_paged_append_bad_pages_lengths_and_rows_behind():
    """A page outside the cache, a sequence longer than its table, lengths below the new tokens: left out, reported,
    and nothing else is touched; tokens behind the last sequence keep their rows."""
    H, d, page = 2, 64, 16
    held, new = [20, 3, 40, 9], [4, 4, 4, 4]
    c = ref.Cache(held, new, H, d, page, seed=3)
    k, v, q = normal((16, H, d), 21), normal((16, H, d), 22), normal((16, 3, d), 23)
    f, _ = qg.rope_frequencies(d)
    table, lens = c.table.clone(), c.seqlens.clone()
    table[0, 1] = c.kpages.shape[0]          # rows 16.. of sequence 0: past the cache
    table[1, 0] = -7
    lens[2] = table.shape[1] * page + 1      # longer than the table
    lens[3] = 3                              # fewer rows than new tokens
    for cu in (None, torch.tensor([0, 4, 8, 12, 16], dtype=torch.int32, device="cuda")):
        kp, vp, out = c.kpages.clone(), c.vpages.clone(), torch.full_like(q, 9.0)
        shape = (lambda x: x.view(4, 4, *x.shape[1:])) if cu is None else (lambda x: x)
        qg.paged_append(shape(k), shape(v), kp, vp, table, lens, cu_new=cu, freqs=f, q=shape(q), out_q=shape(out))
        with pytest.raises(qg.PivotError):
            qg.sync_status()
        assert qg.sync_status() == 0
        assert same_bits(kp, c.kpages) and same_bits(vp, c.vpages) and bool((out == 9).all())
    # tokens behind cu[B], and one empty sequence between
    cu = torch.tensor([0, 4, 4, 8, 12], dtype=torch.int32, device="cuda")
    lens = torch.tensor([24, 3, 44, 13], dtype=torch.int32, device="cuda")
    kp, vp, out = c.kpages.clone(), c.vpages.clone(), torch.full_like(q, 9.0)
    qg.paged_append(k, v, kp, vp, c.table, lens, cu_new=cu, freqs=f, q=q, out_q=out)
    assert qg.sync_status() == 0
    assert bool((out[12:] == 9).all()) and not bool((out[:12] == 9).all(-1).any())
    assert int((kp.view(torch.int16) != c.kpages.view(torch.int16)).any(-1).any(-1).sum()) == 12


# ------------------------------------------------------------------ dense attention over the pages
ATTEND = [  # held, new, Hq, Hk, d, page, itself, ragged
    ([0], [1], 1, 1, 64, 1, True, False),
    ([0], [1], 2, 1, 128, 16, False, False),                       # a query that sees nothing
    ([700, 20, 0, 255], [2, 2, 2, 2], 4, 4, 128, 16, True, False),
    ([130, 1], [3, 3], 10, 2, 64, 64, False, False),               # 15 packed rows
    ([300, 64], [5, 5], 7, 1, 128, 32, True, False),               # 35 packed rows
    ([0, 33, 500, 0], [70, 1, 0, 17], 6, 2, 64, 8, True, True),
    ([3, 0], [129, 257], 3, 3, 128, 128, False, True),
    ([1000], [200], 8, 1, 128, 16, True, True),
    ([0], [300], 2, 2, 64, 256, True, True),
    ([2500, 900], [1, 1], 16, 2, 128, 4, True, False),             # split along the keys, tiny pages
    ([0], [600], 4, 4, 128, 64, True, False),                      # several row tiles, causal inside one key tile
    ([40, 1], [256, 3], 3, 1, 64, 16, False, True),
    ([1500], [37], 8, 1, 128, 32, True, True),                     # matrix tiles, split along the keys
    ([5000, 0], [50, 33], 8, 2, 64, 512, True, True),
    ([127, 128, 129, 255, 256, 257], [1] * 6, 2, 1, 128, 128, True, True),
    ([90], [40], 5, 1, 64, 2, True, True),
    ([1300, 0], [41, 300], 4, 2, 128, 1, True, True),              # matrix tiles over pages of one row
    ([600], [77], 3, 3, 64, 4, False, False),
    (list(range(0, 80, 2)), [1 + i % 2 for i in range(40)], 2, 2, 64, 16, True, True),
]


def attend(c, q, itself, ragged, **kw):
    n, Hq, d = q.shape
    lse = torch.full((n, Hq), 7.0, dtype=torch.float32, device="cuda")
    shape = (lambda x: x) if ragged else (lambda x: x.view(len(c.new), c.new[0], *x.shape[1:]))
    out = qg.paged_attention(shape(q), c.kpages, c.vpages, c.table, c.seqlens, kw.pop("longest", c.longest),
                             cu_q=c.cu if ragged else None, include_self=itself, out_lse=shape(lse), **kw)
    return out.view(q.shape), lse


def check_attention(c, q, out, lse, itself, scale, what=""):
    t = 0
    for s, (h, n) in enumerate(zip(c.held, c.new)):
        lim = [h + i + (1 if itself else 0) for i in range(n)]
        y, z, yb, zb = ref.attention(q[t:t + n], c.k[s], c.v[s], lim, scale)
        ref.close(out[t:t + n], y, yb, f"{what} output of sequence {s}")
        seen = torch.tensor(lim, device="cuda") > 0
        assert bool(torch.isneginf(lse[t:t + n][~seen]).all())
        ref.close(lse[t:t + n][seen], z[seen], zb[seen], f"{what} lse of sequence {s}")
        t += n


@gpu
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"B{len(c[0])}-held{max(c[0])}-new{max(c[1])}-{c[2]}over{c[3]}-d{c[4]}-page{c[5]}")
def test_paged_attention(case):
    held, new, Hq, Hk, d, page, itself, ragged = case
    c = ref.Cache(held, new, Hk, d, page, seed=sum(held) + page)   # rows that no sequence holds are NaN
    q = normal((sum(new), Hq, d), 31)
    out, lse = attend(c, q, itself, ragged)
    assert qg.sync_status() == 0
    check_attention(c, q, out, lse, itself, d ** -0.5)
    again, lse2 = attend(c, q, itself, ragged)
    assert same_bits(out, again) and same_bits(lse, lse2)
    # a loose bound on the lengths, another scale
    out, lse = attend(c, q, itself, ragged, longest=100000, scale=0.31)
    assert qg.sync_status() == 0
    check_attention(c, q, out, lse, itself, 0.31, "scaled")


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,new", [(16, 2), (16, 40), (2, 40)])
def test_paged_attention_masked_values_may_be_anything(page, new, d):
    """A key or value that a query does not see leaves it alone, infinity and NaN included, also where both share a
    tile; the queries that see it take it."""
    H, held = 2, 60
    c = ref.Cache([held], [new], H, d, page, seed=5)
    q = normal((new, H, d), 41)
    clean, _ = attend(c, q, True, True)
    bad = new - 1                                   # the last new token's value and key
    row = held + bad
    pg, sl = int(c.table[0, row // page]), row % page
    for kind in (float("nan"), float("inf")):
        for pages in (c.vpages, c.kpages):
            keep = pages[pg, sl].clone()
            pages[pg, sl] = kind
            out, _ = attend(c, q, True, True)
            assert bool(torch.isfinite(out[:bad]).all())
            check_attention(c_sub(c, bad), q[:bad], out[:bad], qg_lse(c, q)[:bad], True, d ** -0.5, f"{kind}")
            assert not bool(torch.isfinite(out[bad]).all())
            pages[pg, sl] = keep
    assert same_bits(attend(c, q, True, True)[0], clean)


def c_sub(c, n):
    """The cache as its first n new tokens see it."""
    import copy
    s = copy.copy(c)
    s.new = [n]
    return s


def qg_lse(c, q):
    return attend(c, q, True, True)[1]


@gpu
def test_paged_attention_bad_lengths_pages_and_rows_behind():
    H, d, page = 2, 64, 16
    held, new = [30, 5, 50, 12], [3, 3, 3, 3]
    c = ref.Cache(held, new, H, d, page, seed=8)
    q = normal((14, H, d), 51)
    cu = c.cu
    lens = c.seqlens.clone()
    lens[1], lens[2] = 2, 10000
    for ragged in (True, False):
        n = 14 if ragged else 12
        out, lse = torch.full((n, H, d), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((n, H), 9.0, device="cuda")
        shape = (lambda x: x) if ragged else (lambda x: x.view(4, 3, *x.shape[1:]))
        qg.paged_attention(shape(q[:n]), c.kpages, c.vpages, c.table, lens, 10000, cu_q=cu if ragged else None,
                           out=shape(out), out_lse=shape(lse))
        with pytest.raises(qg.PivotError):
            qg.sync_status()
        assert bool((out[3:9] == 0).all()) and bool(torch.isneginf(lse[3:9]).all())   # skipped sequences
        assert bool((out[12:] == 9).all()) and bool((lse[12:] == 9).all())            # tokens of no sequence
        good, _ = attend(c, q[:12], True, True)
        assert qg.sync_status() == 0
        assert same_bits(out[:3], good[:3]) and same_bits(out[9:12], good[9:])
    # offsets that do not fit: told, and the sequences that do fit are right
    odd = cu.clone()
    odd[4] = 40
    out = torch.full((14, H, d), 9.0, dtype=torch.bfloat16, device="cuda")
    qg.paged_attention(q, c.kpages, c.vpages, c.table, c.seqlens, c.longest, cu_q=odd, out=out)
    with pytest.raises(qg.PivotError):
        qg.sync_status()
    assert same_bits(out[:9], good[:9]) and bool((out[9:] == 9).all())
    # a length that does not fit, of a sequence without new tokens
    odd, lens = torch.tensor([0, 3, 3, 6, 9], dtype=torch.int32, device="cuda"), c.seqlens.clone()
    lens[1], lens[2] = 100000, 53
    qg.paged_attention(q, c.kpages, c.vpages, c.table, lens, c.longest, cu_q=odd)
    with pytest.raises(qg.PivotError):
        qg.sync_status()
    # pages outside the cache are left out and reported
    t = c.table.clone()
    t[0, 0], t[3, 0] = -1, c.kpages.shape[0] + 5
    out = qg.paged_attention(q[:12], c.kpages, c.vpages, t, c.seqlens, c.longest, cu_q=cu)
    with pytest.raises(qg.PivotError):
        qg.sync_status()
    assert same_bits(out[3:9], good[3:9]) and bool(torch.isfinite(out).all())


@gpu
def test_paged_attention_many_sequences_one_long():
    """More sequences than a warp, chunks of one token next to one of many, and no new token in most."""
    for new in ([0] * 30 + [200] + [1] * 40 + [0] * 5 + [3], [1] * 3 + [0] * 126 + [5] + [i % 3 for i in range(200)] + [60],
                [30] * 2 + [17 + i % 5 for i in range(140)]):
        held = [i * 7 % 50 + 1 for i in range(len(new))]
        c = ref.Cache(held, new, 1, 64, 32, seed=9)
        q = normal((sum(new), 3, 64), 61)
        out, lse = attend(c, q, True, True)
        assert qg.sync_status() == 0
        check_attention(c, q, out, lse, True, 0.125)


@gpu
@pytest.mark.parametrize("held0", [40, 3000])
@pytest.mark.parametrize("page,d", [(16, 128), (1, 64)])
def test_paged_attention_chunks_among_single_tokens(page, d, held0):
    """A few rows a sequence on average, but some with many: those go to the matrix tiles, the others do not, whatever
    bound on the new tokens is given, and bad lengths among them are told."""
    new = [1] * 20 + [90] + [1] * 25 + [0, 2, 9, 1] + [1] * 84
    held = [(held0 + 37 * i) % (held0 + 50) for i in range(len(new))]
    c = ref.Cache(held, new, 1, d, page, seed=23)
    q = normal((sum(new), 3, d), 63)          # 693 packed rows, 5 a sequence
    out, lse = attend(c, q, True, True)
    assert qg.sync_status() == 0
    check_attention(c, q, out, lse, True, d ** -0.5)
    for bound in (1, 90, 4000):     # 1 is wrong: the choice of kernels follows it, the result does not
        got, lse2 = attend(c, q, True, True, max_q=bound)
        assert qg.sync_status() == 0
        check_attention(c, q, got, lse2, True, d ** -0.5, f"bound {bound}")
    lens = c.seqlens.clone()
    lens[20], lens[47] = 3, 1       # fewer rows than new tokens
    c.seqlens = lens
    bad, _ = attend(c, q, True, True)
    with pytest.raises(qg.PivotError):
        qg.sync_status()
    assert same_bits(bad[:20], out[:20]) and bool((bad[20:110] == 0).all()) and same_bits(bad[110:135], out[110:135])
    assert bool((bad[135:137] == 0).all()) and same_bits(bad[137:], out[137:])


@gpu
@pytest.mark.parametrize("page", [2, 16])
def test_paged_attention_waits_run_out_and_the_next_call_is_exact(page):
    """The waits of the matrix-tile kernels are bounded: under a limit of a nanosecond a call either gives up and says
    so (a wait that is over at its first look does not) or is right, and leaves the device as it was."""
    c = ref.Cache([9000], [64], 2, 128, page, seed=17)
    q = normal((64, 4, 128), 65)
    want, lse = attend(c, q, True, True)
    assert qg.sync_status() == 0
    lib = qg.load_library()
    told = 0
    try:
        lib.pivot_set_wait_limit(1)
        for _ in range(20):
            out, _ = attend(c, q, True, True)
            try:
                assert qg.sync_status() == 0
                assert same_bits(out, want)
            except qg.PivotError as e:
                assert "timed out" in str(e)
                told += 1
    finally:
        lib.pivot_set_wait_limit(0)
    again, lse2 = attend(c, q, True, True)
    assert qg.sync_status() == 0
    assert same_bits(again, want) and same_bits(lse, lse2)
    print(f"{told} of 20 calls gave up")


@gpu
@pytest.mark.parametrize("page", [1, 16])
def test_rows_behind_two_to_the_thirty_one_elements(page):
    """A cache whose last pages lie behind 2^31 elements (2^32 bytes): append, both attentions and the index rows
    address them."""
    H, d, held, g = 4, 128, 300, 2
    near = ref.Cache([held], [g], H, d, page, seed=19, fill=0.0)
    total = (1 << 31) // (page * H * d) + 64 + near.kpages.shape[0]
    kp = torch.empty((total, page, H, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    shift = total - near.kpages.shape[0]
    kp[shift:], vp[shift:] = near.kpages, near.vpages
    table = torch.where(near.table >= 0, near.table + shift, near.table)
    f, _ = qg.rope_frequencies(d)
    k, v = normal((1, g, H, d), 66), normal((1, g, H, d), 67)
    qg.paged_append(k, v, kp, vp, table, near.seqlens, freqs=f)
    qg.paged_append(k, v, near.kpages, near.vpages, near.table, near.seqlens, freqs=f)
    assert same_bits(kp[shift:], near.kpages) and same_bits(vp[shift:], near.vpages)
    q = normal((1, g, H, d), 68)
    idx = torch.arange(250, dtype=torch.int32, device="cuda").expand(1, g, H, 250).contiguous()
    for call in (lambda a, b, t: qg.paged_attention(q, a, b, t, near.seqlens, held + g),
                 lambda a, b, t: qg.paged_attention(normal((1, g, 32 * H, d), 69), a, b, t, near.seqlens, held + g),
                 lambda a, b, t: qg.sparse_attention_paged(q, a, b, t, near.seqlens, idx)):
        assert same_bits(call(kp, vp, table), call(near.kpages, near.vpages, near.table))
    assert qg.sync_status() == 0


# ------------------------------------------------------------------ attention over index rows
@gpu
@pytest.mark.parametrize("page", [1, 16, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_sparse_attention_paged_equals_packed(d, page):
    held, g, H, top_k = [300, 3, 77], 3, 2, 50
    c = ref.Cache(held, [g] * 3, H, d, page, seed=page)
    q = normal((3, g, H, d), 71)
    rng = np.random.default_rng(d)
    idx = -np.ones((3, g, H, top_k), np.int32)
    for b in range(3):
        for i in range(g):
            for h in range(H):
                n = int(rng.integers(0, min(top_k, held[b] + i) + 1))
                idx[b, i, h, :n] = np.sort(rng.choice(held[b] + i, size=n, replace=False))
    idx[0, 0, 0] = -1
    idx = torch.from_numpy(idx).cuda()
    got = qg.sparse_attention_paged(q, c.kpages, c.vpages, c.table, c.seqlens, idx)
    assert qg.sync_status() == 0
    rows = torch.tensor([0] + c.lens).cumsum(0).to(torch.int32).cuda()
    want = qg.sparse_attention(q, torch.cat(c.k), torch.cat(c.v), idx, cu_seqlens=rows, g=g)
    assert bool((got[0, 0, 0] == 0).all())
    for b in range(3):
        for i in range(g):
            for h in range(H):
                j = idx[b, i, h][idx[b, i, h] >= 0].long()
                if j.numel() == 0:
                    assert bool((got[b, i, h] == 0).all())
                    continue
                x = c.k[b][j, h].double() @ q[b, i, h].double() * d ** -0.5
                y = torch.softmax(x, 0) @ c.v[b][j, h].double()
                # fp32 sums over at most 50 keys and 128 channels: d FP32 on scores of a few units, well below 1e-5
                assert float((got[b, i, h].double() - y).abs().max()) <= 1e-5
    ref.close(got, want.double(), torch.full_like(want.double(), 2e-5), "packed")
    # an index outside its sequence, a page outside the cache: left out and reported
    bad = idx.clone()
    bad[1, 0, 0, 0] = c.lens[1]
    bad[1, 0, 0, 1:] = -1
    out = qg.sparse_attention_paged(q, c.kpages, c.vpages, c.table, c.seqlens, bad)
    with pytest.raises(qg.PivotError):
        qg.sync_status()
    assert bool((out[1, 0, 0] == 0).all()) and bool(torch.isfinite(out).all())
    t = c.table.clone()
    t[2] = c.kpages.shape[0]
    out = qg.sparse_attention_paged(q, c.kpages, c.vpages, t, c.seqlens, idx)
    with pytest.raises(qg.PivotError):
        qg.sync_status()
    assert bool((out[2] == 0).all()) and same_bits(out[:2], got[:2])


def check_index_rows(c, q, idx, out, what):
    """Against the definition in 64 bits, every entry as it stands: twice where it stands twice."""
    d = q.shape[-1]
    for b in range(q.shape[0]):
        for i in range(q.shape[1]):
            for h in range(q.shape[2]):
                j = idx[b, i, h][idx[b, i, h] >= 0].long()
                if j.numel() == 0:
                    assert bool((out[b, i, h] == 0).all())
                    continue
                x = c.k[b][j, h].double() @ q[b, i, h].double() * d ** -0.5
                y = torch.softmax(x, 0) @ c.v[b][j, h].double()
                # scores of a few units by fp32 sums of d products, weights and sums in fp32: below 2e-5 of values of a
                # few units
                far = float((out[b, i, h].double() - y).abs().max())
                assert far <= 2e-5, f"{what}: sequence {b}, member {i}, head {h}: {far}"


@gpu
@pytest.mark.parametrize("g", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("d", [64, 128])
def test_sparse_attention_paged_rows_of_every_kind(d, g):
    """Members that share all, some or none of their rows; rows of very different lengths; rows that are not ascending,
    hold an index twice or padding between; few rows (a cluster each) and many."""
    rng = np.random.default_rng(10 * g + d)
    for B, H, top_k, held in ((2, 2, 700, [900, 64]), (3, 1, 65, [70, 300, 1]), (40, 4, 64, [100 + i for i in range(40)])):
        c = ref.Cache(held, [g] * B, H, d, 16, seed=g)
        q = normal((B, g, H, d), 72)
        idx = -np.ones((B, g, H, top_k), np.int32)
        for b in range(B):
            for h in range(H):
                pool = rng.permutation(held[b])
                kind = rng.integers(0, 6)
                for i in range(g):
                    n = int(rng.integers(0, min(top_k, held[b]) + 1)) if rng.random() < 0.5 else min(top_k, held[b])
                    row = np.sort(pool[:n]) if kind == 0 else np.sort(rng.choice(held[b], n, replace=False))
                    if kind == 1 and i % 2:
                        row = row[:3]
                    if kind == 2 and i == 0:
                        row = rng.permutation(row)
                    if kind == 3 and len(row) > 4:
                        row[2] = row[3]
                    if kind == 4 and len(row) > 4:
                        row[1] = -1
                    if kind == 5 and i % 2:
                        row = row + 0 if i % 4 == 1 else row[:0]
                    idx[b, i, h, :len(row)] = row
        idx = torch.from_numpy(idx).cuda()
        out = qg.sparse_attention_paged(q, c.kpages, c.vpages, c.table, c.seqlens, idx)
        assert qg.sync_status() == 0
        check_index_rows(c, q, idx, out, f"B={B}")
        assert same_bits(out, qg.sparse_attention_paged(q, c.kpages, c.vpages, c.table, c.seqlens, idx))


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,top_k", [(1, 40), (60, 90)])
def test_sparse_attention_paged_takes_infinite_values_as_they_are(d, B, top_k):
    """A selected value that is infinite or NaN comes out as the definition has it, channel by channel (a cluster a
    row, and one CTA); a key that is NaN makes its queries NaN; rows that select neither are untouched."""
    H = 12
    c = ref.Cache([120] * B, [1] * B, H, d, 16, seed=21)
    q = normal((B, 1, H, d), 91)
    idx = torch.arange(top_k, dtype=torch.int32, device="cuda").expand(B, 1, H, top_k).contiguous()
    idx[:, :, 1] += 9                                # leaves out rows 0 to 8
    clean = qg.sparse_attention_paged(q, c.kpages, c.vpages, c.table, c.seqlens, idx)
    pg = int(c.table[0, 0])
    c.vpages[pg, 5, 0, 3:6] = torch.tensor([math.inf, -math.inf, math.nan], device="cuda")
    c.vpages[pg, 5, 1, :] = math.nan                 # not selected
    c.kpages[pg, 7, 2, 0] = math.nan
    out = qg.sparse_attention_paged(q, c.kpages, c.vpages, c.table, c.seqlens, idx)
    assert qg.sync_status() == 0
    want = clean.clone()
    want[0, 0, 0, 3:6] = torch.tensor([math.inf, -math.inf, math.nan], device="cuda")
    want[0, 0, 2] = math.nan
    whole = torch.isfinite(want)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(out[torch.isinf(want)], want[torch.isinf(want)])
    ref.close(out[whole], want[whole].double(), torch.full_like(want[whole].double(), 2e-5), "the finite ones")


@gpu
@pytest.mark.parametrize("new", [1, 40])
def test_paged_attention_infinite_values_beside_a_page_that_is_not_there(new):
    """A page outside the cache reads as zeros also in a row that is worked out key by key."""
    H, d, page, held = 2, 64, 16, 70
    c = ref.Cache([held], [new], H, d, page, seed=22)
    q = normal((new, H, d), 92)
    t = c.table.clone()
    t[0, 1] = -1
    pg = int(c.table[0, 0])
    c.vpages[pg, 3, 0, 7] = math.inf
    out = qg.paged_attention(q, c.kpages, c.vpages, t, c.seqlens, c.longest, cu_q=c.cu)
    with pytest.raises(qg.PivotError):
        qg.sync_status()
    k, v = c.k[0].clone(), c.v[0].clone()
    k[page:2 * page] = 0
    v[page:2 * page] = 0
    lim = torch.arange(held + 1, held + new + 1)
    want, _, bound, _ = ref.attention(q, k, v, lim, d ** -0.5)
    assert bool((out[:, 0, 7] == math.inf).all())
    out[:, 0, 7], want[:, 0, 7] = 0, 0
    ref.close(out, want, bound, "the other channels")


@gpu
def test_attention_without_values_or_with_lengths_past_its_range_is_refused():
    c = ref.Cache([30, 5], [2, 2], 2, 64, 16, seed=1)
    q = normal((2, 2, 2, 64), 1)
    idx = torch.zeros((2, 2, 2, 3), dtype=torch.int32, device="cuda")
    for m in (1 << 30, (1 << 32) + 64, -1):
        with pytest.raises(qg.PivotError):
            qg.paged_attention(q, c.kpages, c.vpages, c.table, c.seqlens, m)
    with pytest.raises(qg.PivotError):
        qg.paged_attention(q, c.kpages, None, c.table, c.seqlens, c.longest)
    with pytest.raises(qg.PivotError):
        qg.sparse_attention_paged(q, c.kpages, None, c.table, c.seqlens, idx)
    with pytest.raises(qg.PivotError):
        qg.paged_attention(q, None, None, c.table, c.seqlens, c.longest)


# ------------------------------------------------------------------ together
def step(c, qkv, Hq, H, d, g, freqs, top_k, Kc):
    """One decode step as a serving loop makes it: append, index, attend over the rows and densely."""
    B = len(c.held)
    q, k, v = (x.view(B, g, -1, d) for x in qkv.split([Hq * d, H * d, H * d], dim=-1))
    q = qg.paged_append(k, v, c.kpages, c.vpages, c.table, c.seqlens, freqs=freqs, q=q)
    idx = qg.pivot_decode_index_paged(q, c.kpages, c.table, c.seqlens, g, top_k, Kc, max_seqlen=c.longest)
    o = qg.sparse_attention_paged(q, c.kpages, c.vpages, c.table, c.seqlens, idx)
    dense = qg.paged_attention(q, c.kpages, c.vpages, c.table, c.seqlens, c.longest, include_self=False)
    return q, idx, o, dense


@gpu
def test_a_decode_step_of_them_together():
    """append -> index -> both attentions.  Where top_k covers every key the index rows are all of them, so the
    attention over the rows is the dense one (strictly before each query)."""
    B, g, H, d, page = 4, 2, 2, 64, 16
    c = ref.Cache([90, 17, 250, 64], [g] * B, H, d, page, seed=13, fill=0.0)
    f, _ = qg.rope_frequencies(d)
    qkv = normal((B, g, 3 * H * d), 81)
    q, idx, o, dense = step(c, qkv, H, H, d, g, f, 256, 512)
    assert qg.sync_status() & ~qg.FLAG_FALLBACK == 0
    pos = torch.tensor([[h + i for i in range(g)] for h in c.held], dtype=torch.int32, device="cuda")
    qv, kv, vv = (x.reshape(B, g, H, d) for x in qkv.split([H * d] * 3, dim=-1))
    wq, wk = qg.qk_rope(qv, kv, pos, f)
    assert same_bits(q, wq)
    for b, h in enumerate(c.held):
        k = torch.cat([c.k[b][:h], wk[b]])
        v = torch.cat([c.v[b][:h], vv[b]])
        lim = [h + i for i in range(g)]
        y, _, yb, _ = ref.attention(q[b], k, v, lim, d ** -0.5)
        ref.close(dense[b], y, yb, f"dense {b}")
        for i in range(g):
            assert idx[b, i, 0][:lim[i]].tolist() == list(range(min(lim[i], 256)))
        assert float((o[b].double() - y).abs().max()) <= 1e-4


@gpu
def test_captured_steps_replay_on_new_inputs_and_side_by_side():
    """Two graphs of the step, captured apart and replayed in turn and on two streams at once, each on new inputs put
    into its buffers: what they leave equals the eager step's.  (The indexer's workspace belongs to the stream that it
    was captured on, so the graphs hold the calls around it.)"""
    B, g, H, d, page = 3, 2, 4, 128, 16
    f, _ = qg.rope_frequencies(d)
    made = []
    for n in range(2):
        c = ref.Cache([1500 + n, 40, 333], [g] * B, H, d, page, seed=20 + n, fill=0.0)
        qkv = normal((B, g, 3 * H * d), 90 + n)
        idx = torch.arange(30, dtype=torch.int32, device="cuda").expand(B, g, H, 30).contiguous()

        def calls(c=c, qkv=qkv, idx=idx):
            q, k, v = (x.view(B, g, H, d) for x in qkv.split([H * d] * 3, dim=-1))
            q = qg.paged_append(k, v, c.kpages, c.vpages, c.table, c.seqlens, freqs=f, q=q)
            return (q, qg.paged_attention(q, c.kpages, c.vpages, c.table, c.seqlens, c.longest),
                    qg.sparse_attention_paged(q, c.kpages, c.vpages, c.table, c.seqlens, idx))

        calls()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = calls()
        made.append((c, qkv, calls, graph, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(3):
        want = []
        for n, (c, qkv, calls, graph, out) in enumerate(made):
            qkv.copy_(normal(qkv.shape, 100 + 10 * turn + n))
            want.append([x.clone() for x in calls()])
            for x in out:
                x.fill_(3.0)
        torch.cuda.synchronize()
        for n, (c, qkv, calls, graph, out) in enumerate(made):
            with torch.cuda.stream(streams[n]):
                graph.replay()
        torch.cuda.synchronize()
        for n in range(2):
            for x, y in zip(made[n][4], want[n]):
                assert same_bits(x, y), (turn, n)
    assert qg.sync_status() == 0


@gpu
def test_calls_on_a_given_stream():
    """stream=: the work, and what it allocates, belong to that stream, while the current one is busy or idle."""
    c = ref.Cache([900, 64], [2, 2], 2, 128, 16, seed=33)
    q = normal((4, 4, 128), 95)
    want, _ = attend(c, q, True, False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        junk = torch.full((4, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        outs.append(qg.paged_attention(q.view(2, 2, 4, 128), c.kpages, c.vpages, c.table, c.seqlens, c.longest, stream=s))
        del junk
    f, _ = qg.rope_frequencies(128)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    turned = qg.qk_rope(q, None, pos, f, stream=s)[0]
    s.synchronize()
    for o in outs:
        assert same_bits(o.view(4, 4, 128), want)
    assert same_bits(turned, qg.qk_rope(q, None, pos, f)[0])


@gpu
def test_calls_from_several_threads_at_once():
    """Host threads, each with a stream of its own, over one cache (the calls release the interpreter's lock)."""
    import threading
    H, d, g, page = 4, 128, 2, 16
    c = ref.Cache([900, 64, 333], [g] * 3, H, d, page, seed=31)
    f, _ = qg.rope_frequencies(d)
    pos = torch.arange(3 * g, dtype=torch.int32, device="cuda")
    idx = torch.arange(60, dtype=torch.int32, device="cuda").expand(3, g, H, 60).contiguous()
    qs = [normal((3, g, 2 * H, d), 200 + i) for i in range(4)]

    def calls(q):
        t, _ = qg.qk_rope(q, None, pos, f)
        return (t, qg.paged_attention(t, c.kpages, c.vpages, c.table, c.seqlens, c.longest),
                qg.sparse_attention_paged(t[:, :, :H].contiguous(), c.kpages, c.vpages, c.table, c.seqlens, idx))

    want = [calls(q) for q in qs]
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    got = calls(qs[i])
                    torch.cuda.current_stream().synchronize()
                    if not all(same_bits(a, b) for a, b in zip(got, want[i])):
                        wrong.append(i)
        except Exception as e:       # told by the test below, not lost with the thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(qs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and not wrong
    assert qg.sync_status() == 0


@gpu
def test_the_binding_refuses():
    c = ref.Cache([30, 5], [2, 2], 2, 64, 16, seed=1)
    q, f = normal((2, 2, 4, 64), 1), qg.rope_frequencies(64)[0]
    k = normal((2, 2, 2, 64), 2)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")

    def no(call):
        with pytest.raises(qg.PivotError):
            call()

    A = lambda q=q, kp=c.kpages, vp=c.vpages, t=c.table, s=c.seqlens, m=c.longest, **kw: qg.paged_attention(q, kp, vp, t, s, m, **kw)  # noqa: E731
    no(lambda: A(q=q.float()))
    no(lambda: A(q=q.cpu()))
    no(lambda: A(q=q[:, :, :3]))                                   # not a multiple, nor contiguous
    no(lambda: A(q=q[:, :, :3].contiguous()))
    no(lambda: A(q=q.transpose(0, 1)))
    no(lambda: A(q=q.view(4, 4, 64)))                              # [T, H, d] without cu_q
    no(lambda: A(cu_q=c.cu))                                       # [B, g, H, d] with it
    no(lambda: A(q=q.view(4, 4, 64), cu_q=c.cu[:2]))
    no(lambda: A(q=q.view(4, 4, 64), cu_q=c.cu.long()))
    no(lambda: A(t=c.table.long()))
    no(lambda: A(t=c.table[:1]))
    no(lambda: A(s=c.seqlens.cpu()))
    no(lambda: A(kp=c.kpages[:, :12]))
    no(lambda: A(kp=c.kpages[:, :12].contiguous(), vp=c.vpages[:, :12].contiguous()))
    no(lambda: A(vp=c.vpages[:-1]))
    no(lambda: A(m=0))
    no(lambda: A(q=q.view(4, 4, 64), cu_q=c.cu, max_q=0))
    no(lambda: A(scale=0.0))
    no(lambda: A(out=torch.empty_like(q.float())))
    no(lambda: A(out=q))
    no(lambda: A(out_lse=torch.empty((4, 4), device="cuda")))
    P = lambda k=k, v=k, kp=c.kpages, vp=c.vpages, **kw: qg.paged_append(k, v, kp, vp, c.table, c.seqlens, **{"freqs": f, **kw})  # noqa: E731
    no(lambda: P(v=None))
    no(lambda: P(vp=None))
    no(lambda: P(k=k.float()))                                     # v of another type
    no(lambda: P(k=normal((2, 2, 3, 64), 1), v=normal((2, 2, 3, 64), 1)))
    no(lambda: P(q_weight=k[0, 0, 0]))
    no(lambda: P(out_q=q))
    no(lambda: P(q=q[:1]))
    no(lambda: P(layout="other"))
    no(lambda: P(freqs=f.float()))
    no(lambda: P(freqs=f[:4]))
    no(lambda: P(k=normal((2, 2, 2, 68), 1)[..., :64], v=normal((2, 2, 2, 68), 1)[..., :64]))    # rows off 16 bytes
    no(lambda: P(k=normal((2, 2, 2, 128), 1)[..., ::2], v=normal((2, 2, 2, 128), 1)[..., ::2]))  # channels apart
    no(lambda: P(eps=-1.0))
    R = lambda q=q, k=None, pos=pos, **kw: qg.qk_rope(q, k, pos, f, **kw)  # noqa: E731
    no(lambda: R(q=None))
    no(lambda: R(pos=None))
    no(lambda: R(pos=pos[:3]))
    no(lambda: R(pos=pos.long()))
    no(lambda: R(k_weight=pos))
    no(lambda: R(q_weight=torch.ones(64, device="cuda")))          # fp32 weight of bf16 heads
    no(lambda: R(q=normal((2, 2, 4, 96), 1)))
    no(lambda: R(k=k[:1]))
    no(lambda: qg.sparse_attention_paged(q, c.kpages, c.vpages, c.table, c.seqlens, pos))
    no(lambda: qg.sparse_attention_paged(q, c.kpages, c.vpages, c.table, c.seqlens, torch.zeros((2, 2, 4, 3), dtype=torch.int32, device="cuda")))
    assert qg.sync_status() == 0

// Dense causal attention of a chunk of new tokens over a paged cache.
//
// New token i of sequence b sits at row pos = seqlens[b] - n_b + i of its
// sequence and sees the keys j < lim, lim = pos + 1 (or pos, where a query
// leaves its own key out, as the indexer does).  For query head h, whose keys
// and values are head h / (Hq / Hk) of the cache:
//     o = sum_{j < lim} softmax_j(scale q . k_j) v_j,   lse = log sum_j exp(scale q . k_j)
// and zeros with lse = -inf where lim = 0.  One pass over the keys with the
// running maximum m and sum l of the softmax (in units of log2) in fp32:
//     m' = max(m, max s),  l <- l 2^(m-m') + sum 2^(s-m'),  o <- o 2^(m-m') + 2^(s-m') v.
//
// The query heads of one key head are packed as rows (row r is token r / grp,
// head r % grp of the group), so one read of a key serves them all.  A long
// axis is split: each CTA takes chunk_of(len) keys, and attend_join_kernel adds up
// the parts, o = sum_c w_c o_c, w_c = exp(lse_c - lse).
//
// attend_rows_kernel is the form for few rows per key head (decode): 16 rows
// (one m16n8k16 tile), bound by the bytes of the keys and values.  Each of its
// four warps walks its own 16-key tiles of the chunk with a ring of its own
// (cp.async, no barrier between warps) and its own (m, l, o), which are merged
// at the end: nothing waits for anything but memory.
#pragma once

#include "paged_rows.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace pivot {

struct PagedAttendParams {
  const uint16_t* q;       // [T][Hq][d] bf16
  const uint16_t* kpages;  // [pages][page_size][Hk][d] bf16
  const uint16_t* vpages;
  PagedRows rows;
  int Hq, Hk, grp;         // grp = Hq / Hk
  int self_key;            // 1: a query sees its own key
  int nsplit, min_chunk;   // CTAs along the keys of each row tile; the fewest keys that a part is worth
  int tiles;               // row tiles over all sequences (an upper bound where cu is given)
  float scale_log2;        // scale * log2(e)
  uint16_t* out;           // [T][Hq][d] bf16
  float* lse;              // [T][Hq] natural log, or null
  float* part_o;           // nsplit > 1: [nsplit][T][Hq][d], each part normalised
  float* part_lse;         // nsplit > 1: [nsplit][T][Hq], log2 units
  int* status;
  unsigned long long wait_ns;
};

constexpr float kLn2 = 0.693147180559945309f;

// Keys per part of a sequence of `len` rows: an nsplit-th of it, whatever the
// bound that sized the grid, in whole 128-key tiles, and no less than min_chunk.
__device__ __forceinline__ int chunk_of(int len, const PagedAttendParams& p) {
  return max(p.min_chunk, ((len + p.nsplit - 1) / p.nsplit + 127) & ~127);
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The row tile `flat` of the batch: which sequence, and which of its tiles of
// `rows` packed rows.  One warp; without cu every sequence has the same number
// of tiles, else the sequences' tile counts are summed 32 at a time.  Returns
// -1 behind the last tile.
__device__ __forceinline__ int locate_tile(const PagedRows& p, int grp, int rows, int flat, int lane, int* tile,
                                           int* status) {
  if (!p.cu) {
    const int per = (p.g * grp + rows - 1) / rows;
    *tile = flat % per;
    return flat / per < p.B ? flat / per : -1;
  }
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    int n = 0;
    if (b < p.B) {
      const NewSpan sp = p.span(b);
      n = static_cast<int>((static_cast<long long>(sp.n) * grp + rows - 1) / rows);
      if (!sp.ok) atomicOr(status, kStBadLen);
    }
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + sum > flat);
    if (past) {
      const int l = __ffs(past) - 1;
      *tile = flat - (before + __shfl_sync(0xffffffffu, sum - n, l));
      return b0 + l;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return -1;
}

// One row over the keys [j0, j1) by a whole warp, key after key, reading only
// those keys: lane l holds channels [l * D/32, ...).  For rows whose tile gave
// a value that is not finite: there a masked position's infinity or NaN may
// have come in as 0 * inf, and here it does not.
template <int D>
__device__ __forceinline__ void attend_row_exact(const PagedAttendParams& p, int b, int hk, long long qrow, int j0,
                                              int j1, int lane, float (&o)[D / 32], float* lse2) {
  constexpr int C = D / 32;
  float q[C], m = neg_inf(), l = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    q[c] = __uint_as_float(static_cast<uint32_t>(p.q[qrow * D + lane * C + c]) << 16);
    o[c] = 0.f;
  }
  for (int j = j0; j < j1; ++j) {
    const long long row = p.rows.row(b, j);
    if (row < 0) continue;
    const long long at = (row * p.Hk + hk) * D + lane * C;
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) s = fmaf(q[c], __uint_as_float(static_cast<uint32_t>(p.kpages[at + c]) << 16), s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s);
    const float ms = mn == neg_inf() ? 0.f : mn;
    const float f = fast_exp2(m - ms), e = fast_exp2(s - ms);
    l = l * f + e;
#pragma unroll
    for (int c = 0; c < C; ++c)
      o[c] = fmaf(e, __uint_as_float(static_cast<uint32_t>(p.vpages[at + c]) << 16), o[c] * f);
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] *= inv;
  *lse2 = l == 0.f ? neg_inf() : m + log2f(l);
}

// ------------------------------------------------------------------ few rows
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_m16n8k16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
struct RowsCfg {
  static constexpr int NW = 4;                          // warps, each with keys of its own
  static constexpr int KT = 16;                         // keys a warp's step
  static constexpr int ST = D == 128 ? 3 : 6;           // steps in flight per warp
  static constexpr int TILE = KT * D * 2;               // bytes of a step's keys (its values as many)
  static constexpr int RING = NW * ST * 2 * TILE;
  static constexpr int MERGE = NW * 16 * (D + 4) * 4;   // the warps' (o, m, l) at the end, in the ring's place
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;
};

template <int D>
__global__ void __launch_bounds__(128) attend_rows_kernel(const __grid_constant__ PagedAttendParams p) {
  using C = RowsCfg<D>;
  constexpr int KS = D / 16;       // k-steps of q . k
  constexpr int CH = D / 8;        // 16-byte pieces of a row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int seq_s[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // key heads in the innermost place: neighbouring CTAs read neighbouring heads of the same rows
  const long long bid = blockIdx.x;
  const int hk = static_cast<int>(bid % p.Hk);
  const int split = static_cast<int>(bid / p.Hk % p.nsplit);
  const int flat = static_cast<int>(bid / p.Hk / p.nsplit);
  if (warp == 0) {
    int tile = 0;
    const int b = locate_tile(p.rows, p.grp, 16, flat, lane, &tile, p.status);
    if (lane == 0) seq_s[0] = b, seq_s[1] = tile;
  }
  __syncthreads();
  const int b = seq_s[0], r0 = seq_s[1] * 16;
  if (b < 0) return;
  const NewSpan sp = p.rows.span(b);
  const int nrows = min(16, sp.n * p.grp - r0);
  if (nrows <= 0) return;
  const int pos0 = sp.len - sp.n + p.self_key;             // lim of the sequence's first new token
  auto lim_of = [&](int r) { return sp.ok ? pos0 + (r0 + r) / p.grp : 0; };
  auto row_of = [&](int r) {
    return (static_cast<long long>(sp.tok0) + (r0 + r) / p.grp) * p.Hq + hk * p.grp + (r0 + r) % p.grp;
  };
  if (!sp.ok && threadIdx.x == 0) atomicOr(p.status, kStBadLen);
  const int chunk = chunk_of(sp.len, p);
  const int kbeg = split * chunk;
  const int kend = min(lim_of(nrows - 1), kbeg + chunk);
  if (kbeg >= kend && split > 0) return;                   // the join reads no part a row has no keys in

  const int gr = lane >> 2, gc = lane & 3;                 // row and column group of the mma fragments
  uint32_t qa[KS][4];
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    const int r = gr + 8 * hf;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + row_of(r < nrows ? r : 0) * D) + gc;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      qa[k][hf] = r < nrows ? src[8 * k] : 0u;
      qa[k][2 + hf] = r < nrows ? src[8 * k + 4] : 0u;
    }
  }
  const int lim0 = lim_of(gr), lim1 = lim_of(gr + 8);

  const uint32_t ring = smem_u32(smem) + warp * (C::ST * 2 * C::TILE);
  const int ntiles = (kend - kbeg + C::KT - 1) / C::KT;    // of the CTA; the warp takes every NW-th
  const int mine = ntiles > warp ? (ntiles - warp + C::NW - 1) / C::NW : 0;
  // cache row of the key that lanes l and l + 16 address in tile `it`
  auto key_row = [&](int it) -> long long {
    const int j = kbeg + (warp + it * C::NW) * C::KT + (lane & 15);
    if (it >= mine || j >= kend) return -1;
    const long long row = p.rows.row(b, j);
    if (row < 0) atomicOr(p.status, kStBadPage);
    return row;
  };
  long long next_row = key_row(0);
  auto issue = [&](int it) {
    const long long row = next_row;
    next_row = key_row(it + 1);
    if (it < mine) {
      const uint32_t dst = ring + (it % C::ST) * (2 * C::TILE);
#pragma unroll
      for (int x = 0; x < C::KT * CH / 32; ++x) {
        const int key = (x * 32 + lane) / CH, ch = lane % CH;
        const long long kr = __shfl_sync(0xffffffffu, row, key);
        const long long off = kr < 0 ? 0 : (kr * p.Hk + hk) * D + ch * 8;
        const uint32_t to = dst + key * (D * 2) + ((ch ^ (key & 7)) << 4);
        cp_async_16(to, p.kpages + off, kr < 0 ? 0u : 16u);
        cp_async_16(to + C::TILE, p.vpages + off, kr < 0 ? 0u : 16u);
      }
    }
    cp_async_commit();
  };

  float o[CH][4], m0 = neg_inf(), m1 = neg_inf(), l0 = 0.f, l1 = 0.f;
#pragma unroll
  for (int n = 0; n < CH; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
  for (int s = 0; s < C::ST - 1; ++s) issue(s);
  const int lrow = lane & 7, lmat = lane >> 3;
  for (int it = 0; it < mine; ++it) {
    issue(it + C::ST - 1);
    cp_async_wait<C::ST - 1>();
    __syncwarp();
    const uint32_t kt = ring + (it % C::ST) * (2 * C::TILE), vt = kt + C::TILE;
    float s[2][4] = {};
    {
      const int key = (lmat >> 1) * 8 + lrow;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t kb[4];
        ldmatrix_x4(kt + key * (D * 2) + (((2 * k + (lmat & 1)) ^ (key & 7)) << 4), kb);
        mma_m16n8k16(s[0], qa[k], kb[0], kb[1]);
        mma_m16n8k16(s[1], qa[k], kb[2], kb[3]);
      }
    }
    const int j0 = kbeg + (warp + it * C::NW) * C::KT + 2 * gc;
    float x0 = neg_inf(), x1 = neg_inf();
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = j0 + 8 * n + e;
        s[n][e] = j < lim0 && j < kend ? s[n][e] * p.scale_log2 : neg_inf();
        s[n][2 + e] = j < lim1 && j < kend ? s[n][2 + e] * p.scale_log2 : neg_inf();
        x0 = fmaxf(x0, s[n][e]);
        x1 = fmaxf(x1, s[n][2 + e]);
      }
    }
#pragma unroll
    for (int x = 1; x <= 2; x <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, x));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, x));
    }
    if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
      const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
      const float f0 = m0 == n0 ? 1.f : fast_exp2(m0 - n0), f1 = m1 == n1 ? 1.f : fast_exp2(m1 - n1);
      m0 = n0, m1 = n1;
      l0 *= f0, l1 *= f1;
#pragma unroll
      for (int n = 0; n < CH; ++n) o[n][0] *= f0, o[n][1] *= f0, o[n][2] *= f1, o[n][3] *= f1;
    }
    const float z0 = m0 == neg_inf() ? 0.f : m0, z1 = m1 == neg_inf() ? 0.f : m1;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[n][e] = fast_exp2(s[n][e] - z0);
        s[n][2 + e] = fast_exp2(s[n][2 + e] - z1);
        l0 += s[n][e];
        l1 += s[n][2 + e];
      }
    }
    // the weights go to bf16 for the second product, as its operand type asks; their sum l stays fp32
    const uint32_t pa[4] = {pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]), pack_bf16(s[1][0], s[1][1]),
                            pack_bf16(s[1][2], s[1][3])};
    {
      const int key = (lmat & 1) * 8 + lrow;
#pragma unroll
      for (int n = 0; n < CH; n += 2) {
        uint32_t vb[4];
        ldmatrix_x4_trans(vt + key * (D * 2) + (((n + (lmat >> 1)) ^ (key & 7)) << 4), vb);
        mma_m16n8k16(o[n], pa, vb[0], vb[1]);
        mma_m16n8k16(o[n + 1], pa, vb[2], vb[3]);
      }
    }
    __syncwarp();   // every lane has read the slot that the next step's copies fill
  }
  cp_async_wait<0>();
#pragma unroll
  for (int x = 1; x <= 2; x <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, x);
    l1 += __shfl_xor_sync(0xffffffffu, l1, x);
  }
  __syncthreads();
  // merge the warps' parts: [warp][row][D] and the rows' (m, l) behind them
  float* mo = reinterpret_cast<float*>(smem);
  float* ml = mo + C::NW * 16 * D;
#pragma unroll
  for (int n = 0; n < CH; ++n) {
    float* at = mo + (warp * 16 + gr) * D + 8 * n + 2 * gc;
    *reinterpret_cast<float2*>(at) = make_float2(o[n][0], o[n][1]);
    *reinterpret_cast<float2*>(at + 8 * D) = make_float2(o[n][2], o[n][3]);
  }
  if (gc == 0) {
    *reinterpret_cast<float2*>(ml + (warp * 16 + gr) * 2) = make_float2(m0, l0);
    *reinterpret_cast<float2*>(ml + (warp * 16 + gr + 8) * 2) = make_float2(m1, l1);
  }
  __syncthreads();
  constexpr int CL = D / 32;
  for (int r = warp; r < nrows; r += C::NW) {
    float m = neg_inf(), l = 0.f, acc[CL] = {};
#pragma unroll
    for (int w = 0; w < C::NW; ++w) m = fmaxf(m, ml[(w * 16 + r) * 2]);
    const float z = m == neg_inf() ? 0.f : m;
#pragma unroll
    for (int w = 0; w < C::NW; ++w) {
      const float f = fast_exp2(ml[(w * 16 + r) * 2] - z);
      l = fmaf(f, ml[(w * 16 + r) * 2 + 1], l);
#pragma unroll
      for (int c = 0; c < CL; ++c) acc[c] = fmaf(f, mo[(w * 16 + r) * D + lane * CL + c], acc[c]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    float lse2 = l == 0.f ? neg_inf() : m + log2f(l);
    bool fine = true;
#pragma unroll
    for (int c = 0; c < CL; ++c) {
      acc[c] *= inv;
      fine = fine && fabsf(acc[c]) < __int_as_float(0x7f800000);
    }
    const long long row = row_of(r);
    if (!__all_sync(0xffffffffu, fine))
      attend_row_exact<D>(p, b, hk, row, kbeg, min(kend, lim_of(r)), lane, acc, &lse2);
    if (p.nsplit > 1) {
      const long long at = static_cast<long long>(split) * p.rows.T * p.Hq + row;
#pragma unroll
      for (int c = 0; c < CL; ++c) p.part_o[at * D + lane * CL + c] = acc[c];
      if (lane == 0) p.part_lse[at] = lse2;
    } else {
#pragma unroll
      for (int c = 0; c < CL; c += 2)
        *reinterpret_cast<uint32_t*>(p.out + row * D + lane * CL + c) = pack_bf16(acc[c], acc[c + 1]);
      if (lane == 0 && p.lse) p.lse[row] = lse2 * kLn2;
    }
  }
}

// ------------------------------------------------------------------ joining the parts
// One warp a row: the parts that hold keys of the row are the first
// ceil(lim / chunk_of(len)) (at least one), whichever kernel wrote them.
template <int D>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ PagedAttendParams p) {
  constexpr int CL = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + warp;
  const long long rows = static_cast<long long>(p.rows.T) * p.Hq;
  if (row >= rows) return;
  const int tok = static_cast<int>(row / p.Hq);
  const NewSpan sp = p.rows.span(find_sequence(p.rows, tok, lane));
  if (tok < sp.tok0 || tok >= sp.tok0 + sp.n) return;
  const int lim = sp.ok ? sp.len - sp.n + p.self_key + (tok - sp.tok0) : 0;
  const int chunk = chunk_of(sp.len, p);
  const int parts = max(1, (lim + chunk - 1) / chunk);
  float m = neg_inf();
  for (int s = lane; s < parts; s += 32) m = fmaxf(m, p.part_lse[s * rows + row]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float z = m == neg_inf() ? 0.f : m;
  float l = 0.f, acc[CL] = {};
#pragma unroll 4
  for (int s = 0; s < parts; ++s) {
    const float f = fast_exp2(p.part_lse[s * rows + row] - z);
    const float* o = p.part_o + (s * rows + row) * D + lane * CL;
    l += f;
#pragma unroll
    for (int c = 0; c < CL; ++c) acc[c] = fmaf(f, o[c], acc[c]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int c = 0; c < CL; c += 2)
    *reinterpret_cast<uint32_t*>(p.out + row * D + lane * CL + c) = pack_bf16(acc[c] * inv, acc[c + 1] * inv);
  if (lane == 0 && p.lse) p.lse[row] = l == 0.f ? neg_inf() : (z + log2f(l)) * kLn2;
}

}  // namespace pivot

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
// axis is split: each CTA takes chunk_of(sequence) keys, and attend_join_kernel adds up
// the parts, o = sum_c w_c o_c, w_c = exp(lse_c - lse).
//
// attend_rows_kernel is the form for few rows per key head (decode), bound by
// the bytes of the keys and values.  Each of a CTA's four warps walks its own
// 16-key steps of the chunk with a ring and an (m, l, o) of its own, merged at
// the end, so nothing waits for anything but memory.  The products take the
// keys as the 16 rows of the tile and the queries as its 8 columns:
//     S^T = K q^T (16 keys x 8 queries), o^T += V^T P^T (16 channels x 8),
// half the instructions and accumulators of queries in rows; the weights turn
// from the first product's layout to the second's operand by a transposing
// register move.
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
  int over, upto;          // with cu: the packed rows of the sequences that this launch takes, over < rows <= upto
  int many, nsplit_many;   // sequences of more packed rows than `many` are cut into nsplit_many parts, not nsplit
  float scale_log2;        // scale * log2(e)
  uint16_t* out;           // [T][Hq][d] bf16
  float* lse;              // [T][Hq] natural log, or null
  float* part_o;           // where keys are split: [parts][T][Hq][d], each part normalised; else null
  float* part_lse;         // [parts][T][Hq], log2 units
  int* status;
  unsigned long long wait_ns;
};

constexpr float kLn2 = 0.693147180559945309f;

// Keys per part of a sequence: an nsplit-th of its rows, whatever the bound that
// sized the grid, in whole 128-key tiles, and no less than min_chunk.
__device__ __forceinline__ int chunk_of(const NewSpan& sp, const PagedAttendParams& p) {
  const int parts = sp.n * p.grp > p.many ? p.nsplit_many : p.nsplit;
  return max(p.min_chunk, ((sp.len + parts - 1) / parts + 127) & ~127);
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The row tile `flat` of the batch: which sequence, and which of its tiles of
// `rows` packed rows; -1 where there is none.  One warp.
//  * Without cu every sequence has the same number of tiles.
//  * With cu, sequence b's tiles start at floor(cu[b] grp / rows) + b, which
//    leaves each its own (ceil(n grp / rows) of them fit before the next start)
//    and needs no sums: b is found by 32 probes a round.  Some places stay empty.
//  * A launch for the sequences of many rows alone would leave most places empty:
//    there the tile counts of those are summed, 128 sequences at a time.
__device__ __forceinline__ int locate_tile(const PagedAttendParams& a, int rows, int flat, int lane, int* tile) {
  const PagedRows& p = a.rows;
  if (!p.cu) {
    const int per = (p.g * a.grp + rows - 1) / rows;
    *tile = flat % per;
    return flat / per < p.B ? flat / per : -1;
  }
  if (a.over == 0) {
    auto start = [&](int b) { return static_cast<long long>(p.cu[b]) * a.grp / rows + b; };
    int lo = 0, hi = p.B;   // the answer is in [lo, hi)
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const unsigned votes = __ballot_sync(0xffffffffu, at < hi && start(at) <= flat) | 1u;
      lo += (31 - __clz(votes)) * step;
      hi = min(hi, lo + step);
    }
    const long long t = flat - start(lo);
    if (t < 0 || t > flat || p.new_tokens(lo) * a.grp > a.upto) return -1;
    *tile = static_cast<int>(t);
    return lo;
  }
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 128) {
    int n[4], sum = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int b = b0 + 4 * lane + x;
      const int packed = b < p.B ? p.new_tokens(b) * a.grp : 0;
      n[x] = packed > a.over && packed <= a.upto ? static_cast<int>((static_cast<long long>(packed) + rows - 1) / rows) : 0;
    }
    const int mine = n[0] + n[1] + n[2] + n[3];
    sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + sum > flat);
    if (past) {
      // in the first lane whose sum passes: its first sequence that does
      const int l = __ffs(past) - 1;
      int left = flat - (before + sum - mine), x = 0;
      while (x < 3 && left >= n[0]) {
        left -= n[0];
        n[0] = n[1], n[1] = n[2], n[2] = n[3];
        ++x;
      }
      *tile = __shfl_sync(0xffffffffu, left, l);
      return b0 + 4 * l + __shfl_sync(0xffffffffu, x, l);
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return -1;
}

// ------------------------------------------------------------------ rows that are not finite
// By definition an infinity or NaN among the values that a row sees makes its
// channel so, however small its weight, and one that it does not see leaves it
// alone.  A product over a whole tile does neither by itself: there a value that
// is not seen meets a weight of zero, and a small weight may round to zero.  So
//  * values that some row of a tile does not see are made finite (zeros) where the
//    tile lies in shared memory (cleaned), which costs the last tiles alone;
//  * if that found any, or a row came out not finite though the sum of its weights
//    is (a NaN there is the row's), FirstNonFinite looks the values up and puts in
//    what the row's channels have to be;
//  * what is still not finite had values so large that a sum went past the type's
//    end: attend_row_exact works that row out anew.
// One infinite value at the start of a 4096-token prefill of 16 heads so takes
// 295 us for the 83 without it; every later row key by key took 69 ms.
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __int_as_float(0x7f800000); }
__device__ __forceinline__ float add_weighted(float w, float v, float sum) { return finite(v) ? fmaf(w, v, sum) : sum + v; }

// acc, zero so far, and not zero from the first pair of bf16 values on that is not
// finite (0 times it is NaN).
__device__ __forceinline__ uint32_t odd_so_far(uint32_t acc, uint32_t two) {
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(two), "r"(0u));
  return acc;
}
__device__ __forceinline__ uint32_t odd_so_far(uint32_t acc, const uint4& v) {
  return odd_so_far(odd_so_far(odd_so_far(odd_so_far(acc, v.x), v.y), v.z), v.w);
}
// Eight bf16 values, those that are not finite made zero.
__device__ __forceinline__ uint4 cleaned(uint4 v) {
  auto two = [](uint32_t w) {
    const uint32_t odd = ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;   // an exponent of all ones carries
    return w & ~((odd >> 15) * 0xFFFFu);
  };
  return make_uint4(two(v.x), two(v.y), two(v.z), two(v.w));
}

// A lane's D/32 channels [lane * D/32, ...) of a row of keys or values.
template <int D>
__device__ __forceinline__ void load_lane(const uint16_t* row, int lane, uint32_t (&w)[D / 64]) {
  if constexpr (D == 128) {
    const uint2 u = *reinterpret_cast<const uint2*>(row + lane * 4);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(row + lane * 2);
  }
}

// The first keys whose value is +infinity, -infinity and NaN in each of a lane's channels.
template <int D>
struct FirstNonFinite {
  static constexpr int C = D / 32, NONE = 0x7FFFFFFF;
  int pos[C], neg[C], nan[C];

  // Looks through the values of the keys j0 <= j < j1, by a whole warp; row_of as below.
  template <class P, class RowOf>
  __device__ __forceinline__ void look(const P& p, int heads, int head, int j0, int j1, RowOf row_of, int lane) {
#pragma unroll
    for (int c = 0; c < C; ++c) pos[c] = neg[c] = nan[c] = NONE;
    for (int jb = j0; jb < j1; jb += 32) {
      const int mine = jb + lane < j1 ? static_cast<int>(row_of(jb + lane)) : -1;
      for (int x0 = 0; x0 < 32; x0 += 8) {
        uint32_t w[8][D / 64], odd = 0;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int row = __shfl_sync(0xffffffffu, mine, x0 + x);
#pragma unroll
          for (int h = 0; h < D / 64; ++h) w[x][h] = 0;
          if (row >= 0) load_lane<D>(p.vpages + (static_cast<long long>(row) * heads + head) * D, lane, w[x]);
        }
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
          for (int h = 0; h < D / 64; ++h) odd = odd_so_far(odd, w[x][h]);
        if (!odd) continue;
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const uint32_t v = w[x][c / 2] >> (16 * (c & 1)) & 0xFFFFu;
            const int j = jb + x0 + x;
            pos[c] = min(pos[c], v == 0x7F80u ? j : NONE);
            neg[c] = min(neg[c], v == 0xFF80u ? j : NONE);
            nan[c] = min(nan[c], (v & 0x7FFFu) > 0x7F80u ? j : NONE);
          }
      }
    }
  }
  // What channel c of a row that sees the keys below lim has to be: not finite, or 0 where it may be finite.
  __device__ __forceinline__ float due(int c, int lim) const {
    const bool up = pos[c] < lim, down = neg[c] < lim;
    if (nan[c] < lim || (up && down)) return __int_as_float(0x7fffffff);
    return up ? __int_as_float(0x7f800000) : down ? __int_as_float(0xff800000) : 0.f;
  }
  // Puts what has to be not finite into a row's channels; true where another one is not finite.
  __device__ __forceinline__ bool settle(float (&o)[C], int lim) const {
    bool open = false;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float x = due(c, lim);
      if (x != 0.f)
        o[c] = x;
      else
        open = open || !finite(o[c]);
    }
    return __any_sync(0xffffffffu, open);
  }
};

// One query row over the keys j0 <= j < j1, key j in cache row row_of(j) (-1:
// left out, -2: zeros), by a whole warp, reading only those keys: 32 at a time, a
// key a lane for the scores, then lane l with channels [l * D/32, ...) for the values.
// The weights are taken times kDown, so that no sum of values ends past the type's end.
constexpr float kDown = 0x1p-31f, kUp = 0x1p31f;
template <int D, class P, class RowOf>
__device__ __forceinline__ void attend_row_exact(const P& p, int heads, int head, long long qrow, int j0, int j1,
                                                 RowOf row_of, int lane, float (&o)[D / 32], float* lse2) {
  constexpr int C = D / 32;
  using Bf16 = __nv_bfloat16;
  const Bf16* const q = reinterpret_cast<const Bf16*>(p.q + qrow * D);
  float m = neg_inf(), l = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.f;
  for (int jb = j0; jb < j1; jb += 32) {
    const int mine = jb + lane < j1 ? static_cast<int>(row_of(jb + lane)) : -1;
    float s = 0.f;
    if (mine >= 0) {
      const Bf16* const k = reinterpret_cast<const Bf16*>(p.kpages + (static_cast<long long>(mine) * heads + head) * D);
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        Vec8<Bf16> vk, vq;
        float fk[8], fq[8];
        vk.load(k + 8 * c);
        vq.load(q + 8 * c);
        vk.get(fk);
        vq.get(fq);
#pragma unroll
        for (int x = 0; x < 8; ++x) s = fmaf(fk[x], fq[x], s);
      }
    }
    s = mine == -1 ? neg_inf() : s * p.scale_log2;
    float mn = s;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
    mn = fmaxf(m, mn);
    const float ms = mn == neg_inf() ? 0.f : mn;
    const float f = fast_exp2(m - ms), e = fast_exp2(s - ms);
    float sum = e;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = l * f + sum;
    if (l != l) break;   // all is NaN from here on, whatever follows
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = finite(o[c]) ? o[c] * f : o[c];
    m = mn;
#pragma unroll 8
    for (int x = 0; x < 32; ++x) {
      const int row = __shfl_sync(0xffffffffu, mine, x);
      const float w = __shfl_sync(0xffffffffu, e, x);
      uint32_t v[D / 64] = {};
      if (row >= 0) load_lane<D>(p.vpages + (static_cast<long long>(row) * heads + head) * D, lane, v);
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = add_weighted(w * kDown, c & 1 ? bf16_hi(v[c / 2]) : bf16_lo(v[c / 2]), o[c]);
    }
  }
  const float inv = l == 0.f ? 0.f : kUp / l;
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] *= inv;
  *lse2 = l == 0.f ? neg_inf() : m + log2f(l);
}

// A row that is not finite though the sum of its weights is, or whose values were cleaned: its channels over the keys
// [j0, j1) as they came out, and as they have to be.
template <int D>
struct RowResult {
  float o[D / 32], lse2;
};
template <int D>
__device__ __forceinline__ RowResult<D> settle_row(const PagedAttendParams& p, const SequenceRows rows, int hk, long long row,
                                                int j0, int j1, RowResult<D> r) {
  const int lane = threadIdx.x & 31;
  auto cache_row = [&](int j) { return rows.row_or(j, -2); };
  FirstNonFinite<D> odd;
  odd.look(p, p.Hk, hk, j0, j1, cache_row, lane);
  if (odd.settle(r.o, j1)) attend_row_exact<D>(p, p.Hk, hk, row, j0, j1, cache_row, lane, r.o, &r.lse2);
  return r;
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
// An 8 x 8 tile of 16-bit values, two of a row a lane, turned about its diagonal.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// A warp's ring of 16-key steps: 16 key rows and 16 value rows each, 16 bytes
// apart beyond their length so that the eight rows of a matrix load lie in
// different banks.  Filled by cp.async, 16 bytes a lane: bulk copies of a row
// each need one instruction for 32 rows, but took 19 cycles a copy, twice what
// the memory's rate leaves for 256 bytes.
template <int D>
struct KvRing {
  static constexpr int NW = 4;                          // warps a CTA
  static constexpr int KT = 16;                         // keys a step
  static constexpr int ROW = 2 * D + 16;
  static constexpr int HALF = KT * ROW;                 // the keys; the values as many bytes behind them
  // Steps in flight.  Three CTAs of two steps an SM beat two of three (a decode
  // step of 64 sequences of 8192, 8 key heads: 378 us for 396) and one of five
  // (439): a warp's own chain of loads and products wants company.  At 64
  // channels, four of three beat three of four and five of two (index rows of 32
  // sequences, 16 heads, 512 indices: 39 us for 47 and 41).
  static constexpr int ST = D == 128 ? 2 : 3;
  static constexpr int BYTES = ST * 2 * HALF;           // a warp's ring
  static constexpr int SMEM = NW * BYTES;
  static constexpr int PER_SM = D == 128 ? 3 : 4;       // CTAs that an SM holds
  static_assert(PER_SM * (SMEM + 2048) <= 232448, "shared memory of an SM");

  uint32_t ring;
  const uint8_t *kbase, *vbase;                         // the head's first key and value row, at the lane's 16 bytes
  uint32_t stride;                                      // bytes from a cache row to the next

  __device__ __forceinline__ void init(uint8_t* smem, const uint16_t* kpages, const uint16_t* vpages, int heads, int head,
                                       int warp, int lane) {
    ring = smem_u32(smem) + warp * BYTES + (lane / (D / 8)) * ROW + (lane % (D / 8)) * 16;
    const long long at = static_cast<long long>(head) * D + (lane % (D / 8)) * 8;
    kbase = reinterpret_cast<const uint8_t*>(kpages + at);
    vbase = reinterpret_cast<const uint8_t*>(vpages + at);
    stride = static_cast<uint32_t>(heads) * D * 2;
  }
  // Brings in step `it`: lane l and l + 16 have the cache row of key l, -1
  // where there is none (zeros then: 0 * what the ring held may be NaN).
  // `whole`, the same in every lane: all 16 are there.
  __device__ __forceinline__ void issue(int it, int row, bool whole) {
    const uint32_t dst = ring + (it % ST) * (2 * HALF);
    constexpr int RP = 256 / D;                         // rows that a warp's 32 pieces make
    const int mine = (threadIdx.x & 31) / (D / 8);
    if (whole) {
#pragma unroll
      for (int x = 0; x < KT / RP; ++x) {
        const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(__shfl_sync(0xffffffffu, row, x * RP + mine))) * stride;
        cp_async_16(dst + x * RP * ROW, kbase + off);
        cp_async_16(dst + x * RP * ROW + HALF, vbase + off);
      }
    } else {
#pragma unroll
      for (int x = 0; x < KT / RP; ++x) {
        const int kr = __shfl_sync(0xffffffffu, row, x * RP + mine);
        const uint64_t off = kr < 0 ? 0 : static_cast<uint64_t>(static_cast<uint32_t>(kr)) * stride;
        cp_async_16(dst + x * RP * ROW, kbase + off, kr < 0 ? 0u : 16u);
        cp_async_16(dst + x * RP * ROW + HALF, vbase + off, kr < 0 ? 0u : 16u);
      }
    }
  }
  // Makes the values of step `it` finite from its key `from` on, each lane those that it brought in; true where one was not.
  __device__ __forceinline__ bool clean_values(int it, uint8_t* smem, int from) const {
    uint8_t* const at = smem + (ring - smem_u32(smem)) + (it % ST) * (2 * HALF) + HALF;
    constexpr int RP = 256 / D;
    const int mine = (threadIdx.x & 31) / (D / 8);
    bool any = false;
    for (int x = 0; x < KT / RP; ++x) {
      if (x * RP + mine < from) continue;
      uint4* const v = reinterpret_cast<uint4*>(at + x * RP * ROW);
      if (odd_so_far(0u, *v)) {
        *v = cleaned(*v);
        any = true;
      }
    }
    return any;
  }
  __device__ __forceinline__ uint32_t keys(int it, uint8_t* smem, int warp) const {
    return smem_u32(smem) + warp * BYTES + (it % ST) * (2 * HALF);
  }
};

// S^T of a step: s[0], s[1]: key lane / 4 with queries 2 (lane % 4) and the
// next; s[2], s[3]: key lane / 4 + 8.  Two chains of products, added.
template <int D>
__device__ __forceinline__ void step_scores(uint32_t kt, const uint32_t (&qb)[D / 16][2], int lane, float (&s)[4]) {
  const uint32_t at = kt + ((lane >> 3 & 1) * 8 + (lane & 7)) * KvRing<D>::ROW + (lane >> 4) * 16;
  float t[2][4] = {};
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    uint32_t a[4];
    ldmatrix_x4(at + 32 * k, a);
    mma_m16n8k16(t[k & 1], a, qb[k][0], qb[k][1]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] = t[0][e] + t[1][e];
}
// o^T += V^T P^T: o[n]: channel 16 n + lane / 4 (and + 8), queries as above;
// b0, b1: the weights of keys 0-7 and 8-15, transposed.
template <int D>
__device__ __forceinline__ void step_values(uint32_t vt, uint32_t b0, uint32_t b1, int lane, float (&o)[D / 16][4]) {
  const uint32_t at = vt + ((lane >> 4) * 8 + (lane & 7)) * KvRing<D>::ROW + (lane >> 3 & 1) * 16;
#pragma unroll
  for (int n = 0; n < D / 16; ++n) {
    uint32_t a[4];
    ldmatrix_x4_trans(at + 32 * n, a);
    mma_m16n8k16(o[n], a, b0, b1);
  }
}

// NT tiles of 8 packed rows a CTA.
template <int D, int NT>
__global__ void __launch_bounds__(128) attend_rows_kernel(const __grid_constant__ PagedAttendParams p) {
  using R = KvRing<D>;
  constexpr int KS = D / 16;       // k-steps of q . k, and 16-channel tiles of o
  constexpr int ROWS = 8 * NT;
  constexpr int OS = D + 4;        // floats a row of the merge
  static_assert(R::NW * ROWS * (OS + 2) * 4 <= R::NW * R::BYTES, "the merge takes the rings' place");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int seq_s[2];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  grid_launch_dependents();
  // key heads in the innermost place: neighbouring CTAs read neighbouring heads of the same rows
  const unsigned bid = blockIdx.x;
  const int hk = static_cast<int>(bid % p.Hk);
  const int split = static_cast<int>(bid / p.Hk % p.nsplit);
  const int flat = static_cast<int>(bid / p.Hk / p.nsplit);
  if (warp == 0) {
    int tile = 0;
    const int b = locate_tile(p, ROWS, flat, lane, &tile);
    if (lane == 0) seq_s[0] = b, seq_s[1] = tile;
  }
  __syncthreads();
  const int b = seq_s[0], r0 = seq_s[1] * ROWS;
  if (b < 0) return;
  const NewSpan sp = p.rows.span(b);
  if (!sp.ok && threadIdx.x == 0) atomicOr(p.status, kStBadLen);
  const int nrows = min(ROWS, sp.n * p.grp - r0);
  if (nrows <= 0) return;
  const int pos0 = sp.len - sp.n + p.self_key;             // lim of the sequence's first new token
  auto lim_of = [&](int r) { return sp.ok ? pos0 + (r0 + r) / p.grp : 0; };
  auto row_of = [&](int r) {
    return (static_cast<long long>(sp.tok0) + (r0 + r) / p.grp) * p.Hq + hk * p.grp + (r0 + r) % p.grp;
  };
  const int chunk = chunk_of(sp, p);
  const int kbeg = split * chunk;
  const int kend = min(lim_of(nrows - 1), kbeg + chunk);
  if (kbeg >= kend && split > 0) return;                   // the join reads no part a row has no keys in

  const int ntiles = max(0, (kend - kbeg + R::KT - 1) / R::KT);   // of the CTA; the warp takes every NW-th
  const int mine = ntiles > warp ? (ntiles - warp + R::NW - 1) / R::NW : 0;
  R kv;
  kv.init(smem, p.kpages, p.vpages, p.Hk, hk, warp, lane);
  const SequenceRows rows(p.rows, b);
  // cache row of the key that lanes l and l + 16 address in step `it`
  auto place = [&](int it) -> int {
    const int j = kbeg + (warp + it * R::NW) * R::KT + (lane & 15);
    if (it >= mine || j >= kend) return -1;
    const int row = rows.row(j);
    if (row < 0) atomicOr(p.status, kStBadPage);
    return row;
  };
  int next = place(0);
  auto issue = [&](int it) {
    const int row = next;
    next = place(it + 1);
    if (it < mine) kv.issue(it, row, __all_sync(0xffffffffu, row >= 0));
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < R::ST - 1; ++s) issue(s);

  const int gr = lane >> 2, gc = lane & 3;
  uint32_t qb[NT][KS][2];
  int lim[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = 8 * t + gr;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + row_of(r < nrows ? r : 0) * D) + gc;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      qb[t][k][0] = r < nrows ? src[8 * k] : 0u;
      qb[t][k][1] = r < nrows ? src[8 * k + 4] : 0u;
    }
    lim[t][0] = min(kend, lim_of(8 * t + 2 * gc));
    lim[t][1] = min(kend, lim_of(8 * t + 2 * gc + 1));
  }
  float o[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t][0] = m[t][1] = neg_inf();
    l[t][0] = l[t][1] = 0.f;
#pragma unroll
    for (int n = 0; n < KS; ++n) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.f;
  }
  const int unseen = lim_of(0);    // from here on there are keys that some row does not see
  const int mixed = unseen < kend ? unseen - R::KT : 0x7FFFFFFF;   // ... in the steps whose first key is past this one
  bool dirty = false;              // some of those keys' values were not finite
  for (int it = 0; it < mine; ++it) {
    issue(it + R::ST - 1);
    cp_async_wait<R::ST - 1>();
    const int j0 = kbeg + (warp + it * R::NW) * R::KT, j = j0 + gr;
    if (j0 > mixed) dirty = kv.clean_values(it, smem, unseen - j0) || dirty;
    __syncwarp();
    const uint32_t kt = kv.keys(it, smem, warp);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float s[4];
      step_scores<D>(kt, qb[t], lane, s);
      float x[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[e] = j < lim[t][e] ? s[e] * p.scale_log2 : neg_inf();
        s[2 + e] = j + 8 < lim[t][e] ? s[2 + e] * p.scale_log2 : neg_inf();
        x[e] = fmaxf(s[e], s[2 + e]);
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) x[e] = fmaxf(x[e], __shfl_xor_sync(0xffffffffu, x[e], y));
      }
      if (__any_sync(0xffffffffu, x[0] > m[t][0] || x[1] > m[t][1])) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float n = fmaxf(m[t][e], x[e]);
          f[e] = m[t][e] == n ? 1.f : fast_exp2(m[t][e] - n);
          m[t][e] = n;
          l[t][e] *= f[e];
        }
#pragma unroll
        for (int n = 0; n < KS; ++n)
          o[t][n][0] *= f[0], o[t][n][1] *= f[1], o[t][n][2] *= f[0], o[t][n][3] *= f[1];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float z = m[t][e] == neg_inf() ? 0.f : m[t][e];
        s[e] = fast_exp2(s[e] - z);
        s[2 + e] = fast_exp2(s[2 + e] - z);
        l[t][e] += s[e] + s[2 + e];
      }
      // The weights go to bf16 for the second product, as its operand type asks; their sum l stays fp32.  The roundings
      // average out over the keys (4 sequences of 65536: error against 64 bits 0.001673, of which 0.001672 is the
      // result's own rounding); two bf16 terms a weight took up to 7 % of the time for that.
      step_values<D>(kt + R::HALF, transpose_8x8(pack_bf16(s[0], s[1])), transpose_8x8(pack_bf16(s[2], s[3])), lane, o[t]);
    }
    __syncwarp();   // every lane has read the slot that the next step's copies fill
  }
  cp_async_wait<0>();
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int y = 4; y < 32; y <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], y);
  dirty = __syncthreads_or(dirty);
  // merge the warps' parts: [warp][row][OS] and the rows' (m, l) behind them
  float* mo = reinterpret_cast<float*>(smem);
  float* ml = mo + R::NW * ROWS * OS;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float* at = mo + (warp * ROWS + 8 * t + 2 * gc + (e & 1)) * OS + gr + 8 * (e >> 1);
#pragma unroll
      for (int n = 0; n < KS; ++n) at[16 * n] = o[t][n][e];
    }
    if (gr == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<float2*>(ml + (warp * ROWS + 8 * t + 2 * gc + e) * 2) = make_float2(m[t][e], l[t][e]);
    }
  }
  __syncthreads();
  constexpr int CL = D / 32;
  for (int r = warp; r < nrows; r += R::NW) {
    float rm = neg_inf(), rl = 0.f, acc[CL] = {};
#pragma unroll
    for (int w = 0; w < R::NW; ++w) rm = fmaxf(rm, ml[(w * ROWS + r) * 2]);
    const float z = rm == neg_inf() ? 0.f : rm;
#pragma unroll
    for (int w = 0; w < R::NW; ++w) {
      const float f = fast_exp2(ml[(w * ROWS + r) * 2] - z);
      rl = fmaf(f, ml[(w * ROWS + r) * 2 + 1], rl);
#pragma unroll
      for (int c = 0; c < CL; ++c) acc[c] = fmaf(f, mo[(w * ROWS + r) * OS + lane * CL + c], acc[c]);
    }
    const float inv = rl == 0.f ? 0.f : 1.f / rl;
    float lse2 = rl == 0.f ? neg_inf() : rm + log2f(rl);
    bool fine = true;
#pragma unroll
    for (int c = 0; c < CL; ++c) {
      acc[c] *= inv;
      fine = fine && finite(acc[c]);
    }
    const long long row = row_of(r);
    if (rl == rl && (dirty || !__all_sync(0xffffffffu, fine))) {
      RowResult<D> x;
#pragma unroll
      for (int c = 0; c < CL; ++c) x.o[c] = acc[c];
      x.lse2 = lse2;
      x = settle_row<D>(p, rows, hk, row, kbeg, min(kend, lim_of(r)), x);
#pragma unroll
      for (int c = 0; c < CL; ++c) acc[c] = x.o[c];
      lse2 = x.lse2;
    }
    if (p.part_o) {
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
// The parts that hold keys of the row are the first
// ceil(lim / chunk_of(sequence)) (at least one), whichever kernel wrote them.  Launched
// while that kernel still runs, it looks its row up and then waits for it.
// WIDE: a CTA's four warps share a row's parts (many parts mean few rows: 55
// parts of 32 rows took 15 us by one warp a row).
template <int D, bool WIDE>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ PagedAttendParams p) {
  constexpr int CL = D / 32, NW = WIDE ? 4 : 1;
  __shared__ float sm_l[NW], sm_a[NW][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = WIDE ? warp : 0;
  const long long row = WIDE ? static_cast<long long>(blockIdx.x) : static_cast<long long>(blockIdx.x) * 4 + warp;
  const long long rows = static_cast<long long>(p.rows.T) * p.Hq;
  // every warp waits, those without a row too: what comes behind this kernel in
  // the stream must not find the parts' kernel still running
  const int tok = static_cast<int>(min(row, rows - 1) / p.Hq);
  const NewSpan sp = p.rows.span(find_sequence(p.rows, tok, lane));
  const int lim = sp.ok ? sp.len - sp.n + p.self_key + (tok - sp.tok0) : 0;
  const int chunk = chunk_of(sp, p);
  const int parts = max(1, (lim + chunk - 1) / chunk);
  grid_wait();
  if (row >= rows || tok < sp.tok0 || tok >= sp.tok0 + sp.n) return;
  float m = neg_inf();
  for (int s = lane; s < parts; s += 32) m = fmaxf(m, p.part_lse[s * rows + row]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float z = m == neg_inf() ? 0.f : m;
  float l, acc[CL];
  auto add_up = [&](auto weigh) {
    l = 0.f;
#pragma unroll
    for (int c = 0; c < CL; ++c) acc[c] = 0.f;
#pragma unroll 4
    for (int s = w; s < parts; s += NW) {
      const float f = fast_exp2(p.part_lse[s * rows + row] - z);
      const float* o = p.part_o + (s * rows + row) * D + lane * CL;
      l += f;
#pragma unroll
      for (int c = 0; c < CL; ++c) acc[c] = weigh(f, o[c], acc[c]);
    }
  };
  add_up([](float f, float o, float sum) { return fmaf(f, o, sum); });
  bool fine = true;
#pragma unroll
  for (int c = 0; c < CL; ++c) fine = fine && fabsf(acc[c]) < 0x1p126f;
  // a part's infinity times a weight of zero, or a sum past the type's end (four warps' together)
  if (WIDE) fine = !__syncthreads_or(!fine);
  if (!fine) add_up([](float f, float o, float sum) { return add_weighted(f * kDown, o, sum); });
  if (WIDE) {
    if (lane == 0) sm_l[w] = l;
#pragma unroll
    for (int c = 0; c < CL; ++c) sm_a[w][lane * CL + c] = acc[c];
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int y = 1; y < NW; ++y) {
      l += sm_l[y];
#pragma unroll
      for (int c = 0; c < CL; ++c) acc[c] += sm_a[y][lane * CL + c];
    }
  }
  const float inv = l == 0.f ? 0.f : (fine ? 1.f : kUp) / l;
#pragma unroll
  for (int c = 0; c < CL; c += 2)
    *reinterpret_cast<uint32_t*>(p.out + row * D + lane * CL + c) = pack_bf16(acc[c] * inv, acc[c + 1] * inv);
  if (lane == 0 && p.lse) p.lse[row] = l == 0.f ? neg_inf() : (z + log2f(l)) * kLn2;
}

}  // namespace pivot

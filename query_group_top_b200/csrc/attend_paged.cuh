// The sparse attention over index rows (attend.cuh) on a paged cache: keys and
// values behind a block table, the rows of a decode step.
//
// Bytes: the gathers, 2 * d * 2 an index.  A CTA takes one (query, head); its
// four warps take the row's indices 16 at a time through the ring of
// paged_attend.cuh, so that what is on its way does not hang on registers or on
// the arithmetic.  The index of a step is read two steps before its keys and the
// page one step before, so neither of the two dependent loads is waited for.
// What bounds it is the chain of a step in its warp (rows, product, softmax,
// product), three warps a scheduler: DRAM is at 54 %, the issue slots at 26.  32
// sequences, steps of two, 16 heads of 128, 2048 indices take 155 to 162 us.  Merging the
// rows of two members in a CTA, so that common keys are gathered once (0.68 GB for
// 1.07), was built and took 173 to 182.
//
// The products run as there, keys in the rows and the query in the columns of
// m16n8k16 tiles.  The query stands in all eight columns, so every lane has the
// scores of its two keys; for the second product column 0 holds the upper 8
// bits of each fp32 weight, column 1 the next 8, column 2 the last: one chain of
// products whose three columns add up to the sum under fp32 weights (exact to
// 2^-25 of a weight).  The results stay fp32.
//
// Where the rows are few, a cluster of CTAs shares one row's indices and merges
// over distributed shared memory, so no workspace is needed.
#pragma once

#include <cooperative_groups.h>

#include "paged_attend.cuh"

namespace pivot {

struct AttendPagedParams {
  const uint16_t* q;       // [B][g][H][d] bf16
  const uint16_t* kpages;  // [pages][page_size][H][d]
  const uint16_t* vpages;
  const int32_t* idx;      // [B][g][H][top_k]
  PagedRows rows;
  float* out;              // [B][g][H][d]
  int H, g, top_k;
  int parts;               // CTAs of a cluster, each a part of the row's indices
  float scale_log2;        // d^-1/2 * log2(e)
  int* status;
};

// A row that came out not finite (paged_attend.cuh): thread c has channel c's value and gets it anew.  By the whole CTA;
// kinds: D words of shared memory.
template <int D>
__device__ __noinline__ float sparse_row_not_finite(const AttendPagedParams& p, unsigned rh, int h, const int32_t* row,
                                                    const SequenceRows rows, int len, float value, uint32_t* kinds) {
  constexpr int NW = KvRing<D>::NW, C = D / 32;
  const int c = threadIdx.x, warp = c >> 5, lane = c & 31;
  auto cache_row = [&](int t) {
    const int j = __ldg(row + t);
    return j >= 0 && j < len ? rows.row(j) : -1;
  };
  if (c < D) kinds[c] = 0;   // of a channel's values: bit 0 infinite, 1 its negative, 2 NaN
  __syncthreads();
  FirstNonFinite<D> odd;
  const int share = (p.top_k + NW - 1) / NW;
  odd.look(p, p.H, h, warp * share, min(p.top_k, (warp + 1) * share), cache_row, lane);
#pragma unroll
  for (int x = 0; x < C; ++x) {
    const uint32_t k = (odd.pos[x] != odd.NONE ? 1u : 0u) | (odd.neg[x] != odd.NONE ? 2u : 0u) | (odd.nan[x] != odd.NONE ? 4u : 0u);
    if (k) atomicOr(&kinds[lane * C + x], k);
  }
  __syncthreads();
  const uint32_t k = c < D ? kinds[c] : 0u;
  if (k) value = __int_as_float(k == 1u ? 0x7f800000 : k == 2u ? 0xff800000 : 0x7fffffff);
  if (!__syncthreads_or(!k && !finite(value))) return value;
  if (warp == 0) {
    float o[C], lse2;
    attend_row_exact<D>(p, p.H, h, rh, 0, p.top_k, cache_row, lane, o, &lse2);
#pragma unroll
    for (int x = 0; x < C; ++x) kinds[lane * C + x] = __float_as_uint(o[x]);
  }
  __syncthreads();
  return c < D ? __uint_as_float(kinds[c]) : 0.f;
}

template <int D>
__global__ void __launch_bounds__(128) sparse_attention_paged_kernel(const __grid_constant__ AttendPagedParams p) {
  using R = KvRing<D>;
  constexpr int KS = D / 16;       // k-steps of q . k, and 16-channel tiles of o
  constexpr int OS = D + 4;        // floats a row of the merge
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const unsigned rh = blockIdx.x / p.parts;                // query row and head
  const int rank = static_cast<int>(blockIdx.x % p.parts); // the CTA's rank in its cluster
  const int h = static_cast<int>(rh % p.H);
  const int b = static_cast<int>(rh / p.H / p.g);
  const NewSpan sp = p.rows.span(b);
  const int len = sp.ok ? sp.len : 0;                      // a sequence that does not fit gets zeros
  const int chunk = ((p.top_k + p.parts - 1) / p.parts + 15) & ~15;
  const int tbeg = rank * chunk;
  int tend = min(p.top_k, tbeg + chunk);
  const int32_t* row = p.idx + static_cast<long long>(rh) * p.top_k;
  R kv;
  kv.init(smem, p.kpages, p.vpages, p.H, h, warp, lane);
  {
    // the part ends behind its last index: rows are often padded far beyond their sequence
    __shared__ int last_s[R::NW];
    int last = tbeg;
#pragma unroll 4
    for (int t = tbeg + threadIdx.x; t < tend; t += 128)
      if (__ldg(row + t) >= 0) last = t + 1;
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) last_s[warp] = last;
    __syncthreads();
    tend = max(max(last_s[0], last_s[1]), max(last_s[2], last_s[3]));
  }

  const int ntiles = tend > tbeg ? (tend - tbeg + R::KT - 1) / R::KT : 0;
  const int mine = ntiles > warp ? (ntiles - warp + R::NW - 1) / R::NW : 0;
  // index of the entry that lanes l and l + 16 take of step `it`, then its cache row (-1: none)
  auto entry = [&](int it) -> int {
    const int t = tbeg + (warp + it * R::NW) * R::KT + (lane & 15);
    return it < mine && t < tend ? __ldg(row + t) : -1;
  };
  const SequenceRows rows(p.rows, b);
  auto place = [&](int j) -> int {
    if (j < 0) return -1;
    const int at = j < len ? rows.row(j) : -1;
    if (at < 0 && sp.ok) atomicOr(p.status, kStBadPage);
    return at;
  };
  int next = place(entry(0));
  int next_entry = entry(1);
  uint32_t there[R::ST];                                   // entries that are there, a bit each, of the steps in flight
#pragma unroll
  for (int s = 0; s < R::ST; ++s) there[s] = 0;
  auto issue = [&](int it) {
    const int at = next, e = next_entry;
    next_entry = entry(it + 2);
#pragma unroll
    for (int s = 0; s + 1 < R::ST; ++s) there[s] = there[s + 1];
    there[R::ST - 1] = __ballot_sync(0xffffffffu, at >= 0) & 0xffffu;
    if (it < mine && there[R::ST - 1]) kv.issue(it, at, there[R::ST - 1] == 0xffffu);
    cp_async_commit();
    next = place(e);
  };
#pragma unroll
  for (int s = 0; s < R::ST - 1; ++s) issue(s);

  const int gr = lane >> 2, gc = lane & 3;
  uint32_t qb[KS][2];
  {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + static_cast<long long>(rh) * D) + gc;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      qb[k][0] = src[8 * k];
      qb[k][1] = src[8 * k + 4];
    }
  }
  float o[KS][4], m = neg_inf(), l = 0.f;                  // m: the whole warp's; l: of the lane's keys
#pragma unroll
  for (int n = 0; n < KS; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  for (int it = 0; it < mine; ++it) {
    issue(it + R::ST - 1);
    cp_async_wait<R::ST - 1>();
    __syncwarp();
    const uint32_t mask = there[0];
    if (mask == 0) continue;
    const uint32_t kt = kv.keys(it, smem, warp);
    float s[4];
    step_scores<D>(kt, qb, lane, s);
    const float a = mask >> gr & 1 ? s[0] * p.scale_log2 : neg_inf();
    const float c = mask >> (gr + 8) & 1 ? s[2] * p.scale_log2 : neg_inf();
    float x = fmaxf(a, c);
#pragma unroll
    for (int y = 4; y < 32; y <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, y));
    if (x > m) {                                           // the same in every lane
      const float f = fast_exp2(m - x);
      m = x;
      l *= f;
#pragma unroll
      for (int n = 0; n < KS; ++n) o[n][0] *= f, o[n][1] *= f, o[n][2] *= f, o[n][3] *= f;
    }
    const float z = m == neg_inf() ? 0.f : m;
    const float wa = fast_exp2(a - z), wc = fast_exp2(c - z);
    l += wa + wc;
    const float ha = round_bf16(wa), hc = round_bf16(wc), ma = round_bf16(wa - ha), mc = round_bf16(wc - hc);
    const uint32_t pa = gc == 0 ? pack_bf16(ha, ma) : gc == 1 ? pack_bf16(wa - ha - ma, 0.f) : 0u;
    const uint32_t pc = gc == 0 ? pack_bf16(hc, mc) : gc == 1 ? pack_bf16(wc - hc - mc, 0.f) : 0u;
    step_values<D>(kt + R::HALF, transpose_8x8(pa), transpose_8x8(pc), lane, o);
    __syncwarp();   // every lane has read the slot that the next step's copies fill
  }
  cp_async_wait<0>();
#pragma unroll
  for (int y = 4; y < 32; y <<= 1) l += __shfl_xor_sync(0xffffffffu, l, y);
  __syncthreads();
  // the warps' parts: [warp][OS], then (m, l) of each; the CTA's behind them
  float* mo = reinterpret_cast<float*>(smem);
  float* ml = mo + R::NW * OS;
  float* co = ml + R::NW * 2;
#pragma unroll
  for (int n = 0; n < KS; ++n) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      // columns 0 and 1 are lane gc = 0's, column 2 lane gc = 1's
      const float lo = __shfl_down_sync(0xffffffffu, o[n][e], 1);
      if (gc == 0) mo[warp * OS + 16 * n + gr + 4 * e] = (lo + o[n][e + 1]) + o[n][e];
    }
  }
  if (lane == 0) ml[2 * warp] = m, ml[2 * warp + 1] = l;
  __syncthreads();
  const int c = threadIdx.x;                               // channel
  float cm = neg_inf(), cl = 0.f, acc = 0.f;
  if (c < D) {
#pragma unroll
    for (int w = 0; w < R::NW; ++w) cm = fmaxf(cm, ml[2 * w]);
    const float z = cm == neg_inf() ? 0.f : cm;
#pragma unroll
    for (int w = 0; w < R::NW; ++w) {
      const float f = fast_exp2(ml[2 * w] - z);
      cl = fmaf(f, ml[2 * w + 1], cl);
      acc = fmaf(f, mo[w * OS + c], acc);
    }
  }
  if (p.parts > 1) {
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    if (c < D && rank > 0) {
      co[c] = acc;
      if (c == 0) co[D] = cm, co[D + 1] = cl;
    }
    cluster.sync();
    if (c < D && rank == 0) {
      for (int r = 1; r < p.parts; ++r) {
        const float* ro = cluster.map_shared_rank(co, r);
        const float rm = ro[D], n = fmaxf(cm, rm), z = n == neg_inf() ? 0.f : n;
        const float f = fast_exp2(cm - z), e = fast_exp2(rm - z);
        cl = fmaf(e, ro[D + 1], cl * f);
        acc = fmaf(e, ro[c], acc * f);
        cm = n;
      }
    }
    cluster.sync();   // no CTA leaves while its part is being read
  }
  if (rank > 0) return;
  if (!sp.ok && c == 0) atomicOr(p.status, kStBadLen);     // told here: at the start the whole row would wait for the length
  float value = cl == 0.f ? 0.f : acc / cl;                // 0 in threads without a channel
  // an infinite value under a weight whose lower terms are zero came in as 0 * inf
  if (__syncthreads_or(!finite(value) && cl == cl))
    value = sparse_row_not_finite<D>(p, rh, h, row, SequenceRows(p.rows, b), len, value, reinterpret_cast<uint32_t*>(co));
  if (c < D) p.out[static_cast<long long>(rh) * D + c] = value;
}

}  // namespace pivot

// Dense causal attention over a paged cache for many rows per key head, on the
// 5th-generation tensor cores.  The mathematics and the packing of rows are
// those of paged_attend.cuh.
//
// A CTA takes 256 packed rows (two tiles of 128) of one key head and walks the
// key axis in tiles of 128 keys:
//   warp 0      producer: looks each tile's pages up in the block table and
//               brings keys and values in by TMA, one box per page and 64
//               channels (a page of 128 rows or more: per tile), through one
//               ring of key and value tiles
//   warp 2      goes through the values of the last tiles (mixed), which some rows
//               see in part, between their landing and the products
//   warps 2, 3  the producer for pages of fewer than 8 rows (GATHER), which TMA
//               cannot lay into the swizzled tiles: every key row looked up by
//               itself and copied in 16-byte pieces (cp.async)
//   warp 1      TMEM allocator and MMA issuer (one elected thread):
//               S_t = Q_t K^T (128 x 128 x d), O_t += P_t V (128 x d x 128),
//               P_t read from TMEM, V as it lies (keys in rows: N-major)
//   warps 4-7, 8-11  softmax of tile 0 and tile 1: thread = row.  128 scores in
//               registers, so maximum and sum need no exchange; P_t goes back to
//               TMEM in bf16 over the scores it came from
// While one tile's softmax runs, the tensor cores work for the other.  TMEM:
// S_0, S_1 (128 columns each), O_0, O_1 (d each).
//
// O is rescaled only when a row's maximum has grown by more than 2^40 since the
// last time.  Until then the row's reference stays behind its maximum and the
// weights reach up to 2^40, which fp32 sums and bf16 weights hold as exactly as
// those up to 1 (their sums stay below 2^127 for any length, and a value that
// were to overflow them ends in the row by row form).  With keys of uneven
// length some row of a warp grows by 2^8 in most early tiles: rescaling at that
// took 279 us for 264 (8192-token prefill, 16 heads, 1 % of the keys four times
// as long).  The score tile's commit also tells that the earlier P V product is done
// (one thread issues both), so the softmax warps may change O between it and
// their own arrival.
#pragma once

#include "paged_attend.cuh"

namespace pivot {

template <int D>
struct TcCfg {
  static constexpr int BM = 128, BN = 128;
  static constexpr int ATOMS = D / 64;                   // 64-channel halves of a row
  static constexpr int TILE = BN * D * 2;                // a key, value or query tile
  static constexpr int ATOM = BN * 128;                  // one half of it
  static constexpr int NST = D == 128 ? 5 : 8;           // ring of key and value tiles
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_RING = 2 * TILE;
  static constexpr int OFF_BAR = OFF_RING + NST * TILE;
  static constexpr int SMEM = OFF_BAR + 288 + 1024;      // barriers, alignment slack
  static constexpr int THREADS = 128 + 256;               // three warpgroups
  static constexpr int MIXED = 3;                        // key tiles that some of a CTA's rows see in part
  static constexpr uint32_t S_COL = 0, O_COL = 256;      // + t * 128, + t * D
  // registers a thread: 168 at launch, moved from the first warpgroup to the softmax ones, which hold 128 scores
  static constexpr int REGS_FEW = 72, REGS_MANY = 216;
  static_assert(REGS_FEW + 2 * REGS_MANY <= 3 * 168, "register shares");
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(SMEM > 116 * 1024, "one CTA an SM: each takes the whole TMEM");
};

constexpr float kRescaleLog2 = 40.f;
// Of 16 pairs of weights, how many exp2_poly makes.  At 64 channels the special
// functions bound the loop (half the products for as many weights): 3 of 16
// took 178 us for 197 (4 chunks of 2048 tokens, 16 heads, contexts of 2048);
// at 128 the products do, and any share is within 1 %.
template <int D>
constexpr int kPolyOf16 = D == 64 ? 3 : 0;
constexpr int kEarly = 3;      // quarters of a weight tile that are handed on ahead of the rest

// 2^x of two values in fp32 by arithmetic alone (no special-function unit):
// x = n + f with n whole and |f| <= 1/2, 2^f by its minimax polynomial of
// degree 5 (fitted here by the Remez exchange; relative error 7.5e-8, with the
// coefficients rounded to fp32 1.6e-7, with the arithmetic's roundings below
// 2.2e-7), and n added to the exponent.  x below -127
// gives 0 (a subnormal), x must not be NaN.
__device__ __forceinline__ void exp2_poly(float xa, float xb, float& a, float& b) {
  const float kMagic = 12582912.f;   // 1.5 2^23: adding it rounds to a whole number in the low bits
  const uint64_t magic = pair_f32(kMagic, kMagic), unmagic = pair_f32(-kMagic, -kMagic);
  const uint64_t x = pair_f32(fmaxf(xa, -127.f), fmaxf(xb, -127.f));
  const uint64_t n = add2(x, magic);
  const uint64_t f = fma2(add2(n, unmagic), pair_f32(-1.f, -1.f), x);
  uint64_t r = pair_f32(0x1.5c08e6p-10f, 0x1.5c08e6p-10f);
  r = fma2(r, f, pair_f32(0x1.3d0c52p-7f, 0x1.3d0c52p-7f));
  r = fma2(r, f, pair_f32(0x1.c6b6e4p-5f, 0x1.c6b6e4p-5f));
  r = fma2(r, f, pair_f32(0x1.ebf918p-3f, 0x1.ebf918p-3f));
  r = fma2(r, f, pair_f32(0x1.62e428p-1f, 0x1.62e428p-1f));
  r = fma2(r, f, pair_f32(0x1.000002p+0f, 0x1.000002p+0f));
  float na, nb, ra, rb;
  unpair_f32(n, na, nb);
  unpair_f32(r, ra, rb);
  a = __uint_as_float((__float_as_uint(na) << 23) + __float_as_uint(ra));
  b = __uint_as_float((__float_as_uint(nb) << 23) + __float_as_uint(rb));
}

// Rows that are not finite though the sum of their weights is, or whose values were cleaned (paged_attend.cuh), by a
// softmax warp: a bit of `todo` each, lane x's row.  seq: sequence and tile.  What the kernel knows besides is worked out
// again, so that its loop need not hold it.
template <int D>
__device__ __forceinline__ void settle_rows(const PagedAttendParams& p, const volatile int* seq, unsigned todo) {
  constexpr int CL = D / 32;
  const int lane = threadIdx.x & 31, b = seq[0];
  const int hk = static_cast<int>(blockIdx.x % p.Hk), split = static_cast<int>(blockIdx.x / p.Hk % p.nsplit_many);
  const NewSpan sp = p.rows.span(b);
  const int chunk = chunk_of(sp, p), kbeg = split * chunk;
  // the lane's packed row (rows behind the last have no bit), and the keys that it sees: rows further on see no fewer
  const int pr = min(seq[1] * (2 * TcCfg<D>::BM) + static_cast<int>(threadIdx.x) - 128, sp.n * p.grp - 1), tok = pr / p.grp;
  const long long row = (static_cast<long long>(sp.tok0) + tok) * p.Hq + hk * p.grp + (pr - tok * p.grp);
  const int seen = min(sp.ok ? sp.len - sp.n + p.self_key + tok : 0, kbeg + chunk);
  const SequenceRows rows(p.rows, b);
  auto cache_row = [&](int j) { return rows.row_or(j, -2); };
  FirstNonFinite<D> odd;
  odd.look(p, p.Hk, hk, kbeg, __shfl_sync(0xffffffffu, seen, 31 - __clz(todo)), cache_row, lane);
  for (; todo; todo &= todo - 1) {
    const int x = __ffs(todo) - 1;
    const long long rx = __shfl_sync(0xffffffffu, row, x);
    const int lx = __shfl_sync(0xffffffffu, seen, x);
    const long long ax = static_cast<long long>(split) * p.rows.T * p.Hq + rx;
    float* const part = p.part_o + ax * D + lane * CL;
    uint16_t* const out = p.out + rx * D + lane * CL;
    float o[CL], z;
#pragma unroll
    for (int c = 0; c < CL; ++c) o[c] = p.part_o ? part[c] : __uint_as_float(static_cast<uint32_t>(out[c]) << 16);
    if (odd.settle(o, lx)) {
      attend_row_exact<D>(p, p.Hk, hk, rx, kbeg, lx, cache_row, lane, o, &z);
      if (lane == 0) {
        if (p.part_o)
          p.part_lse[ax] = z;
        else if (p.lse)
          p.lse[rx] = z * kLn2;
      }
    }
    if (p.part_o) {
#pragma unroll
      for (int c = 0; c < CL; ++c) part[c] = o[c];
    } else {
#pragma unroll
      for (int c = 0; c < CL; c += 2) *reinterpret_cast<uint32_t*>(out + c) = pack_bf16(o[c], o[c + 1]);
    }
  }
}

template <int D, bool GATHER>
__global__ void __launch_bounds__(TcCfg<D>::THREADS, 1)
attend_tiles_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ PagedAttendParams p) {
  using C = TcCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t ring = sbase + C::OFF_RING;
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::NST + s); };
  constexpr int B0 = 2 * C::NST;
  const uint32_t q_bar = bar0 + 8u * B0;
  auto s_bar = [&](int t) { return bar0 + 8u * (B0 + 1 + t); };    // scores of tile t are in TMEM
  auto p_bar = [&](int t) { return bar0 + 8u * (B0 + 3 + t); };    // the early weights of tile t are in TMEM
  auto w_bar = [&](int t) { return bar0 + 8u * (B0 + 5 + t); };    // ... the rest of them
  auto o_bar = [&](int t) { return bar0 + 8u * (B0 + 7 + t); };    // the last product of tile t is done
  auto land_bar = [&](int k) { return bar0 + 8u * (B0 + 9 + k); }; // the values of the k-th mixed tile have landed
  const uint32_t done_bar = bar0 + 8u * (B0 + 9 + C::MIXED);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 240);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 244);
  int* seq_s = reinterpret_cast<int*>(smem + C::OFF_BAR + 248);
  volatile int* dirty_flag = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 256);   // some were not finite

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  grid_launch_dependents();
  // key heads innermost (neighbouring CTAs share pages), the longest row tiles first
  const unsigned bid = blockIdx.x;
  const int hk = static_cast<int>(bid % p.Hk);
  const int split = static_cast<int>(bid / p.Hk % p.nsplit_many);
  const int flat = p.tiles - 1 - static_cast<int>(bid / p.Hk / p.nsplit_many);
  if (warp == 0) {
    int tile = 0;
    const int b = locate_tile(p, 2 * C::BM, flat, lane, &tile);
    // a barrier a lane, in their order above
    constexpr int BARS = B0 + 10 + C::MIXED;
    static_assert(BARS <= 30, "a barrier a lane, below the words at 240");
    if (lane < BARS)
      mbar_init(bar0 + 8u * lane, lane < C::NST ? (GATHER ? 64 : 1) : lane == B0 ? 256 : lane >= B0 + 3 && lane < B0 + 7 ? 4 : 1);
    if (lane == 0) {
      seq_s[0] = b;
      seq_s[1] = tile;
      *abort_flag = 0;
      *dirty_flag = 0;
    }
    fence_barrier_init();
  }
  __syncthreads();
  const int b = seq_s[0], r0 = seq_s[1] * (2 * C::BM);
  if (b < 0) return;
  const NewSpan sp = p.rows.span(b);
  const int total = sp.n * p.grp;                           // packed rows of the sequence
  if (!sp.ok && threadIdx.x == 0) atomicOr(p.status, kStBadLen);
  if (r0 >= total) return;
  const int pos0 = sp.len - sp.n + p.self_key;
  auto lim_of = [&](int r) { return sp.ok ? pos0 + r / p.grp : 0; };
  const int chunk = chunk_of(sp, p);
  const int kbeg = split * chunk;
  // keys of the part that the last row of tile t sees; its key tiles
  int kend[2], nk[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = r0 + t * C::BM, last = min(first + C::BM, total) - 1;
    kend[t] = first < total ? min(lim_of(last), kbeg + chunk) : 0;
    nk[t] = max(0, (kend[t] - kbeg + C::BN - 1) / C::BN);
  }
  const int n = max(nk[0], nk[1]), end = max(kend[0], kend[1]);
  // From the first key on that some row does not see, and from its tile (256 rows
  // see keys at most 255 apart, so C::MIXED tiles), the values are gone through
  // between landing and the products: made finite and, behind the last key that
  // anyone sees, zeros (0 * NaN is not 0).
  auto first_unseen = [&]() { return lim_of(r0); };
  auto first_mixed = [&](int unseen) { return max(0, (unseen - kbeg) / C::BN); };
  if (n == 0 && split > 0) return;                          // the join reads no part a row has no keys in

  // the shares move inside each side's branch: ahead of it, the whole of both sides gets the smaller one
  if (warp < 4) {
    regs_dec<C::REGS_FEW>();
  }
  if (!GATHER && warp == 0) {
    // ------------------------------------------------------------ producer
    const int page_rows = min(1 << p.rows.log2_page, C::BN);
    const int boxes = C::BN / page_rows;                    // pages (or parts of one) a tile: at most 16
    const int out_row = p.rows.num_pages << p.rows.log2_page;   // past the cache: TMA fills zeros
    // cache row of the page's part that lane l loads of tile i
    auto box_row = [&](int i) -> int {
      const int j = kbeg + i * C::BN + lane * page_rows;
      if (lane >= boxes || i >= n || j >= end) return out_row;
      const long long row = p.rows.row(b, j);
      if (row < 0) {
        atomicOr(p.status, kStBadPage);
        return out_row;
      }
      return static_cast<int>(row);
    };
    int use = 0;
    bool ok = true;
    const int mixed = first_mixed(first_unseen());
    // the barrier of tile i's values
    auto value_bar = [&](int i, int s) { return i < mixed ? full_bar(s) : land_bar(i - mixed); };
    // the next slot of the ring, empty, its barrier told of a tile (of values, or of keys: i < 0); -1: given up
    auto slot = [&](int i) -> int {
      const int s = use % C::NST, u = use / C::NST;
      if (u > 0) {
        ok = ok && mbar_wait(empty_bar(s), (u - 1) & 1, abort_flag, p.status, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) return -1;
      if (lane == 0) mbar_arrive_expect_tx(i < 0 ? full_bar(s) : value_bar(i, s), C::TILE);
      __syncwarp();
      ++use;
      return s;
    };
    auto load = [&](const CUtensorMap* tm, int s, uint32_t bar, int row) {
      if (lane < boxes) {
#pragma unroll
        for (int a = 0; a < C::ATOMS; ++a)
          tma_load_3d(ring + s * C::TILE + a * C::ATOM + lane * page_rows * 128, tm, bar, a * 64, hk, row);
      }
    };
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    int next = box_row(0);
    for (int i = 0; i < n; ++i) {
      const int row = next;
      next = box_row(i + 1);
      int s = slot(-1);
      if (s < 0) break;
      load(&tm_k, s, full_bar(s), row);
      s = slot(i);
      if (s < 0) break;
      load(&tm_v, s, value_bar(i, s), row);
    }
    // never leave the CTA with a copy still landing in its shared memory
    for (int u = max(0, use - C::NST); u < use; ++u) {
      const int s = u % C::NST;
      if (u % 2 == 1 && u / 2 >= mixed)
        mbar_wait_cleanup(land_bar(u / 2 - mixed), 0);
      else
        mbar_wait_cleanup(full_bar(s), (u / C::NST) & 1);
    }
  } else if (!GATHER && warp == 2) {
    // ------------------------------------------------------------ values of the mixed tiles
    const int unseen = first_unseen(), mixed = first_mixed(unseen);
    for (int i = mixed; i < n; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait<true>(land_bar(i - mixed), 0, abort_flag, p.status, p.wait_ns))) break;
      const int s = (2 * i + 1) % C::NST, j0 = kbeg + i * C::BN;
      uint4* const at = reinterpret_cast<uint4*>(smem + C::OFF_RING + s * C::TILE);
      // rows [from, upto) hold what some see, those behind it nothing; in 16-byte pieces, eight a row and atom
      const int from = max(0, unseen - j0) * 8, upto = min(C::BN, end - j0) * 8;
      for (int x = upto + lane; x < C::BN * 8; x += 32)
#pragma unroll
        for (int a = 0; a < C::ATOMS; ++a) at[a * (C::ATOM / 16) + x] = make_uint4(0, 0, 0, 0);
      constexpr int STEP = 8 / C::ATOMS;                    // eight loads in flight
      bool any = false;
      for (int x0 = from + lane; x0 < upto; x0 += 32 * STEP) {
        uint4 v[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) v[y] = at[y % C::ATOMS * (C::ATOM / 16) + min(x0 + y / C::ATOMS * 32, upto - 1)];
        uint32_t odd = 0;
#pragma unroll
        for (int y = 0; y < 8; ++y) odd = odd_so_far(odd, v[y]);
        if (!odd) continue;
        any = true;
#pragma unroll
        for (int y = 0; y < 8; ++y)
          at[y % C::ATOMS * (C::ATOM / 16) + min(x0 + y / C::ATOMS * 32, upto - 1)] = cleaned(v[y]);
      }
      if (any) *dirty_flag = 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full_bar(s));
    }
  } else if (GATHER && (warp == 2 || warp == 3)) {
    // ------------------------------------------------------------ producers, row by row
    constexpr int CH = D / 8, RP = 32 / CH;                 // pieces of a row, rows that a warp's 32 pieces make
    const int unseen = first_unseen(), mixed = first_mixed(unseen);
    const int ch = lane % CH, kw = (warp - 2) * 64;         // the lane's piece; the warp's first key of a tile
    const uint16_t* kb = p.kpages + static_cast<long long>(hk) * D + ch * 8;
    const uint16_t* vb = p.vpages + static_cast<long long>(hk) * D + ch * 8;
    const long long stride = static_cast<long long>(p.Hk) * D;
    // cache row of key kw + 32 half + lane of tile i, -1: none (its rows become zeros)
    auto key_row = [&](int i, int half) -> int {
      const int j = kbeg + i * C::BN + kw + 32 * half + lane;
      if (i >= n || j >= end) return -1;
      const long long row = p.rows.row(b, j);
      if (row < 0) atomicOr(p.status, kStBadPage);
      return static_cast<int>(row);
    };
    int use = 0;
    bool ok = true;
    // from: the first key of the tile whose piece is gone through (values alone)
    auto fill = [&](const uint16_t* base, int r0_, int r1_, int from) {
      const int s = use % C::NST, u = use / C::NST;
      if (u > 0) {
        ok = mbar_wait(empty_bar(s), (u - 1) & 1, abort_flag, p.status, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
      }
      const uint32_t dst = ring + s * C::TILE + (ch >> 3) * C::ATOM;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll 8
        for (int x = 0; x < 32 / RP; ++x) {
          const int k = x * RP + lane / CH, key = kw + 32 * half + k;
          const int row = __shfl_sync(0xffffffffu, half ? r1_ : r0_, k);
          cp_async_16(dst + key * 128 + (((ch & 7) ^ (key & 7)) << 4), base + max(row, 0) * stride, row < 0 ? 0u : 16u);
        }
      }
      if (from < C::BN) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        bool any = false;
        for (int key = kw + lane / CH; key < kw + 64; key += RP) {
          if (key < from) continue;
          uint4* const v = reinterpret_cast<uint4*>(smem + C::OFF_RING + s * C::TILE + (ch >> 3) * C::ATOM + key * 128 +
                                                    (((ch & 7) ^ (key & 7)) << 4));
          if (odd_so_far(0u, *v)) {
            *v = cleaned(*v);
            any = true;
          }
        }
        if (any) *dirty_flag = 1;
        mbar_arrive(full_bar(s));
      } else {
        cp_async_arrive_noinc(full_bar(s));
      }
      ++use;
    };
    int n0 = key_row(0, 0), n1 = key_row(0, 1);
    for (int i = 0; i < n && ok; ++i) {
      const int c0 = n0, c1 = n1;
      n0 = key_row(i + 1, 0);
      n1 = key_row(i + 1, 1);
      fill(kb, c0, c1, C::BN);
      if (ok) fill(vb, c0, c1, i < mixed ? C::BN : max(0, unseen - (kbeg + i * C::BN)));
    }
    // never leave the CTA with a copy still landing in its shared memory
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop and one lane issues: a loop of one lane
    // would move every descriptor from vector to uniform registers, which took
    // longer than the products (73 cycles an instruction for 64 of work).
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
    tc_fence_before();
    named_barrier(1, 32 + 256);                              // its address, to the softmax warps
    tc_fence_after();
    if (n > 0) {
      constexpr uint32_t idesc_s = umma_idesc_bf16(C::BM, C::BN);
      constexpr uint32_t idesc_o = umma_idesc_bf16(C::BM, D) | kIdescBNMajor;
      const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_slot, 0);
      const int nu = __shfl_sync(0xffffffffu, n, 0);
      const int n0 = __shfl_sync(0xffffffffu, nk[0], 0), n1 = __shfl_sync(0xffffffffu, nk[1], 0);
      const uint64_t qd = sw128_kmajor_desc(sbase + C::OFF_Q), kd = sw128_kmajor_desc(ring);
      const uint64_t vd = sw128_nmajor_desc(ring, C::ATOM);
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait<GATHER>(bar, parity, abort_flag, p.status, p.wait_ns)) != 0;
      };
      // slot and phase of the ring's next tile (key tile i, then value tile i, ...)
      int slot = 0;
      uint32_t phase = 0;
      auto advance = [&]() {
        if (++slot == C::NST) slot = 0, phase ^= 1;
      };
      auto scores = [&](int t, int ks) {
        const uint64_t a = qd + static_cast<uint64_t>(t * (C::TILE >> 4)), b_ = kd + static_cast<uint64_t>(ks * (C::TILE >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = ((kk >> 2) * C::ATOM + (kk & 3) * 32) >> 4;
          umma_bf16(tm + C::S_COL + t * C::BN, a + off, b_ + off, idesc_s, kk > 0 ? 1u : 0u);
        }
        umma_commit(s_bar(t));
      };
      auto products = [&](int t, int vs, int k0, int k1, bool first) {
        const uint64_t b_ = vd + static_cast<uint64_t>(vs * (C::TILE >> 4));
#pragma unroll
        for (int kk = k0; kk < k1; ++kk)
          umma_bf16_ts(tm + C::O_COL + t * D, tm + C::S_COL + t * C::BN + kk * 8, b_ + static_cast<uint64_t>(kk * (2048 >> 4)),
                       idesc_o, first && kk == 0 ? 0u : 1u);
      };
      bool ok = wait(q_bar, 0) && wait(full_bar(0), 0);
      if (ok) {
        if (GATHER) fence_proxy_async_smem();               // the rows were written by threads, the products read them
        tc_fence_after();
        if (elect_one()) {
          if (n0 > 0) scores(0, 0);
          if (n1 > 0) scores(1, 0);
          umma_commit(empty_bar(0));
        }
        __syncwarp();
      }
      advance();
      for (int i = 0; i < nu && ok; ++i) {
        // the tile's values and the next tile's keys, nearly always landed: both asked in one vote
        const int vs = slot;
        const uint32_t vph = phase;
        advance();
        const int ks = slot;
        const uint32_t kph = phase;
        const bool more = i + 1 < nu;
        if (more) advance();
        const bool v_in = mbar_try_wait(full_bar(vs), vph), k_in = !more || mbar_try_wait(full_bar(ks), kph);
        if (!__all_sync(0xffffffffu, v_in && k_in)) {
          ok = wait(full_bar(vs), vph) && (!more || wait(full_bar(ks), kph));
          if (!ok) break;
        }
        if (GATHER) fence_proxy_async_smem();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int nt = t == 0 ? n0 : n1;
          if (i >= nt) continue;
          ok = ok && wait(p_bar(t), i & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) products(t, vs, 0, 2 * kEarly, i == 0);
          __syncwarp();
          ok = wait(w_bar(t), i & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            products(t, vs, 2 * kEarly, 8, i == 0);
            if (i + 1 < nt)
              scores(t, ks);
            else
              umma_commit(o_bar(t));
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) {
          umma_commit(empty_bar(vs));
          if (i + 1 < nu) umma_commit(empty_bar(ks));
        }
        __syncwarp();
      }
      // all products must be complete before TMEM is given back
      if (elect_one()) umma_commit(done_bar);
      __syncwarp();
      mbar_wait_cleanup(done_bar, 0);
    }
  } else if (warp >= 4) {
    regs_inc<C::REGS_MANY>();
    // ------------------------------------------------------------ softmax
    const int tid = threadIdx.x - 128;
    const int t = tid >> 7;
    const int r = (warp & 3) * 32 + lane;                   // row of the tile = TMEM lane
    // both query tiles into shared memory in the swizzled layout: a thread takes
    // one 16-byte piece of every RS-th row (rows behind the last repeat it: they
    // go nowhere), all of its loads in flight
    constexpr int CH = D / 8, RS = 256 / CH;
    {
      const int ch = tid % CH, row0 = tid / CH;
      int tok = (r0 + row0) / p.grp, rem = (r0 + row0) % p.grp;   // of the packed row at hand
      const int dtok = RS / p.grp, drem = RS % p.grp;
      const int ltok = (total - 1) / p.grp, lrem = p.grp - 1;      // of the last one
      const uint16_t* qb = p.q + (static_cast<long long>(sp.tok0) * p.Hq + hk * p.grp) * D + ch * 8;
      uint4 v[CH];
#pragma unroll
      for (int y = 0; y < CH; ++y) {
        const bool in = tok <= ltok;
        v[y] = __ldg(reinterpret_cast<const uint4*>(
            qb + (static_cast<long long>(in ? tok : ltok) * p.Hq + (in ? rem : lrem)) * D));
        tok += dtok;
        rem += drem;
        if (rem >= p.grp) rem -= p.grp, ++tok;
      }
#pragma unroll
      for (int y = 0; y < CH; ++y) {
        const int row = row0 + RS * y;
        *reinterpret_cast<uint4*>(smem + C::OFF_Q + (row >> 7) * C::TILE + (ch >> 3) * C::ATOM + (row & 127) * 128 +
                                  (((ch & 7) ^ (row & 7)) << 4)) = v[y];
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(q_bar);
    named_barrier(1, 32 + 256);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int pr = r0 + t * C::BM + r;                      // packed row
    // row of q and out, -1 behind the last
    const int qrow = pr < total ? (sp.tok0 + pr / p.grp) * p.Hq + hk * p.grp + pr % p.grp : -1;
    const int lim = lim_of(min(pr, total - 1));
    // the warp's first row sees the fewest keys (rows behind the last repeat it and go nowhere)
    const int wlim = lim_of(min(r0 + t * C::BM + (warp & 3) * 32, total - 1));
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + C::S_COL + t * C::BN;
    const uint32_t to = tmem + lane_base + C::O_COL + t * D;
    float m = neg_inf(), l = 0.f;                           // reference maximum (raw scores), sum of weights
    float dl = 0.f;                                         // what rounding the heaviest weight of each tile adds
    bool ok = true;
    const int mine = t == 0 ? nk[0] : nk[1];
    for (int i = 0; i < mine; ++i) {
      ok = mbar_wait(s_bar(t), i & 1, abort_flag, p.status, p.wait_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      uint32_t s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(ts + 32 * c, s + 32 * c);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 128; ++c) reg_fence(s[c]);
      const int j0 = kbeg + i * C::BN;
      if (j0 + C::BN > wlim) {
        const int seen = lim - j0;
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= seen) s[c] = 0xff800000u;
      }
      float mx4[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) mx4[c] = max3_nan(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]), neg_inf());
#pragma unroll
      for (int c = 8; c < 128; c += 2)
        mx4[(c >> 1) & 3] = max3_nan(mx4[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
      const float tile_mx = max3_nan(max3_nan(mx4[0], mx4[1], mx4[2]), mx4[3], neg_inf());
      // NaN where a score is: the reference and with it the whole row then become NaN
      const float mx = max3_nan(tile_mx, m, neg_inf());
      if (i == 0) {
        m = mx;
      } else if (__any_sync(0xffffffffu, !((mx - m) * p.scale_log2 <= kRescaleLog2))) {
        const float f = mx == neg_inf() ? 1.f : fast_exp2((m - mx) * p.scale_log2);
        m = mx;
        l *= f;
        dl *= f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(to + 32 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            reg_fence(o[x]);
            o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
          }
          tmem_st_32x32b_x32(to + 32 * c, o);
        }
      }
      // no key seen yet: every weight is 0; an infinite score: every weight is NaN
      const float off = fabsf(m) < __int_as_float(0x7f800000) ? -m * p.scale_log2 : m == neg_inf() ? 0.f : __int_as_float(0x7fffffff);
      const uint64_t scale2 = pair_f32(p.scale_log2, p.scale_log2), off2 = pair_f32(off, off);
      uint64_t l2[2] = {0, 0};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint64_t x = pair_f32(__uint_as_float(s[32 * h + 2 * c]), __uint_as_float(s[32 * h + 2 * c + 1]));
          float a, e;
          unpair_f32(fma2(x, scale2, off2), a, e);
          if (c * kPolyOf16<D> % 16 < kPolyOf16<D> && kPolyOf16<D> > 0) {
            exp2_poly(a, e, a, e);
          } else {
            a = fast_exp2(a);
            e = fast_exp2(e);
          }
          l2[c & 1] = add2(l2[c & 1], pair_f32(a, e));
          w[c] = pack_bf16(a, e);
        }
        tmem_st_32x32b_x16(ts + 16 * h, w);
        if (h == kEarly - 1) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_bar(t));
        }
      }
      float la, lb;
      unpair_f32(add2(l2[0], l2[1]), la, lb);
      l += la + lb;
      const float top = fast_exp2(fmaf(tile_mx, p.scale_log2, off));
      dl += round_bf16(top) - top;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(w_bar(t));
    }
    if (ok && mine > 0) ok = mbar_wait(o_bar(t), 0, abort_flag, p.status, p.wait_ns);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      // The result is normalised by the sum of the weights as the second product had them.  Rounding each
      // moves it by up to 2^-8, which averages out unless a few weights make up the sum; so of every tile the
      // heaviest one's rounding is taken along (error of the 8192-token prefill's output against 64 bits: 0.0018; 0.0023
      // without it; summing every rounded weight as well took 7 % of the time).
      // A row that sees no key of the part keeps its reference at -inf; its sum is 0 only up to exp2_poly's
      // subnormals, over which it would come out NaN (and, though right, worked out key by key: 6 us).
      const bool sees = mine > 0 && m != neg_inf();
      const float inv = sees ? 1.f / (l + dl) : 0.f;
      const float lse2 = sees ? fmaf(m, p.scale_log2, log2f(l)) : neg_inf();
      const bool row_ok = qrow >= 0;
      const long long row = max(qrow, 0);
      const long long at = static_cast<long long>(split) * p.rows.T * p.Hq + row;
      bool fine = true;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (mine > 0) {
          tmem_ld_32x32b_x32(to + 32 * c, o);
          tmem_ld_wait();
        }
        float f[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          if (mine > 0) reg_fence(o[x]);
          f[x] = mine > 0 ? __uint_as_float(o[x]) * inv : 0.f;
          fine = fine && finite(f[x]);
        }
        if (!row_ok) continue;
        if (p.part_o) {
#pragma unroll
          for (int x = 0; x < 32; x += 4)
            *reinterpret_cast<float4*>(p.part_o + at * D + 32 * c + x) = make_float4(f[x], f[x + 1], f[x + 2], f[x + 3]);
        } else {
#pragma unroll
          for (int x = 0; x < 32; x += 8) store8_bf16(p.out + row * D + 32 * c + x, f + x);
        }
      }
      if (row_ok) {
        if (p.part_o)
          p.part_lse[at] = lse2;
        else if (p.lse)
          p.lse[row] = lse2 * kLn2;
      }
      // rows that are not finite though their sum is, or whose values were cleaned
      __syncwarp();   // (their first result, written by the row's own lane, comes before)
      unsigned todo = __ballot_sync(0xffffffffu, row_ok && (!fine || *dirty_flag) && l == l);
      if (todo) settle_rows<D>(p, seq_s, todo);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, 512);
  }
}

}  // namespace pivot

// Norm and rotary position of query and key heads in one pass, and the same
// pass writing keys and values into the pages of a paged cache.
//
// For a head row x (d channels) of a token at position pos:
//   norm (where a weight is given):  x_c <- x_c (mean_c x_c^2 + eps)^-1/2 w_c
//   rotation of the first rot channels: each pair (a, b) becomes
//     A (a cos t - b sin t), A (b cos t + a sin t),  t = pos f_i,
//   pair i being channels (i, i + rot/2) ("half") or (2i, 2i+1)
//   ("interleaved"); A is the amplitude of the frequencies' scaling.
// All in fp32 and rounded once, to bf16, when the row is stored.  The angle is
// taken in revolutions in fp64 and reduced there: at position 10^6 an fp32
// product would be off by 0.03 rad.
//
// Bound by memory (each channel read once, written once), and next to it by
// instructions, so the work of a head row is kept to its loads, stores and
// paired arithmetic: a block takes a few tokens and makes their rot/2 cosines
// and sines in shared memory (once a token, not once a head: the fp64 product
// and the sine cost as much as turning some ten heads).  d/16 lanes then take a
// head row, 16 channels a lane in 16-byte loads, the pair's two halves in the
// same lane, so that the only exchange is the norm's sum over those lanes; they
// stay with their token, whose cosines they hold in registers, and walk its
// heads, so that the next row's address is one addition away and its loads run
// ahead of the arithmetic.  Blocks of 128 threads, seven an SM: 8192 tokens of
// 32 heads of 128, normed and turned, take 29 us, a plain copy of the same bytes
// 25; 27 of them are the kernel without norm and rotation.  32768 tokens of 40
// heads: 123 us, the copy 113.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_rows.cuh"
#include "ptx.cuh"

namespace pivot {

struct HeadRows {
  const void* x;            // [T][n][d], strides in elements, channels adjacent
  const void* weight;       // [d] norm weight of x's type, or null: no norm
  long long token_stride, head_stride;
  int n;                    // heads (0: absent)
};

struct RopeParams {
  HeadRows q, k, v;
  const double* freqs;      // [rot/2] radians a position (rot = 0: unused)
  const int32_t* positions; // [T]; null: the tokens' cache rows (paged)
  uint16_t* out_q;          // [T][q.n][d]
  uint16_t* out_k;          // [T][k.n][d]; null: into the pages
  uint16_t* kpages;         // [pages][page_size][k.n][d]
  uint16_t* vpages;
  PagedRows rows;           // paged: where the tokens' rows lie
  int T, rot, tokens_per_block;
  float amplitude, eps;
  bool clear;               // paged: queries of tokens that are left out become zeros, else they stay
  int* status;
};

constexpr int kRopeNT = 128;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float round_bf16(float x) { return __uint_as_float(pack_bf16(x, 0.f) << 16); }

// Eight channels as they lie in memory, and as fp32.
template <class T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  }
};
template <>
struct Vec8<__half> {
  uint4 u;
  __device__ __forceinline__ void load(const __half* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};

__device__ __forceinline__ void store8_bf16(uint16_t* p, const float* f) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// T: type of x and the weights; HALF: channel pairs (i, i + rot/2), else (2i, 2i+1).
template <int D, bool HALF, class T>
__global__ void __launch_bounds__(kRopeNT, sizeof(T) == 2 ? 7 : 6) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LG = D / 16;              // lanes a head row
  constexpr int GROUPS = kRopeNT / LG;
  extern __shared__ float2 cs[];          // [tokens][rot / 2]
  __shared__ int pos_s[GROUPS];
  __shared__ long long row_s[GROUPS];     // cache row of the token; -1: leave the token out
  __shared__ float4 w_s[2][4][LG];        // norm weights of q and k, a lane's 16 in four pieces

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tb = p.tokens_per_block, gpt = GROUPS / tb;   // groups a token
  const int t0 = blockIdx.x * tb;
  const int nt = min(tb, p.T - t0);
  const bool paged = p.kpages != nullptr;
  const int half = p.rot >> 1;
  const int sub = threadIdx.x % LG, group = threadIdx.x / LG;
  const int tok = group / gpt, g = group % gpt;           // the group's token of the block, its place there
  const bool turns = sub < (p.rot >> 4);
  const int ca = HALF && turns ? 8 * sub : 16 * sub;      // the lane's two runs of 8 channels
  const int cb = HALF && turns ? 8 * sub + half : 16 * sub + 8;
  const long long t = t0 + min(tok, nt - 1);

  // A group walks rows g, g + gpt, ... of the token's queries, then keys, then
  // values, in rounds that are the same for all lanes of a warp (for the norm's
  // shuffles); behind a kind's last row it repeats its first and drops the
  // result.  The next row is loaded before the one at hand is worked on.
  auto first = [&](const HeadRows& src) {
    return static_cast<const T*>(src.x) + t * src.token_stride + min(g, src.n - 1) * src.head_stride;
  };
  const T* const q0 = p.q.n ? first(p.q) : nullptr;
  const T* const k0 = p.k.n ? first(p.k) : nullptr;
  const T* const v0 = p.v.n ? first(p.v) : nullptr;
  Vec8<T> va, vb;
  auto load = [&](const T* row) {
    va.load(row + ca);
    vb.load(row + cb);
  };
  load(q0 ? q0 : k0);   // on its way while the positions and angles are worked out
  const double freq0 = half ? p.freqs[threadIdx.x % half] : 0.0;
  if (threadIdx.x < 2 * LG) {
    const T* w = static_cast<const T*>(threadIdx.x < LG ? p.q.weight : p.k.weight);
    if (w != nullptr) {
      Vec8<T> wa, wb;
      float f[16];
      wa.load(w + ca);
      wb.load(w + cb);
      wa.get(f);
      wb.get(f + 8);
#pragma unroll
      for (int c = 0; c < 4; ++c)   // in the order of the register pairs below
        w_s[threadIdx.x / LG][c][sub] = HALF ? make_float4(f[2 * c], f[2 * c + 1], f[8 + 2 * c], f[9 + 2 * c])
                                             : make_float4(f[4 * c], f[4 * c + 2], f[4 * c + 1], f[4 * c + 3]);
    }
  }

  // lengths that do not fit are told of every sequence, those without new tokens too; at the end, the first ones'
  // being on their way from here
  const long long b0 = static_cast<long long>(blockIdx.x) * kRopeNT + threadIdx.x;
  NewSpan told{0, 0, 0, true};
  if (paged && b0 < p.rows.B) told = p.rows.span(static_cast<int>(b0));
  for (int i = warp; i < nt; i += kRopeNT / 32) {
    const int ti = t0 + i;
    int pos = 0;
    long long row = 0;
    if (paged) {
      const int b = find_sequence(p.rows, ti, lane);
      const NewSpan s = p.rows.span(b);
      row = -1;
      if (ti >= s.tok0 && ti < s.tok0 + s.n) {   // tokens behind the last sequence belong to none
        pos = s.len - s.n + (ti - s.tok0);
        if (s.ok) {
          row = p.rows.row(b, pos);
          if (row < 0 && lane == 0) atomicOr(p.status, kStBadPage);
        }
      }
    } else if (p.rot) {
      pos = p.positions[ti];
    }
    if (lane == 0) {
      pos_s[i] = pos;
      row_s[i] = row;
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < nt * half; x += kRopeNT) {
    const int i = x / half, c = x - i * half;
    const double freq = x < kRopeNT ? freq0 : p.freqs[c];
    double rev = static_cast<double>(pos_s[i]) * (freq * 0.15915494309189533577);   // 1 / (2 pi)
    rev -= rint(rev);
    float sn, co;
    sincospif(static_cast<float>(2.0 * rev), &sn, &co);
    cs[x] = make_float2(co * p.amplitude, sn * p.amplitude);
  }
  __syncthreads();

  const long long row = tok < nt ? row_s[tok] : -1;
  uint64_t co2[4] = {}, si2[4] = {};                      // of the lane's 8 pairs, two a register pair
  if (turns && tok < nt) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 x = cs[tok * half + 8 * sub + 2 * c], y = cs[tok * half + 8 * sub + 2 * c + 1];
      co2[c] = pair_f32(x.x, y.x);
      si2[c] = pair_f32(x.y, y.y);
    }
  }
  // One kind's rows: src from row0 on, to dst + head * D; next: the first row of the kind behind it.
  // put: the token's rows are written, as zeros where it is left out.
  auto walk = [&](const HeadRows& src, const T* row0, uint16_t* dst, bool put, bool turn, const float4 (*w)[LG],
                  const T* next) {
    const long long step = gpt * src.head_stride;
    const T* at = row0;
    dst += g * D;
    for (int h = g, left = (src.n + gpt - 1) / gpt; left > 0; --left, h += gpt, dst += gpt * D) {
      float f[16];
      va.get(f);
      vb.get(f + 8);
      at += step;
      if (left > 1)
        load(h + gpt < src.n ? at : row0);
      else if (next)
        load(next);
      // channels in register pairs: those of a lane's a halves, then its b halves
      uint64_t a[4], b[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        a[c] = HALF ? pair_f32(f[2 * c], f[2 * c + 1]) : pair_f32(f[4 * c], f[4 * c + 2]);
        b[c] = HALF ? pair_f32(f[8 + 2 * c], f[9 + 2 * c]) : pair_f32(f[4 * c + 1], f[4 * c + 3]);
      }
      if (src.weight != nullptr) {
        uint64_t s2 = mul2(a[0], a[0]);
#pragma unroll
        for (int c = 1; c < 4; ++c) s2 = fma2(a[c], a[c], s2);
#pragma unroll
        for (int c = 0; c < 4; ++c) s2 = fma2(b[c], b[c], s2);
        float lo, hi;
        unpair_f32(s2, lo, hi);
        float ss = lo + hi;
#pragma unroll
        for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        const uint64_t r2 = pair_f32(r, r);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float4 g4 = w[c][sub];
          a[c] = mul2(mul2(a[c], r2), pair_f32(g4.x, g4.y));
          b[c] = mul2(mul2(b[c], r2), pair_f32(g4.z, g4.w));
        }
      }
      if (turn) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint64_t y = a[c], z = b[c];
          a[c] = fma2(y, co2[c], mul2(z, si2[c] ^ 0x8000000080000000ull));   // the sines' signs turned
          b[c] = fma2(y, si2[c], mul2(z, co2[c]));
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (HALF) {
          unpair_f32(a[c], f[2 * c], f[2 * c + 1]);
          unpair_f32(b[c], f[8 + 2 * c], f[9 + 2 * c]);
        } else {
          unpair_f32(a[c], f[4 * c], f[4 * c + 2]);
          unpair_f32(b[c], f[4 * c + 1], f[4 * c + 3]);
        }
      }
      if (put && h < src.n) {
        if (row < 0) {
#pragma unroll
          for (int c = 0; c < 16; ++c) f[c] = 0.f;
        }
        store8_bf16(dst + ca, f);
        store8_bf16(dst + cb, f + 8);
      }
    }
  };
  const bool in = row >= 0;
  if (q0) walk(p.q, q0, p.out_q + t * p.q.n * D, in || (p.clear && tok < nt), turns, w_s[0], k0);
  if (k0) walk(p.k, k0, paged ? p.kpages + row * p.k.n * D : p.out_k + t * p.k.n * D, in, turns, w_s[1], v0);
  if (v0) walk(p.v, v0, p.vpages + row * p.v.n * D, in, false, nullptr, nullptr);
  for (long long b = b0 + static_cast<long long>(gridDim.x) * kRopeNT; paged && b < p.rows.B;
       b += static_cast<long long>(gridDim.x) * kRopeNT)
    if (!p.rows.span(static_cast<int>(b)).ok) atomicOr(p.status, kStBadLen);
  if (!told.ok) atomicOr(p.status, kStBadLen);
}

}  // namespace pivot

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
// Bound by memory (each channel read once, written once).  A block takes a few
// tokens: it first makes their rot/2 cosines and sines in shared memory (once
// a token, not once a head: the fp64 product and the sine cost as much as
// turning some ten heads), then d/16 lanes take one head each, 16 channels a
// lane in 16-byte loads, the pair's two halves in the same lane, so that the
// only exchange is the norm's sum over those lanes.
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
  int* status;
};

constexpr int kRopeNT = 256;
constexpr int kRopeMaxTok = 16;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

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
__global__ void __launch_bounds__(kRopeNT) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LG = D / 16;              // lanes a head
  constexpr int GROUPS = kRopeNT / LG;
  __shared__ float2 cs[kRopeMaxTok * D / 2];
  __shared__ int pos_s[kRopeMaxTok];
  __shared__ long long row_s[kRopeMaxTok];  // cache row of the token; -1: leave the token out

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * p.tokens_per_block;
  const int nt = min(p.tokens_per_block, p.T - t0);
  const bool paged = p.kpages != nullptr;

  for (int i = warp; i < nt; i += kRopeNT / 32) {
    const int t = t0 + i;
    int pos = 0;
    long long row = 0;
    if (paged) {
      const int b = find_sequence(p.rows, t, lane);
      const NewSpan s = p.rows.span(b);
      row = -1;
      if (t >= s.tok0 && t < s.tok0 + s.n) {   // tokens behind the last sequence belong to none
        pos = s.len - s.n + (t - s.tok0);
        if (s.ok) {
          row = p.rows.row(b, pos);
          if (row < 0 && lane == 0) atomicOr(p.status, kStBadPage);
        } else if (lane == 0) {
          atomicOr(p.status, kStBadLen);
        }
      } else if (!s.ok && lane == 0) {
        atomicOr(p.status, kStBadLen);
      }
    } else if (p.rot) {
      pos = p.positions[t];
    }
    if (lane == 0) {
      pos_s[i] = pos;
      row_s[i] = row;
    }
  }
  __syncthreads();
  const int half = p.rot >> 1;
  for (int x = threadIdx.x; x < nt * half; x += kRopeNT) {
    const int i = x / half, c = x - i * half;
    double rev = static_cast<double>(pos_s[i]) * (p.freqs[c] * 0.15915494309189533577);  // 1 / (2 pi)
    rev -= rint(rev);
    float sn, co;
    sincospif(static_cast<float>(2.0 * rev), &sn, &co);
    cs[x] = make_float2(co * p.amplitude, sn * p.amplitude);
  }
  __syncthreads();

  const int sub = threadIdx.x % LG;
  const bool turns = sub < (p.rot >> 4);
  const int ca = HALF && turns ? 8 * sub : 16 * sub;            // the lane's two runs of 8 channels
  const int cb = HALF && turns ? 8 * sub + half : 16 * sub + 8;
  const int heads = p.q.n + p.k.n + p.v.n;
  // whole lane groups share a job; every lane of a warp runs the same number of rounds, for the shuffles
  const int jobs = nt * heads;
  for (int j0 = (threadIdx.x & ~31) / LG; j0 < jobs; j0 += GROUPS) {
    const int j = j0 + lane / LG;
    const bool on = j < jobs;
    const int i = on ? j / heads : 0;
    const int h = on ? j - i * heads : 0;
    const int kind = h < p.q.n ? 0 : h < p.q.n + p.k.n ? 1 : 2;
    const HeadRows& src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    const int hh = kind == 0 ? h : kind == 1 ? h - p.q.n : h - p.q.n - p.k.n;
    const T* x = static_cast<const T*>(src.x) + (t0 + i) * src.token_stride + hh * src.head_stride;
    float f[16];
    {
      Vec8<T> va, vb;
      va.load(x + ca);
      vb.load(x + cb);
      va.get(f);
      vb.get(f + 8);
    }
    if (p.q.weight != nullptr || p.k.weight != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int c = 0; c < 16; ++c) ss = fmaf(f[c], f[c], ss);
#pragma unroll
      for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (src.weight != nullptr) {
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        const T* w = static_cast<const T*>(src.weight);
        float g[16];
        Vec8<T> va, vb;
        va.load(w + ca);
        vb.load(w + cb);
        va.get(g);
        vb.get(g + 8);
#pragma unroll
        for (int c = 0; c < 16; ++c) f[c] = f[c] * r * g[c];
      }
    }
    if (turns && kind != 2) {
      const float2* t = cs + i * half + 8 * sub;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int ia = HALF ? c : 2 * c, ib = HALF ? c + 8 : 2 * c + 1;
        const float a = f[ia], b = f[ib];
        f[ia] = a * t[c].x - b * t[c].y;
        f[ib] = b * t[c].x + a * t[c].y;
      }
    }
    if (!on || row_s[i] < 0) continue;
    uint16_t* dst;
    if (kind == 0)
      dst = p.out_q + (static_cast<long long>(t0 + i) * p.q.n + hh) * D;
    else if (!paged)
      dst = p.out_k + (static_cast<long long>(t0 + i) * p.k.n + hh) * D;
    else
      dst = (kind == 1 ? p.kpages : p.vpages) + (row_s[i] * src.n + hh) * D;
    store8_bf16(dst + ca, f);
    store8_bf16(dst + cb, f + 8);
  }
}

}  // namespace pivot

// RMS norm of every query and key head with the rotary position in the same pass, and its
// gradients. For a row x of d elements (one token, one head) at position p:
//   r = 1 / sqrt(mean(x^2) + eps),  z = x r w,  y = z with the pairs of its first `rot` elements
//   turned by the angle of p: (a, b) -> (a c - b s, b c + a s), c and s from the caller's table.
// Backward: dz = dy turned back (s -> -s), dw = sum over rows of dz (x r),
//   dx = r (dz w - x r mean(dz w x r)).
// All arithmetic is fp32 with one rounding to bf16 at the end; dw is summed per lane in fp32 over
// its rows and across CTAs in fp64, in a fixed order.
//
// Bound: HBM. A row is read once and written once (backward: two reads, one write); 8-10 flops an
// element are far below the FMA rate. D / 8 lanes hold one row in 16-byte pieces, so a pair of
// the half-split rotation sits in two lanes (one shuffle per element) and the sum of squares is a
// 3- or 4-step butterfly. A warp takes kIter rows of each lane group of one token, all loads
// issued before the first use, and reads the token's table row once for all of them.
#include <cmath>

#include "common.cuh"
#include "launch.h"

namespace moba {

namespace {

constexpr int kNormThreads = 256;
constexpr int kIter = 4;  // rows per lane group in flight

// Rotation of the lane's eight elements with weights folded in. An element pairs with its partner
// o: y = x cx + o co in units of the normed row. Forward: cx = w c, co = w_o (-+ s), w_o the
// partner's weight; without weights (backward): cx = c, co = -+ s.
struct Rope {
  float cx[8], co[8];
};

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p + 4));
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// Table row of one position for the lane that holds elements 8l .. 8l+7. Elements at or behind
// `rot` are not turned. Half-split: element e < rot/2 pairs with e + rot/2, both read entry
// e mod rot/2; rot is a multiple of 16, so a lane's elements lie in one half and their partners in
// lane l +- rot/16. Adjacent: (2i, 2i+1), in the lane itself. dir = -1 turns back.
template <bool ADJ>
__device__ __forceinline__ Rope load_rope(const float* __restrict__ row, int l, int rot,
                                          float dir) {
  Rope R;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    R.cx[e] = 1.f;
    R.co[e] = 0.f;
  }
  if (8 * l < rot) {
    const int half = rot >> 1;
    if (ADJ) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + 4 * l));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + 4 * l));
      const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        R.cx[e] = cv[e >> 1];
        R.co[e] = (e & 1) ? dir * sv[e >> 1] : -dir * sv[e >> 1];
      }
    } else {
      const bool second = 8 * l >= half;
      const int at = 8 * l - (second ? half : 0);
      const float sign = second ? dir : -dir;
      load8(row + at, R.cx);
      load8(row + half + at, R.co);
#pragma unroll
      for (int e = 0; e < 8; ++e) R.co[e] *= sign;
    }
  }
  return R;
}

// Lane that holds the partners of this lane's elements (half-split form; itself otherwise).
template <bool ADJ>
__device__ __forceinline__ int partner_of(int l, int rot) {
  const int hl = rot >> 4;  // lanes of one half
  return ADJ || 8 * l >= rot ? l : l < hl ? l + hl : l - hl;
}

// The partner's eight elements: four packed pairs, exchanged between lanes or within them.
template <bool ADJ>
__device__ __forceinline__ uint4 swap_pairs(const uint4& u, int lane) {
  if (ADJ)
    return make_uint4(__byte_perm(u.x, 0, 0x1032), __byte_perm(u.y, 0, 0x1032),
                      __byte_perm(u.z, 0, 0x1032), __byte_perm(u.w, 0, 0x1032));
  return make_uint4(__shfl_sync(0xffffffffu, u.x, lane), __shfl_sync(0xffffffffu, u.y, lane),
                    __shfl_sync(0xffffffffu, u.z, lane), __shfl_sync(0xffffffffu, u.w, lane));
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct NormArgs {
  const __nv_bfloat16 *q, *k, *dyq, *dyk;
  long long q_ld, k_ld;  // elements between tokens of q and k (their heads are packed)
  const float *wq, *wk, *rope;
  const int32_t* pos;
  __nv_bfloat16 *oq, *ok;  // y (forward) or dx (backward), packed
  float* part;             // backward: [CTAs][2][D] sums for the weights
  int T, Hq, Hkv, n_pos, rot, qchunks, chunks;
  float eps;
};

// A chunk is kIter * (32 / LPR) consecutive heads of q, or of k.
template <int D>
struct ChunkRows {
  static constexpr int kRows = kIter * (32 / (D / 8));
};

// y = r (x (w c) + x_o (w_o s)): the partner's bf16 pairs are exchanged as they were loaded, and
// the weights go into the token's rotation once for all of the warp's rows.
template <int D, bool ADJ>
__global__ void __launch_bounds__(kNormThreads, 5) qk_norm_rope_kernel(const NormArgs A) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const unsigned unit = blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const unsigned tok = unit / static_cast<unsigned>(A.chunks);
  if (tok >= static_cast<unsigned>(A.T)) return;  // uniform over the warp
  const long long t = tok;
  int chunk = static_cast<int>(unit - tok * A.chunks);
  const bool isq = chunk < A.qchunks;
  if (!isq) chunk -= A.qchunks;
  const int H = isq ? A.Hq : A.Hkv, h0 = chunk * kIter * RPW + sub;
  const __nv_bfloat16* src = (isq ? A.q + t * A.q_ld : A.k + t * A.k_ld) + l * 8;
  __nv_bfloat16* dst = (isq ? A.oq : A.ok) + t * H * D + l * 8;
  uint4 raw[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int h = h0 + i * RPW;
    raw[i] = h < H ? __ldcs(reinterpret_cast<const uint4*>(src + static_cast<size_t>(h) * D))
                   : make_uint4(0, 0, 0, 0);
  }
  const int p = __ldg(A.pos + t);
  const bool known = p >= 0 && p < A.n_pos;
  Rope R = load_rope<ADJ>(A.rope + static_cast<size_t>(known ? p : 0) * A.rot, l, A.rot, 1.f);
  const int pl = partner_of<ADJ>(l, A.rot), partner = lane - l + pl;
  const float* wp = isq ? A.wq : A.wk;
  {
    float w[8], wo[8];
    load8(wp + l * 8, w);
    load8(wp + pl * 8, wo);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      R.cx[e] *= w[e];
      R.co[e] *= ADJ ? w[e ^ 1] : wo[e];
    }
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    float x[8], o[8];
    unpack8(raw[i], x);
    unpack8(swap_pairs<ADJ>(raw[i], partner), o);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
    ss = row_sum<LPR>(ss);
    // a position outside the table has no angle: the row becomes NaN instead of a wrong number
    const float r = known ? rsqrtf(ss * (1.f / D) + A.eps) : __int_as_float(0x7fffffff);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], R.cx[e], o[e] * R.co[e]) * r;
    const int h = h0 + i * RPW;
    if (h < H) __stcs(reinterpret_cast<uint4*>(dst + static_cast<size_t>(h) * D), pack8(x));
  }
}

// Persistent: warp g of G (G a multiple of the chunks per token) takes units g, g + G, ..., all of
// the same chunk, so its weights stay in registers and its dw sums belong to q or to k alone.
template <int D, bool ADJ>
__global__ void __launch_bounds__(kNormThreads) qk_norm_rope_bwd_kernel(const NormArgs A) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, NW = kNormThreads / 32;
  __shared__ float red[NW][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, sub = lane / LPR;
  const long long G = static_cast<long long>(gridDim.x) * NW / A.chunks * A.chunks;
  const long long g = static_cast<long long>(blockIdx.x) * NW + warp;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  int chunk = static_cast<int>(g % A.chunks);
  const bool isq = chunk < A.qchunks;
  if (!isq) chunk -= A.qchunks;
  const int H = isq ? A.Hq : A.Hkv, h0 = chunk * kIter * RPW + sub;
  if (g < G) {
    const int partner = lane - l + partner_of<ADJ>(l, A.rot);
    float w[8];
    load8((isq ? A.wq : A.wk) + l * 8, w);
    for (long long t = g / A.chunks; t < A.T; t += G / A.chunks) {
      const __nv_bfloat16* xs = (isq ? A.q + t * A.q_ld : A.k + t * A.k_ld) + l * 8;
      const __nv_bfloat16* ys = (isq ? A.dyq : A.dyk) + t * H * D + l * 8;
      __nv_bfloat16* dst = (isq ? A.oq : A.ok) + t * H * D + l * 8;
      uint4 xr[kIter], yr[kIter];
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const int h = h0 + i * RPW;
        const bool in = h < H;
        const size_t at = static_cast<size_t>(h) * D;
        xr[i] = in ? __ldcs(reinterpret_cast<const uint4*>(xs + at)) : make_uint4(0, 0, 0, 0);
        yr[i] = in ? __ldcs(reinterpret_cast<const uint4*>(ys + at)) : make_uint4(0, 0, 0, 0);
      }
      const int p = __ldg(A.pos + t);
      const bool known = p >= 0 && p < A.n_pos;
      const Rope R =
          load_rope<ADJ>(A.rope + static_cast<size_t>(known ? p : 0) * A.rot, l, A.rot, -1.f);
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        float x[8], z[8], o[8];
        unpack8(xr[i], x);
        unpack8(yr[i], z);
        unpack8(swap_pairs<ADJ>(yr[i], partner), o);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = fmaf(z[e], R.cx[e], o[e] * R.co[e]);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
        ss = row_sum<LPR>(ss);
        const float r = known ? rsqrtf(ss * (1.f / D) + A.eps) : __int_as_float(0x7fffffff);
        float dot = 0.f;
        const bool in = h0 + i * RPW < H;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= r;  // x r
          if (in) acc[e] = fmaf(z[e], x[e], acc[e]);
          z[e] *= w[e];
          dot = fmaf(z[e], x[e], dot);
        }
        dot = row_sum<LPR>(dot) * (1.f / D);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = r * fmaf(-x[e], dot, z[e]);
        if (in)
          __stcs(reinterpret_cast<uint4*>(dst + static_cast<size_t>(h0 + i * RPW) * D), pack8(x));
      }
    }
  }
  // lanes of the same columns, then the CTA's warps of q and of k
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
    if (sub == 0) red[warp][l * 8 + e] = acc[e];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < 2 * D; x += kNormThreads) {
    const int which = x / D;  // 0: q, 1: k
    float s = 0.f;
    for (int i = 0; i < NW; ++i) {
      const long long gi = static_cast<long long>(blockIdx.x) * NW + i;
      const int ci = static_cast<int>(gi % A.chunks);
      if (gi < G && (ci < A.qchunks) == (which == 0)) s += red[i][x % D];
    }
    A.part[static_cast<size_t>(blockIdx.x) * 2 * D + x] = s;
  }
}

// dw[x] = sum of the CTAs' parts: 32 interleaved fp64 sums, joined in order. One launch of a few
// CTAs, so each thread has all its loads in flight at once.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const float* __restrict__ part, int n,
                                                          int D, float* __restrict__ dwq,
                                                          float* __restrict__ dwk) {
  __shared__ double red[32][33];
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5, x = blockIdx.x * 32 + c;
  double s = 0.;
#pragma unroll 20
  for (int i = w; i < n; i += 32)
    s += static_cast<double>(part[static_cast<size_t>(i) * 2 * D + x]);
  red[w][c] = s;
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += red[i][c];
    (x < D ? dwq[x] : dwk[x - D]) = static_cast<float>(s);
  }
}

NormArgs args_of(const NormLaunch& L) {
  NormArgs A{};
  A.q = static_cast<const __nv_bfloat16*>(L.q);
  A.k = static_cast<const __nv_bfloat16*>(L.k);
  A.dyq = static_cast<const __nv_bfloat16*>(L.dyq);
  A.dyk = static_cast<const __nv_bfloat16*>(L.dyk);
  A.q_ld = L.q_ld; A.k_ld = L.k_ld;
  A.wq = L.wq; A.wk = L.wk; A.rope = L.rope; A.pos = L.pos;
  A.oq = static_cast<__nv_bfloat16*>(L.oq);
  A.ok = static_cast<__nv_bfloat16*>(L.ok);
  A.part = L.part;
  A.T = L.T; A.Hq = L.Hq; A.Hkv = L.Hkv; A.n_pos = L.n_pos; A.rot = L.rot;
  const int rows = L.d == 64 ? ChunkRows<64>::kRows : ChunkRows<128>::kRows;
  A.qchunks = (L.Hq + rows - 1) / rows;
  A.chunks = A.qchunks + (L.Hkv + rows - 1) / rows;
  A.eps = L.eps;
  return A;
}

}  // namespace

// CTAs of the backward kernel: four per SM, enough warps for every chunk of a token.
int qk_norm_bwd_ctas(int Hq, int Hkv, int d, int sms) {
  const int rows = d == 64 ? ChunkRows<64>::kRows : ChunkRows<128>::kRows;
  const int chunks = (Hq + rows - 1) / rows + (Hkv + rows - 1) / rows;
  const int nw = kNormThreads / 32;
  return (4 * sms > (chunks + nw - 1) / nw) ? 4 * sms : (chunks + nw - 1) / nw;
}

cudaError_t launch_qk_norm(const NormLaunch& L, cudaStream_t s) {
  const NormArgs A = args_of(L);
  const long long warps = static_cast<long long>(A.T) * A.chunks;
  const unsigned grid = static_cast<unsigned>((warps + kNormThreads / 32 - 1) / (kNormThreads / 32));
  if (L.d == 64) {
    if (L.adjacent) qk_norm_rope_kernel<64, true><<<grid, kNormThreads, 0, s>>>(A);
    else qk_norm_rope_kernel<64, false><<<grid, kNormThreads, 0, s>>>(A);
  } else {
    if (L.adjacent) qk_norm_rope_kernel<128, true><<<grid, kNormThreads, 0, s>>>(A);
    else qk_norm_rope_kernel<128, false><<<grid, kNormThreads, 0, s>>>(A);
  }
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_bwd(const NormLaunch& L, int ctas, cudaStream_t s) {
  const NormArgs A = args_of(L);
  if (L.d == 64) {
    if (L.adjacent) qk_norm_rope_bwd_kernel<64, true><<<ctas, kNormThreads, 0, s>>>(A);
    else qk_norm_rope_bwd_kernel<64, false><<<ctas, kNormThreads, 0, s>>>(A);
  } else {
    if (L.adjacent) qk_norm_rope_bwd_kernel<128, true><<<ctas, kNormThreads, 0, s>>>(A);
    else qk_norm_rope_bwd_kernel<128, false><<<ctas, kNormThreads, 0, s>>>(A);
  }
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_dw(const float* part, int n, int d, float* dwq, float* dwk,
                              cudaStream_t s) {
  qk_norm_dw_kernel<<<2 * d / 32, 1024, 0, s>>>(part, n, d, dwq, dwk);
  return cudaGetLastError();
}

}  // namespace moba

// RMS norm of every query and key head with the rotary position in the same pass, and its
// gradients. For a row x of d elements (one token, one head) at position p:
//   r = 1 / sqrt(mean(x^2) + eps),  z = x r w,  y = z with the pairs of its first `rot` elements
//   turned by the angle of p: (a, b) -> (a c - b s, b c + a s), c and s from the caller's table.
// Backward: dz = dy turned back (s -> -s), dw = sum over rows of dz (x r),
//   dx = r (dz w - x r mean(dz w x r)).
// All arithmetic is fp32 with one rounding to bf16 at the end; dw is summed per lane in fp32 over
// its rows and across CTAs in fp64, in a fixed order.
//
// Bound: HBM; a row is read once and written once (backward: two reads, one write). The arithmetic
// is only ~10 flops an element, but at 23 bytes per clock and SM the instructions around it count:
// the lanes of a row (d / 8 of them) hold both elements of each of their pairs, so a rotation needs
// no exchange; products go two to an instruction; the sums of squares of a chunk's rows are reduced
// together. Persistent: every warp takes a chunk of 2 KB (8 or 16 heads of one token) at a time
// through a private ring in shared memory (16-byte cp.async, with the token's table row).
// One CTA of 8 warps per SM and two rows at a time: fewer, longer streams suit HBM better than more
// warps (128K tokens, 32 / 8 heads of 128, 2.7 GB: 403-407 us in a replayed graph = 6.7 TB/s, 440 as
// back-to-back calls on inputs that change; two CTAs 467, three 465, four rows at a time 440; gradients
// at 65521 tokens, 16 / 16 heads of 64: 121-127 us, back to back 133, two CTAs 138).
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace moba {

namespace {

constexpr int kNormThreads = 256, kNormWarps = kNormThreads / 32;
constexpr int kIter = 4;  // 16-byte pieces of a chunk per lane
constexpr int kChunkBytes = kIter * 512, kRopeBytes = 512;

__host__ __device__ constexpr int stage_bytes(bool bwd) {
  return (bwd ? 2 : 1) * kChunkBytes + kRopeBytes;
}
constexpr int norm_stages(bool bwd) { return bwd ? 3 : 4; }
constexpr int norm_smem(bool bwd) { return kNormWarps * norm_stages(bwd) * stage_bytes(bwd); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;  // 0 bytes read: the destination is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}

// Multiplies and adds two to an instruction (f32x2).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// A lane's eight elements of a row: the first and the second elements of its four pairs.
struct Elems {
  float2 a[2], b[2];
};

// Where they lie. Lane l < rot/8 has pairs 4l .. 4l+3, the other lanes the elements behind rot.
// Half-split: elements A .. A+3 and B .. B+3. Adjacent: elements A .. A+7, pairs neighbours.
template <bool ADJ>
struct Place {
  int A, B;
  __device__ __forceinline__ Place(int l, int rot) {
    const bool turned = 8 * l < rot;
    A = ADJ || !turned ? 8 * l : 4 * l;
    B = ADJ || !turned ? 8 * l + 4 : (rot >> 1) + 4 * l;
  }
  __device__ __forceinline__ int col(bool second, int i) const {  // of element i of a or b
    return ADJ ? A + 2 * i + second : (second ? B : A) + i;
  }
};

__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <bool ADJ>
__device__ __forceinline__ Elems read_row(const uint8_t* row, const Place<ADJ>& P) {
  Elems x;
  if (ADJ) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + 2 * P.A);
    x.a[0] = make_float2(lo_f(u.x), lo_f(u.y));
    x.a[1] = make_float2(lo_f(u.z), lo_f(u.w));
    x.b[0] = make_float2(hi_f(u.x), hi_f(u.y));
    x.b[1] = make_float2(hi_f(u.z), hi_f(u.w));
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(row + 2 * P.A);
    const uint2 v = *reinterpret_cast<const uint2*>(row + 2 * P.B);
    x.a[0] = make_float2(lo_f(u.x), hi_f(u.x));
    x.a[1] = make_float2(lo_f(u.y), hi_f(u.y));
    x.b[0] = make_float2(lo_f(v.x), hi_f(v.x));
    x.b[1] = make_float2(lo_f(v.y), hi_f(v.y));
  }
  return x;
}

template <bool ADJ>
__device__ __forceinline__ void write_row(__nv_bfloat16* row, const Place<ADJ>& P,
                                          const Elems& x) {
  if (ADJ) {
    __stcs(reinterpret_cast<uint4*>(row + P.A),
           make_uint4(pack2(x.a[0].x, x.b[0].x), pack2(x.a[0].y, x.b[0].y),
                      pack2(x.a[1].x, x.b[1].x), pack2(x.a[1].y, x.b[1].y)));
  } else {
    __stcs(reinterpret_cast<uint2*>(row + P.A),
           make_uint2(pack2(x.a[0].x, x.a[0].y), pack2(x.a[1].x, x.a[1].y)));
    __stcs(reinterpret_cast<uint2*>(row + P.B),
           make_uint2(pack2(x.b[0].x, x.b[0].y), pack2(x.b[1].x, x.b[1].y)));
  }
}

template <bool ADJ>
__device__ __forceinline__ Elems read_weights(const float* w, const Place<ADJ>& P) {
  Elems x;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x.a[i] = make_float2(w[P.col(false, 2 * i)], w[P.col(false, 2 * i + 1)]);
    x.b[i] = make_float2(w[P.col(true, 2 * i)], w[P.col(true, 2 * i + 1)]);
  }
  return x;
}

// Cosines and sines of the lane's four pairs; 1 and 0 behind rot.
struct Angle {
  float2 c[2], s[2];
};
__device__ __forceinline__ Angle read_angle(const float* row, int l, int rot, bool all) {
  Angle R;
  const int at = all || 8 * l < rot ? 4 * l : 0;
  const float4 c = *reinterpret_cast<const float4*>(row + at);
  const float4 s = *reinterpret_cast<const float4*>(row + (rot >> 1) + at);
  R.c[0] = make_float2(c.x, c.y);
  R.c[1] = make_float2(c.z, c.w);
  R.s[0] = make_float2(s.x, s.y);
  R.s[1] = make_float2(s.z, s.w);
  if (!all && 8 * l >= rot) {
    R.c[0] = R.c[1] = make_float2(1.f, 1.f);
    R.s[0] = R.s[1] = make_float2(0.f, 0.f);
  }
  return R;
}
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

// Sums of N values over the LPR lanes of a row, all at once: on the way down a lane keeps half of
// its values and hands over the other half, so that after log2 N steps it holds one value and the
// shuffles are N - 1 + log2(LPR / N) instead of N log2 LPR. Lane l ends with the sum of value
// l / (LPR / N).
template <int LPR, int N>
__device__ __forceinline__ float reduce_rows(float (&v)[N], int l) {
  int n = N;
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        if (i < n) {
          const float give = (l & o) ? v[i] : v[i + n], keep = (l & o) ? v[i + n] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
  return v[0];
}
// The way back: every lane of the row gets all N values.
template <int LPR, int N>
__device__ __forceinline__ void gather_rows(float mine, float (&v)[N], int l) {
  v[0] = mine;
  int n = 1;
#pragma unroll
  for (int o = LPR / N; o < LPR; o <<= 1) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      if (i < n) {
        const float other = __shfl_xor_sync(0xffffffffu, v[i], o);
        v[i + n] = (l & o) ? v[i] : other;
        v[i] = (l & o) ? other : v[i];
      }
    n <<= 1;
  }
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

// A chunk is kIter * (32 / LPR) consecutive heads of q, or of k: 2 KB.
__host__ __device__ constexpr int chunk_rows(int d) { return kChunkBytes / (2 * d); }

// Warp g of G (G a multiple of the chunks per token) takes units g, g + G, ..., all of the same
// chunk, so that its weights stay in registers and its dw sums belong to q or to k alone.
// Forward: y_a = r (x_a (w_a c) - x_b (w_b s)), y_b = r (x_b (w_b c) + x_a (w_a s)), the weights
// multiplied into the token's angle once for all rows of the chunk. Backward: as stated at the top.
template <int D, bool ADJ, bool BWD>
__global__ void __launch_bounds__(kNormThreads, 1) qk_norm_rope_kernel(const NormArgs A) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, kStage = stage_bytes(BWD);
  constexpr int kStages = norm_stages(BWD);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[BWD ? kNormWarps : 1][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, sub = lane / LPR;
  const int G = static_cast<int>(gridDim.x) * kNormWarps / A.chunks * A.chunks;
  const int g = static_cast<int>(blockIdx.x) * kNormWarps + warp;
  int chunk = g % A.chunks;
  const bool isq = chunk < A.qchunks;
  if (!isq) chunk -= A.qchunks;
  const int H = isq ? A.Hq : A.Hkv, h0 = chunk * chunk_rows(D) + sub;
  const Place<ADJ> P(l, A.rot);
  wait_previous_kernel();
  Elems acc;
#pragma unroll
  for (int e = 0; e < 2; ++e) acc.a[e] = acc.b[e] = make_float2(0.f, 0.f);
  const int step = G / A.chunks, t0 = g / A.chunks;  // tokens t0, t0 + step, ...
  if (g < G && t0 < A.T) {
    const long long x_step = (isq ? A.q_ld : A.k_ld) * step;
    const long long y_step = static_cast<long long>(H) * D * step;
    // where this lane's 16 bytes of the chunk's first rows come from, and its row goes to
    const size_t at = static_cast<size_t>(h0) * D;
    const __nv_bfloat16* xs = (isq ? A.q : A.k) + at + l * 8 + (isq ? A.q_ld : A.k_ld) * t0;
    const __nv_bfloat16* ys =
        BWD ? (isq ? A.dyq : A.dyk) + at + l * 8 + static_cast<size_t>(t0) * H * D : nullptr;
    __nv_bfloat16* dst = (isq ? A.oq : A.ok) + at + static_cast<size_t>(t0) * H * D;
    const Elems w = read_weights<ADJ>(isq ? A.wq : A.wk, P);
    uint8_t* ring = smem + warp * (kStages * kStage);
    const bool all = A.rot == D;
    const int rot16 = A.rot >> 2;  // 16-byte pieces of a table row
    bool in[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) in[i] = h0 + i * RPW < H;
    // lane x fetches the position of the warp's unit n0 + x; 32 units at a time
    auto positions = [&](int n0) {
      const long long t = t0 + static_cast<long long>(n0 + lane) * step;
      return t < A.T ? A.pos[t] : -1;
    };
    const int units = (A.T - t0 + step - 1) / step;
    int pos = positions(0);
    const uint32_t lane_dst = smem_u32(ring) + lane * 16;
    auto issue = [&](int n, int stage) {  // copies of the warp's unit n
      if (n < units) {
        const uint32_t d = lane_dst + stage * kStage;
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          copy16(d + i * 512, xs + (in[i] ? i * RPW * D : 0), in[i]);
          if (BWD) copy16(d + kChunkBytes + i * 512, ys + (in[i] ? i * RPW * D : 0), in[i]);
        }
        const int p = __shfl_sync(0xffffffffu, pos, n & 31);
        const bool known = p >= 0 && p < A.n_pos;
        if (lane < rot16)
          copy16(d + kStage - kRopeBytes,
                 A.rope + static_cast<size_t>(known ? p : 0) * A.rot + lane * 4, true);
        xs += x_step;
        if (BWD) ys += y_step;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, i);
    int was = pos;  // positions of the 32 units that the one in work belongs to
    int stage = 0;
    for (int n = 0; n < units; ++n) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();  // the unit is there; the stage of the last one is free
      if ((n & 31) == 0) was = pos;
      if (((n + kStages - 1) & 31) == 0) pos = positions(n + kStages - 1);
      issue(n + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
      const int p = __shfl_sync(0xffffffffu, was, n & 31);
      const bool known = p >= 0 && p < A.n_pos;
      const uint8_t* s = ring + stage * kStage;
      stage = stage + 1 == kStages ? 0 : stage + 1;
      const Angle R =
          read_angle(reinterpret_cast<const float*>(s + kStage - kRopeBytes), l, A.rot, all);
      Elems wc, ws;  // forward: weights times cosine, times sine (w_b's negative)
      if (!BWD)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          wc.a[e] = mul2(w.a[e], R.c[e]);
          wc.b[e] = mul2(w.b[e], R.c[e]);
          ws.a[e] = mul2(w.a[e], R.s[e]);
          ws.b[e] = mul2(neg2(w.b[e]), R.s[e]);
        }
      s += sub * 2 * D;
      constexpr int NB = 2, N = BWD ? 4 : 2;  // rows and sums of a batch
#pragma unroll
      for (int i0 = 0; i0 < kIter; i0 += NB) {
        // the rows' sums first, all together, so that their shuffles overlap
        Elems x[NB], z[BWD ? NB : 1];  // backward: z = dz
        float v[N];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          x[i] = read_row<ADJ>(s + (i0 + i) * 512, P);
          float2 sq = mul2(x[i].a[0], x[i].a[0]);
          sq = fma2(x[i].a[1], x[i].a[1], sq);
          sq = fma2(x[i].b[0], x[i].b[0], sq);
          sq = fma2(x[i].b[1], x[i].b[1], sq);
          v[i] = sq.x + sq.y;
          if constexpr (BWD) {
            const Elems y = read_row<ADJ>(s + kChunkBytes + (i0 + i) * 512, P);
            float2 dt = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              z[i].a[e] = fma2(y.a[e], R.c[e], mul2(y.b[e], R.s[e]));
              z[i].b[e] = fma2(y.b[e], R.c[e], mul2(neg2(y.a[e]), R.s[e]));
              dt = fma2(mul2(z[i].a[e], w.a[e]), x[i].a[e], dt);
              dt = fma2(mul2(z[i].b[e], w.b[e]), x[i].b[e], dt);
            }
            v[NB + i] = dt.x + dt.y;  // times r: sum of dz w (x r)
          }
        }
        float sum = reduce_rows<LPR, N>(v, l);
        // the lanes that hold a sum of squares turn it into r; a position outside the table has
        // no angle: the row becomes NaN, not a wrong number
        if (!BWD || l < LPR / 2)
          sum = known ? rsqrtf(sum * (1.f / D) + A.eps) : __int_as_float(0x7fffffff);
        gather_rows<LPR, N>(sum, v, l);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const float2 r2 = make_float2(v[i], v[i]);
          Elems y;
          if constexpr (!BWD) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              y.a[e] = mul2(fma2(x[i].a[e], wc.a[e], mul2(x[i].b[e], ws.b[e])), r2);
              y.b[e] = mul2(fma2(x[i].b[e], wc.b[e], mul2(x[i].a[e], ws.a[e])), r2);
            }
          } else {
            const float dot = -v[NB + i] * v[i] * (1.f / D);
            const float2 d2 = make_float2(dot, dot);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 xa = mul2(x[i].a[e], r2), xb = mul2(x[i].b[e], r2);
              if (in[i0 + i]) {
                acc.a[e] = fma2(z[i].a[e], xa, acc.a[e]);
                acc.b[e] = fma2(z[i].b[e], xb, acc.b[e]);
              }
              y.a[e] = mul2(r2, fma2(xa, d2, mul2(z[i].a[e], w.a[e])));
              y.b[e] = mul2(r2, fma2(xb, d2, mul2(z[i].b[e], w.b[e])));
            }
          }
          if (in[i0 + i]) write_row<ADJ>(dst + (i0 + i) * RPW * D, P, y);
        }
      }
      dst += y_step;
    }
  }
  if constexpr (BWD) {
    // lanes of the same columns, then the CTA's warps of q and of k
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 pr = e < 4 ? acc.a[(e >> 1) & 1] : acc.b[(e >> 1) & 1];
      float f = e & 1 ? pr.y : pr.x;
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
      if (sub == 0) red[warp][P.col(e >= 4, e & 3)] = f;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * D; x += kNormThreads) {
      float s = 0.f;
      for (int i = 0; i < kNormWarps; ++i) {
        const int gi = static_cast<int>(blockIdx.x) * kNormWarps + i;
        if (gi < G && (gi % A.chunks < A.qchunks) == (x < D)) s += red[i][x % D];
      }
      A.part[static_cast<size_t>(blockIdx.x) * 2 * D + x] = s;
    }
  }
}

// The same for ONE of q and k with few heads for the rows of a chunk: a chunk is then consecutive
// (token, head) rows across tokens, so that it stays full, and every row has an angle of its own.
// Those come straight from the table into registers one unit ahead (their positions two ahead).
struct RowsArgs {
  const __nv_bfloat16 *x, *dy;
  long long ld;
  const float *w, *rope;
  const int32_t* pos;
  __nv_bfloat16* out;
  float* part;          // backward: [CTAs][2][D]
  int rows, H, n_pos, rot;
  uint32_t magic;       // row / H = umulhi(row, magic) >> shift for rows < 2^31, H > 1
  int shift, which;     // which: 0 for q, 1 for k
  float eps;
};

template <int D, bool ADJ, bool BWD>
__global__ void __launch_bounds__(kNormThreads, BWD ? 1 : 2) norm_rope_rows_kernel(const RowsArgs A) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, kRows = chunk_rows(D);
  constexpr int kStage = (BWD ? 2 : 1) * kChunkBytes, kStages = BWD ? 4 : 6;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[BWD ? kNormWarps : 1][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, sub = lane / LPR;
  const int G = static_cast<int>(gridDim.x) * kNormWarps;
  const int g = static_cast<int>(blockIdx.x) * kNormWarps + warp;
  const Place<ADJ> P(l, A.rot);
  const bool all = A.rot == D;
  wait_previous_kernel();
  Elems acc;
#pragma unroll
  for (int e = 0; e < 2; ++e) acc.a[e] = acc.b[e] = make_float2(0.f, 0.f);
  const int chunks = (A.rows + kRows - 1) / kRows;
  const int units = g < chunks ? (chunks - g + G - 1) / G : 0;
  if (units > 0) {
    const Elems w = read_weights<ADJ>(A.w, P);
    uint8_t* ring = smem + warp * (kStages * kStage);
    const uint32_t lane_dst = smem_u32(ring) + lane * 16;
    // row of piece i of unit n, below 2^31 + a grid's worth; its token
    auto row_of = [&](int n, int i) {
      return (static_cast<uint32_t>(g) + static_cast<uint32_t>(n) * G) * kRows + i * RPW + sub;
    };
    auto token_of = [&](uint32_t r) {
      return A.H == 1 ? r : __umulhi(r, A.magic) >> A.shift;
    };
    auto issue = [&](int n, int stage) {
      if (n < units) {
        const uint32_t d = lane_dst + stage * kStage;
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const uint32_t r = row_of(n, i);
          const bool in = r < static_cast<uint32_t>(A.rows);
          const uint32_t t = token_of(in ? r : 0);
          const long long at = t * A.ld + static_cast<long long>((in ? r : 0) - t * A.H) * D;
          copy16(d + i * 512, A.x + at + l * 8, in);
          if (BWD)
            copy16(d + kChunkBytes + i * 512, A.dy + static_cast<size_t>(in ? r : 0) * D + l * 8,
                   in);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto fetch_pos = [&](int n, int (&p)[kIter]) {
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const uint32_t r = row_of(n, i);
        p[i] = n < units && r < static_cast<uint32_t>(A.rows) ? A.pos[token_of(r)] : -1;
      }
    };
    auto fetch_angles = [&](const int (&p)[kIter], Angle (&R)[kIter]) {
#pragma unroll
      for (int i = 0; i < kIter; ++i)
        R[i] = read_angle(
            A.rope + static_cast<size_t>(p[i] >= 0 && p[i] < A.n_pos ? p[i] : 0) * A.rot, l, A.rot,
            all);
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, i);
    int p0[kIter], p1[kIter];  // positions of the unit in work and of the next
    Angle R1[kIter];           // angles of the next
    fetch_pos(0, p1);
    fetch_angles(p1, R1);
    int p2[kIter];
    fetch_pos(1, p2);
    int stage = 0;
    for (int n = 0; n < units; ++n) {
      Angle R[kIter];
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        R[i] = R1[i];
        p0[i] = p1[i];
        p1[i] = p2[i];
      }
      if (n + 1 < units) fetch_angles(p1, R1);
      fetch_pos(n + 2, p2);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();
      issue(n + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
      const uint8_t* s = ring + stage * kStage + sub * 2 * D;
      stage = stage + 1 == kStages ? 0 : stage + 1;
      constexpr int NB = 2, N = BWD ? 4 : 2;
#pragma unroll
      for (int i0 = 0; i0 < kIter; i0 += NB) {
        Elems x[NB], z[BWD ? NB : 1];
        float v[N];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          x[i] = read_row<ADJ>(s + (i0 + i) * 512, P);
          float2 sq = mul2(x[i].a[0], x[i].a[0]);
          sq = fma2(x[i].a[1], x[i].a[1], sq);
          sq = fma2(x[i].b[0], x[i].b[0], sq);
          sq = fma2(x[i].b[1], x[i].b[1], sq);
          v[i] = sq.x + sq.y;
          if constexpr (BWD) {
            const Elems y = read_row<ADJ>(s + kChunkBytes + (i0 + i) * 512, P);
            float2 dt = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              z[i].a[e] = fma2(y.a[e], R[i0 + i].c[e], mul2(y.b[e], R[i0 + i].s[e]));
              z[i].b[e] = fma2(y.b[e], R[i0 + i].c[e], mul2(neg2(y.a[e]), R[i0 + i].s[e]));
              dt = fma2(mul2(z[i].a[e], w.a[e]), x[i].a[e], dt);
              dt = fma2(mul2(z[i].b[e], w.b[e]), x[i].b[e], dt);
            }
            v[NB + i] = dt.x + dt.y;
          }
        }
        float sum = reduce_rows<LPR, N>(v, l);
        if (!BWD || l < LPR / 2) sum = rsqrtf(sum * (1.f / D) + A.eps);
        gather_rows<LPR, N>(sum, v, l);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const uint32_t row = row_of(n, i0 + i);
          const bool in = row < static_cast<uint32_t>(A.rows);
          // a position outside the table: NaN
          const float r =
              p0[i0 + i] >= 0 && p0[i0 + i] < A.n_pos ? v[i] : __int_as_float(0x7fffffff);
          const float2 r2 = make_float2(r, r);
          Elems y;
          if constexpr (!BWD) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 xa = mul2(x[i].a[e], w.a[e]), xb = mul2(x[i].b[e], w.b[e]);
              y.a[e] = mul2(fma2(xa, R[i0 + i].c[e], mul2(neg2(xb), R[i0 + i].s[e])), r2);
              y.b[e] = mul2(fma2(xb, R[i0 + i].c[e], mul2(xa, R[i0 + i].s[e])), r2);
            }
          } else {
            const float dot = -v[NB + i] * r * (1.f / D);
            const float2 d2 = make_float2(dot, dot);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 xa = mul2(x[i].a[e], r2), xb = mul2(x[i].b[e], r2);
              if (in) {
                acc.a[e] = fma2(z[i].a[e], xa, acc.a[e]);
                acc.b[e] = fma2(z[i].b[e], xb, acc.b[e]);
              }
              y.a[e] = mul2(r2, fma2(xa, d2, mul2(z[i].a[e], w.a[e])));
              y.b[e] = mul2(r2, fma2(xb, d2, mul2(z[i].b[e], w.b[e])));
            }
          }
          if (in) write_row<ADJ>(A.out + static_cast<size_t>(row) * D, P, y);
        }
      }
    }
  }
  if constexpr (BWD) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 pr = e < 4 ? acc.a[(e >> 1) & 1] : acc.b[(e >> 1) & 1];
      float f = e & 1 ? pr.y : pr.x;
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
      if (sub == 0) red[warp][P.col(e >= 4, e & 3)] = f;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * D; x += kNormThreads) {
      float s = 0.f;
      if (x / D == A.which)
        for (int i = 0; i < kNormWarps; ++i) s += red[i][x % D];
      A.part[static_cast<size_t>(blockIdx.x) * 2 * D + x] = s;
    }
  }
}

// dw[x] = sum of the CTAs' parts: 32 interleaved fp64 sums, joined in order. One launch of a few
// CTAs, so each thread has all its loads in flight at once.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const float* part, int n, int D,
                                                          float* dwq, float* dwk) {
  __shared__ double red[32][33];
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5, x = blockIdx.x * 32 + c;
  wait_previous_kernel();
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
  A.eps = L.eps;
  return A;
}

// Where a tensor's heads leave chunks half empty or more and there are tokens enough that a second
// launch does not matter, its rows go through the kernel that packs them, whose angles cost more per
// row. Measured by tokens : by rows (graph replays, us; the tokens that the rule begins at and 65536):
//   H / H heads of 128 (8 to a chunk)   forward 16384, 65536        gradients 4096, 65536
//     1 / 1                             18.6 :  6.9,  68.6 :  18.1  11.9 :  8.1, 113.0 :  31.2
//     2 / 2                             18.4 : 10.7,  68.9 :  36.9  11.9 :  9.1, 112.7 :  61.0
//     4 / 4 (the last by rows)          18.7 : 17.9,  70.9 :  66.4  12.0 : 13.0, 115.3 : 112.3
//     5 / 5                             19.6 : 19.3,  75.2 :  79.2  12.2 : 15.7, 117.7 : 137.6
//     7 / 7                             21.2 : 27.7,  80.0 : 109.5  12.3 : 18.3, 119.0 : 188.4
//     9 / 9 (two chunks)                39.4 : 39.5, 149.8 : 137.8  19.4 : 18.9, 232.1 : 234.4
// Heads of 64 (16 to a chunk) alike: 8 / 8 forward 70.2 : 65.4, 9 / 9 74.2 : 70.2, 10 / 10 74.3 : 77.6.
// With 4 / 1 heads of 128 the two meet at 4096 tokens forward (5.9 : 5.9) and below 2000 in the
// gradients; 4 / 4 meet at 10000 and 8192.
bool packed(int H, int d, int T, bool bwd) {
  return 2 * H <= chunk_rows(d) && T >= (bwd ? 4096 : 16384);
}
int chunks_of(int H, int d) { return (H + chunk_rows(d) - 1) / chunk_rows(d); }

// What a call launches: the kernel by tokens for q and / or k, the kernel by rows for the others.
struct Launches {
  int qchunks, kchunks;       // by tokens
  bool q_rows, k_rows;        // by rows
  int ctas, q_ctas, k_ctas;   // one per SM at most (by rows, forward: two, whose rings both fit), a
                              // warp for every chunk of a token at least
};
Launches launches_of(int Hq, int Hkv, int d, int T, bool bwd) {
  Launches N{};
  N.q_rows = packed(Hq, d, T, bwd);
  N.k_rows = packed(Hkv, d, T, bwd);
  N.qchunks = N.q_rows ? 0 : chunks_of(Hq, d);
  N.kchunks = N.k_rows ? 0 : chunks_of(Hkv, d);
  auto fit = [](long long chunks, int per_sm) {
    return static_cast<int>(
        std::min<long long>((chunks + kNormWarps - 1) / kNormWarps, per_sm * kNumSms));
  };
  const int c = N.qchunks + N.kchunks;
  if (c)
    N.ctas = std::max(fit(static_cast<long long>(T) * c, 1), (c + kNormWarps - 1) / kNormWarps);
  const int rows = chunk_rows(d);
  if (N.q_rows) N.q_ctas = fit((static_cast<long long>(T) * Hq + rows - 1) / rows, bwd ? 1 : 2);
  if (N.k_rows) N.k_ctas = fit((static_cast<long long>(T) * Hkv + rows - 1) / rows, bwd ? 1 : 2);
  return N;
}

template <class K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<int> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(1, std::memory_order_relaxed);
  return e;
}

template <int D, bool ADJ, bool BWD>
cudaError_t launch(const NormLaunch& L, cudaStream_t s) {
  const Launches N = launches_of(L.Hq, L.Hkv, D, L.T, BWD);
  NormArgs A = args_of(L);
  if (N.ctas) {
    static std::atomic<int> done[64];
    cudaError_t e = allow_smem(qk_norm_rope_kernel<D, ADJ, BWD>, norm_smem(BWD), done);
    if (e != cudaSuccess) return e;
    A.qchunks = N.qchunks;
    A.chunks = N.qchunks + N.kchunks;
    e = launch_early(qk_norm_rope_kernel<D, ADJ, BWD>, dim3(static_cast<unsigned>(N.ctas)),
                     kNormThreads, norm_smem(BWD), 1, s, A);
    if (e != cudaSuccess) return e;
  }
  for (int which = 0; which < 2; ++which) {
    if (!(which ? N.k_rows : N.q_rows)) continue;
    constexpr int smem = kNormWarps * (BWD ? 8 : 6) * kChunkBytes;
    static std::atomic<int> done[64];
    cudaError_t e = allow_smem(norm_rope_rows_kernel<D, ADJ, BWD>, smem, done);
    if (e != cudaSuccess) return e;
    RowsArgs R{};
    R.x = which ? A.k : A.q;
    R.dy = which ? A.dyk : A.dyq;
    R.ld = which ? A.k_ld : A.q_ld;
    R.w = which ? A.wk : A.wq;
    R.rope = A.rope; R.pos = A.pos;
    R.out = which ? A.ok : A.oq;
    R.H = which ? L.Hkv : L.Hq;
    R.rows = L.T * R.H;
    R.n_pos = A.n_pos; R.rot = A.rot; R.eps = A.eps; R.which = which;
    int lg = 0;
    while ((1 << lg) < R.H) ++lg;
    if (R.H > 1) {
      R.magic = static_cast<uint32_t>((1ull << (31 + lg)) / R.H + 1);
      R.shift = lg - 1;
    }
    R.part = BWD ? L.part + static_cast<size_t>(N.ctas + (which ? N.q_ctas : 0)) * 2 * D : nullptr;
    e = launch_early(norm_rope_rows_kernel<D, ADJ, BWD>,
                     dim3(static_cast<unsigned>(which ? N.k_ctas : N.q_ctas)), kNormThreads, smem,
                     1, s, R);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <bool BWD>
cudaError_t launch_any(const NormLaunch& L, cudaStream_t s) {
  if (L.d == 64)
    return L.adjacent ? launch<64, true, BWD>(L, s) : launch<64, false, BWD>(L, s);
  return L.adjacent ? launch<128, true, BWD>(L, s) : launch<128, false, BWD>(L, s);
}

}  // namespace

int qk_norm_bwd_parts(int Hq, int Hkv, int d, int T) {
  const Launches N = launches_of(Hq, Hkv, d, T, true);
  return N.ctas + N.q_ctas + N.k_ctas;
}

int qk_norm_bwd_max_parts(int Hq, int Hkv, int d) {
  // by tokens at most one per SM (or what the chunks of one token take), by rows one per SM for each
  return std::max(kNumSms, (chunks_of(Hq, d) + chunks_of(Hkv, d) + kNormWarps - 1) / kNormWarps) +
         2 * kNumSms;
}

cudaError_t launch_qk_norm(const NormLaunch& L, cudaStream_t s) { return launch_any<false>(L, s); }

cudaError_t launch_qk_norm_bwd(const NormLaunch& L, cudaStream_t s) {
  return launch_any<true>(L, s);
}

cudaError_t launch_qk_norm_dw(const float* part, int n, int d, float* dwq, float* dwk,
                              cudaStream_t s) {
  return launch_early(qk_norm_dw_kernel, dim3(2 * d / 32), 1024, 0, 1, s, part, n, d, dwq, dwk);
}

}  // namespace moba

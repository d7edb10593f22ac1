// A paged key-value cache: new rows written into their pages (rounded to 8 bits when the cache is
// e4m3), the key sum of every MoBA block kept as its rows arrive, and the cached rows read back
// packed.
//
// Pool layout: k, v [num_pages, Hkv, page_size, d], so that the rows of one page and kv head are
// contiguous (what the attention over them reads). Token u of sequence s lives in page
// page_table[s, u / page_size], slot u % page_size.
// e4m3 rows carry one power-of-two scale, stored as its biased exponent byte b (the value is
// code * 2^(b - 127)): the smallest 2^(b - 127) >= 2^-126 that keeps the row's largest magnitude
// within 448. e4m3 has its own exponent, so a power of two costs at most one binade of its range
// against amax / 448 and none of its 3 mantissa bits; scaling by it is exact, so a code is the
// value rounded once (to nearest even), and code * scale is exact in bf16.
// The sum of block j of a sequence lives at the block's first page, sums [num_pages, Hkv, d] fp32,
// of the keys as given (before the rounding to 8 bits), which the gate scores; the mean differs by
// the factor 1 / block_size, common to all blocks that it ranks.
//
// Bound: HBM (each row read once, written once). One cluster per (sequence, block that the call
// touches, group of kv heads) walks the block's new rows; d / 8 lanes hold one head's row, so the
// row maximum is a 3- or 4-step butterfly. The CTAs of a cluster take consecutive parts of the
// rows and rank 0 adds their column sums in rank order through distributed shared memory: no
// atomics, the same sum every time. Measured: 101K ragged rows of 8 heads of 128 into e4m3 pages,
// 0.62 GB, 109 us in a replayed graph (5.7 TB/s; about 190 instructions per two rows share the SM with
// the copies), 117 as back-to-back calls; the same rows into bf16 pages, 0.83 GB, 139 us (6.0 TB/s);
// 64 single rows 4.0 us (latency). Reading e4m3 rows back packed, 1.3 GB: 212 us (6.1 TB/s), 215.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace cg = cooperative_groups;

namespace moba {

namespace {

constexpr int kCacheThreads = 256;
constexpr int kAppendStages = 5;  // 40 KB a CTA, four CTAs an SM
constexpr int kAppendSmem = kAppendStages * 2 * kCacheThreads * 16;

// Packed arithmetic: an 8-bit row costs about as many instructions as HBM has clocks for it, so
// maxima are taken on bf16 pairs as loaded and sums and products go two to an instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 sum2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
struct Row8 {
  float2 p[4];
};
__device__ __forceinline__ Row8 unpack8(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  Row8 x;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    x.p[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
  return x;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;  // 0 bytes read: the destination is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}

// Largest magnitude of eight bf16 as bf16 bits: without its sign a float orders as an integer.
__device__ __forceinline__ uint32_t max_magnitude(const uint4& u) {
  const uint32_t m = max_u16x2(max_u16x2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                              max_u16x2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// Scale byte of a row whose largest magnitude has the bf16 bits m (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_byte(uint32_t m) {
  return max(static_cast<int>(m >> 7) - 8 + ((m & 0x7fu) > 0x60u ? 1 : 0), 1);
}

__device__ __forceinline__ uint2 to_e4m3(const Row8& x, int b) {
  const float f = __uint_as_float(static_cast<uint32_t>(254 - b) << 23);
  const float2 inv = make_float2(f, f);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = __nv_cvt_float2_to_fp8x2(mul2(x.p[e], inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
}

struct CacheView {
  uint8_t *k, *v, *ks, *vs;
  float* sums;
  const int32_t *page_table, *seq_lens;
  int nseq, max_pages, num_pages, page_log, G, B;
};

struct AppendArgs {
  CacheView C;
  const __nv_bfloat16 *k, *v;
  long long k_ld, v_ld;
  const int32_t* cuq;
  int Tq, heads;  // heads: kv heads per CTA
};

// Largest s in [0, n) with key(s) <= x (key non-decreasing, key(0) <= x): 32 probes at a time, so
// two or three dependent loads where halving would take log2 n. All lanes of the warp call it.
template <class F>
__device__ __forceinline__ int last_not_above(int n, int x, F key) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned ok = __ballot_sync(0xffffffffu, at < hi && key(at) <= x);
    const int p = max(31 - __clz(ok), 0);
    lo += p * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// First unit of sequence s: a sequence with n new rows touches at most n / B + 2 blocks, and
// cuq[s] / B + 2 s leaves room for that without a scan over the sequences before it.
__device__ __forceinline__ int first_unit(int cuq_s, int s, int B) { return cuq_s / B + 2 * s; }

template <int D, bool FP8>
__global__ void __launch_bounds__(kCacheThreads, 4) cache_append_kernel(const AppendArgs A) {
  constexpr int LPR = D / 8;               // lanes per row
  constexpr int SLOTS = kCacheThreads / LPR;
  __shared__ float red[SLOTS][D];          // column sums per slot, then per head in red[head]
  extern __shared__ __align__(128) uint8_t ring[];  // [kAppendStages][K, V][threads] x 16 bytes
  const CacheView& C = A.C;
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int unit = blockIdx.x / CS;
  wait_previous_kernel();
  const int s = last_not_above(C.nseq, unit, [&](int x) {
    return first_unit(A.cuq[x], x, C.B);
  });
  const int c0 = A.cuq[s], c1 = A.cuq[s + 1];
  const int L = C.seq_lens[s];
  // host and device copies may disagree: rows outside the buffers are never touched
  const int n = (c0 >= 0 && c1 >= c0 && c1 <= A.Tq) ? c1 - c0 : 0;
  const int p0 = max(L - n, 0);  // first new position
  const int b = p0 / C.B + unit - first_unit(c0, s, C.B);
  const int cap = static_cast<int>(
      min(static_cast<long long>(C.max_pages) << C.page_log, 0x7fffffffll));
  const int u0 = max(static_cast<int>(min(static_cast<long long>(b) * C.B, 0x7fffffffll)), p0);
  const int u1 = static_cast<int>(min(static_cast<long long>(b + 1) * C.B,
                                      static_cast<long long>(min(L, cap))));
  if (u1 <= u0) return;  // the whole cluster
  const int32_t* pages = C.page_table + static_cast<size_t>(s) * C.max_pages;
  const int per = (u1 - u0 + CS - 1) / CS;
  const int a0 = u0 + rank * per, a1 = min(u1, a0 + per);
  const int g0 = blockIdx.y * A.heads, nh = min(A.heads, C.G - g0);
  const int slot = threadIdx.x / LPR, l = threadIdx.x % LPR;
  const int TP = SLOTS / A.heads;  // rows per pass
  const int hh = slot % A.heads, tt = slot / A.heads;
  const bool mine = hh < nh && tt < TP;
  const int g = g0 + hh;
  Row8 sum;
#pragma unroll
  for (int e = 0; e < 4; ++e) sum.p[e] = make_float2(0.f, 0.f);
  const int mask = (1 << C.page_log) - 1;
  // A thread's 16 bytes of K and V of its slot's rows a0 + tt, a0 + tt + TP, ... pass through a ring
  // that it alone reads, kAppendStages - 1 rows ahead; no barrier.
  const int iters = (a1 - a0 + TP - 1) / TP;  // uniform over the CTA: shuffles below
  const uint32_t my_ring = smem_u32(ring) + threadIdx.x * 16;
  const __nv_bfloat16* ksrc = A.k + (c0 + (a0 + tt - (L - n))) * A.k_ld + g * D + l * 8;
  const __nv_bfloat16* vsrc = A.v + (c0 + (a0 + tt - (L - n))) * A.v_ld + g * D + l * 8;
  const long long k_step = TP * A.k_ld, v_step = TP * A.v_ld;
  int ahead = a0 + tt;  // row of the next copy
  auto issue = [&](int stage) {
    const bool in = mine && ahead < a1;
    const uint32_t d = my_ring + stage * (2 * kCacheThreads * 16);
    copy16(d, in ? ksrc : A.k, in);
    copy16(d + kCacheThreads * 16, in ? vsrc : A.v, in);
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead += TP;
    ksrc += k_step;
    vsrc += v_step;
  };
#pragma unroll
  for (int i = 0; i < kAppendStages - 1; ++i) issue(i);
  int x = a0 + tt, stage = 0;
  auto page_of = [&](int u) { return mine && u < a1 ? pages[u >> C.page_log] : -1; };
  int pid = page_of(x);
  for (int it = 0; it < iters; ++it, x += TP) {
    issue(stage == 0 ? kAppendStages - 1 : stage - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kAppendStages - 1) : "memory");
    const uint8_t* from = ring + stage * (2 * kCacheThreads * 16) + threadIdx.x * 16;
    const uint4 kr = *reinterpret_cast<const uint4*>(from);
    const uint4 vr = *reinterpret_cast<const uint4*>(from + kCacheThreads * 16);
    stage = stage + 1 == kAppendStages ? 0 : stage + 1;
    const bool ok = pid >= 0 && pid < C.num_pages;  // false when the row is not ours
    const size_t at = ((static_cast<size_t>(ok ? pid : 0) * C.G + g) << C.page_log) + (x & mask);
    pid = page_of(x + TP);
    const Row8 kx = unpack8(kr);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum.p[e] = sum2(sum.p[e], kx.p[e]);
    if (FP8) {
      // both maxima in one butterfly: the key row's in the low half, the value row's in the high
      uint32_t top = max_magnitude(kr) | max_magnitude(vr) << 16;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1)
        top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int kb = scale_byte(top & 0xffffu), vb = scale_byte(top >> 16);
      if (ok) {
        *reinterpret_cast<uint2*>(C.k + at * D + l * 8) = to_e4m3(kx, kb);
        *reinterpret_cast<uint2*>(C.v + at * D + l * 8) = to_e4m3(unpack8(vr), vb);
        if (l == 0) {
          C.ks[at] = static_cast<uint8_t>(kb);
          C.vs[at] = static_cast<uint8_t>(vb);
        }
      }
    } else if (ok) {
      *reinterpret_cast<uint4*>(C.k + (at * D + l * 8) * 2) = kr;
      *reinterpret_cast<uint4*>(C.v + (at * D + l * 8) * 2) = vr;
    }
  }
  if (!C.sums) return;  // uniform over the grid
#pragma unroll
  for (int e = 0; e < 8; ++e)
    red[slot][l * 8 + e] = mine ? (e & 1 ? sum.p[e >> 1].y : sum.p[e >> 1].x) : 0.f;
  __syncthreads();
  // red[h] <- sum over the row slots of head h, slots in order
  for (int x = threadIdx.x; x < nh * D; x += kCacheThreads) {
    const int h = x / D, col = x % D;
    float f = red[h][col];
    for (int i = 1; i < TP; ++i) f += red[i * A.heads + h][col];
    red[h][col] = f;
  }
  cluster.sync();
  if (rank == 0) {
    const int home = pages[(static_cast<long long>(b) * C.B) >> C.page_log];
    if (home >= 0 && home < C.num_pages) {
      const bool fresh = static_cast<long long>(b) * C.B >= p0;  // the block begins with new rows
      for (int x = threadIdx.x; x < nh * D; x += kCacheThreads) {
        float* dst = C.sums + (static_cast<size_t>(home) * C.G + g0) * D + x;
        float f = fresh ? 0.f : *dst;
        for (int r = 0; r < CS; ++r) f += *cluster.map_shared_rank(&red[x / D][x % D], r);
        *dst = f;
      }
    }
  }
  cluster.sync();  // peers' shared memory stays until rank 0 has read it
}

struct ReadArgs {
  CacheView C;
  __nv_bfloat16 *k, *v;  // [T, G, D]
  const int32_t* cu;
  int T;
};

// kReadRows consecutive packed rows per CTA; lane t of its first warp finds row t's sequence, page
// and slot, then d / 8 lanes copy one head's row.
constexpr int kReadRows = 32;  // a warp

template <int D, bool FP8>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const ReadArgs A) {
  constexpr int LPR = D / 8, SLOTS = kCacheThreads / LPR, U = 4;
  __shared__ long long at[kReadRows];  // (page * G) << page_log plus slot; -1: zeros, -2: NaN
  const CacheView& C = A.C;
  const int r0 = blockIdx.x * kReadRows;
  const int nr = min(kReadRows, A.T - r0);
  wait_previous_kernel();
  if (threadIdx.x < 32) {  // kReadRows rows, one per lane
    const int s0 = last_not_above(C.nseq, r0, [&](int x) { return A.cu[x]; });
    const int r = r0 + threadIdx.x;
    int lo = s0;  // the rows of a CTA mostly lie in one sequence
    while (lo + 1 < C.nseq && A.cu[lo + 1] <= r) ++lo;
    const long long u = static_cast<long long>(r) - A.cu[lo];
    long long x = -1;
    if (r < A.T && u >= 0 && u < C.seq_lens[lo] && r < A.cu[lo + 1]) {
      x = -2;
      if ((u >> C.page_log) < C.max_pages) {
        const int pid = C.page_table[static_cast<size_t>(lo) * C.max_pages + (u >> C.page_log)];
        if (pid >= 0 && pid < C.num_pages)
          x = ((static_cast<long long>(pid) * C.G) << C.page_log) +
              (u & ((1 << C.page_log) - 1));
      }
    }
    at[threadIdx.x] = x;
  }
  __syncthreads();
  const int slot = threadIdx.x / LPR, l = threadIdx.x % LPR;
  const int total = nr * C.G;  // (row, head) pairs, heads fastest
  for (int x0 = slot; x0 < total; x0 += U * SLOTS) {
    uint4 kr[U], vr[U];
    float kf[U], vf[U];
    long long base[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int x = x0 + i * SLOTS;
      base[i] = -1;
      kr[i] = vr[i] = make_uint4(0, 0, 0, 0);
      kf[i] = vf[i] = 0.f;
      if (x < total) {
        base[i] = at[x / C.G];
        if (base[i] >= 0) {
          const size_t row = static_cast<size_t>(base[i]) +
                             (static_cast<size_t>(x % C.G) << C.page_log);
          if (FP8) {
            const uint2 a = __ldcs(reinterpret_cast<const uint2*>(C.k + row * D) + l);
            const uint2 b = __ldcs(reinterpret_cast<const uint2*>(C.v + row * D) + l);
            kr[i].x = a.x; kr[i].y = a.y;
            vr[i].x = b.x; vr[i].y = b.y;
            kf[i] = __uint_as_float(static_cast<uint32_t>(C.ks[row]) << 23);
            vf[i] = __uint_as_float(static_cast<uint32_t>(C.vs[row]) << 23);
          } else {
            kr[i] = __ldcs(reinterpret_cast<const uint4*>(C.k + row * D * 2) + l);
            vr[i] = __ldcs(reinterpret_cast<const uint4*>(C.v + row * D * 2) + l);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int x = x0 + i * SLOTS;
      if (x >= total) break;
      auto widen = [&](uint4 u, float f) {
        if (base[i] == -2) return make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        if (!FP8) return u;
        uint32_t w[4];
        const uint32_t c[2] = {u.x, u.y};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
              static_cast<__nv_fp8x2_storage_t>(c[e >> 1] >> (16 * (e & 1))), __NV_E4M3);
          const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h));
          const __nv_bfloat162 r = __floats2bfloat162_rn(p.x * f, p.y * f);
          w[e] = *reinterpret_cast<const uint32_t*>(&r);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
      };
      const size_t dst = (static_cast<size_t>(r0) * C.G + x) * D + l * 8;
      __stcs(reinterpret_cast<uint4*>(A.k + dst), widen(kr[i], kf[i]));
      __stcs(reinterpret_cast<uint4*>(A.v + dst), widen(vr[i], vf[i]));
    }
  }
}

CacheView view_of(const PagedCache& P) {
  CacheView C;
  C.k = static_cast<uint8_t*>(P.k); C.v = static_cast<uint8_t*>(P.v);
  C.ks = P.k_scale; C.vs = P.v_scale; C.sums = P.sums;
  C.page_table = P.page_table; C.seq_lens = P.seq_lens;
  C.nseq = P.nseq; C.max_pages = P.max_pages; C.num_pages = P.num_pages;
  C.page_log = P.page_log; C.G = P.G; C.B = P.B;
  return C;
}

template <int D, bool FP8>
cudaError_t append(const PagedCache& P, AppendArgs A, int sms, cudaStream_t s) {
  constexpr int SLOTS = kCacheThreads / (D / 8);
  // Without block sums the block size only cuts the work.
  if (!A.C.sums) A.C.B = 1024;
  const int B = A.C.B;
  const long long units = A.Tq / B + 2ll * P.nseq;
  // Rows a touched block brings on average, cut so that a CTA keeps at least 64 of them.
  const long long rows = std::min<long long>(B, std::max<long long>(1, A.Tq / P.nseq));
  int cs = 1;
  while (cs < 8 && rows / (2 * cs) >= 64) cs *= 2;
  // As many kv heads per CTA as fit its threads (their rows are neighbours in the input); where a
  // CTA has several passes of rows to write, fewer while the grid would not fill the SMs.
  int heads = std::min(P.G, SLOTS);
  const long long busy = std::max<long long>(1, A.Tq / B + P.nseq) * cs;
  while (heads > 1 && rows / cs > 8 && busy * ((P.G + heads - 1) / heads) < 12ll * sms)
    heads = (heads + 1) / 2;
  A.heads = heads;
  return launch_early(cache_append_kernel<D, FP8>,
                      dim3(static_cast<unsigned>(units * cs), (P.G + heads - 1) / heads),
                      kCacheThreads, kAppendSmem, cs, s, A);
}

}  // namespace

cudaError_t launch_cache_append(const PagedCache& P, const void* k, const void* v, long long k_ld,
                                long long v_ld, const int32_t* cuq, int Tq, int sms,
                                cudaStream_t s) {
  AppendArgs A{};
  A.C = view_of(P);
  A.k = static_cast<const __nv_bfloat16*>(k);
  A.v = static_cast<const __nv_bfloat16*>(v);
  A.k_ld = k_ld; A.v_ld = v_ld; A.cuq = cuq; A.Tq = Tq;
  if (P.d == 64) return P.fp8 ? append<64, true>(P, A, sms, s) : append<64, false>(P, A, sms, s);
  return P.fp8 ? append<128, true>(P, A, sms, s) : append<128, false>(P, A, sms, s);
}

cudaError_t launch_cache_read(const PagedCache& P, void* k, void* v, const int32_t* cu, int T,
                              cudaStream_t s) {
  ReadArgs A{};
  A.C = view_of(P);
  A.k = static_cast<__nv_bfloat16*>(k);
  A.v = static_cast<__nv_bfloat16*>(v);
  A.cu = cu; A.T = T;
  const dim3 grid((T + kReadRows - 1) / kReadRows);
  auto kernel = P.d == 64 ? (P.fp8 ? cache_read_kernel<64, true> : cache_read_kernel<64, false>)
                          : (P.fp8 ? cache_read_kernel<128, true> : cache_read_kernel<128, false>);
  return launch_early(kernel, grid, kCacheThreads, 0, 1, s, A);
}

}  // namespace moba

// Attention of the newest rows of cached sequences over a paged key-value cache: over every cached
// key (dense), or over the blocks that the MoBA gate selects. Pages and scales as in kv_cache.cu.
//
// A segment is (sequence s, kv head g, row tile): up to kRows = 8 NT of the rows_per_seq * (Hq/Hkv)
// rows that share kv head g. Its keys are cut into tiles of 8 KB (e4m3: 4 KB) of K
// and as much of V. The tiles of
// all segments form one line, split evenly over the warps of a grid of one CTA per SM, so one
// long sequence, many short ones and a ragged batch all load every SM alike (the host need not
// know the lengths). Each warp is on its own: it streams its tiles through a private ring in
// shared memory (16-byte cp.async, two tiles ahead of the one in work, across segment borders)
// and keeps the running maximum and sum of the softmax in registers. A segment that one warp has
// whole is written at once; otherwise each of its warps leaves a normalised fp32 partial with its
// (max, sum), and paged_merge_kernel joins them in warp order.
//
// Products on mma.sync m16n8k16 with the KEYS as the 16-row operand: S^T = K Q^T (16 keys x 8
// rows), O^T = V^T P^T (16 columns of d x 8 rows). A decode step has 1 to 16 rows per kv head, so
// the 128-row tile of tcgen05.mma would be 1/8 full at best; here a row tile of 8 wastes at most
// 7 rows, and the tensor pipe stays far below the memory time: 16 cached bf16 rows of K and V at
// d = 128 are 8 KB = ~350 clocks of one SM's share of HBM against 24 mma of 16 clocks over four tensor
// units. Bound: HBM, each selected key and value row once. Measured, 32 / 8 heads of 128, in a replayed
// graph (and as back-to-back calls): 8 x 128K tokens of which the heads of a kv group select 26 of 32
// blocks of 4096, 3.6 GB, 528 us (527; 6.8 TB/s); a ragged batch of 32 with 0.69 GB, 113 us (115;
// 6.1 TB/s); 1000 tokens, 9.3 us (9.8; latency).
//
// e4m3 caches: codes widen exactly to f16, products run in f16 with fp32 accumulation. q is bf16
// and becomes f16 after a power-of-two scaling of its row (exactly for elements down to 2^-30 of the
// row's largest; those below 2^-39 of it become zero); a key's scale multiplies its logit z in fp32.
// A value's scale 2^e goes into the weight: w = 2^(z + e - max(z + e) + 15), so that whatever the
// scales of a sequence are, the terms that matter most to a sum are the normal f16 numbers up to 2^15
// and terms below 2^-29 of them lose digits, while the sum of the weights keeps a maximum of its own
// (per lane, joined at the segment's end).
// Rounding: a bf16 cache's weights enter the second product as two bf16 numbers, the second what the
// first's rounding left, so that 2^-16 of a weight is lost and not 2^-8 (a decode over a packed cache
// keeps fp32 weights; the values' bf16 fixes the tensor cores' other operand). The second product of
// each tile costs 0-1 % where a segment has 8 rows or fewer, 4 % at 16 (8 x up to 20K tokens, 4 rows:
// 55.7 -> 58.0 us). An e4m3 cache's weights are f16, off by 2^-11 at most, beside codes that were
// rounded by 2^-4: there a second product costs 6-10 % (8 x 128K tokens 347 -> 369 us, 16 rows a tile
// 95 -> 104), as instructions bound the kernel, and the error against 64 bits stays that of the bf16
// output. Logits, maxima, sums (of the unrounded weights) and outputs are fp32 until the final bf16.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace cg = cooperative_groups;

namespace moba {

namespace {

// Warps of a CTA and bytes of K (and of V) per stage: 192 KB of ring either way. An e4m3 tile takes
// about 930 instructions per 64 keys, a third of them widening codes, so one warp per scheduler
// cannot keep up with HBM on its dependent steps; two with half the tile can (8 x 128K tokens, 32 / 8
// heads of 128: 328 us in short bursts, 6.6 TB/s, and 347-374 in longer runs under the power cap; 365
// with 4 warps and 8 KB).
__host__ __device__ constexpr int paged_warps(bool fp8) { return fp8 ? 8 : 4; }
__host__ __device__ constexpr int tile_bytes(bool fp8) { return fp8 ? 4096 : 8192; }
constexpr int kStages = 3;
// CTAs of a cluster that joins a segment, at most: its warps' partials are one to a lane there.
__host__ __device__ constexpr int join_most(bool fp8) { return fp8 ? 2 : 8; }
static_assert(join_most(false) * paged_warps(false) <= 32 &&
                  join_most(true) * paged_warps(true) <= 32,
              "a cluster's partials are more than the lanes of a warp");
constexpr int kNoLimit = 0x7fffffff;

// ------------------------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;  // 0 bytes read: the destination is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async16_all(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two e4m3 codes (the low or high 16 bits) -> two f16, exact
__device__ __forceinline__ uint32_t widen_lo(uint32_t codes) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}"
      : "=r"(r)
      : "r"(codes));
  return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t codes) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}"
      : "=r"(r)
      : "r"(codes));
  return r;
}
// 2^x to 2 ulp; results below 2^-126 are 0
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// ---------------------------------------------------------------------------------- arguments
struct PagedArgs {
  const __nv_bfloat16* q;  // [nseq * rows, Hq, D]
  const uint8_t *k, *v, *ks, *vs;
  const float* sums;
  const int32_t *page_table, *seq_lens;
  int nseq, max_pages, num_pages, page_log, G, B;
  int rows, Hq, group, nrt, nseg;  // nrt row tiles per (sequence, kv head); nseg segments
  int topk, nb_cap, ent_cap, tiles_per_block;
  int join;  // CTAs of the cluster that has one segment to itself; 0: all segments on one line
  float scale_log2;
  // workspace
  int2* seg_desc;        // [nseg] first worker of a segment, its workers (1: written directly)
  // partials, [2 workers][kRows]: worker w's of a segment that began before it at 2 w, of one that
  // it begins and another finishes at 2 w + 1
  float* part_o;         // x D
  float2* part_ml;
  int* seg_tiles;        // sparse: [nseg] tiles, -1: a page outside the pool
  int2* entries;         // sparse: [nseg][ent_cap] (block, rows that selected it)
  unsigned long long* keys;  // sparse: [nseg][rows of a tile][nb_cap] order keys (large caches)
  unsigned int* marks;       // sparse: [nseg][nb_cap] rows that selected a block (large caches)
  int32_t* idx;          // sparse, nullable: [Hq, nseq * rows, topk]
  __nv_bfloat16* o;
  float* lse;
};

struct Seg { int s, g, rt; };
__device__ __forceinline__ Seg seg_of(const PagedArgs& A, int seg) {
  Seg x;
  x.rt = seg % A.nrt;
  const int sg = seg / A.nrt;
  x.g = sg % A.G;
  x.s = sg / A.G;
  return x;
}

// Cached tokens of sequence s, cut to what its row of the page table can hold (a longer sequence
// is reported as bad by the callers).
__device__ __forceinline__ int seq_len(const PagedArgs& A, int s, bool* over) {
  const int L = max(A.seq_lens[s], 0);
  const long long cap = static_cast<long long>(A.max_pages) << A.page_log;
  *over = L > cap;
  return static_cast<int>(min(static_cast<long long>(L), cap));
}

// ------------------------------------------------------------------------------------- layout
// Byte offset of 16-byte piece c of row r in a tile of rows of RB bytes. Eight consecutive rows'
// pieces c fall into eight different 16-byte columns of the 128-byte bank line (ldmatrix reads
// them without conflicts).
template <int RB>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if (RB == 64) return static_cast<uint32_t>(r) * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  return static_cast<uint32_t>(r) * RB + ((c ^ (r & 7)) << 4);
}

template <int D, bool FP8>
struct Tile {
  static constexpr int kWarps = paged_warps(FP8), kThreads = 32 * kWarps;
  static constexpr int kTileBytes = tile_bytes(FP8);
  static constexpr int RB = D * (FP8 ? 1 : 2);  // bytes of a row
  static constexpr int KT = kTileBytes / RB;    // keys: 32 or 64
  static constexpr int kScaleBytes = FP8 ? 2 * KT : 0;
  static constexpr int kStage = 2 * kTileBytes + kScaleBytes;
  static constexpr int kWarpBytes = kStages * kStage;
};

// Keys of one softmax step. 64 where the registers allow: four independent chains of products
// instead of two, and half the maxima, shuffles and rescaling checks per key.
template <int D, bool FP8, int NT>
struct Sub {
  static constexpr int value = (NT == 1 && Tile<D, FP8>::KT >= 64) ? 64 : 32;
};

// ------------------------------------------------------------------------------ attention
// Worker w of n takes tiles [w U / n, (w + 1) U / n).
__device__ __forceinline__ long long range_start(long long U, int w, int n) {
  return U * w / n;
}

template <int D, bool FP8, int NT, bool SPARSE>
__global__ void __launch_bounds__(Tile<D, FP8>::kThreads, 1) paged_attn_kernel(const PagedArgs A) {
  using TL = Tile<D, FP8>;
  constexpr int kPagedWarps = TL::kWarps, kPagedThreads = TL::kThreads;
  constexpr int kTileBytes = TL::kTileBytes;
  constexpr int RB = TL::RB, KT = TL::KT, kRows = 8 * NT, CPR = RB / 16;
  constexpr int KS = D / 16;
  constexpr int SUB = Sub<D, FP8, NT>::value, MT = SUB / 16;  // keys per softmax step, m-tiles
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ long long prefix[kPagedThreads + 1];
  __shared__ int4 ring[kPagedWarps][4];  // tiles in flight: segment, first key, keys | flags, rows
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = lane & 3, n4 = lane >> 2;
  allow_next_kernel();
  wait_previous_kernel();

  // Tiles of one segment.
  auto tiles_of = [&](int seg) -> int {
    if (SPARSE) return max(A.seg_tiles[seg], 0);
    bool over;
    return (seq_len(A, seg / (A.G * A.nrt), &over) + KT - 1) / KT;
  };
  int workers, me, seg0 = 0;
  long long U, ub, ue, seg_begin = 0;
  if (A.join) {  // this cluster's segment, split over its warps
    seg0 = blockIdx.x / A.join;
    U = tiles_of(seg0);
    workers = static_cast<int>(min(static_cast<long long>(A.join) * kPagedWarps, U));
    // neighbouring tiles go to different CTAs, so that few tiles still use all of them
    me = warp * A.join + static_cast<int>(blockIdx.x % A.join);
    ub = me < workers ? range_start(U, me, workers) : 0;
    ue = me < workers ? range_start(U, me + 1, workers) : 0;
  } else {
    // Prefix sums: thread t owns a run of segments.
    const int per = (A.nseg + kPagedThreads - 1) / kPagedThreads;
    {
      long long mine = 0;
      const int a = min(A.nseg, tid * per), b = min(A.nseg, a + per);
      for (int i = a; i < b; ++i) mine += tiles_of(i);
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) prefix[warp] = incl;
      __syncthreads();
      long long before = 0, all = 0;
      for (int w = 0; w < kPagedWarps; ++w) {
        const long long x = prefix[w];
        if (w < warp) before += x;
        all += x;
      }
      __syncthreads();
      prefix[tid] = before + incl - mine;
      if (tid == 0) prefix[kPagedThreads] = all;
      __syncthreads();
    }
    U = prefix[kPagedThreads];
    // Neighbouring workers sit on different SMs, so that few tiles still use many of them.
    workers = static_cast<int>(min(static_cast<long long>(gridDim.x) * kPagedWarps, U));
    me = warp * gridDim.x + blockIdx.x;
    if (me >= workers) return;  // no block-wide barrier below on this path
    ub = range_start(U, me, workers);
    ue = range_start(U, me + 1, workers);

    // Segment of tile ub: the run that holds it, then 32 segments at a time.
    {
      int run = 0;
      for (int x = lane; x < kPagedThreads; x += 32)
        if (prefix[x] <= ub) run = x;  // ascending in x per lane
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) run = max(run, __shfl_xor_sync(0xffffffffu, run, o));
      long long at = prefix[run];
      const int last = min(A.nseg, (run + 1) * per);
      for (int i = run * per; i < last; i += 32) {
        const int cnt = i + lane < last ? tiles_of(i + lane) : 0;
        long long incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, at + incl > ub);
        if (hit) {
          const int src = __ffs(hit) - 1;
          seg0 = i + src;
          seg_begin = at + __shfl_sync(0xffffffffu, incl - cnt, src);
          break;
        }
        at += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
  }

  uint8_t* wbase = smem + warp * TL::kWarpBytes;
  const uint32_t wsm = smem_u32(wbase);

  // ---- loader: walks the tiles ahead of the consumer
  int l_seg = seg0, l_tile = static_cast<int>(ub - seg_begin), l_tiles = tiles_of(seg0);
  long long l_left = ue - ub;
  Seg l_id = seg_of(A, seg0);
  bool l_over;
  int l_len = seq_len(A, l_id.s, &l_over);
  int4 pend = make_int4(-1, 0, 0, 0);  // tile whose page ids are in my_pid
  int pend_g = 0, my_pid = -1;
  auto look_up = [&]() {  // next tile's place and pages
    pend.x = -1;
    if (l_left == 0) return;
    while (l_tile >= l_tiles) {
      if (++l_seg >= A.nseg) {  // lengths changed under the call: nothing more to copy
        l_left = 0;
        return;
      }
      l_tile = 0;
      l_tiles = tiles_of(l_seg);
      if (l_tiles) {
        l_id = seg_of(A, l_seg);
        l_len = seq_len(A, l_id.s, &l_over);
      }
    }
    int kpos = l_tile * KT, end = l_len;
    unsigned rows = 0xffffffffu;
    if (SPARSE) {
      const int e = l_tile / A.tiles_per_block;
      const int2 ent = A.entries[static_cast<size_t>(l_seg) * A.ent_cap + e];
      kpos = ent.x * A.B + (l_tile - e * A.tiles_per_block) * KT;
      end = static_cast<int>(min(static_cast<long long>(end),
                                 (static_cast<long long>(ent.x) + 1) * A.B));
      rows = static_cast<unsigned>(ent.y);
    }
    const int nk = min(KT, end - kpos);
    my_pid = 0;
    bool bad = l_over;
    if (lane < KT / 16 && lane * 16 < nk) {
      my_pid = A.page_table[static_cast<size_t>(l_id.s) * A.max_pages +
                             ((kpos + lane * 16) >> A.page_log)];
      if (my_pid < 0 || my_pid >= A.num_pages) {
        bad = true;
        my_pid = -1;
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    pend = make_int4(l_seg, kpos, nk | (bad ? 1 << 16 : 0), static_cast<int>(rows));
    pend_g = l_id.g;
    ++l_tile;
    --l_left;
  };
  // This lane's 16-byte pieces of 16 rows: piece i is row i * kRowsPer + lane / CPR, column
  // lane % CPR. Its swizzled place is that of piece 0 with the row's bits above lane / CPR flipped
  // in, so a full tile costs one xor and two copies per piece.
  constexpr int kPieces = 16 * CPR / 32, kRowsPer = 32 / CPR;
  constexpr int kBits = RB == 64 ? 0 : 7;  // bits of a row that the swizzle sees, above my_row's
  const int my_row = lane / CPR, my_col = lane % CPR;
  const uint32_t my_dst = swz<RB>(my_row, my_col), my_src = my_row * RB + my_col * 16;
  auto issue = [&](int stage, int slot4) {  // copies of the pending tile into `stage`
    if (pend.x >= 0) {
      if (lane == 0) ring[warp][slot4] = pend;
      const int nk = pend.z & 0xffff, mask = (1 << A.page_log) - 1;
      const uint32_t kd = wsm + stage * TL::kStage;
      if (pend.z == KT) {  // all keys there, all pages good
        const uint8_t *ks = nullptr, *vs = nullptr;
        const uint8_t* ss = nullptr;
#pragma unroll
        for (int gq = 0; gq < KT / 16; ++gq) {  // 16 keys of one page
          const int at = (pend.y + gq * 16) & mask;
          if (gq == 0 || at == 0) {
            const int pid = __shfl_sync(0xffffffffu, my_pid, gq);
            const size_t row = ((static_cast<size_t>(pid) * A.G + pend_g) << A.page_log) + at;
            ks = A.k + row * RB + my_src - gq * 16 * RB;
            vs = A.v + row * RB + my_src - gq * 16 * RB;
            if (FP8) ss = (lane ? A.vs : A.ks) + row - gq * 16;
          }
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const uint32_t d = kd + gq * 16 * RB + i * kRowsPer * RB +
                               (my_dst ^ (((i * kRowsPer) & kBits) << 4));
            cp_async16_all(d, ks + (gq * 16 + i * kRowsPer) * RB);
            cp_async16_all(d + kTileBytes, vs + (gq * 16 + i * kRowsPer) * RB);
          }
          if (FP8 && lane < 2)  // 16 scale bytes of K (lane 0) and V (lane 1)
            cp_async16_all(kd + 2 * kTileBytes + lane * KT + gq * 16, ss + gq * 16);
        }
      } else {
#pragma unroll 1
        for (int gq = 0; gq < KT / 16; ++gq) {
          const int pid = __shfl_sync(0xffffffffu, my_pid, gq);
          const size_t row =
              ((static_cast<size_t>(max(pid, 0)) * A.G + pend_g) << A.page_log) +
              ((pend.y + gq * 16) & mask);
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const bool ok = pid >= 0 && gq * 16 + i * kRowsPer + my_row < nk;
            const size_t off = ok ? (row + i * kRowsPer) * RB + my_src : 0;
            const uint32_t d = kd + gq * 16 * RB + i * kRowsPer * RB +
                               (my_dst ^ (((i * kRowsPer) & kBits) << 4));
            cp_async16(d, A.k + off, ok);
            cp_async16(d + kTileBytes, A.v + off, ok);
          }
          if (FP8 && lane < 2) {
            const bool ok = pid >= 0 && gq * 16 < nk;
            cp_async16(kd + 2 * kTileBytes + lane * KT + gq * 16,
                       (lane ? A.vs : A.ks) + (ok ? row : 0), ok);
          }
        }
      }
    }
    cp_async_commit();
  };

  const int ntiles = static_cast<int>(ue - ub);
  look_up();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    issue(i, i);
    look_up();
  }

  // ---- consumer state
  int seg = -1, first_tile_of_seg = 0;
  Seg id{0, 0, 0};
  uint32_t qf[KS][NT][2];
  float acc[KS][NT][4];
  // m: maximum of the logits z, in log2 units (e4m3: of z + the value scale's exponent); l: sum of
  // 2^(z - m) (e4m3: of 2^(z - r), r this lane's own maximum of z)
  float m[NT][2], l[NT][2], r[NT][2], cmul[NT][2];
  int lim[NT][2];
  bool bad = false;
  long long cur_begin = seg_begin;  // first tile of the current segment on the line
  int cur_tiles = 0;

  auto begin = [&](int sg) {
    id = seg_of(A, sg);
    bool over;
    const int L = seq_len(A, id.s, &over);
    bad = over;
    const int R = A.rows * A.group;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int rr = id.rt * kRows + nt * 8 + n4;  // row whose elements this lane holds
      const bool in = rr < R;
      const __nv_bfloat16* src =
          A.q + (static_cast<size_t>(id.s) * A.rows + (in ? rr / A.group : 0)) * A.Hq * D +
          (static_cast<size_t>(id.g) * A.group + (in ? rr % A.group : 0)) * D;
      // the pairs of d that a lane's two B registers hold: 2c and 2c + 8 of each 16 columns, or
      // 4c and 4c + 2 where the keys' bytes come four to a lane
      constexpr int kFirst = FP8 ? 4 : 2, kSecond = FP8 ? 2 : 8;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qf[ks][nt][0] = in ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + kFirst * c) : 0u;
        qf[ks][nt][1] =
            in ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + kFirst * c + kSecond) : 0u;
      }
      float f = A.scale_log2;
      if (FP8) {
        uint32_t top = 0;  // largest magnitude of the row, as bf16 bits
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            top = max(top, max(qf[ks][nt][h] & 0x7fffu, (qf[ks][nt][h] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // times 2^(13 - exponent): the largest element lies in [2^13, 2^14)
        // (2^126 at most, whose inverse is a normal number too)
        const int up = min(253, max(1, 267 - static_cast<int>(top >> 7)));
        const float mul = __uint_as_float(static_cast<uint32_t>(up) << 23);
        // never 0: a hidden key's -inf times it has to stay -inf
        f = fmaxf(f * __uint_as_float(static_cast<uint32_t>(254 - up) << 23), FLT_MIN);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            qf[ks][nt][h] = pack_f16(__uint_as_float(qf[ks][nt][h] << 16) * mul,
                                     __uint_as_float(qf[ks][nt][h] & 0xffff0000u) * mul);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        cmul[nt][j] = FP8 ? __shfl_sync(0xffffffffu, f, (2 * c + j) * 4) : f;
        const int rc = id.rt * kRows + nt * 8 + 2 * c + j;  // row of this lane's result columns
        // keys it may see; a column of padding (q = 0, never written) needs no mask
        lim[nt][j] = rc < R ? L - A.rows + rc / A.group + 1 : kNoLimit;
        m[nt][j] = r[nt][j] = -INFINITY;
        l[nt][j] = 0.f;
      }
#pragma unroll
      for (int ds = 0; ds < KS; ++ds)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[ds][nt][x] = 0.f;
    }
  };

  auto finish = [&](int sg, int t0, int t1) {  // this warp had tiles [t0, t1) of the segment
    const bool whole = t0 == 0 && t1 == cur_tiles && !A.join;
    const int R = A.rows * A.group;
    const size_t slot = 2 * static_cast<size_t>(me) + (t0 == 0 ? 1 : 0);
    // partials: in the workspace, or in this warp's own (now idle) ring for the cluster to join
    float* po = A.join ? reinterpret_cast<float*>(wbase) : A.part_o + slot * kRows * D;
    float2* pml = A.join ? reinterpret_cast<float2*>(wbase + kRows * D * 4)
                         : A.part_ml + slot * kRows;
    if (t1 == cur_tiles && lane == 0 && !A.join) {
      int w0 = me;
      if (!whole) {  // worker of the segment's first tile
        w0 = static_cast<int>(cur_begin * workers / U);
        while (range_start(U, w0 + 1, workers) <= cur_begin) ++w0;
        while (range_start(U, w0, workers) > cur_begin) --w0;
      }
      A.seg_desc[sg] = make_int2(w0, me - w0 + 1);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float nan = __int_as_float(0x7fffffff);
        float s = l[nt][j], top = m[nt][j], mul;
        if (FP8) {
          top = r[nt][j];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          if (s != 0.f) s *= ex2(r[nt][j] - top);  // a lane without keys: 0, and r = -inf
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        mul = s > 0.f ? 1.f / s : 0.f;
        // e4m3: times 2^(m - 15 - top), down to 2^-141: half of the exponent in each of two factors,
        // as the whole would be 0 where the values' scales are all small
        float lead = 1.f;
        if (FP8 && s > 0.f) {
          lead = ex2(0.5f * (m[nt][j] - 15.f - top));
          mul *= lead;
        }
        // The maxima pass over a NaN logit, the sum keeps it. A row that sees a key and ends
        // without a sum had logits of -inf alone.
        const bool gone = bad || s != s || (whole && lim[nt][j] > 0 && !(s > 0.f));
        if (gone) mul = top = nan;
        const int col = nt * 8 + 2 * c + j, rr = id.rt * kRows + col;
        if (rr >= R) continue;
        if (whole) {
          const int tok = rr / A.group, h = id.g * A.group + rr % A.group;
          const size_t row = static_cast<size_t>(id.s) * A.rows + tok;
          __nv_bfloat16* dst = A.o + (row * A.Hq + h) * D;
#pragma unroll
          for (int ds = 0; ds < KS; ++ds) {
            const int d0 = ds * 16 + (FP8 ? 2 * n4 : n4), d1 = d0 + (FP8 ? 1 : 8);
            dst[d0] = __float2bfloat16_rn(acc[ds][nt][j] * lead * mul);
            dst[d1] = __float2bfloat16_rn(acc[ds][nt][2 + j] * lead * mul);
          }
          if (n4 == 0)
            A.lse[static_cast<size_t>(h) * A.nseq * A.rows + row] =
                gone ? nan : s > 0.f ? (top + log2f(s)) * 0.69314718055994531f : -INFINITY;
        } else {
          float* dst = po + col * D;
#pragma unroll
          for (int ds = 0; ds < KS; ++ds) {
            const int d0 = ds * 16 + (FP8 ? 2 * n4 : n4), d1 = d0 + (FP8 ? 1 : 8);
            dst[d0] = acc[ds][nt][j] * lead * mul;
            dst[d1] = acc[ds][nt][2 + j] * lead * mul;
          }
          if (n4 == 0) pml[col] = make_float2(top, s);
        }
      }
  };

  // ---- tiles. The descriptor of tile `it` was written two iterations ago, before a __syncwarp;
  // a new segment's q is fetched while its first tile is still on its way.
  __syncwarp();
  int stage = 0, next_tile = static_cast<int>(ub - seg_begin);
  for (int it = 0; it < ntiles; ++it) {
    const int4 t = ring[warp][it & 3];
    if (t.x != seg) {
      if (seg >= 0) {
        finish(seg, first_tile_of_seg, cur_tiles);
        cur_begin += cur_tiles;
        next_tile = 0;
      }
      seg = t.x;
      cur_tiles = tiles_of(seg);
      first_tile_of_seg = next_tile;
      begin(seg);
    }
    cp_async_wait<kStages - 2>();
    __syncwarp();
    // the stage that was consumed in the last iteration takes the next tile
    issue(stage == 0 ? kStages - 1 : stage - 1, (it + kStages - 1) & 3);
    look_up();
    ++next_tile;
    const int nk = t.z & 0xffff;
    bad |= (t.z >> 16) != 0;
    const unsigned rows = static_cast<unsigned>(t.w);
    const uint32_t kb = wsm + stage * TL::kStage, vb = kb + kTileBytes;
    const uint8_t* sc = wbase + stage * TL::kStage + 2 * kTileBytes;
    int klim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        klim[nt][j] =
            lim[nt][j] == kNoLimit ? kNoLimit
            : (!SPARSE || ((rows >> (nt * 8 + 2 * c + j)) & 1)) ? min(lim[nt][j], t.y + nk) : 0;
    bool masked = false;  // a key of the tile is hidden from a row
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) masked |= klim[nt][j] < t.y + KT;
    masked = __any_sync(0xffffffffu, masked);
#pragma unroll 1
    for (int sub = 0; sub < KT / SUB; ++sub) {
      if (sub * SUB >= nk) break;
      float sacc[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) sacc[mt][nt][x] = 0.f;
      // S^T = K Q^T
      const int krow = sub * SUB + (lane & 15);
      if (!FP8) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t a[4];
            ldsm4(a, kb + swz<RB>(krow + mt * 16, ks * 2 + (lane >> 4)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<false>(sacc[mt][nt], a, qf[ks][nt][0], qf[ks][nt][1]);
          }
      } else {
#pragma unroll
        for (int k2 = 0; k2 < KS / 2; ++k2)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            // matrices: (keys 0-7, 16 columns), (keys 8-15, same), then the next 16 columns
            uint32_t b[4];
            ldsm4(b, kb + swz<RB>(krow + mt * 16, k2 * 2 + (lane >> 4)));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t a[4];
              a[0] = widen_lo(b[2 * h]);
              a[1] = widen_lo(b[2 * h + 1]);
              a[2] = widen_hi(b[2 * h]);
              a[3] = widen_hi(b[2 * h + 1]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816<true>(sacc[mt][nt], a, qf[2 * k2 + h][nt][0], qf[2 * k2 + h][nt][1]);
            }
          }
      }
      // softmax: this lane holds keys n4 + 8 x of each 16, columns 2c, 2c + 1
      float ve[MT][2];  // exponent of the value's scale
      if (FP8) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int key = sub * SUB + mt * 16 + x * 8 + n4;
            const float f = __uint_as_float(static_cast<uint32_t>(sc[key]) << 23);
            ve[mt][x] = static_cast<float>(static_cast<int>(sc[KT + key]) - 127);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              sacc[mt][nt][2 * x] *= f;
              sacc[mt][nt][2 * x + 1] *= f;
            }
          }
      }
      if (masked) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = t.y + sub * SUB + mt * 16 + (x >> 1) * 8 + n4;
              if (key >= klim[nt][x & 1]) sacc[mt][nt][x] = -INFINITY;
            }
      }
      float corr[NT][2];
      bool grew = false;
      uint32_t pf[MT][NT][2];  // P^T as the second operand: 8 x 8 pieces turned within the warp
      uint32_t pl[FP8 ? 1 : MT][NT][2];  // bf16: what its rounding leaves
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[MT][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float cm = cmul[nt][j];
          float best = -INFINITY, own = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float z = sacc[mt][nt][2 * x + j];  // before the factor cm > 0
              if (FP8) {
                own = fmaxf(own, z);
                w[mt][2 * x + j] = fmaf(z, cm, ve[mt][x]);
                best = fmaxf(best, w[mt][2 * x + j]);
              } else {
                best = fmaxf(best, z);
              }
            }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
          if (!FP8) best *= cm;
          const float mn = fmaxf(m[nt][j], best);
          corr[nt][j] = mn > m[nt][j] ? ex2(m[nt][j] - mn) : 1.f;  // 0 for the first keys
          grew |= mn > m[nt][j];
          m[nt][j] = mn;
          // no key yet: any finite reference gives weights of 0
          const float ref = mn == -INFINITY ? 0.f : mn;
          float sum = 0.f;
          if (FP8) {
            const float rn = fmaxf(r[nt][j], own * cm);
            const float rref = rn == -INFINITY ? 0.f : rn;
            const float keep = rn > r[nt][j] ? ex2(r[nt][j] - rn) : 1.f;
            r[nt][j] = rn;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                sum += ex2(fmaf(sacc[mt][nt][2 * x + j], cm, -rref));
                w[mt][2 * x + j] = ex2(w[mt][2 * x + j] - (ref - 15.f));
              }
            l[nt][j] = fmaf(l[nt][j], keep, sum);
          } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float p = ex2(fmaf(sacc[mt][nt][2 * x + j], cm, -ref));
                w[mt][2 * x + j] = p;
                sum += p;
              }
            l[nt][j] = fmaf(l[nt][j], corr[nt][j], sum);
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float w0 = w[mt][2 * x], w1 = w[mt][2 * x + 1];
            const uint32_t high = FP8 ? pack_f16(w0, w1) : pack_bf16(w0, w1);
            pf[mt][nt][x] = transpose8x8(high);
            if constexpr (!FP8)
              pl[mt][nt][x] = transpose8x8(pack_bf16(w0 - __uint_as_float(high << 16),
                                                     w1 - __uint_as_float(high & 0xffff0000u)));
          }
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int ds = 0; ds < KS; ++ds)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[ds][nt][x] *= corr[nt][x & 1];
      }
      // O^T += V^T P^T
      if (!FP8) {
        const int vrow = sub * SUB + ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
        // four accumulators in turn: a product waits for the one four before it
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int d0 = 0; d0 < KS; d0 += 4) {
            uint32_t a[4][4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              ldsm4t(a[x], vb + swz<RB>(vrow + mt * 16, (d0 + x) * 2 + half));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                mma16816<false>(acc[d0 + x][nt], a[x], pf[mt][nt][0], pf[mt][nt][1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                mma16816<false>(acc[d0 + x][nt], a[x], pl[FP8 ? 0 : mt][nt][0],
                                pl[FP8 ? 0 : mt][nt][1]);
          }
      } else {
        // matrices: (keys 0-7, 16 columns), (keys 8-15, same), then the next 16 columns; a
        // register holds columns 2i, 2i + 1 of keys 2c, 2c + 1
        const int vrow = sub * SUB + (((lane >> 3) & 1) << 3) + (lane & 7);
#pragma unroll
        for (int d2 = 0; d2 < KS / 2; ++d2)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t b[4];
            ldsm4t(b, vb + swz<RB>(vrow + mt * 16, d2 * 2 + (lane >> 4)));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t lo = __byte_perm(b[2 * h], 0, 0x3120);
              const uint32_t hi = __byte_perm(b[2 * h + 1], 0, 0x3120);
              uint32_t a[4];
              a[0] = widen_lo(lo);  // column 2i of keys 2c, 2c + 1
              a[1] = widen_hi(lo);  // column 2i + 1
              a[2] = widen_lo(hi);  // keys 8 + 2c, 8 + 2c + 1
              a[3] = widen_hi(hi);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816<true>(acc[2 * d2 + h][nt], a, pf[mt][nt][0], pf[mt][nt][1]);
            }
          }
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  if (A.join) __syncwarp();  // all copies into the ring have landed: it takes the partial
  if (seg >= 0) finish(seg, first_tile_of_seg, next_tile);
  if (!A.join) return;

  // ---- the cluster joins its segment. CTA r takes rows r, r + CTAs, ...: a warp per row and slice
  // of the partials, lanes over d, eight partials in flight; the slices meet in shared memory.
  float2* my_ml = reinterpret_cast<float2*>(wbase + kRows * D * 4);
  if (seg < 0 && lane < kRows) my_ml[lane] = make_float2(-INFINITY, 0.f);
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  constexpr int PER = D / 32;
  float* slices = reinterpret_cast<float*>(smem + kRows * D * 4 + kRows * 8);  // [warps][D]
  const Seg js = seg_of(A, seg0);
  bool over;
  const int jlen = seq_len(A, js.s, &over);
  if (SPARSE) over |= A.seg_tiles[seg0] < 0;
  const int crank = blockIdx.x % A.join;
  const int nrow = min(kRows, A.rows * A.group - js.rt * kRows);
  const int mine = (nrow - crank + A.join - 1) / A.join;  // rows of this CTA
  int nr = 1;  // rows at once
  while (nr < mine && nr < kPagedWarps) nr *= 2;
  const int parts = A.join * kPagedWarps;  // at most 32
  const int nslice = kPagedWarps / nr, each = parts / nslice, slice = warp / nr;
  for (int k0 = 0; k0 < mine; k0 += nr) {  // uniform over the CTA
    const int k = k0 + warp % nr, row = crank + k * A.join;
    const bool on = k < mine;
    auto part = [&](int i) {  // partial i in the memory of its CTA
      return cluster.map_shared_rank(smem + (i / A.join) * TL::kWarpBytes, i % A.join);
    };
    float pm = -INFINITY, pl = 0.f, o[PER];  // partial `lane`
    if (on && lane < parts) {
      const float2 ml = reinterpret_cast<const float2*>(part(lane) + kRows * D * 4)[row];
      pm = ml.x;
      pl = ml.y;
    }
    bool nan = __any_sync(0xffffffffu, over || !(pm <= FLT_MAX));
    float top = pm;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    pl = pl > 0.f ? pl * ex2(pm - top) : 0.f;
    float sum = pl;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    // a row with a position and without a sum: logits of -inf alone
    nan |= !(sum > 0.f) && jlen - A.rows + (js.rt * kRows + row) / A.group >= 0;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = 0.f;
    for (int i0 = slice * each; i0 < (slice + 1) * each; i0 += 8) {
      float w[8], v[8][PER];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = min(i0 + i, parts - 1);
        const float wi = __shfl_sync(0xffffffffu, pl, at);
        w[i] = i0 + i >= (slice + 1) * each ? 0.f : wi;
        const float* src = reinterpret_cast<const float*>(part(at)) + row * D + lane * PER;
#pragma unroll
        for (int e = 0; e < PER; ++e) v[i][e] = on ? src[e] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < PER; ++e)  // a warp without tiles has left no values
          o[e] = w[i] > 0.f ? fmaf(w[i], v[i][e], o[e]) : o[e];
    }
    if (nslice > 1) {
#pragma unroll
      for (int e = 0; e < PER; ++e) slices[warp * D + lane * PER + e] = o[e];
      __syncthreads();
      if (slice == 0)
        for (int x = 1; x < nslice; ++x)
#pragma unroll
          for (int e = 0; e < PER; ++e) o[e] += slices[(x * nr + warp) * D + lane * PER + e];
    }
    if (slice == 0 && on) {
      const int rr = js.rt * kRows + row, h = js.g * A.group + rr % A.group;
      const size_t at = static_cast<size_t>(js.s) * A.rows + rr / A.group;
      const float inv = nan ? __int_as_float(0x7fffffff) : sum > 0.f ? 1.f / sum : 0.f;
      uint32_t* dst = reinterpret_cast<uint32_t*>(A.o + (at * A.Hq + h) * D + lane * PER);
#pragma unroll
      for (int e = 0; e < PER; e += 2)
        dst[e / 2] = nan ? 0x7fff7fffu : pack_bf16(o[e] * inv, o[e + 1] * inv);
      if (lane == 0)
        A.lse[static_cast<size_t>(h) * A.nseq * A.rows + at] =
            nan ? inv : sum > 0.f ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
    }
    if (nslice > 1) __syncthreads();  // slices before the next rows
  }
  cluster.sync();  // peers' partials stay until everyone has read them
}

// ------------------------------------------------------------------------------------- merge
// One CTA per (sequence, row, head): the partials of its segment, its warps taking every NW-th,
// joined in a fixed order. Bound by latency: two dependent loads (the segment's description, then
// the partials), so a warp has kMergeBatch partials in flight at once and the host gives a CTA
// more warps the fewer segments share the partials. Rows without keys get o = 0, lse = -inf; a
// row whose sequence names a page outside the pool gets NaN, and so does one whose query is not
// finite.
constexpr int kMergeBatch = 8;
constexpr int kMergeWarps = 16;  // at most

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) paged_merge_kernel(const PagedArgs A,
                                                                       int kRows, bool sparse) {
  __shared__ float sm[kMergeWarps], sl[kMergeWarps], so[kMergeWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, NW = blockDim.x >> 5;
  constexpr int PER = D / 32;
  const int h = blockIdx.x % A.Hq, row = blockIdx.x / A.Hq;
  const int s = row / A.rows, r = row % A.rows, g = h / A.group;
  const int rr = r * A.group + h % A.group, rt = rr / kRows, col = rr % kRows;
  const int seg = (s * A.G + g) * A.nrt + rt;
  wait_previous_kernel();
  bool over;
  const int L = seq_len(A, s, &over);
  // written for every segment that has tiles
  const int2 desc = A.seg_desc[seg];
  const int tiles = sparse ? A.seg_tiles[seg] : L;
  const int count = tiles > 0 ? desc.y : 0;
  bool bad = over || tiles < 0;
  if (count == 1) return;  // written by the warp that had all of it
  float m = -INFINITY, l = 0.f, acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  for (int i0 = warp; i0 < count; i0 += NW * kMergeBatch) {
    float2 ml[kMergeBatch];
    float o[kMergeBatch][PER];
#pragma unroll
    for (int x = 0; x < kMergeBatch; ++x) {
      const int i = i0 + x * NW;
      ml[x] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < PER; ++e) o[x][e] = 0.f;
      if (i < count) {
        const size_t at = (2 * static_cast<size_t>(desc.x + i) + (i == 0 ? 1 : 0)) * kRows + col;
        ml[x] = A.part_ml[at];
        const float* src = A.part_o + at * D + lane * PER;
        if constexpr (PER == 4) {
          const float4 f = *reinterpret_cast<const float4*>(src);
          o[x][0] = f.x; o[x][1] = f.y; o[x][2] = f.z; o[x][3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(src);
          o[x][0] = f.x; o[x][1] = f.y;
        }
      }
    }
#pragma unroll
    for (int x = 0; x < kMergeBatch; ++x) {
      bad |= !(ml[x].x <= FLT_MAX);  // NaN: a bad page or a logit that is NaN
      if (ml[x].y > 0.f) {
        const float mn = fmaxf(m, ml[x].x), a = exp2f(m - mn), b = exp2f(ml[x].x - mn) * ml[x].y;
        l = fmaf(l, a, b);
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = fmaf(acc[e], a, b * o[x][e]);
        m = mn;
      }
    }
  }
  if (lane == 0) {
    sm[warp] = bad ? __int_as_float(0x7fffffff) : m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < PER; ++e) so[warp][lane * PER + e] = acc[e];
  __syncthreads();
  float M = -INFINITY, Lsum = 0.f;
  bool any_bad = false;
  for (int w = 0; w < NW; ++w) {
    any_bad |= sm[w] != sm[w];
    M = fmaxf(M, sm[w]);
  }
  for (int w = 0; w < NW; ++w)
    if (sl[w] > 0.f) Lsum = fmaf(exp2f(sm[w] - M), sl[w], Lsum);
  // a row with a position and without a sum: logits of -inf alone
  any_bad |= !(Lsum > 0.f) && L - A.rows + r >= 0;
  const float inv = any_bad ? __int_as_float(0x7fffffff) : Lsum > 0.f ? 1.f / Lsum : 0.f;
  for (int x = threadIdx.x; x < D; x += blockDim.x) {
    float o = 0.f;
    for (int w = 0; w < NW; ++w)
      if (sl[w] > 0.f) o = fmaf(exp2f(sm[w] - M), so[w][x], o);
    A.o[(static_cast<size_t>(row) * A.Hq + h) * D + x] = __float2bfloat16_rn(o * inv);
  }
  if (threadIdx.x == 0)
    A.lse[static_cast<size_t>(h) * A.nseq * A.rows + row] =
        any_bad ? __int_as_float(0x7fffffff)
                : Lsum > 0.f ? (M + log2f(Lsum)) * 0.69314718055994531f : -INFINITY;
}

// -------------------------------------------------------------------------------------- gate
// Routing of one segment's rows: scores of the past blocks, the exact top (topk - 1) of each row,
// and the list of blocks that any of the rows selected, with the rows that did.
// Scores are q . (block sum): the mean's 1 / B is common to the past blocks, which are all full.
// They are accumulated in fp64 (products of bf16 and fp32 are exact there), so the selection does
// not hang on the order of the sum; fp64 runs at half the fp32 rate here and the scores are a
// small part of the step. Equal scores: the lower block first.
//
// Bound by latency (a chain of page id, sum, score, selection, list), so: one cluster of up to 8
// CTAs per segment, eight lanes to a block's sum so that a CTA of 8 warps has 32 blocks in flight;
// the page ids and q are fetched before the sequence's length is known; all rows' partial sums of
// a block are reduced together, a lane keeping half of its values at each step; and the selection is
// ranking by 32 shuffles (at most 32 past blocks), one warp per row with its keys in registers (at
// most 256), or one CTA per row (beyond; keys in registers up to 2048). The latter two are a radix
// selection on order-preserving 64-bit keys whose 256 bins span only the range still in question:
// usually two sweeps instead of the eight that fixed bytes of an fp64 key would take.
// Measured inside the kernel, in clocks: 31 past blocks and 4 rows, 10,000 (lengths and q 2,600,
// scores 3,000, selection 2,300, list 2,200; a step runs once, so much of it is the first fetch of
// its instructions); 1791 blocks of d = 64 and one row over 4 CTAs, 20,000.
constexpr int kGateThreads = 256;
constexpr int kGateWarps = kGateThreads / 32;
constexpr int kGateInRegs = 8;  // keys a thread holds in a selection
constexpr int kGateWords = kMaxBlocksPerSeq / 32;
constexpr int kGateSmem = 65536;  // for keys and marks

__device__ __forceinline__ unsigned long long order_key64(double x) {
  if (x != x) return 0ull;  // NaN: behind every number
  const unsigned long long u =
      static_cast<unsigned long long>(__double_as_longlong(x + 0.0));  // -0 -> +0
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// Sum over groups of eight lanes of each of RR values per lane. At each step a lane keeps half of
// its values and hands over the other half, so lane x of a group ends with the sums of values
// first(x) .. first(x) + max(1, RR / 8) - 1 in v[0] ..., and RR < 8 leaves 8 / RR lanes with the same.
template <int RR>
__device__ __forceinline__ void reduce_rows8(double (&v)[RR], int lane) {
  int n = RR;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    if (n > 1) {
      const bool up = lane & o;
      n >>= 1;
#pragma unroll
      for (int i = 0; i < RR / 2; ++i)
        if (i < n) {
          const double give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
}

// One bin of a radix pass: the highest bin that brings the count from the top to `want`.
// Returns the bin, the keys in it (0 when the bins hold fewer than `want`) and the keys above it;
// every lane of the warp gets them.
__device__ __forceinline__ void pick_bin(const int* hist, int want, int lane, int* bin, int* cnt,
                                         int* above) {
  int bins[8], mine = 0;  // lane 0 has the eight highest bins
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    bins[x] = hist[255 - (lane * 8 + x)];
    mine += bins[x];
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, incl >= want)) - 1;
  int ab = incl - mine, b = 0, c = 0;
#pragma unroll
  for (int x = 0; x < 8; ++x)
    if (c == 0) {
      if (ab + bins[x] >= want) { b = 255 - (lane * 8 + x); c = bins[x]; }
      else ab += bins[x];
    }
  *bin = __shfl_sync(0xffffffffu, b, src & 31);
  *cnt = src < 0 ? 0 : __shfl_sync(0xffffffffu, c, src & 31);
  *above = __shfl_sync(0xffffffffu, ab, src & 31);
}

// State of a radix selection of the `want` largest keys: keys above thr are in, and the first
// need_eq (lowest blocks) of those equal to it.
struct Radix {
  unsigned long long thr, range;
  int want, need_eq;
  __device__ __forceinline__ int shift() const {
    return max(0, 56 - __clzll(static_cast<long long>(range)));
  }
  __device__ __forceinline__ void all(unsigned long long lo, unsigned long long hi) {
    thr = lo;
    range = hi - lo;
  }
  // The search begins in the four binades below a positive largest score, where the largest keys
  // nearly always are: bins over all keys would be as wide as sixteen binades and put most of the
  // keys into a few of them. all() starts again where that range holds too few.
  __device__ __forceinline__ void start(unsigned long long lo, unsigned long long hi) {
    all(lo, hi);
    if (hi > 0x8000000000000000ull) {
      const double top = __longlong_as_double(static_cast<long long>(hi ^ 0x8000000000000000ull));
      const unsigned long long from = order_key64(top * 0.0625);
      if (from > lo && from < hi) all(from, hi);
    }
  }
  // Narrows to the picked bin; true when the selection is settled.
  __device__ __forceinline__ bool narrow(int bin, int cnt, int above) {
    const int sh = shift();
    const unsigned long long step = static_cast<unsigned long long>(bin) << sh;
    want -= above;
    thr += step;
    if (cnt == want) { need_eq = 0x7fffffff; return true; }  // the whole bin
    if (sh == 0) { need_eq = want; return true; }            // one key value
    range = min(range - step, (1ull << sh) - 1);
    return false;
  }
};

template <int D, int RR>
__global__ void __launch_bounds__(kGateThreads, 2) paged_gate_kernel(const PagedArgs A, int kRows,
                                                                  int KT, int in_smem) {
  constexpr int NV = D / 32;  // 16-byte pieces of a sum per lane (eight lanes have a block)
  constexpr int U = RR >= 8 ? 1 : RR >= 4 || D == 128 ? 2 : 4;  // blocks in flight per eight lanes
  extern __shared__ __align__(1024) uint8_t smem[];
  unsigned long long* skeys = reinterpret_cast<unsigned long long*>(smem);  // [RR][nb_cap]
  __shared__ double qd[RR][D];
  __shared__ int hist[kGateWarps][256];
  __shared__ unsigned int bits[2][kGateWords];
  __shared__ int sbad, scan[kGateWarps], stot;
  __shared__ unsigned long long slo[kGateWarps], shi[kGateWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int seg = blockIdx.x / CS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  allow_next_kernel();
  wait_previous_kernel();
  auto sync_all = [&]() {  // the segment's CTAs
    if (CS > 1) cluster.sync(); else __syncthreads();
  };
  const Seg id = seg_of(A, seg);
  const int R = A.rows * A.group, row0 = id.rt * kRows;
  const int nrow = min(kRows, R - row0);  // rows of this tile (<= RR)
  const int32_t* pages = A.page_table + static_cast<size_t>(id.s) * A.max_pages;
  bool over;
  const int L = seq_len(A, id.s, &over);
  // eight lanes per block: this group's blocks are first, first + stride, ...
  const int first = (rank * kGateWarps + warp) * 4 + (lane >> 3), stride = CS * kGateWarps * 4;
  auto page_of = [&](int j) {
    return j < A.nb_cap ? pages[(static_cast<long long>(j) * A.B) >> A.page_log] : -1;
  };
  int pid[U];
#pragma unroll
  for (int u = 0; u < U; ++u) pid[u] = A.topk > 1 ? page_of(first + u * stride) : -1;
  for (int r = warp; r < RR; r += kGateWarps) {  // q as fp64
    const int rr = row0 + r;
    const __nv_bfloat16* src =
        A.q + ((static_cast<size_t>(id.s) * A.rows + rr / A.group) * A.Hq +
               static_cast<size_t>(id.g) * A.group + rr % A.group) * D;
#pragma unroll
    for (int x = lane; x < D; x += 32)
      qd[r][x] = r < nrow ? static_cast<double>(__bfloat162float(src[x])) : 0.;
  }
  const int last = L > 0 ? (L - 1) / A.B : -1;  // current block of the newest row
  unsigned long long* keys =
      in_smem ? skeys : A.keys + static_cast<size_t>(seg) * min(kRows, R) * A.nb_cap;
  unsigned int* marks = in_smem ? reinterpret_cast<unsigned int*>(skeys + RR * A.nb_cap)
                                : A.marks + static_cast<size_t>(seg) * A.nb_cap;
  if (tid == 0) sbad = 0;
  if (RR > 1)
    for (int j = rank * kGateThreads + tid; j <= last; j += CS * kGateThreads) marks[j] = 0;
  const bool scored = A.topk > 1 && A.topk - 1 < last;
  if (scored) {
    __syncthreads();
    const int l8 = lane & 7;
    // the warp's four blocks are neighbours: all its lanes leave the loop together
    for (int j0 = first; j0 - (lane >> 3) < last; j0 += U * stride) {
      float4 c[U][NV];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = j0 + u * stride < last, ok = pid[u] >= 0 && pid[u] < A.num_pages;
        const float4* src = reinterpret_cast<const float4*>(
            A.sums + (static_cast<size_t>(ok ? pid[u] : 0) * A.G + id.g) * D);
#pragma unroll
        for (int x = 0; x < NV; ++x)
          c[u][x] = in && ok ? src[l8 + 8 * x] : make_float4(0.f, 0.f, 0.f, 0.f);
        if (in && !ok) sbad = 1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) pid[u] = page_of(j0 + (U + u) * stride);
      // all of the round's chains side by side (an fp64 step takes tens of clocks); blocks behind
      // the last are computed and dropped
      double v[U][RR];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < RR; ++r) v[u][r] = 0.;
#pragma unroll
      for (int x = 0; x < NV; ++x)
#pragma unroll
        for (int r = 0; r < RR; ++r) {
          const double2* qp = reinterpret_cast<const double2*>(&qd[r][(l8 + 8 * x) * 4]);
          const double2 a = qp[0], b = qp[1];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            v[u][r] = fma(a.x, static_cast<double>(c[u][x].x), v[u][r]);
            v[u][r] = fma(a.y, static_cast<double>(c[u][x].y), v[u][r]);
            v[u][r] = fma(b.x, static_cast<double>(c[u][x].z), v[u][r]);
            v[u][r] = fma(b.y, static_cast<double>(c[u][x].w), v[u][r]);
          }
        }
#pragma unroll
      for (int u = 0; u < U; ++u) reduce_rows8<RR>(v[u], lane);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * stride;
        if (j < last) {
          if constexpr (RR >= 8) {
#pragma unroll
            for (int i = 0; i < RR / 8; ++i) {
              const int r = l8 * (RR / 8) + i;
              if (r < nrow) keys[static_cast<size_t>(r) * A.nb_cap + j] = order_key64(v[u][i]);
            }
          } else {
            const int r = l8 / (8 / RR);
            if (l8 % (8 / RR) == 0 && r < nrow)
              keys[static_cast<size_t>(r) * A.nb_cap + j] = order_key64(v[u][0]);
          }
        }
      }
    }
  }
  sync_all();

  // ---- selection. select(row, where) writes its results through these.
  int2* ent = A.entries + static_cast<size_t>(seg) * A.ent_cap;
  auto place = [&](int r, int* pos_block) -> int32_t* {  // row's output, and its current block
    const int rr = row0 + r, tok = rr / A.group, h = id.g * A.group + rr % A.group;
    const int pos = L - A.rows + tok;
    *pos_block = pos >= 0 && !over ? pos / A.B : -1;
    return A.idx ? A.idx + (static_cast<size_t>(h) * A.nseq * A.rows +
                            static_cast<size_t>(id.s) * A.rows + tok) * A.topk
                 : nullptr;
  };
  auto take = [&](int32_t* out, int r, int at, int j) {
    if (out) out[at] = j;
    if (RR > 1) atomicOr(marks + j, 1u << r);
    else ent[at] = make_int2(j, 1);
  };
  if (last <= 32) {
    // row r by warp r / CS of rank r % CS, a block per lane, ranked by its score. (Its own code, as
    // short as it gets: at one pass through it, fetching instructions is what takes the time.)
    for (int r = rank + CS * warp; r < nrow; r += CS * kGateWarps) {
      int i;
      int32_t* out = place(r, &i);
      const int want = min(A.topk - 1, max(i, 0));
      int before = 0;  // blocks selected before this lane's
      if (want > 0 && want < i) {
        const unsigned long long k =
            lane < i ? keys[static_cast<size_t>(r) * A.nb_cap + lane] : 0ull;
#pragma unroll 4
        for (int x = 0; x < i; ++x) {
          const unsigned long long other = __shfl_sync(0xffffffffu, k, x);
          before += other > k || (other == k && x < lane);
        }
      }
      const bool sel = lane < i && before < want;
      const unsigned sels = __ballot_sync(0xffffffffu, sel);
      if (sel) take(out, r, __popc(sels & ((1u << lane) - 1)), lane);
      if (i >= 0 && lane == 0) take(out, r, want, i);
      if (out)
        for (int x = (i >= 0 ? want + 1 : 0) + lane; x < A.topk; x += 32) out[x] = -1;
      if (RR == 1 && lane == 0) stot = i >= 0 ? want + 1 : 0;
    }
  } else if (last <= 32 * kGateInRegs) {
    // row r by warp r / CS of rank r % CS
    for (int r = rank + CS * warp; r < nrow; r += CS * kGateWarps) {
      int i;
      int32_t* out = place(r, &i);
      const int want = min(A.topk - 1, max(i, 0));
      unsigned long long kk[kGateInRegs];
      Radix S{0ull, 0ull, want, want};
      if (want > 0 && want < i) {
        const unsigned long long* kr = keys + static_cast<size_t>(r) * A.nb_cap;
#pragma unroll
        for (int x = 0; x < kGateInRegs; ++x)
          kk[x] = x * 32 + lane < i ? kr[x * 32 + lane] : 0ull;
        unsigned long long lo = ~0ull, hi = 0;
#pragma unroll
        for (int x = 0; x < kGateInRegs; ++x)
          if (x * 32 + lane < i) {
            lo = min(lo, kk[x]);
            hi = max(hi, kk[x]);
          }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
          hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        S.start(lo, hi);
        if (S.range)
          while (true) {
            const int sh = S.shift();
#pragma unroll
            for (int x = 0; x < 8; ++x) hist[warp][x * 32 + lane] = 0;
            __syncwarp();
#pragma unroll
            for (int x = 0; x < kGateInRegs; ++x) {
              const unsigned long long d = kk[x] - S.thr;  // wraps above range for lower keys
              if (x * 32 + lane < i && d <= S.range)
                atomicAdd(&hist[warp][static_cast<int>(d >> sh)], 1);
            }
            __syncwarp();
            int bin, cnt, above;
            pick_bin(hist[warp], S.want, lane, &bin, &cnt, &above);
            if (cnt == 0) S.all(lo, hi);
            else if (S.narrow(bin, cnt, above)) break;
            __syncwarp();
          }
      }
      int at = 0, eq = 0;
      if (want > 0) {
#pragma unroll
        for (int x = 0; x < kGateInRegs; ++x) {
          const int j = x * 32 + lane;
          if (x * 32 >= i) break;
          bool sel = j < i && (want == i || kk[x] > S.thr);
          if (want < i) {
            const bool same = j < i && kk[x] == S.thr;
            const unsigned eqs = __ballot_sync(0xffffffffu, same);
            if (same) sel = eq + __popc(eqs & ((1u << lane) - 1)) < S.need_eq;
            eq += __popc(eqs);
          }
          const unsigned sels = __ballot_sync(0xffffffffu, sel);
          if (sel) take(out, r, at + __popc(sels & ((1u << lane) - 1)), j);
          at += __popc(sels);
        }
      }
      if (i >= 0 && lane == 0) take(out, r, want, i);
      if (out)
        for (int x = (i >= 0 ? want + 1 : 0) + lane; x < A.topk; x += 32) out[x] = -1;
      if (RR == 1 && lane == 0) stot = i >= 0 ? want + 1 : 0;
    }
  } else {
    for (int r = rank; r < nrow; r += CS) {  // uniform over the CTA
      int i;
      int32_t* out = place(r, &i);
      const int want = min(A.topk - 1, max(i, 0));
      if (want > 0) {  // want < i here: i is near `last`, far above the largest topk
        const unsigned long long* kr = keys + static_cast<size_t>(r) * A.nb_cap;
        const bool in_regs = i <= kGateThreads * kGateInRegs;
        unsigned long long kk[kGateInRegs];
        if (in_regs) {
#pragma unroll
          for (int x = 0; x < kGateInRegs; ++x)
            kk[x] = x * kGateThreads + tid < i ? kr[x * kGateThreads + tid] : 0ull;
        }
        // f(j, key) for this thread's blocks tid, tid + 256, ...
        auto each = [&](auto f) {
          if (in_regs) {
#pragma unroll
            for (int x = 0; x < kGateInRegs; ++x)
              if (x * kGateThreads + tid < i) f(x * kGateThreads + tid, kk[x]);
          } else {
#pragma unroll 8
            for (int j = tid; j < i; j += kGateThreads) f(j, kr[j]);
          }
        };
        unsigned long long lo = ~0ull, hi = 0;
        each([&](int, unsigned long long k) {
          lo = min(lo, k);
          hi = max(hi, k);
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
          hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        if (lane == 0) {
          slo[warp] = lo;
          shi[warp] = hi;
        }
        hist[0][tid] = 0;
        __syncthreads();
        for (int w = 0; w < kGateWarps; ++w) {
          lo = min(lo, slo[w]);
          hi = max(hi, shi[w]);
        }
        Radix S{0ull, 0ull, want, want};
        S.start(lo, hi);
        if (S.range)
          while (true) {
            const int sh = S.shift();
            each([&](int, unsigned long long k) {
              const unsigned long long d = k - S.thr;  // wraps above range for lower keys
              if (d <= S.range) atomicAdd(&hist[0][static_cast<int>(d >> sh)], 1);
            });
            __syncthreads();
            int bin, cnt, above;
            pick_bin(hist[0], S.want, lane, &bin, &cnt, &above);  // every warp alike
            __syncthreads();
            if (cnt == 0) S.all(lo, hi);
            else if (S.narrow(bin, cnt, above)) break;
            hist[0][tid] = 0;
            __syncthreads();
          }
        // selected blocks as bits, 32 blocks to a word
        const bool all_eq = S.need_eq == 0x7fffffff;
        for (int x = tid; x < 2 * kGateWords; x += kGateThreads) (&bits[0][0])[x] = 0;
        __syncthreads();
        each([&](int j, unsigned long long k) {
          if (k > S.thr || (all_eq && k == S.thr)) atomicOr(&bits[0][j >> 5], 1u << (j & 31));
          else if (k == S.thr) atomicOr(&bits[1][j >> 5], 1u << (j & 31));
        });
        __syncthreads();
        if (!all_eq && tid == 0) {  // several blocks of the border's score: the lowest ones
          int left = S.need_eq;
          for (int w = 0; left > 0; ++w) {
            unsigned e = bits[1][w];
            while (e && left > 0) {
              bits[0][w] |= e & (0u - e);
              e &= e - 1;
              --left;
            }
          }
        }
        __syncthreads();
        // thread t emits words 4t .. 4t + 3
        int mine = 0;
#pragma unroll
        for (int w = 0; w < kGateWords / kGateThreads; ++w)
          mine += __popc(bits[0][tid * (kGateWords / kGateThreads) + w]);
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        int at = incl - mine;
        for (int w = 0; w < warp; ++w) at += scan[w];
#pragma unroll
        for (int w = 0; w < kGateWords / kGateThreads; ++w) {
          const int word = tid * (kGateWords / kGateThreads) + w;
          for (unsigned e = bits[0][word]; e; e &= e - 1) take(out, r, at++, word * 32 + __ffs(e) - 1);
        }
      }
      if (i >= 0 && tid == 0) take(out, r, want, i);
      if (out)
        for (int x = (i >= 0 ? want + 1 : 0) + tid; x < A.topk; x += kGateThreads) out[x] = -1;
      if (RR == 1 && tid == 0) stot = i >= 0 ? want + 1 : 0;
      __syncthreads();  // shared arrays before the next row
    }
  }
  if (RR > 1) sync_all();      // all rows' marks
  else __syncthreads();        // stot (rank 0 has the one row)
  if (rank == 0) {  // the blocks that a row selected, ascending
    const int few = last < 32 * kGateInRegs;  // one warp lists them, without barriers
    int total = 0, has_last = 0;
    if (RR == 1) {
      total = last >= 0 ? stot : 0;
      has_last = total > 0;  // the one row is the newest
    } else if (few) {
      if (warp > 0) total = -1;  // not this warp's
      for (int j0 = 0; j0 <= last && warp == 0; j0 += 32) {
        const unsigned int mk = j0 + lane <= last ? marks[j0 + lane] : 0u;
        const unsigned b = __ballot_sync(0xffffffffu, mk != 0);
        if (mk)
          ent[total + __popc(b & ((1u << lane) - 1))] = make_int2(j0 + lane, static_cast<int>(mk));
        total += __popc(b);
        if (last < j0 + 32) has_last = (b >> (last - j0)) & 1;
      }
    } else {
      for (int j0 = 0; j0 <= last; j0 += kGateThreads) {
        const int j = j0 + tid;
        const unsigned int mk = j <= last ? marks[j] : 0u;
        const unsigned b = __ballot_sync(0xffffffffu, mk != 0);
        if (lane == 0) scan[warp] = __popc(b);
        if (j == last) stot = mk != 0;
        __syncthreads();
        int before = total;
#pragma unroll
        for (int w = 0; w < kGateWarps; ++w) {
          before += w < warp ? scan[w] : 0;
          total += scan[w];
        }
        if (mk) ent[before + __popc(b & ((1u << lane) - 1))] = make_int2(j, static_cast<int>(mk));
        __syncthreads();
      }
      has_last = stot;
    }
    if (tid == 0) {
      bool bad = over || sbad != 0;
      for (int r = 1; r < CS; ++r) bad |= *cluster.map_shared_rank(&sbad, r) != 0;
      const int tail = L - max(last, 0) * A.B;
      A.seg_tiles[seg] = bad ? -1
                             : (total - has_last) * A.tiles_per_block +
                                   (has_last ? (tail + KT - 1) / KT : 0);
    }
  }
  if (CS > 1) cluster.sync();  // peers' flags stay until rank 0 has read them
}

// -------------------------------------------------------------------------------------- host
PagedArgs args_of(const PagedLaunch& L) {
  PagedArgs A{};
  const PagedCache& P = L.cache;
  A.q = static_cast<const __nv_bfloat16*>(L.q);
  A.k = static_cast<const uint8_t*>(P.k);
  A.v = static_cast<const uint8_t*>(P.v);
  A.ks = P.k_scale; A.vs = P.v_scale; A.sums = P.sums;
  A.page_table = P.page_table; A.seq_lens = P.seq_lens;
  A.nseq = P.nseq; A.max_pages = P.max_pages; A.num_pages = P.num_pages;
  A.page_log = P.page_log; A.G = P.G; A.B = P.B;
  A.rows = L.rows; A.Hq = L.Hq; A.group = L.Hq / P.G;
  A.nrt = L.shape.nrt; A.nseg = L.shape.nseg;
  A.topk = L.topk; A.nb_cap = L.shape.nb_cap; A.ent_cap = L.shape.ent_cap;
  const int kt = tile_bytes(P.fp8) / (P.d * (P.fp8 ? 1 : 2));
  A.tiles_per_block = L.topk ? (P.B + kt - 1) / kt : 0;
  A.join = L.shape.join;
  A.scale_log2 = L.scale * 1.4426950408889634f;
  A.seg_desc = reinterpret_cast<int2*>(L.seg_desc);
  A.part_o = L.part_o; A.part_ml = reinterpret_cast<float2*>(L.part_ml);
  A.seg_tiles = L.seg_tiles; A.entries = reinterpret_cast<int2*>(L.entries);
  A.keys = L.keys; A.marks = L.marks;
  A.idx = L.idx;
  A.o = static_cast<__nv_bfloat16*>(L.o);
  A.lse = L.lse;
  return A;
}

// Launch attributes are set once per device and kernel (a driver call that a decode step of a few
// microseconds would notice).
template <class K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<int> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_relaxed) >= bytes)
    return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(bytes, std::memory_order_relaxed);
  return e;
}

template <int D, bool FP8, int NT, bool SPARSE>
cudaError_t attn(const PagedArgs& A, const PagedLaunch& L, cudaStream_t s) {
  static std::atomic<int> done[64];
  constexpr int smem = Tile<D, FP8>::kWarps * Tile<D, FP8>::kWarpBytes;
  cudaError_t e = allow_smem(paged_attn_kernel<D, FP8, NT, SPARSE>, smem, done);
  if (e != cudaSuccess) return e;
  return launch_early(paged_attn_kernel<D, FP8, NT, SPARSE>,
                      dim3(static_cast<unsigned>(A.join ? A.nseg * A.join : L.shape.ctas)),
                      Tile<D, FP8>::kThreads, smem, A.join ? A.join : 1, s, A);
}

template <int D, int RR>
cudaError_t gate(const PagedArgs& A, const PagedLaunch& L, cudaStream_t s) {
  static std::atomic<int> done[64];
  const int in_smem = !L.shape.gate_global;
  const size_t smem = in_smem ? static_cast<size_t>(A.nb_cap) * (RR * 8 + 4) : 0;
  cudaError_t e = allow_smem(paged_gate_kernel<D, RR>, kGateSmem, done);
  if (e != cudaSuccess) return e;
  const int kt = tile_bytes(L.cache.fp8) / (D * (L.cache.fp8 ? 1 : 2));
  return launch_early(paged_gate_kernel<D, RR>,
                      dim3(static_cast<unsigned>(A.nseg) * L.shape.gate_ctas), kGateThreads, smem,
                      L.shape.gate_ctas, s, A, L.shape.rows_per_tile, kt, in_smem);
}

template <int D>
cudaError_t merge(const PagedArgs& A, const PagedLaunch& L, cudaStream_t s) {
  // Warps for the partials that a segment has on average, eight to a warp. More would only fill the
  // SMs with rows that wait: 25 sequences of 4 rows, 16 heads, took 11 us longer with eight.
  const long long partials =
      static_cast<long long>(L.shape.ctas) * paged_warps(L.cache.fp8) / A.nseg + 2;
  int warps = 1;
  while (warps < kMergeWarps && warps * kMergeBatch < partials) warps *= 2;
  return launch_early(paged_merge_kernel<D>,
                      dim3(static_cast<unsigned>(A.nseq) * A.rows * A.Hq), 32 * warps, 0, 1, s, A,
                      L.shape.rows_per_tile, L.topk > 0);
}

}  // namespace

PagedShape paged_shape(const PagedCache& P, int rows, int Hq, int topk, int sms) {
  PagedShape S{};
  const int R = rows * (Hq / P.G);
  S.rows_per_tile = R <= 8 ? 8 : 16;
  S.nrt = (R + S.rows_per_tile - 1) / S.rows_per_tile;
  S.gate_rows = std::min(R, S.rows_per_tile);
  S.nseg = static_cast<long long>(P.nseq) * P.G * S.nrt;
  const int kt = tile_bytes(P.fp8) / (P.d * (P.fp8 ? 1 : 2));
  const int warps = paged_warps(P.fp8);
  const long long cap = static_cast<long long>(P.max_pages) << P.page_log;
  const long long tiles = S.nseg * ((cap + kt - 1) / kt);
  S.ctas = static_cast<int>(std::min<long long>(sms, (tiles + warps - 1) / warps));
  S.slots = 2ll * S.ctas * warps;
  long long seg_tiles = (cap + kt - 1) / kt;  // of a segment at most
  if (topk) {
    S.nb_cap = static_cast<int>((cap + P.B - 1) / P.B);
    S.ent_cap = static_cast<int>(std::min<long long>(
        S.nb_cap, static_cast<long long>(std::min(R, S.rows_per_tile)) * topk));
    S.gate_ctas = 1;
    // A CTA scores 32 blocks at a time. More CTAs per segment while they nearly all run at once: two
    // fit an SM, 30 clusters of 8 the measured GPU (1024 blocks, 31 or 32 segments: one row 24-26 us of
    // a call with 8 CTAs, 22 with 4, 4 rows 45 : 43, 16 rows 113 : 119). Keys and marks of a single
    // CTA stay in its shared memory where they fit.
    while (S.gate_ctas < 8 && S.nb_cap > 64 * S.gate_ctas &&
           S.nseg * S.gate_ctas * 2 <= 256)  // up to 32 clusters of 8, 64 of 4
      S.gate_ctas *= 2;
    seg_tiles = std::min(seg_tiles, static_cast<long long>(S.ent_cap) * ((P.B + kt - 1) / kt));
    S.gate_global = S.gate_ctas > 1 ||
                    static_cast<long long>(S.nb_cap) * (S.gate_rows * 16 + 4) > kGateSmem;
  }
  // Few and short segments: a cluster has each to itself and joins it in its own memory, one launch
  // instead of two. Only while all clusters run at once, and while a warp then has little more to do
  // than with the tiles spread over every SM: a bf16 tile takes a warp about 1 us, the merge kernel
  // 3; e4m3 tiles take longer and their 8 warps make more partials, so its margin is smaller and its
  // clusters at most two. Measured, d = 128, 32 / 8 heads, joined against spread and merged:
  // 16 x 500 tokens 10.4 us : 16 (either type), 1 x 4000 bf16 12.3 : 12.9, 1 x 8000 bf16 (4.4 tiles
  // more per warp) 16.1 : 14.9, 4 x 1000 e4m3 (1.1 more) 12.5 : 12.0.
  // At once means 14 clusters of 8, 32 of 4 or 72 of 2: a cluster lies within one of the GPU's groups
  // of SMs, whose sizes vary; the measured GPU runs 15, 33 and 74, and one cluster more waits for a
  // whole other to end (2100 tokens, 15 segments joined by 8 CTAs each 11.1 us, 16 segments 20.7, 16
  // spread and merged 12.1).
  // Over 1-64 sequences of 100-16000 tokens, 32 / 8, 8 / 1 and 4 / 1 heads of 128, 16 / 16 and 8 / 2 of
  // 64 (one row a sequence, tables as wide as the sequences) the path taken is within 5 % of the
  // better of the two in 302 of 336 cases over bf16 caches and in 269 of 336 over e4m3. The worst are
  // 15 x 2000 bf16 at 32 / 8 heads, 29.8 us spread where a join takes 25.0, and 15 x 1000 e4m3,
  // 19.2 : 13.1; e4m3 sequences of 250 (d = 64: 500) tokens take 10.6 us where a join takes 8.7.
  // The plan takes the table's width for the lengths: short sequences behind a wide table are spread
  // and merged.
  if (S.nseg <= sms) {
    const int most = join_most(P.fp8);
    const double margin = P.fp8 ? 0.75 : 3.0;
    auto at_once = [](int c) { return c == 2 ? 72 : c == 4 ? 32 : 14; };
    int cs = 1;
    while (cs < most && S.nseg <= at_once(2 * cs) &&
           seg_tiles > static_cast<long long>(cs) * warps)
      cs *= 2;
    const double joined = static_cast<double>(seg_tiles) / (cs * warps);
    const double spread = static_cast<double>(seg_tiles) * S.nseg / (sms * warps);
    if (joined <= spread + margin) S.join = cs;
  }
  return S;
}

cudaError_t launch_paged_gate(const PagedLaunch& L, cudaStream_t s) {
  const PagedArgs A = args_of(L);
  const int R = L.shape.gate_rows;
#define MOBA_GATE(D)                                     \
  return R <= 1   ? gate<D, 1>(A, L, s)                  \
         : R <= 2 ? gate<D, 2>(A, L, s)                  \
         : R <= 4 ? gate<D, 4>(A, L, s)                  \
         : R <= 8 ? gate<D, 8>(A, L, s) : gate<D, 16>(A, L, s)
  if (L.cache.d == 64) MOBA_GATE(64);
  MOBA_GATE(128);
#undef MOBA_GATE
}

cudaError_t launch_paged_attn(const PagedLaunch& L, cudaStream_t s) {
  const PagedArgs A = args_of(L);
  const bool two = L.shape.rows_per_tile == 16, sparse = L.topk > 0;
#define MOBA_ATTN(D, F)                                                              \
  return two ? (sparse ? attn<D, F, 2, true>(A, L, s) : attn<D, F, 2, false>(A, L, s)) \
             : (sparse ? attn<D, F, 1, true>(A, L, s) : attn<D, F, 1, false>(A, L, s))
  if (L.cache.d == 64) {
    if (L.cache.fp8) MOBA_ATTN(64, true);
    MOBA_ATTN(64, false);
  }
  if (L.cache.fp8) MOBA_ATTN(128, true);
  MOBA_ATTN(128, false);
#undef MOBA_ATTN
}

cudaError_t launch_paged_merge(const PagedLaunch& L, cudaStream_t s) {
  const PagedArgs A = args_of(L);
  return L.cache.d == 64 ? merge<64>(A, L, s) : merge<128>(A, L, s);
}

}  // namespace moba

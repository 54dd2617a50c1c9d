// Paged decode attention, the streaming part: every (sequence, kv head) with
// its own rows (and, where the prefix is not worth a launch of its own, the
// prefix rows in front of them).
//
// Work is cut by tiles of 64 rows, not by sequences: the tiles of all units
// (sequence, kv head) stand in one line, CTA c of n takes those from
// c * total / n on, and a unit that spans CTAs is joined by the merge kernel
// from one partial state per (CTA, unit).  A ragged batch thus loads every SM
// alike, whatever its lengths.  A CTA's tile range is found from a scan of
// the lengths, which every CTA does for itself.
//
// One warp copies: lane i looks up the pages of the CTA's i-th next tile, so
// that the table's latency is paid once per 32 tiles, and issues that tile's
// copies, a lane a copy (codes by TMA with the swizzle of the row length, metadata
// and the unit's query rows by bulk copies), when its stage is free.  Four
// warps compute, 16 rows of a tile each, with the arithmetic of
// the contiguous cache's decode (decode_tc.cuh): transposed products on
// mma.sync m16n8k16 with 16 rows of keys or channels of values on the wide
// side and the heads on the narrow one (Columns), keys
// as exact codes with one fp32 accumulator per 32 channels.
// A page holds whole 16-row blocks, so a block is on one page: a bad page id
// takes its blocks out.
//
// Bound by instruction issue for packed rows: 33 ragged sequences up to 16K of 8
// kv heads of 64, 8-bit pages of 16 rows, 288 MB in 88 us (48% of the measured
// copy rate; issue 57% active, ALU pipe 50%), of which the copies of 1 KB and 64
// bytes without any product take four fifths (metadata in 16-byte pieces by the
// copying lanes: the same here, 2 us more on pages of 64); codes converted to
// fp16 integers took 90.  120 sequences of five heads a kv
// head, 4-bit, 71 MB in 53 us, where a second column tile for heads 5 to 8 took
// 81.  For fp16 rows by the latency of short runs (67 MB in 21 us).  The same
// products on tcgen05.mma (rows of the cache on the 128-row side, unpacked to
// shared memory by their own warps) were right and slower, 186 and 178 us: every
// role is long straight code run by one warp per scheduler, and instructions
// did not arrive in time.
#pragma once

#include "decode_tc.cuh"
#include "paged.cuh"

namespace kvq {

constexpr int kPartPad = 4;   // partial row: D accumulators, max, sum, 2 pad

// Tiles of 64 rows of a part of `len` rows behind `cols` page-table entries (its length cut to them).
struct Part {
  int len, tiles;
};
__device__ __forceinline__ Part part_of(int len, int cols, int page_log2, int* status) {
  long long room = (long long)cols << page_log2;
  Part p;
  p.len = max(len, 0);
  if (p.len > room) {
    p.len = (int)room;
    if (status) set_pool_status(status, KVQ_DEV_BAD_PAGE);
  }
  p.tiles = (p.len + 63) >> 6;
  return p;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* m) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(m)) : "memory");
}
// Barrier `id` over `threads` threads of the CTA.
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// CTAs of a grid that share `total` tiles: every one of them has some.
__device__ __forceinline__ int busy_ctas(long long total, int grid) { return (int)(total < grid ? total : grid); }

// How the query heads lie in the eight columns of a product.  A 16-bit query is
// exact in fp16 (after a power of two per head); a softmax weight is not, and
// enters as fp16 part and residual where a column pair per head is free, or
// where the output's own fp16 rounding would not cover its error.
enum Columns : int {
  kPairs = 0,     // up to four heads: column 2 j the head j's fp16 part, 2 j + 1 the residual
  kSingles = 1,   // five to eight heads, bf16 output: a column each
  kTwoTiles = 2,  // five to eight heads, fp16 output: two tiles of pairs
};

template <int D, int F, int M> struct OwnShape {
  static constexpr int HT = M == kTwoTiles ? 2 : 1;          // column tiles
  static constexpr int kHeads = M == kPairs ? 4 : 8;
  static constexpr int kBits = FmtBits<F>::v;
  static constexpr int kRow = D * kBits / 8;
  static constexpr bool kAff = F != F_FP16;
  static constexpr int kNgMax = kAff ? D / 32 : 0;
  static constexpr int kCodes = 64 * kRow;
  static constexpr int kMeta = 64 * kNgMax * 4;
  static constexpr int kQ = kHeads * D * 2;
  static constexpr int kStage = (2 * kCodes + 2 * kMeta + kQ + 1023) / 1024 * 1024;
  static constexpr int kWarps = 4;                 // computing warps
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kAcc = kWarps * kHeads * (D + 8) * 4;   // the warps' states at a unit's end
  // CTAs per SM: as many as keep three stages each, four at most (registers; two or three with two
  // column tiles' accumulators)
  static constexpr int kBySmem = kStage > 24 * 1024 ? 2 : (kStage > 12 * 1024 ? 3 : 4);
  static constexpr int kCtas = HT == 1 ? kBySmem : (D == 128 ? 2 : (kBySmem > 3 ? 3 : kBySmem));
  static constexpr int kRaw = (225 * 1024 / kCtas - 4096 - kAcc) / kStage;
  static constexpr int kStages = kRaw < 2 ? 2 : (kRaw > 8 ? 8 : kRaw);
};

struct OwnArgs {
  BatchView batch;
  const void* q;
  void* out;
  float* parts;      // [grid + n_seqs * Hkv] states of [G][D + kPartPad]
  int* starts;       // [n_seqs + 1] tiles of one kv head in front of each sequence, for the merge
  int io_dtype;
  int Hq, G;
  float qscale;
  int with_prefix;   // the units' rows begin with the prefix's
  int joined;        // further states come from elsewhere: no unit is final here
  unsigned stall_tx; // test hook, as DecodeArgs
};

// Four stored bytes (u - 128 as signed bytes) as exact fp16 pairs of u - 128: byte
// b ^ 0x80 in the mantissa of 1024, less 1152.
__device__ __forceinline__ void signed_bytes(uint32_t x, __half2& lo, __half2& hi) {
  const __half2 off = u2h(0x64806480u);
  bytes_to_h2_1024(x ^ 0x80808080u, lo, hi);
  lo = __hsub2(lo, off);
  hi = __hsub2(hi, off);
}

// A code u in the low bits of an fp16 word is the subnormal number u * 2^-24, exact
// in a product; u sixteen times as large sits four bits up.
constexpr float kSubnormal = 0x1p-24f;
__device__ __forceinline__ void low_bytes(uint32_t x, __half2& lo, __half2& hi) {   // u - 128 as signed bytes
  x ^= 0x80808080u;
  lo = u2h(__byte_perm(x, 0u, 0x4140u));
  hi = u2h(__byte_perm(x, 0u, 0x4342u));
}
__device__ __forceinline__ void low_nibbles(uint32_t w, __half2 (&h)[4]) {   // as nibbles_to_h2, 16 u in h[1] and h[3]
  const uint32_t w8 = w >> 8;
  h[0] = u2h(w & 0x000F000Fu);
  h[1] = u2h(w & 0x00F000F0u);
  h[2] = u2h(w8 & 0x000F000Fu);
  h[3] = u2h(w8 & 0x00F000F0u);
}

// How codes of values enter a product.
enum ValueCodes : int {
  kDecoded = 0,   // times scale plus zero, rounded to fp16
  kSigned = 1,    // u - 8 or u - 128: half the size, where weights have no residual
  kRaw = 2,       // u * 2^-24 (4-bit: 16 u * 2^-24 on rows 8 to 15 of an m-tile)
};

// O^T += V^T . P^T for one 16-row block and every column tile, as pvt_mma
// (decode_tc.cuh): words A, B, C, E of the thread's rows 2t, 2t + 1, 2t + 8, 2t
// + 9 feed m-tiles mo on.
template <int KB, int HT, int NW, int MT, int VC>
__device__ __forceinline__ void value_products(float (&oacc)[HT][MT][4], const uint32_t (&pb)[HT][2], int mo,
                                               const uint32_t (&A)[NW], const uint32_t (&B)[NW],
                                               const uint32_t (&C)[NW], const uint32_t (&E)[NW], __half2 sAB,
                                               __half2 zAB, __half2 sCD, __half2 zCD) {
  auto both = [&](int mt, const uint32_t(&va)[4]) {
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) mma_f16(oacc[ht][mt], va, pb[ht][0], pb[ht][1]);
  };
#pragma unroll
  for (int wi = 0; wi < NW; ++wi) {
    if constexpr (KB == 16) {
      const uint32_t va[4] = {__byte_perm(A[wi], B[wi], 0x5410u), __byte_perm(A[wi], B[wi], 0x7632u),
                              __byte_perm(C[wi], E[wi], 0x5410u), __byte_perm(C[wi], E[wi], 0x7632u)};
      both(mo + wi, va);
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if constexpr (KB == 4) {
          const uint32_t sel = half ? 0x7632u : 0x5410u;
          __half2 h0[4], h1[4];   // h0[i]: channel 8 wi + 4 half + i of rows A, B
          auto unpack = [](uint32_t w, __half2(&h)[4]) {
            if constexpr (VC == kRaw) low_nibbles(w, h);
            else nibbles_to_h2<VC == kDecoded ? 0 : 8>(w, h);
          };
          unpack(__byte_perm(A[wi], B[wi], sel), h0);
          unpack(__byte_perm(C[wi], E[wi], sel), h1);
          if constexpr (VC == kDecoded) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              h0[i] = __hfma2(h0[i], sAB, zAB);
              h1[i] = __hfma2(h1[i], sCD, zCD);
            }
          }
#pragma unroll
          for (int pp = 0; pp < 2; ++pp) {
            const uint32_t va[4] = {h2u(h0[2 * pp]), h2u(h0[2 * pp + 1]), h2u(h1[2 * pp]), h2u(h1[2 * pp + 1])};
            both(mo + 4 * wi + 2 * half + pp, va);
          }
        } else {
          const uint32_t sel = half ? 0x7362u : 0x5140u;   // channels 4 wi + 2 half + 0 / 1
          __half2 l0, h0, l1, h1;
          if constexpr (VC == kRaw) {
            low_bytes(__byte_perm(A[wi], B[wi], sel), l0, h0);
            low_bytes(__byte_perm(C[wi], E[wi], sel), l1, h1);
          } else if constexpr (VC == kDecoded) {
            bytes_to_h2(__byte_perm(A[wi], B[wi], sel) ^ 0x80808080u, l0, h0);
            bytes_to_h2(__byte_perm(C[wi], E[wi], sel) ^ 0x80808080u, l1, h1);
            l0 = __hfma2(l0, sAB, zAB); h0 = __hfma2(h0, sAB, zAB);
            l1 = __hfma2(l1, sCD, zCD); h1 = __hfma2(h1, sCD, zCD);
          } else {
            signed_bytes(__byte_perm(A[wi], B[wi], sel), l0, h0);
            signed_bytes(__byte_perm(C[wi], E[wi], sel), l1, h1);
          }
          const uint32_t va[4] = {h2u(l0), h2u(h0), h2u(l1), h2u(h1)};
          both(mo + 2 * wi + half, va);
        }
      }
    }
  }
}

template <int D, int F, int M>
__global__ void __launch_bounds__(OwnShape<D, F, M>::kThreads, OwnShape<D, F, M>::kCtas)
    paged_own_kernel(const __grid_constant__ PoolView p, const __grid_constant__ OwnArgs a) {
  using S = OwnShape<D, F, M>;
  constexpr int KB = S::kBits, ROW = S::kRow, NST = S::kStages, NCW = S::kWarps;
  constexpr int KS = D / 16, NB = D / 32, MT = D / 16, VCH = D / 8, VTB = ROW / 8;
  constexpr bool AFF = S::kAff;
  constexpr int NACC = AFF ? NB : 1;
  constexpr int HT = S::HT, NS = M == kPairs ? 1 : 2;   // column tiles; heads whose state a thread holds
  // Codes of keys enter raw, those of values under one scale and zero a row raw or less kOff (zeros as z +
  // kOff * s).  Queries enter below 2^kUp, so that the smaller channels next to a subnormal code stay exact.
  constexpr int VFOLD = M == kSingles ? kSigned : kRaw, kOff = VFOLD == kRaw ? 0 : (KB == 4 ? 8 : 128);
  constexpr int kUp = AFF ? 13 : 0;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float(*sm_acc)[S::kHeads][D + 8] = reinterpret_cast<float(*)[S::kHeads][D + 8]>(smem + NST * S::kStage);
  int* sm_start = reinterpret_cast<int*>(smem + NST * S::kStage + S::kAcc);   // [n_seqs + 1]
  __shared__ __align__(8) uint64_t full[NST], empty[NST];
  __shared__ float sm_m[NCW][S::kHeads], sm_l[NCW][S::kHeads];
  __shared__ int s_bad[NST], s_issued[NST], s_scan[NCW + 1];
  __shared__ volatile int s_fail;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    s_fail = 0;
    for (int s = 0; s < NST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], NCW);
      s_issued[s] = -1;
    }
    fence_mbar_init();
  }
  // Behind the prefix kernel this one does not wait for it: that kernel let it
  // start only after its own wait, when all that came before was done, and the
  // two share nothing.  The first CTA waits at its end instead, so that the
  // merge, which waits for this grid, has both.
  if (!a.joined) grid_dependency_wait();
  grid_launch_dependents();

  // ---- tiles in front of each sequence (of one kv head)
  const int n = a.batch.n_seqs;
  const bool lead = blockIdx.x == 0;
  Part pre{0, 0};
  if (a.with_prefix) pre = part_of(a.batch.prefix_len[0], a.batch.max_prefix_pages, p.page_log2, lead ? p.status : nullptr);
  {
    const int per = (n + S::kThreads - 1) / S::kThreads;
    const int i0 = min(threadIdx.x * per, n), i1 = min(i0 + per, n);
    int sum = 0;
    for (int i = i0; i < i1; ++i)
      sum += pre.tiles + part_of(a.batch.lens[i], a.batch.max_pages, p.page_log2, lead ? p.status : nullptr).tiles;
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    int at = inc - sum;
    for (int w = 0; w < warp; ++w) at += s_scan[w];
    for (int i = i0; i < i1; ++i) {
      sm_start[i] = at;
      at += pre.tiles + part_of(a.batch.lens[i], a.batch.max_pages, p.page_log2, nullptr).tiles;
    }
    if (threadIdx.x == 0) {
      int all = 0;
      for (int w = 0; w <= NCW; ++w) all += s_scan[w];
      sm_start[n] = all;
    }
    __syncthreads();
    if (lead)
      for (int i = threadIdx.x; i <= n; i += S::kThreads) a.starts[i] = sm_start[i];
  }
  const long long total = (long long)sm_start[n] * p.Hkv;
  const int ctas = busy_ctas(total, gridDim.x);
  if (blockIdx.x >= ctas) {
    if (a.joined && lead) grid_dependency_wait();
    return;
  }
  const long long t0 = total * blockIdx.x / ctas, t1 = total * (blockIdx.x + 1) / ctas;
  const int ntile = (int)(t1 - t0);   // at least one

  // Sequence, kv head and tile of the unit that tile x of the line belongs to.
  struct At {
    int b, kvh, j, tiles;
  };
  auto locate = [&](long long x) {
    int lo = 0, hi = n;   // the last b with sm_start[b] * Hkv <= x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)sm_start[mid] * p.Hkv <= x) lo = mid;
      else hi = mid;
    }
    At r;
    r.b = lo;
    r.tiles = sm_start[lo + 1] - sm_start[lo];
    const int rest = (int)(x - (long long)sm_start[lo] * p.Hkv);
    r.kvh = rest / r.tiles;
    r.j = rest - r.kvh * r.tiles;
    return r;
  };

  const int kng = p.k.n_groups, vng = p.v.n_groups;
  if (warp == NCW) {
    // ------------------------------------------------------------- copies
    for (int base = 0; base < ntile && !s_fail; base += 32) {
      const bool mine = base + lane < ntile;
      int ids[4] = {-1, -1, -1, -1}, kvh = 0, b = 0, off = 0, np = 0;
      bool first = false;
      if (mine) {
        const At u = locate(t0 + base + lane);
        b = u.b;
        kvh = u.kvh;
        const bool in_pre = u.j < pre.tiles;
        const int j = in_pre ? u.j : u.j - pre.tiles;
        const int len = in_pre ? pre.len : part_of(a.batch.lens[b], a.batch.max_pages, p.page_log2, nullptr).len;
        const int* pages = in_pre ? a.batch.prefix_pages : a.batch.table + (size_t)b * a.batch.max_pages;
        const int rows = min(64, len - j * 64);
        np = p.page_log2 >= 6 ? 1 : (rows + (1 << p.page_log2) - 1) >> p.page_log2;
        off = (j * 64) & ((1 << p.page_log2) - 1);
        first = u.j == 0 || base + lane == 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < np) ids[i] = pages[((j * 64) >> p.page_log2) + i];
      }
      const int cnt = min(32, ntile - base);
      for (int s = 0; s < cnt; ++s) {
        const int it = base + s, stg = it % NST;
        if (it >= NST) {
          if (s_fail || !__all_sync(0xffffffffu, mbar_wait_bounded(&empty[stg], ((it / NST) - 1) & 1))) {
            s_fail = 1;
            break;
          }
        }
        // the tile's pages, a lane a copy: lane 4 i + k takes plane k of page i, lane 16 the queries
        const int n_pg = __shfl_sync(0xffffffffu, np, s), row0 = __shfl_sync(0xffffffffu, off, s);
        const int head = __shfl_sync(0xffffffffu, kvh, s), seq = __shfl_sync(0xffffffffu, b, s);
        const bool begins = __shfl_sync(0xffffffffu, first, s);
        int id = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = __shfl_sync(0xffffffffu, ids[i], s);
          if ((lane >> 2) == i && i < n_pg) id = x;
        }
        const bool ok = (unsigned)id < (unsigned)p.n_pages;
        const unsigned good = __ballot_sync(0xffffffffu, ok);          // four lanes a page
        uint8_t* st = smem + stg * S::kStage;
        const int rows = min(64, 1 << p.page_log2);   // of one copy
        const uint32_t qb = begins ? (uint32_t)(a.G * D * 2) : 0u;
        if (lane == 0) {
          int bad = 0;
          for (int i = 0; i < n_pg; ++i)
            if (!((good >> (4 * i)) & 1)) bad |= ((1 << (rows >> 4)) - 1) << (i * (rows >> 4));
          if (bad) set_pool_status(p.status, KVQ_DEV_BAD_PAGE);
          s_bad[stg] = bad;
          s_issued[stg] = (it / NST) & 1;
          mbar_expect_tx(&full[stg], (uint32_t)((__popc(good) >> 2) * rows * (2 * ROW + 4 * (kng + vng))) + qb +
                                         (it == 0 ? a.stall_tx : 0u));
        }
        __syncwarp();
        fence_async_smem();   // the stage's readers are done: order the copies behind them
        if (ok) {
          const int i = lane >> 2, k = lane & 3;
          const int row = (int)((((long long)id * p.Hkv + head) << p.page_log2) + row0);
          if (k == 0) tma_rows<ROW>(st + i * rows * ROW, &p.kmap, row, &full[stg]);
          else if (k == 1) tma_rows<ROW>(st + S::kCodes + i * rows * ROW, &p.vmap, row, &full[stg]);
          else if (AFF && k == 2)
            bulk_copy(st + 2 * S::kCodes + i * rows * 4 * kng, p.k.meta + (size_t)row * kng, (uint32_t)(rows * 4 * kng),
                      &full[stg]);
          else if (AFF)
            bulk_copy(st + 2 * S::kCodes + S::kMeta + i * rows * 4 * vng, p.v.meta + (size_t)row * vng,
                      (uint32_t)(rows * 4 * vng), &full[stg]);
        }
        if (lane == 16 && begins)
          bulk_copy(st + 2 * S::kCodes + 2 * S::kMeta,
                    static_cast<const uint16_t*>(a.q) + ((size_t)seq * a.Hq + (size_t)head * a.G) * D, qb, &full[stg]);
        __syncwarp();
      }
    }
  } else {
    // ---------------------------------------------------------- products
    const int g = lane >> 2, t = lane & 3;
    const int blk = warp * 16;
    const int rk[2] = {blk + tau<ROW>(g), blk + tau<ROW>(g + 8)};
    const int rr[4] = {blk + tau<ROW>(2 * t), blk + tau<ROW>(2 * t + 1), blk + tau<ROW>(2 * t + 8),
                       blk + tau<ROW>(2 * t + 9)};
    const int vgi = AFF ? (g * VCH) / p.v.group : 0;
    const bool vfold = AFF && vng == 1;
    // what brings the two halves of an m-tile back to size
    const float up0 = vfold && VFOLD == kRaw ? 1.0f / kSubnormal : 1.0f, up1 = KB == 4 && up0 != 1.0f ? up0 / 16 : up0;
    // the states of the thread's heads: 4 s + t in pairs, 2 t + s in singles
    float m_run[NS], l_part[NS], zacc[NS], qmul[NS];
    float oacc[HT][MT][4];
    auto head_of = [&](int s) { return M == kSingles ? 2 * t + s : 4 * s + t; };
    auto clear = [&]() {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        m_run[s] = neg_inf();
        l_part[s] = zacc[s] = 0.0f;
      }
#pragma unroll
      for (int ht = 0; ht < HT; ++ht)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) oacc[ht][mt][0] = oacc[ht][mt][1] = oacc[ht][mt][2] = oacc[ht][mt][3] = 0.0f;
    };
    clear();
    uint32_t qf[HT][KS][2];
    float qg[NS][NB];
    At u = locate(t0);
    bool first = true, begun_here = u.j == 0;
    int own_len = part_of(a.batch.lens[u.b], a.batch.max_pages, p.page_log2, nullptr).len;

    for (int it = 0; it < ntile; ++it) {
      const int stg = it % NST;
      if (s_fail || !__all_sync(0xffffffffu, mbar_wait_bounded(&full[stg], (it / NST) & 1))) s_fail = 1;
      const uint8_t* kst = smem + stg * S::kStage;
      const uint8_t* vst = kst + S::kCodes;
      const uint8_t* kmt = kst + 2 * S::kCodes;
      const uint8_t* vmt = kmt + S::kMeta;
      if (first) {
        first = false;
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
          const int hq = M == kSingles ? g : 4 * ht + (g >> 1);   // the head of column g
          const bool live = hq < a.G;
          float xq[KS][4];
          load_query_channels<D, KB>(vmt + S::kMeta, (size_t)(live ? hq : 0) * D, a.io_dtype, t, live, xq);
          // a power of two brings the head's largest magnitude under 2^kUp (bf16's range in fp16)
          float big = 0.0f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int i = 0; i < 4; ++i) big = fmaxf(big, fabsf(xq[ks][i]));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          int ex = 0;
          if (big > 0.0f && big < __int_as_float(0x7f800000)) frexpf(big, &ex);
          ex = max(min(ex, 126), kUp - 126);
          const float down = __int_as_float((127 + kUp - ex) << 23);
          const float mul = __int_as_float((127 + ex) << 23) * a.qscale;
          float qb[NB];
#pragma unroll
          for (int i = 0; i < NB; ++i) qb[i] = 0.0f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = xq[ks][i] * down;
            if constexpr (AFF) qb[ks >> 1] += (x[0] + x[1]) + (x[2] + x[3]);
            // (exact: an odd column of a pair, the queries' residual, is zero)
            const bool zero = M != kSingles && (g & 1);
            if (KB == 4 && (ks & 1))   // these channels' codes are 16 u
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] *= 0.0625f;
            qf[ht][ks][0] = zero ? 0u : h2u(__floats2half2_rn(x[0], x[1]));
            qf[ht][ks][1] = zero ? 0u : h2u(__floats2half2_rn(x[2], x[3]));
          }
          if constexpr (AFF) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              qb[i] += __shfl_xor_sync(0xffffffffu, qb[i], 1);
              qb[i] = (qb[i] + __shfl_xor_sync(0xffffffffu, qb[i], 2)) * kSubnormal;
            }
          }
          // for the thread's own heads: the sums of q over each key group, and what brings scores back to scale
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            if (M != kTwoTiles || s == ht) {
              const int from = M == kSingles ? 8 * t + 4 * s : 8 * t;
              qmul[s] = __shfl_sync(0xffffffffu, mul, from);
              if constexpr (AFF) {
#pragma unroll
                for (int i = 0; i < NB; ++i) qg[s][i] = __shfl_sync(0xffffffffu, qb[i], from);
                if (2 * kng == NB) {
#pragma unroll
                  for (int j = 0; j < NB / 2; ++j) qg[s][j] = qg[s][2 * j] + qg[s][2 * j + 1];
                } else if (kng == 1) {
#pragma unroll
                  for (int j = 1; j < NB; ++j) qg[s][0] += qg[s][j];
                }
              }
            }
          }
        }
      }
      const bool in_pre = u.j < pre.tiles;
      const int nv = in_pre ? pre.len - u.j * 64 : own_len - (u.j - pre.tiles) * 64;   // live rows of the tile
      auto block = [&](auto masked) {
        constexpr bool MASK = decltype(masked)::value;
        float acc[HT][NACC][4];
#pragma unroll
        for (int ht = 0; ht < HT; ++ht)
#pragma unroll
          for (int i = 0; i < NACC; ++i) acc[ht][i][0] = acc[ht][i][1] = acc[ht][i][2] = acc[ht][i][3] = 0.0f;
        if constexpr (KB == 4) {
#pragma unroll
          for (int pb = 0; pb < NB; ++pb) {
            __half2 h0[4], h1[4];
            low_nibbles(*reinterpret_cast<const uint32_t*>(kst + swz_off<ROW>(rk[0], 16 * pb + 4 * t)), h0);
            low_nibbles(*reinterpret_cast<const uint32_t*>(kst + swz_off<ROW>(rk[1], 16 * pb + 4 * t)), h1);
            const uint32_t ka0[4] = {h2u(h0[0]), h2u(h1[0]), h2u(h0[2]), h2u(h1[2])};
            const uint32_t ka1[4] = {h2u(h0[1]), h2u(h1[1]), h2u(h0[3]), h2u(h1[3])};
#pragma unroll
            for (int ht = 0; ht < HT; ++ht) {
              mma_f16(acc[ht][pb], ka0, qf[ht][2 * pb][0], qf[ht][2 * pb][1]);
              mma_f16(acc[ht][pb], ka1, qf[ht][2 * pb + 1][0], qf[ht][2 * pb + 1][1]);
            }
          }
        } else if constexpr (KB == 8) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            __half2 l0, h0, l1, h1;
            low_bytes(*reinterpret_cast<const uint32_t*>(kst + swz_off<ROW>(rk[0], 16 * ks + 4 * t)), l0, h0);
            low_bytes(*reinterpret_cast<const uint32_t*>(kst + swz_off<ROW>(rk[1], 16 * ks + 4 * t)), l1, h1);
            const uint32_t ka[4] = {h2u(l0), h2u(l1), h2u(h0), h2u(h1)};
#pragma unroll
            for (int ht = 0; ht < HT; ++ht) mma_f16(acc[ht][ks >> 1], ka, qf[ht][ks][0], qf[ht][ks][1]);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const uint2 v0 = *reinterpret_cast<const uint2*>(kst + swz_off<ROW>(rk[0], 32 * ks + 8 * t));
            const uint2 v1 = *reinterpret_cast<const uint2*>(kst + swz_off<ROW>(rk[1], 32 * ks + 8 * t));
            const uint32_t ka[4] = {v0.x, v1.x, v0.y, v1.y};
#pragma unroll
            for (int ht = 0; ht < HT; ++ht) mma_f16(acc[ht][0], ka, qf[ht][ks][0], qf[ht][ks][1]);
          }
        }
        // s * sum(q u) + z * sum(q) per scale group of 32, 64 or 128 channels
        bool vk[2];
        float sc[NS][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          vk[e] = !MASK || rk[e] < nv;
          [[maybe_unused]] float2 sz[NB];
          if constexpr (AFF) {
            const uint8_t* mrow = kmt + rk[e] * (4 * kng);
            uint32_t ws[4] = {0u, 0u, 0u, 0u};
            if (kng == 4) {
              const uint4 w = *reinterpret_cast<const uint4*>(mrow);
              ws[0] = w.x; ws[1] = w.y; ws[2] = w.z; ws[3] = w.w;
            } else if (kng == 2) {
              const uint2 w = *reinterpret_cast<const uint2*>(mrow);
              ws[0] = w.x; ws[1] = w.y;
            } else {
              ws[0] = *reinterpret_cast<const uint32_t*>(mrow);
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) sz[j] = __half22float2(u2h(ws[j]));
          }
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            // the head's column (a pair's second one holds nothing)
            auto got = [&](int nb) { return acc[M == kTwoTiles ? s : 0][nb][2 * e + (M == kSingles ? s : 0)]; };
            float v = 0.0f;
            if constexpr (AFF) {
              float x[NB];
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) x[nb] = got(nb);
              if (kng == 4) {
#pragma unroll
                for (int j = 0; j < NB; ++j) v = fmaf(sz[j].x, x[j], fmaf(sz[j].y, qg[s][j], v));
              } else if (kng == 2) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  v = fmaf(sz[j].x, NB == 4 ? x[2 * j] + x[2 * j + 1] : x[j], fmaf(sz[j].y, qg[s][j], v));
              } else {
#pragma unroll
                for (int j = 1; j < NB; ++j) x[0] += x[j];
                v = fmaf(sz[0].x, x[0], sz[0].y * qg[s][0]);
              }
            } else {
              v = got(0);
            }
            if constexpr (AFF) v *= 1.0f / (kSubnormal * (1 << kUp));   // (qmul alone may be near fp32's largest)
            sc[s][e] = vk[e] ? v * qmul[s] : neg_inf();
          }
        }
        // online softmax (log2); the block's first row is live
        float pr[NS][2];
        bool over = false;
#pragma unroll
        for (int s = 0; s < NS; ++s) over |= fmaxf(sc[s][0], sc[s][1]) > m_run[s];
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            float mb = fmaxf(sc[s][0], sc[s][1]);
            mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 4));
            mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 8));
            mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 16));
            const float mn = fmaxf(m_run[s], mb);
            if (mn > m_run[s]) {
              const float alpha = fast_exp2(m_run[s] - mn);
              l_part[s] *= alpha;
              zacc[s] *= alpha;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                if constexpr (M == kSingles) {
                  oacc[0][mt][s] *= alpha;
                  oacc[0][mt][2 + s] *= alpha;
                } else {
                  constexpr int kNone = 0;
                  float(&o)[4] = oacc[M == kTwoTiles ? s : kNone][mt];
                  o[0] *= alpha; o[1] *= alpha; o[2] *= alpha; o[3] *= alpha;
                }
              }
              m_run[s] = mn;
            }
          }
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const float base = m_run[s] == neg_inf() ? 0.0f : m_run[s];   // scores of -inf alone weigh nothing
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            pr[s][e] = fast_exp2(sc[s][e] - base);
            l_part[s] += pr[s][e];
          }
        }
        // Rows past the end hold whatever the page holds: weight 0, and scale and
        // zero (or fp16 values) zeroed so that no NaN reaches the products.
        bool vok[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) vok[i] = !MASK || rr[i] < nv;
        __half2 sAB = u2h(0u), zAB = u2h(0u), sCD = u2h(0u), zCD = u2h(0u);
        if constexpr (AFF) {
          const uint32_t* vm = reinterpret_cast<const uint32_t*>(vmt);
          if (vfold) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float2 sz = __half22float2(u2h(vm[rk[e]]));
              if (!vk[e]) sz = make_float2(0.0f, 0.0f);
              if constexpr (kOff != 0) sz.y = fmaf((float)kOff, sz.x, sz.y);
#pragma unroll
              for (int s = 0; s < NS; ++s) {
                zacc[s] = fmaf(pr[s][e], sz.y, zacc[s]);
                pr[s][e] *= sz.x;
              }
            }
          } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = vok[i] ? vm[rr[i] * vng + vgi] : 0u;
            sAB = u2h(__byte_perm(w[0], w[1], 0x5410u));
            zAB = u2h(__byte_perm(w[0], w[1], 0x7632u));
            sCD = u2h(__byte_perm(w[2], w[3], 0x5410u));
            zCD = u2h(__byte_perm(w[2], w[3], 0x7632u));
          }
        }
        uint32_t pb[HT][2];
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
          if constexpr (M == kSingles) {
            pb[ht][0] = movmatrix_t(h2u(__floats2half2_rn(pr[0][0], pr[1][0])));
            pb[ht][1] = movmatrix_t(h2u(__floats2half2_rn(pr[0][1], pr[1][1])));
          } else {
            const __half2 ph = __floats2half2_rn(pr[ht][0], pr[ht][1]);
            const float2 pf = __half22float2(ph);
            const __half2 pl = __floats2half2_rn(pr[ht][0] - pf.x, pr[ht][1] - pf.y);
            pb[ht][0] = movmatrix_t(h2u(__lows2half2(ph, pl)));
            pb[ht][1] = movmatrix_t(h2u(__highs2half2(ph, pl)));
          }
        }
        constexpr int NWT = VTB / 4;
        constexpr int NW = NWT > 4 ? 4 : NWT;
#pragma unroll
        for (int w0 = 0; w0 < NWT; w0 += NW) {
          if (w0 > 0) asm volatile("" ::: "memory");   // the next run's loads stay behind these products
          uint32_t A[NW], B[NW], C[NW], E[NW];
          lds_row_words<ROW, NW>(A, vst, rr[0], g * VTB + 4 * w0);
          lds_row_words<ROW, NW>(B, vst, rr[1], g * VTB + 4 * w0);
          lds_row_words<ROW, NW>(C, vst, rr[2], g * VTB + 4 * w0);
          lds_row_words<ROW, NW>(E, vst, rr[3], g * VTB + 4 * w0);
          if constexpr (KB == 16) {
            if (MASK) {
#pragma unroll
              for (int w = 0; w < NW; ++w) {
                A[w] = vok[0] ? A[w] : 0u;
                B[w] = vok[1] ? B[w] : 0u;
                C[w] = vok[2] ? C[w] : 0u;
                E[w] = vok[3] ? E[w] : 0u;
              }
            }
          }
          const int mo = w0 * (MT / NWT);
          if (AFF && !vfold) value_products<KB, HT, NW, MT, kDecoded>(oacc, pb, mo, A, B, C, E, sAB, zAB, sCD, zCD);
          else value_products<KB, HT, NW, MT, VFOLD>(oacc, pb, mo, A, B, C, E, sAB, zAB, sCD, zCD);
        }
      };
      const bool take = blk < nv && !s_fail && !((s_bad[stg] >> (warp & 3)) & 1);   // warp-uniform
      if (take) {
        if (blk + 16 <= nv) block(std::false_type{});
        else block(std::true_type{});
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stg]);

      // ---- the unit's last tile here: join the warps' states, write, start over
      const bool ends = u.j + 1 == u.tiles;
      if (ends || it + 1 == ntile) {
#pragma unroll
        for (int s = 0; s < NS; ++s) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            l_part[s] += __shfl_xor_sync(0xffffffffu, l_part[s], o);
            zacc[s] += __shfl_xor_sync(0xffffffffu, zacc[s], o);
          }
          const int head = head_of(s);
          constexpr int kNone = 0;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float(&o)[4] = oacc[M == kTwoTiles ? s : kNone][mt];
            sm_acc[warp][head][(2 * mt) * 8 + g] = fmaf(M == kSingles ? o[s] : o[0] + o[1], up0, zacc[s]);
            sm_acc[warp][head][(2 * mt + 1) * 8 + g] = fmaf(M == kSingles ? o[2 + s] : o[2] + o[3], up1, zacc[s]);
          }
          if (g == 0) {
            sm_m[warp][head] = m_run[s];
            sm_l[warp][head] = l_part[s];
          }
        }
        named_sync(1, 32 * NCW);
        const bool final = !a.joined && begun_here && ends;
        const long long unit = (long long)u.b * p.Hkv + u.kvh;
        // a warp a head: lane i holds channels D / 32 * i on
#pragma unroll 1
        for (int head = warp; head < a.G; head += NCW) {
          const int i = lane;
          float mm = neg_inf(), ll = 0.0f, w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) mm = fmaxf(mm, sm_m[k][head]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            w[k] = sm_l[k][head] == 0.0f ? 0.0f : fast_exp2(sm_m[k][head] - mm);
            ll = fmaf(sm_l[k][head], w[k], ll);
          }
          constexpr int C = D / 32;
          float o[C];
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int d = (i & 31) * C + c;
            o[c] = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (w[k] != 0.0f) o[c] = fmaf(w[k], sm_acc[k][head][(d % VCH) * 8 + d / VCH], o[c]);
          }
          if (final) {
            const float r = ll == 0.0f ? 0.0f : 1.0f / ll;
            const size_t at = ((size_t)u.b * a.Hq + (size_t)u.kvh * a.G + head) * D + (i & 31) * C;
#pragma unroll
            for (int c = 0; c < C; ++c) store_io(a.out, at + c, a.io_dtype, o[c] * r);
          } else {
            float* dst = a.parts + ((size_t)(blockIdx.x + unit) * a.G + head) * (D + kPartPad);
#pragma unroll
            for (int c = 0; c < C; ++c) dst[(i & 31) * C + c] = o[c];
            if ((i & 31) == 0) {
              dst[D] = mm;
              dst[D + 1] = ll;
            }
          }
        }
        named_sync(1, 32 * NCW);
        clear();
        first = true;
      }
      if (++u.j == u.tiles) {
        u.j = 0;
        begun_here = true;
        if (++u.kvh == p.Hkv) {
          u.kvh = 0;
          if (it + 1 < ntile) {
            do {
              ++u.b;
              u.tiles = sm_start[u.b + 1] - sm_start[u.b];
            } while (u.tiles == 0);
            own_len = part_of(a.batch.lens[u.b], a.batch.max_pages, p.page_log2, nullptr).len;
          }
        }
      }
    }
  }
  __syncthreads();
  if (s_fail && threadIdx.x == 0) {
    // a stage never arrived: say so, and wait (bounded) for the copies still in flight
    set_pool_status(p.status, KVQ_DEV_TIMEOUT);
    for (int s = 0; s < NST; ++s)
      if (s_issued[s] >= 0) mbar_wait_bounded(&full[s], s_issued[s]);
  }
  if (a.joined && lead) grid_dependency_wait();
}

}  // namespace kvq

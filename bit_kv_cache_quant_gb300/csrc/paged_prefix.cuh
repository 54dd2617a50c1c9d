// Decode attention over a prefix that a whole batch shares: the query rows of
// all sequences stand against each tile of keys, so the prefix is read,
// decoded and multiplied once for the batch.
//
// For a kv head the B * G query rows (G query heads a kv head) are the 128-row
// side of tcgen05.mma.  A CTA takes one or two such row tiles and a run of
// 128-row tiles of the prefix; runs of different CTAs are joined by the merge.
//   S = Q K^T   [128 x 128], Q and K from shared memory, fp32 in tensor memory
//   P = 2^(S c - m) as fp16, written back over S by the softmax warps
//   O += P V    P from tensor memory, V from shared memory, fp32 in tensor memory
// Warps 0-3 (and 4-7 for the second row tile) own the softmax, a thread a
// row; the next four bring keys and values into shared memory in the order the
// matrix unit wants (128-byte swizzle): fp16 pages by TMA, 8- and 4-bit pages
// decoded to fp16 on the way (one rounding of u * s + z); one thread of the last
// warp issues the products.  While one row tile is in its softmax the other's
// products run.
//
// The running maximum of a row moves only when a tile exceeds it by more than
// 2^kSlack (weights up to 2^kSlack are exact enough in fp16 and fp32), so that
// the accumulators in tensor memory are almost never rescaled.
//
// Queries enter as fp16 after a power of two per row brings the row's largest
// magnitude under one, so that bf16's range is kept; the power goes back in
// with the softmax scale.
#pragma once

#include "paged_own.cuh"

namespace kvq {

constexpr float kSlack = 8.0f;

struct PrefixArgs {
  BatchView batch;
  const void* q;
  float* part_o;     // [Hkv][nsplit][rows][D]
  float2* part_ml;   // [Hkv][nsplit][rows] (max, sum)
  int io_dtype;
  int Hq, G, rows;   // rows = n_seqs * G
  int nsplit;        // runs per (kv head, row tiles) at most
  float qscale;
};

// Runs a prefix of `tiles` tiles is cut into.
__device__ __forceinline__ int prefix_runs(int tiles, int nsplit) { return tiles < nsplit ? tiles : nsplit; }

// ------------------------------------------------------------- tensor memory --

__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* m) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(smem_u32(m))
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// 32 columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,"
      "%31,%32};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Shared-memory operand descriptor: 128-byte swizzle; strides in bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// Instruction descriptor of kind::f16: fp16 operands, fp32 accumulators, A rows along K; b_mn: B along N.
__host__ __device__ constexpr uint32_t mma_desc(int m, int n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

// 128 bytes of TMA box columns from byte x of rows y .. of a 2-d code-plane map.
__device__ __forceinline__ void tma_columns(void* dst, const CUtensorMap* map, int x, int y, uint64_t* m) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(m))
      : "memory");
}

template <int D, int F, int NQ> struct PrefixShape {
  static constexpr int kHalves = D / 64;             // 64-channel halves of a row, 128 bytes each
  static constexpr int kTile = 128 * D * 2;          // a 128-row fp16 tile
  static constexpr int kStages = 2;                  // of keys and of values
  static constexpr int kSmem = NQ * kTile + 2 * kStages * kTile + 1024;
  static constexpr int kSoft = 4 * NQ;               // softmax warps
  static constexpr int kThreads = 32 * (kSoft + 5);
  static constexpr uint32_t kCols = NQ == 2 ? 512 : 256;   // tensor memory: 128 S + 128 O per row tile
};

// Byte offset of 16-byte chunk c (of D / 8) of row r in a swizzled tile.
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  return (uint32_t)((c >> 3) * 16384 + r * 128 + (((c ^ r) & 7) << 4));
}

// Decodes 16-byte-chunk-ordered fp16 of one stored row from its raw words: chunk c
// holds channels 8 c .. 8 c + 7, for 4-bit codes in the order 0 4 1 5 2 6 3 7
// (queries are laid out, and outputs read, the same way).
template <int D, int F>
__device__ __forceinline__ void store_decoded(uint8_t* tile, int r, const uint32_t* raw, const uint32_t* meta, int ng) {
  constexpr int KB = FmtBits<F>::v;
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    uint4 o;
    if constexpr (KB == 16) {
      o = make_uint4(raw[4 * c], raw[4 * c + 1], raw[4 * c + 2], raw[4 * c + 3]);
    } else {
      // the chunk's (scale, zero): the groups of a row are 32, 64 or 128 channels
      const uint32_t m = ng == 1 ? meta[0] : (ng == D / 64 ? meta[c >> 3] : meta[c >> 2]);
      const __half2 s = u2h(__byte_perm(m, m, 0x1010u)), z = u2h(__byte_perm(m, m, 0x3232u));
      __half2 h[4];
      if constexpr (KB == 4) {
        nibbles_to_h2(raw[c], h);
      } else {
        bytes_to_h2(raw[2 * c] ^ 0x80808080u, h[0], h[1]);
        bytes_to_h2(raw[2 * c + 1] ^ 0x80808080u, h[2], h[3]);
      }
      o = make_uint4(h2u(__hfma2(h[0], s, z)), h2u(__hfma2(h[1], s, z)), h2u(__hfma2(h[2], s, z)),
                     h2u(__hfma2(h[3], s, z)));
    }
    *reinterpret_cast<uint4*>(tile + tile_off(r, c)) = o;
  }
}

template <int D, int F, int NQ>
__global__ void __launch_bounds__(PrefixShape<D, F, NQ>::kThreads, 1)
    paged_prefix_kernel(const __grid_constant__ PoolView p, const __grid_constant__ PrefixArgs a) {
  using S = PrefixShape<D, F, NQ>;
  constexpr int KB = FmtBits<F>::v, ROW = D * KB / 8, RAW = ROW / 4, NST = S::kStages;
  constexpr bool AFF = F != F_FP16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = smem;
  uint8_t* sk = smem + NQ * S::kTile;
  uint8_t* sv = sk + NST * S::kTile;
  __shared__ __align__(8) uint64_t q_full, k_full[NST], k_empty[NST], v_full[NST], v_empty[NST], s_full[NQ], p_full[NQ],
      o_full[NQ];
  __shared__ uint32_t s_tmem;
  __shared__ uint32_t s_mask[4][4];   // live rows of tile j in ring slot j & 3
  __shared__ float s_scale[NQ * 128];
  __shared__ volatile int s_fail;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kvh = blockIdx.y, row0 = blockIdx.z * (128 * NQ);
  if (threadIdx.x == 0) {
    s_fail = 0;
    mbar_init(&q_full, 128);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&k_full[i], 128);
      mbar_init(&v_full[i], 128);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
    }
    fence_mbar_init();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  const Part pre = part_of(a.batch.prefix_len[0], a.batch.max_prefix_pages, p.page_log2,
                           threadIdx.x == 0 && blockIdx.x + blockIdx.y + blockIdx.z == 0 ? p.status : nullptr);
  const int tiles = (pre.len + 127) >> 7;
  const int runs = prefix_runs(tiles, a.nsplit);
  if ((int)blockIdx.x >= runs) return;   // the whole CTA, before any tensor memory is held
  const int j0 = (int)((long long)tiles * blockIdx.x / runs), j1 = (int)((long long)tiles * (blockIdx.x + 1) / runs);
  const int n = j1 - j0;
  if (warp == S::kSoft + 4) tmem_alloc(&s_tmem, S::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // every wait is bounded; once one runs out the others return at once, the loops
  // keep their counts and the results are marked by the status word
  auto wait = [&](uint64_t* m, uint32_t parity) {
    if (!s_fail && !mbar_wait_bounded(m, parity)) s_fail = 1;
  };

  if (warp < S::kSoft) {
    // ------------------------------------------------------------- softmax
    const int t = warp >> 2;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // 32 lanes a warp, lane number from bit 16 on
    const uint32_t ts = tmem + lanes + t * 256, to = ts + 128;
    const int r = (warp & 3) * 32 + lane;
    wait(&q_full, 0);
    const float c = s_scale[t * 128 + r] * a.qscale;
    float m = neg_inf(), l = 0.0f;
    for (int j = 0; j < n; ++j) {
      wait(&s_full[t], j & 1);
      tc_fence_after();
      uint32_t live[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) live[i] = s_mask[j & 3][i];
      float top = neg_inf();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t x[32];
        tmem_ld32(x, ts + 32 * i);
        tmem_wait_ld();
        if (live[i] != 0xffffffffu) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((live[i] >> e) & 1)) x[e] = 0xff800000u;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(x[e]));
      }
      top *= c;
      const float lift = j == 0 ? 0.0f : kSlack;
      if (__any_sync(0xffffffffu, top > m + lift)) {
        const bool up = top > m + lift;
        const float mn = up ? top : m;
        const float alpha = up ? fast_exp2(m - mn) : 1.0f;
        if (j > 0) {   // (the first tile's product overwrites the accumulators)
          l *= alpha;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t x[32];
            tmem_ld32(x, to + 32 * i);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * alpha);
            tmem_st32(to + 32 * i, x);
          }
        }
        m = mn;
      }
      const float base = m == neg_inf() ? 0.0f : m;   // no live row yet: every weight is 2^-inf
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t x[32], w[16];
        tmem_ld32(x, ts + 32 * i);
        tmem_wait_ld();
        if (live[i] != 0xffffffffu) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((live[i] >> e) & 1)) x[e] = 0xff800000u;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float p0 = fast_exp2(fmaf(__uint_as_float(x[2 * e]), c, -base));
          const float p1 = fast_exp2(fmaf(__uint_as_float(x[2 * e + 1]), c, -base));
          sum += p0 + p1;
          w[e] = h2u(__floats2half2_rn(p0, p1));
        }
        tmem_st16(ts + 16 * i, w);   // over scores this thread has read
      }
      l += sum;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[t]);
    }
    wait(&o_full[t], 0);
    tc_fence_after();
    const int row = row0 + t * 128 + r;
    const bool mine = row < a.rows && !s_fail;
    const size_t at = ((size_t)kvh * a.nsplit + blockIdx.x) * a.rows + row;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t x[32];
      tmem_ld32(x, to + 32 * i);
      tmem_wait_ld();
      if (mine) {
        float* dst = a.part_o + at * D + 32 * i;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          // channels in order again: eight of a chunk sit as 0 4 1 5 2 6 3 7 for 4-bit values
          uint32_t y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = KB == 4 ? x[e + 2 * (k & 3) + (k >> 2)] : x[e + k];
          reinterpret_cast<uint4*>(dst + e)[0] = make_uint4(y[0], y[1], y[2], y[3]);
          reinterpret_cast<uint4*>(dst + e)[1] = make_uint4(y[4], y[5], y[6], y[7]);
        }
      }
    }
    if (mine) a.part_ml[at] = make_float2(m, l);
  } else if (warp < S::kSoft + 4) {
    // -------------------------------------------- queries, keys and values
    const int r = threadIdx.x - 32 * S::kSoft;   // a thread a row
    for (int t = 0; t < NQ; ++t) {
      const int row = row0 + t * 128 + r;
      uint4 w[D / 8];
      float big = 0.0f;
      const bool have = row < a.rows;
      if (have) {
        const int b = row / a.G;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(a.q) + ((size_t)b * a.Hq + (size_t)kvh * a.G + (row - b * a.G)) * D);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) w[i] = src[i];
      }
      const bool bf = a.io_dtype == KVQ_DTYPE_BF16;
      auto value = [&](int i) {   // channel i (compile-time) of the row
        const uint4 v = w[i >> 3];
        const uint32_t word = (i & 7) < 2 ? v.x : (i & 7) < 4 ? v.y : (i & 7) < 6 ? v.z : v.w;
        const uint32_t h = (i & 1) ? word >> 16 : word & 0xffffu;
        return bf ? __uint_as_float(h << 16) : __half2float(__ushort_as_half((unsigned short)h));
      };
      if (have) {
#pragma unroll
        for (int i = 0; i < D; ++i) big = fmaxf(big, fabsf(value(i)));
      }
      // a power of two at or above the largest magnitude
      int e = 0;
      if (big > 0.0f && big < __int_as_float(0x7f800000)) frexpf(big, &e);
      e = max(min(e, 126), -126);
      const float down = __int_as_float((127 - e) << 23);
      s_scale[t * 128 + r] = __int_as_float((127 + e) << 23);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        __half2 h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c0 = KB == 4 ? k : 2 * k, c1 = KB == 4 ? k + 4 : 2 * k + 1;
          h[k] = have ? __floats2half2_rn(value(8 * i + c0) * down, value(8 * i + c1) * down) : u2h(0u);
        }
        *reinterpret_cast<uint4*>(sq + t * S::kTile + tile_off(r, i)) = make_uint4(h2u(h[0]), h2u(h[1]), h2u(h[2]), h2u(h[3]));
      }
    }
    fence_async_smem();
    mbar_arrive(&q_full);

    // the page of this thread's row of tile j (-1: none)
    auto page_of = [&](int j) {
      const int tok = (j0 + j) * 128 + r;
      return j < n && tok < pre.len ? a.batch.prefix_pages[tok >> p.page_log2] : -1;
    };
    int id = page_of(0);
    for (int j = 0; j < n; ++j) {
      const int next = page_of(j + 1);
      const int tok = (j0 + j) * 128 + r;
      const bool ok = (unsigned)id < (unsigned)p.n_pages;
      if (!ok && tok < pre.len) set_pool_status(p.status, KVQ_DEV_BAD_PAGE);
      const size_t row = ok ? ((((size_t)id * p.Hkv) + kvh) << p.page_log2) + (tok & (p.page - 1)) : 0;
      const uint32_t votes = __ballot_sync(0xffffffffu, ok);
      const int stg = j % NST;
      const uint32_t par = ((j / NST) & 1) ^ 1;
      uint32_t raw[RAW], meta[4];
      // A tile of live rows of fp16 goes by TMA.  The four warps agree on it through the mask.
      auto load = [&](const PoolSide& s) {
        const uint4* src = reinterpret_cast<const uint4*>(s.codes + row * ROW);
#pragma unroll
        for (int i = 0; i < RAW / 4; ++i) {
          const uint4 v = ok ? src[i] : make_uint4(0u, 0u, 0u, 0u);
          raw[4 * i] = v.x;
          raw[4 * i + 1] = v.y;
          raw[4 * i + 2] = v.z;
          raw[4 * i + 3] = v.w;
        }
        if constexpr (AFF) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            meta[i] = ok && i < s.n_groups ? reinterpret_cast<const uint32_t*>(s.meta)[row * s.n_groups + i] : 0u;
        }
      };
      if (lane == 0) s_mask[j & 3][r >> 5] = votes;
      load(p.k);
      if (j >= NST) wait(&k_empty[stg], par);
      store_decoded<D, F>(sk + stg * S::kTile, r, raw, meta, p.k.n_groups);
      fence_async_smem();
      mbar_arrive(&k_full[stg]);
      load(p.v);
      if (j >= NST) wait(&v_empty[stg], par);
      store_decoded<D, F>(sv + stg * S::kTile, r, raw, meta, p.v.n_groups);
      fence_async_smem();
      mbar_arrive(&v_full[stg]);
      id = next;
    }
  } else if (lane == 0) {
    // ------------------------------------------------------------ products
    constexpr uint32_t kQK = mma_desc(128, 128, false), kPV = mma_desc(128, D, true);
    auto scores = [&](int t, int j) {
      const uint32_t qa = smem_u32(sq + t * S::kTile), ka = smem_u32(sk + (j % NST) * S::kTile);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
        tc_mma_ss(tmem + t * 256, operand_desc(qa + off, 16, 1024), operand_desc(ka + off, 16, 1024), kQK, k > 0);
      }
      tc_commit(&s_full[t]);
    };
    wait(&q_full, 0);
    wait(&k_full[0], 0);
    tc_fence_after();
    for (int t = 0; t < NQ; ++t) scores(t, 0);
    tc_commit(&k_empty[0]);
    for (int j = 0; j < n; ++j) {
      const int stg = j % NST;
      for (int t = 0; t < NQ; ++t) {
        wait(&p_full[t], j & 1);
        if (t == 0) wait(&v_full[stg], (j / NST) & 1);
        tc_fence_after();
        const uint32_t va = smem_u32(sv + stg * S::kTile);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc_mma_ts(tmem + t * 256 + 128, tmem + t * 256 + 8 * k, operand_desc(va + k * 2048, 16384, 1024), kPV,
                    j > 0 || k > 0);
        if (j + 1 == n) tc_commit(&o_full[t]);
        if (t + 1 == NQ) tc_commit(&v_empty[stg]);
        if (j + 1 < n) {
          if (t == 0) {
            wait(&k_full[(j + 1) % NST], ((j + 1) / NST) & 1);
            tc_fence_after();
          }
          scores(t, j + 1);
          if (t + 1 == NQ) tc_commit(&k_empty[(j + 1) % NST]);
        }
      }
    }
    // the last product is done before the tensor memory goes back
    for (int t = 0; t < NQ; ++t) mbar_wait_bounded(&o_full[t], 0);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == S::kSoft + 4) tmem_free(tmem, S::kCols);
  if (s_fail && threadIdx.x == 0) set_pool_status(p.status, KVQ_DEV_TIMEOUT);
}

}  // namespace kvq

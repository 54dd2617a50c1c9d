// Decode attention over a prefix that a whole batch shares: the query rows of
// all sequences stand against each tile of keys, so the prefix is read,
// decoded and multiplied once for the batch.
//
// For a kv head the B * G query rows (G query heads a kv head) are the 128-row
// side of tcgen05.mma.  A CTA takes one or two such row tiles and a run of
// 128-row tiles of the prefix, as two streams: with two row tiles each stream
// has its own queries and both take every tile, with one they share the
// queries and take tiles in turn.  Streams of all CTAs are joined by the merge.
//   S = Q K^T   [128 x 128], Q and K from shared memory, fp32 in tensor memory
//   P = 2^(S c - m) as fp16, written back over S by the softmax warps
//   O += P V    P from tensor memory, V from shared memory, fp32 in tensor memory
// Warps 0-3 and 4-7 own the streams' softmax, a thread a row; the next four
// bring keys and the four after them values into shared
// memory in the order the matrix unit wants (128-byte swizzle): fp16 pages by
// TMA, 8- and 4-bit pages (and tiles with rows to leave out) by a thread a row,
// decoded to fp16 on the way (one rounding of u * s + z).  A stream's first
// warp issues its products, which its warps would wait for anyway; while one
// stream is in its softmax the other's products run.  The loading warps hand
// registers to the softmax warps.
//
// The running maximum of a row moves only when a tile exceeds it by more than
// 2^kSlack (weights up to 2^kSlack are exact enough in fp16 and fp32), so that
// the accumulators in tensor memory are almost never rescaled.
//
// 64 sequences of 32 heads behind 32K rows of 8 kv heads of 128, fp16: 44 us for
// 134 MB and 34 GFLOP (30% of the measured copy rate and 40% of the measured
// bf16 rate at once; tensor pipe active 36%).  Bound by the dependent chain of a
// stream's tile (scores, 1400 cycles of softmax, weights back, products): 3000
// to 3900 cycles where the products of both streams alone are 2100.  Measured on
// the way there: keys and values by one warp group 60; an extra pass for the
// maximum and spilled scores 70; a separate issuing warp 48; operands in vector
// registers (about 100 cycles a product to issue) 53; without turns 47.
//
// Queries enter as fp16 after a power of two per row brings the row's largest
// magnitude under one, so that bf16's range is kept; the power goes back in
// with the softmax scale.
//
// What is rounded: weights to fp16 (at most 2^-11 of each), and 8- and 4-bit keys
// and values to fp16 (2^-11 of each again; a score then carries the sum of its
// channels' errors), because kind::f16 takes 16-bit operands and exact codes would
// need an accumulator per group of channels.  Measured in the 2-norm against 64
// bits: bf16 outputs 1.7e-3 for all formats (1.65e-3 is the output's own rounding),
// fp16 outputs 2.8e-4 for fp16 pages and 4.7e-4 to 6.5e-4 for 8- and 4-bit ones
// (own rounding 2.1e-4).  Keys as two fp16 parts would take half as many products
// again, in the chain that bounds the kernel.
#pragma once

#include "paged_own.cuh"

namespace kvq {

constexpr float kSlack = 8.0f;

struct PrefixArgs {
  BatchView batch;
  const void* q;
  float* part_o;     // [Hkv][nsplit * streams][rows][D]
  float2* part_ml;   // [Hkv][nsplit * streams][rows] (max, sum)
  int io_dtype;
  int Hq, G, rows;   // rows = n_seqs * G
  int nsplit;        // CTAs per (kv head, row tiles) at most
  int streams;       // states a CTA leaves per row: 1, or 2 where its streams share the rows
  float qscale;
  unsigned stall_tx; // test hook, as DecodeArgs
};

// CTAs that share a prefix of `tiles` tiles.
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
// Waits for the loads into r (and all before them); r is an operand, so that no use of it moves up past the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
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
  static constexpr int kSoft = 8;                    // softmax warps
  static constexpr int kThreads = 32 * (kSoft + 8);
  static constexpr uint32_t kCols = 512;             // tensor memory: 128 S + 128 O per stream
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
    {
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

// Registers a thread: of 16 warps with 128 each, 8 go down to 88 and 8 up to 168.
template <int N> __device__ __forceinline__ void raise_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N> __device__ __forceinline__ void lower_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// One lane of the warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
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
  __shared__ __align__(8) uint64_t q_full, k_full[NST], k_empty[NST], v_full[NST], v_empty[NST], s_full[2], o_full[2],
      issued[2];
  __shared__ uint32_t s_tmem;
  // Live rows of tile j, in ring slot j & 7.  A slot is written again when the scores of the fourth and
  // third tile before are known to be done, hence the softmax of every tile up to the fifth before.
  __shared__ uint32_t s_mask[8][4];
  __shared__ float s_scale[NQ * 128];
  __shared__ volatile int s_fail;

  // (from one lane, so that what follows from the warp's number is known to be uniform: a product's
  // operands then live in uniform registers)
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int kvh = blockIdx.y, row0 = blockIdx.z * (128 * NQ);
  if (threadIdx.x == 0) {
    s_fail = 0;
    mbar_init(&q_full, 128 * NQ);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&k_full[i], 128);
      mbar_init(&v_full[i], 128);
      mbar_init(&k_empty[i], NQ);   // streams that read the tile
      mbar_init(&v_empty[i], NQ);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&issued[i], 1);
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
  if (warp == S::kSoft + 7) tmem_alloc(&s_tmem, S::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  // every wait is bounded; once one runs out the others return at once, the loops
  // keep their counts and the results are marked by the status word
  auto wait = [&](uint64_t* m, uint32_t parity) {
    if (!s_fail && !mbar_wait_bounded(m, parity)) s_fail = 1;
  };

  if (warp < S::kSoft) {
    // ------------------------------------------------------------- softmax
    raise_registers<168>();
    const int t = warp >> 2;                       // the stream
    const int qt = NQ == 2 ? t : 0;                // its row tile
    const int mine_n = NQ == 2 ? n : (n + 1 - t) >> 1;   // its tiles
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // 32 lanes a warp, lane number from bit 16 on
    const uint32_t ts = tmem + lanes + t * 256, to = ts + 128;
    const int r = (warp & 3) * 32 + lane;
    // Products are issued by the stream's first warp, when its four warps have met.
    constexpr uint32_t kQK = mma_desc(128, 128, false), kPV = mma_desc(128, D, true);
    const uint64_t qd = operand_desc(smem_u32(sq + qt * S::kTile), 16, 1024);
    auto scores = [&](int j) {   // S = the stream's queries against keys of tile j
      const uint64_t kd = operand_desc(smem_u32(sk + (j % NST) * S::kTile), 16, 1024);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
        tc_mma_ss(tmem + t * 256, qd + off, kd + off, kQK, k > 0);
      }
      tc_commit(&s_full[t]);
      tc_commit(&k_empty[j % NST]);
    };
    auto values = [&](int j, bool add) {   // O += the weights times values of tile j
      const uint64_t vd = operand_desc(smem_u32(sv + (j % NST) * S::kTile), 16384, 1024);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        tc_mma_ts(tmem + t * 256 + 128, tmem + t * 256 + 64 + 8 * k, vd + ((k * 2048) >> 4), kPV, add || k > 0);
      tc_commit(&v_empty[j % NST]);
    };
    const bool leads = (warp & 3) == 0;
    wait(&q_full, 0);
    if (leads && mine_n > 0) {
      const int j = NQ == 2 ? 0 : t;
      wait(&k_full[j], 0);
      tc_fence_after();
      if (elect_one()) scores(j);
      __syncwarp();
    }
    const float c = fmaxf(s_scale[qt * 128 + r] * a.qscale, 0x1p-149f);   // (never 0: -inf * c stays -inf)
    float m = neg_inf(), l = 0.0f;   // the row's reference maximum (unscaled) and sum
#pragma unroll 1
    for (int k = 0; k < mine_n; ++k) {
      const int j = NQ == 2 ? k : 2 * k + t;
      wait(&s_full[t], k & 1);
      tc_fence_after();
      volatile const uint32_t* live = s_mask[j & 7];
      // Scores in quarters of 32 columns, the next one on its way while one is used.  Weights against the
      // row's reference maximum are kept back until all 128 scores have shown that it stands.
      uint32_t xa[32], xb[32];
      float t0 = neg_inf(), t1 = neg_inf();
      float2 sum = make_float2(0.0f, 0.0f);
      const float2 c2 = make_float2(c, c);
      auto mask = [&](uint32_t(&x)[32], int i) {
        const uint32_t word = live[i];
        if (word != 0xffffffffu) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((word >> e) & 1)) x[e] = 0xff800000u;
        }
      };
      auto highest = [&](uint32_t(&x)[32]) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          t0 = fmaxf(fmaxf(t0, __uint_as_float(x[e])), __uint_as_float(x[e + 1]));
          t1 = fmaxf(fmaxf(t1, __uint_as_float(x[e + 2])), __uint_as_float(x[e + 3]));
        }
      };
      // (the difference first: a scaled maximum's own rounding would count in whole powers at huge scores)
      auto weigh = [&](uint32_t(&x)[32], uint32_t* w, float2 base2) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2 v = mul2(add2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), base2), c2);
          v.x = fast_exp2(v.x);
          v.y = fast_exp2(v.y);
          sum = add2(sum, v);
          w[e] = h2u(__floats2half2_rn(v.x, v.y));
        }
      };
      bool stands = k > 0;
      if (stands) {   // (the same for the whole warp)
        uint32_t w0[32], w1[32];
        const float base = m == neg_inf() ? 0.0f : m;
        const float2 base2 = make_float2(-base, -base);
        tmem_ld32(xa, ts);
        tmem_wait_ld(xa);
        tmem_ld32(xb, ts + 32);
        mask(xa, 0);
        highest(xa);
        weigh(xa, w0, base2);
        tmem_wait_ld(xb);
        tmem_ld32(xa, ts + 64);
        mask(xb, 1);
        highest(xb);
        weigh(xb, w0 + 16, base2);
        tmem_wait_ld(xa);
        tmem_ld32(xb, ts + 96);
        mask(xa, 2);
        highest(xa);
        weigh(xa, w1, base2);
        tmem_wait_ld(xb);
        mask(xb, 3);
        highest(xb);
        weigh(xb, w1 + 16, base2);
        // (a row that has had no live score yet has no reference to keep)
        stands = !__any_sync(0xffffffffu, m == neg_inf() || (fmaxf(t0, t1) - base) * c > kSlack);
        if (stands) {   // over scores this thread has read
          tmem_st32(ts + 64, w0);
          tmem_st32(ts + 96, w1);
        }
      }
      if (!stands) {   // the first tile, or a new maximum: the scores are still there
        t0 = t1 = neg_inf();
        sum = make_float2(0.0f, 0.0f);
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          tmem_ld32(xa, ts + 32 * i);
          tmem_wait_ld(xa);
          mask(xa, i);
          highest(xa);
        }
        const float top = fmaxf(t0, t1);
        const bool up = top > m;
        const float mn = up ? top : m;
        if (k > 0) {   // (the first tile's product overwrites the accumulators)
          const float alpha = up ? fast_exp2((m - mn) * c) : 1.0f;
          l *= alpha;
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) {
            tmem_ld32(xa, to + 32 * i);
            tmem_wait_ld(xa);
#pragma unroll
            for (int e = 0; e < 32; ++e) xa[e] = __float_as_uint(__uint_as_float(xa[e]) * alpha);
            tmem_st32(to + 32 * i, xa);
          }
        }
        m = mn;
        const float base = m == neg_inf() ? 0.0f : m;   // no live row yet: every weight is 2^-inf
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {   // quarters 3, 2, 0, 1: weights go where scores have been read twice
          const int at = i < 2 ? 3 - i : i - 2;
          uint32_t w[16];
          tmem_ld32(xa, ts + 32 * at);
          tmem_wait_ld(xa);
          mask(xa, at);
          weigh(xa, w, make_float2(-base, -base));
          tmem_st16(ts + 64 + 16 * at, w);
        }
      }
      l += sum.x + sum.y;
      tmem_wait_st();
      tc_fence_before();
      named_sync(1 + t, 128);
      if (leads) {
        const int next = NQ == 2 ? j + 1 : j + 2;
        const bool more = k + 1 < mine_n;
        wait(&v_full[j % NST], (j / NST) & 1);
        // The streams take turns at the matrix unit: sharing it they fall into step, both in their
        // softmax and then both waiting for products.
        if (t == 1) wait(&issued[0], k & 1);
        else if (k > 0) wait(&issued[1], (k - 1) & 1);
        tc_fence_after();
        if (elect_one()) {
          values(j, k > 0);
          if (!more) tc_commit(&o_full[t]);
        }
        __syncwarp();
        if (more) {
          wait(&k_full[next % NST], (next / NST) & 1);
          tc_fence_after();
          if (elect_one()) scores(next);
        }
        if (lane == 0) mbar_arrive(&issued[t]);
      }
      __syncwarp();
    }
    if (mine_n > 0 && !mbar_wait_bounded(&o_full[t], 0)) s_fail = 1;   // the last product is done, whatever ran out
    tc_fence_after();
    const int row = row0 + qt * 128 + r;
    const bool mine = row < a.rows && !s_fail;
    const int slot = NQ == 2 ? blockIdx.x : 2 * blockIdx.x + t;
    const size_t at = ((size_t)kvh * a.nsplit * a.streams + slot) * a.rows + row;
    if (mine) a.part_ml[at] = make_float2(m * c, l);
    if (mine_n > 0) {
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
        uint32_t x[32];
        tmem_ld32(x, to + 32 * i);
        tmem_wait_ld(x);
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
    }
  } else {
    // -------------------------------------------- queries, keys and values
    lower_registers<88>();
    const bool keys = warp < S::kSoft + 4;
    const int r = (threadIdx.x - 32 * S::kSoft) & 127;   // a thread a row
    if (keys || NQ == 2) {   // the key warps lay out the first row tile, the value warps the second
      const int t = keys ? 0 : 1;
      const int row = row0 + t * 128 + r;
      float big = 0.0f;
      const bool have = row < a.rows;
      const int b = have ? row / a.G : 0;
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(a.q) + ((size_t)b * a.Hq + (size_t)kvh * a.G + (have ? row - b * a.G : 0)) * D);
      const bool bf = a.io_dtype == KVQ_DTYPE_BF16;
      auto pair = [&](uint32_t w) {
        return bf ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)) : __half22float2(u2h(w));
      };
      if (have) {
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          const uint4 v = src[i];
          const float2 f0 = pair(v.x), f1 = pair(v.y), f2 = pair(v.z), f3 = pair(v.w);
          big = fmaxf(big, fmaxf(fmaxf(fmaxf(fabsf(f0.x), fabsf(f0.y)), fmaxf(fabsf(f1.x), fabsf(f1.y))),
                                 fmaxf(fmaxf(fabsf(f2.x), fabsf(f2.y)), fmaxf(fabsf(f3.x), fabsf(f3.y)))));
        }
      }
      // a power of two at or above the largest magnitude
      int e = 0;
      if (big > 0.0f && big < __int_as_float(0x7f800000)) frexpf(big, &e);
      e = max(min(e, 126), -126);
      const float down = __int_as_float((127 - e) << 23);
      s_scale[t * 128 + r] = __int_as_float((127 + e) << 23);
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        uint4 o = make_uint4(0u, 0u, 0u, 0u);
        if (have) {
          const uint4 v = src[i];
          float2 f[4] = {pair(v.x), pair(v.y), pair(v.z), pair(v.w)};
#pragma unroll
          for (int k = 0; k < 4; ++k) f[k] = make_float2(f[k].x * down, f[k].y * down);
          // 4-bit keys come as channels 0 4 1 5 2 6 3 7
          o = KB == 4 ? make_uint4(h2u(__floats2half2_rn(f[0].x, f[2].x)), h2u(__floats2half2_rn(f[0].y, f[2].y)),
                                   h2u(__floats2half2_rn(f[1].x, f[3].x)), h2u(__floats2half2_rn(f[1].y, f[3].y)))
                      : make_uint4(h2u(__floats2half2_rn(f[0].x, f[0].y)), h2u(__floats2half2_rn(f[1].x, f[1].y)),
                                   h2u(__floats2half2_rn(f[2].x, f[2].y)), h2u(__floats2half2_rn(f[3].x, f[3].y)));
        }
        *reinterpret_cast<uint4*>(sq + t * S::kTile + tile_off(r, i)) = o;
      }
      fence_async_smem();
      mbar_arrive(&q_full);
    }

    const PoolSide& side = keys ? p.k : p.v;
    const CUtensorMap* map = keys ? &p.kcols : &p.vcols;
    uint64_t* full = keys ? k_full : v_full;
    uint64_t* empty = keys ? k_empty : v_empty;
    uint8_t* ring = keys ? sk : sv;
    // the page of this thread's row of tile j (-1: none)
    auto page_of = [&](int j) {
      const int tok = (j0 + j) * 128 + r;
      return j < n && tok < pre.len ? a.batch.prefix_pages[tok >> p.page_log2] : -1;
    };
    uint32_t raw[AFF ? RAW : 1], meta[4];
    int id = page_of(0), next = page_of(1);
    size_t row = 0;
    bool ok = false, tma = false;
    auto place = [&](int j) {   // the thread's row of tile j, which warps take it by TMA
      const int tok = (j0 + j) * 128 + r;
      ok = (unsigned)id < (unsigned)p.n_pages;
      if (!ok && j < n && tok < pre.len) set_pool_status(p.status, KVQ_DEV_BAD_PAGE);
      row = ok ? ((((size_t)id * p.Hkv) + kvh) << p.page_log2) + (tok & (p.page - 1)) : 0;
      tma = !AFF && __all_sync(0xffffffffu, ok);   // a warp's 32 rows, each warp for itself
    };
    auto load = [&]() {   // 8- and 4-bit rows into registers, ahead of their stage
      if constexpr (AFF) {
        const uint4* src = reinterpret_cast<const uint4*>(side.codes + row * ROW);
#pragma unroll
        for (int i = 0; i < RAW / 4; ++i) {
          const uint4 v = ok ? src[i] : make_uint4(0u, 0u, 0u, 0u);
          raw[4 * i] = v.x;
          raw[4 * i + 1] = v.y;
          raw[4 * i + 2] = v.z;
          raw[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          meta[i] = ok && i < side.n_groups ? reinterpret_cast<const uint32_t*>(side.meta)[row * side.n_groups + i] : 0u;
      }
    };
    place(0);
    load();
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const int stg = j % NST;
      const uint32_t votes = __ballot_sync(0xffffffffu, ok);
      if (keys && lane == 0) s_mask[j & 7][r >> 5] = votes;
      if (j >= NST) wait(&empty[stg], ((j / NST) & 1) ^ 1);
      uint8_t* tile = ring + stg * S::kTile;
      if (tma) {
        // The warp's 32 rows: one box of 32, or two of 16 rows on pages of 16, for each half.
        const int box = min(p.page, 32);
        fence_async_smem();
        if (lane == 0) mbar_expect_tx(&full[stg], 32 * ROW + (j == 0 && keys && r == 0 ? a.stall_tx : 0u));
        else mbar_arrive(&full[stg]);
        __syncwarp();
        if (lane % box == 0) {   // this lane's row is a box's first
#pragma unroll
          for (int h = 0; h < S::kHalves; ++h)
            tma_columns(tile + h * 16384 + r * 128, map, h * 128, (int)row, &full[stg]);
        }
      } else {
        if constexpr (AFF) {
          store_decoded<D, F>(tile, r, raw, meta, side.n_groups);
        } else {
          const uint4* src = reinterpret_cast<const uint4*>(side.codes + row * ROW);
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c)
            *reinterpret_cast<uint4*>(tile + tile_off(r, c)) = ok ? src[c] : make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async_smem();
        if (a.stall_tx && j == 0 && keys && r == 0) mbar_expect_tx(&full[stg], a.stall_tx);
        else mbar_arrive(&full[stg]);
      }
      id = next;
      next = page_of(j + 2);
      place(j + 1);
      if (j + 1 < n) load();
    }
    // no copy is left in flight when the CTA ends, whatever else ran out
    if (!AFF)
      for (int j = max(n - NST, 0); j < n; ++j) mbar_wait_bounded(&full[j % NST], (j / NST) & 1);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == S::kSoft + 7) tmem_free(tmem, S::kCols);
  if (s_fail && threadIdx.x == 0) set_pool_status(p.status, KVQ_DEV_TIMEOUT);
}

}  // namespace kvq

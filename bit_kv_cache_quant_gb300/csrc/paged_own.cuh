// Paged decode attention, the streaming part: every (sequence, kv head) with
// its own rows (and, where the prefix is not worth a launch of its own, the
// prefix rows in front of them).
//
// Work is cut by tiles of 128 rows, not by sequences: the tiles of all units
// (sequence, kv head) stand in one line, CTA c of n takes those from
// c * total / n on, and a unit that spans CTAs is joined by the merge kernel
// from one partial state per (CTA, unit).  A ragged batch thus loads every SM
// alike, whatever its lengths.  A CTA's tile range is found from a scan of
// the lengths, which every CTA does for itself.
//
// Both products are taken transposed, with the cache on the 128-row side of
// tcgen05.mma and the up to eight query heads, as (fp16 part, residual), in
// 16 columns:
//   S^T [128 rows x 16] = K Q^T, one block of columns per scale group of keys
//   O^T [D x 16] += V^T P^T, one block of columns per scale group of values
// Stored codes enter as the integers they are (exact in fp16; u - 128 or
// u - 8), so the rounding of scale and zero never meets the tensor core: a
// thread per row puts the groups' scores together as s * sum(q u') + z' *
// sum(q) in fp32, and its softmax weight enters the second product times each
// value group's scale, again as (fp16 part, residual); the zeros' share, sum(p
// z'), is kept apart in fp32 per head and group.  With D = 64 the second
// product stacks rows 0-63 and 64-127 of a tile on its 128 rows against two
// sets of columns.
//
// Warps 0-3: softmax, a thread a row of the tile, and the joined state's way
// out.  Warps 4-7 bring keys, warps 8-11 values: a thread a row, several tiles
// ahead in registers, unpacked into the swizzled layout of the products (fp16
// rows go by TMA).  One thread of warp 12 issues the products, a tile's scores
// while the tile before is in its softmax.
//
// Bound by HBM for fp16 and 8-bit rows; for 4-bit rows by shared memory, where
// each unpacked tile is written once and read once.
#pragma once

#include "paged_tc.cuh"

namespace kvq {

constexpr int kPartPad = 4;   // partial row: D accumulators, max, sum, 2 pad

// CTAs of a grid that share `total` tiles: every one of them has some.
__device__ __forceinline__ int busy_ctas(long long total, int grid) { return (int)(total < grid ? total : grid); }

template <int D, int F> struct OwnShape {
  static constexpr int kBits = FmtBits<F>::v;
  static constexpr int kRow = D * kBits / 8;
  static constexpr bool kAff = F != F_FP16;
  static constexpr int kNg = kAff ? D / 32 : 1;      // scale groups of a row, at most
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kStages = 2;                  // of keys and of values
  static constexpr int kQTile = 16 * D * 2;
  static constexpr int kP = 128 * 16 * kNg * 2;      // a tile's weights
  static constexpr int kMeta = 128 * 2 * kNg * 4;    // a tile's (scale, zero) pairs of keys and values
  static constexpr int kAhead = kRow <= 64 ? 3 : 2;  // tiles in a loading thread's registers
  static constexpr int oK = 0, oV = kStages * kTile, oP = oV + kStages * kTile, oQ = oP + 2 * kP,
                       oMeta = oQ + 2 * kQTile, oRed = oMeta + (kAff ? 4 * kMeta : 0),
                       oHalf = oRed + 4 * 8 * (1 + kNg) * 4, oStart = oHalf + (D == 64 ? 64 * 8 * 4 : 0);
  static constexpr int kThreads = 13 * 32;
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

// 16-byte chunk c of a stored row as eight fp16 integers: u - 128 in order, or
// u - 8 in the order 0 4 1 5 2 6 3 7.
template <int KB>
__device__ __forceinline__ uint4 integers(const uint32_t* raw, int c) {
  __half2 h[4];
  if constexpr (KB == 4) {
    nibbles_to_h2<8>(raw[c], h);
  } else {
    const __half2 off = u2h(0x64806480u);   // 1024 + 128
    bytes_to_h2_1024(raw[2 * c] ^ 0x80808080u, h[0], h[1]);
    bytes_to_h2_1024(raw[2 * c + 1] ^ 0x80808080u, h[2], h[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __hsub2(h[i], off);
  }
  return make_uint4(h2u(h[0]), h2u(h[1]), h2u(h[2]), h2u(h[3]));
}

// Whether `any` holds for some thread of the four softmax warps (a barrier of theirs).
__device__ __forceinline__ bool any_of_128(bool any) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)any)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void sync_128() { asm volatile("barrier.cta.sync 1, 128;\n" ::: "memory"); }

template <int D, int F>
__global__ void __launch_bounds__(OwnShape<D, F>::kThreads, 1)
    paged_own_kernel(const __grid_constant__ PoolView p, const __grid_constant__ OwnArgs a) {
  using S = OwnShape<D, F>;
  constexpr int KB = S::kBits, ROW = S::kRow, RAW = ROW / 4, NST = S::kStages, NG = S::kNg;
  constexpr bool AFF = S::kAff;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint32_t* sm_meta = reinterpret_cast<uint32_t*>(smem + S::oMeta);   // [4][2 NG][128]
  float* sm_red = reinterpret_cast<float*>(smem + S::oRed);           // [4 warps][8][1 + NG]
  float* sm_half = reinterpret_cast<float*>(smem + S::oHalf);         // [64][8] (D = 64)
  int* sm_start = reinterpret_cast<int*>(smem + S::oStart);           // [n_seqs + 1]
  int* sm_len = sm_start + a.batch.n_seqs + 1;                        // [n_seqs]
  __shared__ __align__(8) uint64_t k_full[NST], k_empty[NST], v_full[NST], v_empty[NST], s_full[2], p_full[2];
  __shared__ uint32_t s_tmem;
  __shared__ uint32_t s_mask[4][4];        // live rows of tile j in ring slot j & 3
  __shared__ float s_qsum[4][8][4];        // sum of q of a head over each 32-channel block, slot unit & 3
  __shared__ float s_qmul[4][8];           // what brings a head's scores back to scale
  __shared__ float s_top[4][8];
  __shared__ int s_scan[13];
  __shared__ volatile int s_fail;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    s_fail = 0;
    for (int i = 0; i < NST; ++i) {
      mbar_init(&k_full[i], 128);
      mbar_init(&v_full[i], 128);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
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
    for (int i = i0; i < i1; ++i) {
      const Part own = part_of(a.batch.lens[i], a.batch.max_pages, p.page_log2, lead ? p.status : nullptr);
      sm_len[i] = own.len;
      sum += pre.tiles + own.tiles;
    }
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
      at += pre.tiles + ((sm_len[i] + 127) >> 7);
    }
    if (threadIdx.x == 0) {
      int all = 0;
      for (int w = 0; w < 13; ++w) all += s_scan[w];
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
  const int kng = AFF ? p.k.n_groups : 1, vng = AFF ? p.v.n_groups : 1;
  const int scols = 16 * NG;          // columns of one tile's scores; the outputs' follow two of them
  constexpr uint32_t kCols = 4 * 16 * NG <= 32 ? 32 : (4 * 16 * NG <= 64 ? 64 : (4 * 16 * NG <= 128 ? 128 : 256));
  if (warp == 12) tmem_alloc(&s_tmem, kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem, tmem_o = tmem + 2 * scols;

  // The unit of a tile, and the step to the next tile's.
  struct At {
    int b, kvh, j, tiles, len;   // len: own rows
  };
  At u;
  {
    int lo = 0, hi = n;   // the last b with sm_start[b] * Hkv <= t0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)sm_start[mid] * p.Hkv <= t0) lo = mid;
      else hi = mid;
    }
    u.b = lo;
    u.tiles = sm_start[lo + 1] - sm_start[lo];
    u.len = sm_len[lo];
    const int rest = (int)(t0 - (long long)sm_start[lo] * p.Hkv);
    u.kvh = rest / u.tiles;
    u.j = rest - u.kvh * u.tiles;
  }
  auto step = [&](At& v) {
    if (++v.j < v.tiles) return;
    v.j = 0;
    if (++v.kvh < p.Hkv) return;
    v.kvh = 0;
    do {
      ++v.b;
      v.tiles = v.b < n ? sm_start[v.b + 1] - sm_start[v.b] : 1;   // (behind the last unit nothing is used)
    } while (v.tiles == 0);
    v.len = v.b < n ? sm_len[v.b] : 0;
  };
  // every wait is bounded; once one runs out the others return at once, the loops
  // keep their counts and the results are marked by the status word
  auto wait = [&](uint64_t* m, uint32_t parity) {
    if (!s_fail && !mbar_wait_bounded(m, parity)) s_fail = 1;
  };

  if (warp < 4) {
    // ------------------------------------------------------------- softmax
    const int r = threadIdx.x;
    const uint32_t lanes = (uint32_t)warp << 21;
    // the thread's channel of the outputs: D = 64 tiles keep rows 64-127 in lanes and columns of their own
    const int place = D == 64 ? r & 63 : r;
    const int vgrp = AFF ? p.v.group : D;
    const int og = (D == 64 ? (warp & 1) * 32 : warp * 32) / vgrp;   // its value group: one per warp
    const uint32_t to = tmem_o + lanes + (D == 64 ? (warp >> 1) * 16 * vng : 0) + 16 * og;
    float top[8], l[8], z[8][NG];
    bool fresh = true, whole = u.j == 0;   // the unit's state is empty; its first tile was this CTA's
    int unit = 0;
#pragma unroll 1
    for (int it = 0; it < ntile; ++it) {
      const int stg = it & 1;
      wait(&s_full[stg], (it >> 1) & 1);
      tc_fence_after();
      const bool live = (s_mask[it & 3][r >> 5] >> lane) & 1;
      const uint32_t* mk = sm_meta + (it & 3) * (2 * NG * 128) + r;
      float v[8];
#pragma unroll
      for (int h = 0; h < 8; ++h) v[h] = 0.0f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (g < kng) {
          uint32_t x[16];
          tmem_ld16(x, tmem + lanes + stg * scols + 16 * g);
          float2 sz = make_float2(1.0f, 0.0f);
          if constexpr (AFF) {
            sz = __half22float2(u2h(mk[g * 128]));
            sz.y = fmaf(KB == 8 ? 128.0f : 8.0f, sz.x, sz.y);
          }
          tmem_wait_ld(x);
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            const float s = __uint_as_float(x[h]) + __uint_as_float(x[8 + h]);
            if constexpr (AFF) v[h] = fmaf(sz.x, s, fmaf(sz.y, s_qsum[unit & 3][h][g], v[h]));
            else v[h] = s;
          }
        }
      }
      bool over = fresh;
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        v[h] = live ? v[h] * s_qmul[unit & 3][h] : neg_inf();
        if (h >= a.G) v[h] = neg_inf();
        if (!fresh) over |= v[h] > top[h] + kSlack;
      }
      if (any_of_128(over)) {
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          float w = v[h];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, o));
          if (lane == 0) s_top[warp][h] = w;
        }
        sync_128();
        float alpha[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const float w = fmaxf(fmaxf(s_top[0][h], s_top[1][h]), fmaxf(s_top[2][h], s_top[3][h]));
          const float up = fresh ? w : fmaxf(top[h], w);
          alpha[h] = fresh || up == neg_inf() ? 1.0f : fast_exp2(top[h] - up);
          top[h] = up;
        }
        if (fresh) {
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            l[h] = 0.0f;
#pragma unroll
            for (int g = 0; g < NG; ++g) z[h][g] = 0.0f;
          }
        } else {   // the accumulators, once the product before has gone into them
          wait(&v_empty[stg ^ 1], ((it - 1) >> 1) & 1);
          tc_fence_after();
          uint32_t x[16];
          tmem_ld16(x, to);
          tmem_wait_ld(x);
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            x[h] = __float_as_uint(__uint_as_float(x[h]) * alpha[h]);
            x[8 + h] = __float_as_uint(__uint_as_float(x[8 + h]) * alpha[h]);
            l[h] *= alpha[h];
#pragma unroll
            for (int g = 0; g < NG; ++g) z[h][g] *= alpha[h];
          }
          tmem_st16(to, x);
          tmem_wait_st();
        }
        fresh = false;
      }
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        v[h] = fast_exp2(v[h] - (top[h] == neg_inf() ? 0.0f : top[h]));
        l[h] += v[h];
      }
      // the weights' buffer is free once the product of two tiles ago has read it
      if (it >= 2) wait(&v_empty[stg], ((it >> 1) & 1) ^ 1);
      uint8_t* pt = smem + S::oP + stg * S::kP;
      const int span = D == 64 ? 2 : 1;   // sets of columns
      const int kb = (D == 64 ? r & 63 : r) >> 3, set = D == 64 ? r >> 6 : 0;
      uint4* pw = reinterpret_cast<uint4*>(pt + kb * (span * 2 * vng * 128) + set * (2 * vng * 128) + (r & 7) * 16);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (g < vng) {
          float2 sz = make_float2(1.0f, 0.0f);
          if constexpr (AFF) {
            sz = __half22float2(u2h(mk[(NG + g) * 128]));
            sz.y = fmaf(KB == 8 ? 128.0f : 8.0f, sz.x, sz.y);
            if (!live) sz = make_float2(0.0f, 0.0f);   // whatever a dead row's page holds
          }
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float w0 = v[2 * k] * sz.x, w1 = v[2 * k + 1] * sz.x;
            const __half2 h2 = __floats2half2_rn(w0, w1);
            const float2 f = __half22float2(h2);
            hi[k] = h2u(h2);
            lo[k] = h2u(__floats2half2_rn(w0 - f.x, w1 - f.y));
            if constexpr (AFF) {
              z[2 * k][g] = fmaf(v[2 * k], sz.y, z[2 * k][g]);
              z[2 * k + 1][g] = fmaf(v[2 * k + 1], sz.y, z[2 * k + 1][g]);
            }
          }
          pw[(2 * g) * 8] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          pw[(2 * g + 1) * 8] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(&p_full[stg]);

      // ---- the unit's last tile here: its state goes out
      const bool ends = u.j + 1 == u.tiles;
      if (ends || it + 1 == ntile) {
        // sums over the tile rows of the maxima's weights and of the zeros' shares
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          if (h < a.G) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
              l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
#pragma unroll
              for (int g = 0; g < NG; ++g)
                if (AFF && g < vng) z[h][g] += __shfl_xor_sync(0xffffffffu, z[h][g], o);
            }
            if (lane == 0) {
              sm_red[(warp * 8 + h) * (1 + NG)] = l[h];
#pragma unroll
              for (int g = 0; g < NG; ++g)
                if (AFF && g < vng) sm_red[(warp * 8 + h) * (1 + NG) + 1 + g] = z[h][g];
            }
          }
        }
        wait(&v_empty[stg], (it >> 1) & 1);
        tc_fence_after();
        uint32_t x[16];
        tmem_ld16(x, to);
        tmem_wait_ld(x);
        float o[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) o[h] = __uint_as_float(x[h]) + __uint_as_float(x[8 + h]);
        if (D == 64 && warp >= 2) {
#pragma unroll
          for (int h = 0; h < 8; ++h) sm_half[place * 8 + h] = o[h];
        }
        sync_128();
        if (D == 128 || warp < 2) {
          const bool final = !a.joined && whole && ends;
          const long long id = (long long)u.b * p.Hkv + u.kvh;
          // 4-bit rows hold the channels of an eight as 0 4 1 5 2 6 3 7
          const int ch = KB == 4 ? (place & ~7) + ((place & 7) >> 1) + 4 * (place & 1) : place;
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            if (h < a.G) {
              float sum = 0.0f, zero = 0.0f;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                sum += sm_red[(w * 8 + h) * (1 + NG)];
                if (AFF) zero += sm_red[(w * 8 + h) * (1 + NG) + 1 + og];
              }
              float y = o[h] + zero;
              if (D == 64) y += sm_half[place * 8 + h];
              if (final) {
                store_io(a.out, ((size_t)u.b * a.Hq + (size_t)u.kvh * a.G + h) * D + ch, a.io_dtype,
                         sum == 0.0f ? 0.0f : y / sum);
              } else {
                float* dst = a.parts + ((size_t)(blockIdx.x + id) * a.G + h) * (D + kPartPad);
                dst[ch] = y;
                if (r == 0) {
                  dst[D] = top[h];
                  dst[D + 1] = sum;
                }
              }
            }
          }
        }
        sync_128();   // before the next unit's sums
        tc_fence_before();
        fresh = true;
        ++unit;
        whole = true;
      }
      step(u);
    }
  } else if (warp < 12) {
    // -------------------------------------------------- keys and values
    const bool keys = warp < 8;
    const int r = threadIdx.x & 127;   // a thread a row
    const PoolSide& side = keys ? p.k : p.v;
    const CUtensorMap* map = keys ? &p.kcols : &p.vcols;
    uint64_t* full = keys ? k_full : v_full;
    uint64_t* empty = keys ? k_empty : v_empty;
    uint8_t* ring = smem + (keys ? S::oK : S::oV);
    constexpr int AH = S::kAhead;
    uint32_t raw[AH][AFF ? RAW : 1], meta[AH][AFF ? 2 * NG : 1];
    uint4 qw[AH];
    size_t row[AH];
    unsigned flags[AH];   // bit 0: the row is live, 1: the warp's rows go by TMA, 2: the tile begins a unit here
    At w = u;             // the tile whose page ids are on their way
    int ids = -1, head = 0;
    auto look = [&](const At& v, int it) {   // page of this thread's row of v's tile, -1: none
      if (it >= ntile) return -1;
      const bool in_pre = v.j < pre.tiles;
      const int tok = (in_pre ? v.j : v.j - pre.tiles) * 128 + r;
      if (tok >= (in_pre ? pre.len : v.len)) return -1;
      const int id = (in_pre ? a.batch.prefix_pages : a.batch.table + (size_t)v.b * a.batch.max_pages)[tok >> p.page_log2];
      return (unsigned)id < (unsigned)p.n_pages ? id : -2;
    };
    auto fetch = [&](int s) {   // tile `head` into slot s; the ids of the next one
      const bool ok = ids >= 0;
      if (ids == -2) set_pool_status(p.status, KVQ_DEV_BAD_PAGE);
      row[s] = ok ? ((((size_t)ids * p.Hkv) + w.kvh) << p.page_log2) + (r & (p.page - 1)) : 0;
      const bool first = head < ntile && (w.j == 0 || head == 0);
      flags[s] = (ok ? 1u : 0u) | (!AFF && __all_sync(0xffffffffu, ok) ? 2u : 0u) | (first ? 4u : 0u);
      if constexpr (AFF) {
        const uint4* src = reinterpret_cast<const uint4*>(side.codes + row[s] * ROW);
#pragma unroll
        for (int i = 0; i < RAW / 4; ++i) {
          const uint4 x = ok ? src[i] : make_uint4(0u, 0u, 0u, 0u);
          raw[s][4 * i] = x.x;
          raw[s][4 * i + 1] = x.y;
          raw[s][4 * i + 2] = x.z;
          raw[s][4 * i + 3] = x.w;
        }
        if (keys) {   // the key warps bring both sides' (scale, zero) for the softmax
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            meta[s][i] = ok && i < kng ? reinterpret_cast<const uint32_t*>(p.k.meta)[row[s] * kng + i] : 0u;
            meta[s][NG + i] = ok && i < vng ? reinterpret_cast<const uint32_t*>(p.v.meta)[row[s] * vng + i] : 0u;
          }
        }
      }
      if (keys && first && r < D && r / (D / 8) < a.G)   // eight channels of one head's query
        qw[s] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                               ((size_t)w.b * a.Hq + (size_t)w.kvh * a.G) * D)[r];
      else
        qw[s] = make_uint4(0u, 0u, 0u, 0u);
      ++head;
      step(w);
      ids = look(w, head);
    };
    ids = look(w, 0);
#pragma unroll
    for (int s = 0; s < AH; ++s) fetch(s);
    int unit = -1;
#pragma unroll 1
    for (int base = 0; base < ntile; base += AH) {
#pragma unroll
      for (int s = 0; s < AH; ++s) {
        const int it = base + s;
        if (it < ntile) {
          const int stg = it % NST;
          if (it >= NST) wait(&empty[stg], ((it / NST) & 1) ^ 1);
          uint8_t* tile = ring + stg * S::kTile;
          if (keys) {
            const uint32_t votes = __ballot_sync(0xffffffffu, flags[s] & 1);
            if (lane == 0) s_mask[it & 3][r >> 5] = votes;
            if constexpr (AFF) {
#pragma unroll
              for (int i = 0; i < 2 * NG; ++i) sm_meta[((it & 3) * 2 * NG + i) * 128 + r] = meta[s][i];
            }
            if (flags[s] & 4) {
              // The unit's queries: each head brought under one by a power of two (bf16's range),
              // then fp16 part in rows 0-7 and residual in rows 8-15 of the tile.
              ++unit;
              const int h = r / (D / 8), c = r % (D / 8);
              const bool bf = a.io_dtype == KVQ_DTYPE_BF16;
              auto pair = [&](uint32_t x) {
                return bf ? make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)) : __half22float2(u2h(x));
              };
              float2 f[4] = {pair(qw[s].x), pair(qw[s].y), pair(qw[s].z), pair(qw[s].w)};
              float big = 0.0f;
#pragma unroll
              for (int i = 0; i < 4; ++i) big = fmaxf(big, fmaxf(fabsf(f[i].x), fabsf(f[i].y)));
#pragma unroll
              for (int o = 1; o < D / 8; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
              int e = 0;
              if (big > 0.0f && big < __int_as_float(0x7f800000)) frexpf(big, &e);
              e = max(min(e, 126), -126);
              const float down = __int_as_float((127 - e) << 23);
              float sum = 0.0f;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                f[i] = make_float2(f[i].x * down, f[i].y * down);
                sum += f[i].x + f[i].y;
              }
              // sums over each scale group of keys
              const int width = D / kng / 8;
#pragma unroll
              for (int o = 1; o < D / 8; o <<= 1)
                if (o < width) sum += __shfl_xor_sync(0xffffffffu, sum, o);
              if (r < D) {
                if (c % width == 0) s_qsum[unit & 3][h][c / width] = sum;
                if (c == 0) s_qmul[unit & 3][h] = __int_as_float((127 + e) << 23) * a.qscale;
                if (KB == 4) {   // as the codes come: 0 4 1 5 2 6 3 7
                  const float2 t0 = f[0], t1 = f[1], t2 = f[2], t3 = f[3];
                  f[0] = make_float2(t0.x, t2.x);
                  f[1] = make_float2(t0.y, t2.y);
                  f[2] = make_float2(t1.x, t3.x);
                  f[3] = make_float2(t1.y, t3.y);
                }
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const __half2 h2 = __floats2half2_rn(f[i].x, f[i].y);
                  const float2 g = __half22float2(h2);
                  hi[i] = h2u(h2);
                  lo[i] = h2u(__floats2half2_rn(f[i].x - g.x, f[i].y - g.y));
                }
                uint8_t* qt = smem + S::oQ + (unit & 1) * S::kQTile + (c >> 3) * 2048;
                *reinterpret_cast<uint4*>(qt + h * 128 + (((c ^ h) & 7) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(qt + (8 + h) * 128 + (((c ^ h) & 7) << 4)) =
                    make_uint4(lo[0], lo[1], lo[2], lo[3]);
              }
            }
          }
          const uint32_t stall = keys && it == 0 && r == 0 ? a.stall_tx : 0u;
          if (!AFF && (flags[s] & 2)) {
            const int box = min(p.page, 32);   // the warp's 32 rows: one box, or two on pages of 16
            fence_async_smem();
            if (lane == 0) mbar_expect_tx(&full[stg], 32 * ROW + stall);
            else mbar_arrive(&full[stg]);
            __syncwarp();
            if (lane % box == 0) {
#pragma unroll
              for (int h = 0; h < S::kHalves; ++h)
                tma_columns(tile + h * 16384 + r * 128, map, h * 128, (int)row[s], &full[stg]);
            }
          } else {
            if constexpr (AFF) {
#pragma unroll
              for (int c = 0; c < D / 8; ++c) *reinterpret_cast<uint4*>(tile + tile_off(r, c)) = integers<KB>(raw[s], c);
            } else {
              const uint4* src = reinterpret_cast<const uint4*>(side.codes + row[s] * ROW);
#pragma unroll 4
              for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4*>(tile + tile_off(r, c)) = (flags[s] & 1) ? src[c] : make_uint4(0u, 0u, 0u, 0u);
            }
            fence_async_smem();
            if (stall) mbar_expect_tx(&full[stg], stall);
            else mbar_arrive(&full[stg]);
          }
          fetch(s);
        }
      }
    }
    // no copy is left in flight when the CTA ends, whatever else ran out
    if (!AFF)
      for (int it = max(ntile - NST, 0); it < ntile; ++it) mbar_wait_bounded(&full[it % NST], (it / NST) & 1);
  } else if (lane == 0) {
    // ------------------------------------------------------------ products
    constexpr uint32_t kQK = mma_desc(128, 16, false, false);
    const uint32_t kPV = mma_desc(128, (D == 64 ? 32 : 16) * vng, true, true);
    const int gsteps = D / 16 / kng;   // k-steps of a scale group of keys
    int unit = -1;
    At w = u;   // the next tile to be scored
    auto scores = [&](int it) {
      const int stg = it % NST;
      if (w.j == 0 || it == 0) ++unit;
      wait(&k_full[stg], (it / NST) & 1);
      tc_fence_after();
      const uint32_t ka = smem_u32(smem + S::oK + stg * S::kTile), qa = smem_u32(smem + S::oQ + (unit & 1) * S::kQTile);
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t in = (k & 3) * 32;
        tc_mma_ss(tmem + (it & 1) * scols + 16 * (k / gsteps), operand_desc(ka + (k >> 2) * 16384 + in, 16, 1024),
                  operand_desc(qa + (k >> 2) * 2048 + in, 16, 1024), kQK, k % gsteps > 0);
      }
      tc_commit(&s_full[it & 1]);
      tc_commit(&k_empty[stg]);
      step(w);
    };
    scores(0);
    if (ntile > 1) scores(1);
    At v = u;   // the tile whose values come next
    for (int it = 0; it < ntile; ++it) {
      const int stg = it % NST;
      const bool begins = v.j == 0 || it == 0;
      wait(&p_full[it & 1], (it >> 1) & 1);
      wait(&v_full[stg], (it / NST) & 1);
      tc_fence_after();
      const uint32_t va = smem_u32(smem + S::oV + stg * S::kTile), pa = smem_u32(smem + S::oP + (it & 1) * S::kP);
      const uint32_t lead_p = (D == 64 ? 2 : 1) * 2 * vng * 128;   // bytes of eight rows of weights
#pragma unroll
      for (int k = 0; k < (D == 64 ? 4 : 8); ++k)
        tc_mma_ss(tmem_o, operand_desc(va + k * 2048, D == 64 ? 8192 : 16384, 1024),
                  operand_desc(pa + k * 2 * lead_p, lead_p, 128, kPlain), kPV, !begins || k > 0);
      tc_commit(&v_empty[stg]);
      if (it + 2 < ntile) scores(it + 2);
      step(v);
    }
    // the last product is done before the tensor memory goes back
    mbar_wait_bounded(&v_empty[(ntile - 1) % NST], ((ntile - 1) / NST) & 1);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_free(tmem, kCols);
  if (s_fail && threadIdx.x == 0) set_pool_status(p.status, KVQ_DEV_TIMEOUT);
  if (a.joined && lead) grid_dependency_wait();
}

}  // namespace kvq

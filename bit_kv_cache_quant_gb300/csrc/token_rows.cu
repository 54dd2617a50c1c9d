// Rotary positions, per-head norms and the paged append.
//
// Two kernels.  token_rows_kernel takes any layout: one warp per token and
// run of head rows, lane l the channels [l E, l E + E) with E = head_dim / 32,
// partners of a pair found by shuffles.  token_chunks_kernel takes rows whose
// starts are 16-byte aligned: a lane holds two runs of eight channels, c and
// c + D / 2 on, so that both channels of a pair sit in one lane (half layout
// over the whole head, or interleaved) and D / 16 lanes make a row.  The
// rotation of a 32K prompt (40 heads of 128, bf16, 671 MB) takes 281 us in the
// first form and 100 us in the second (6.7 TB/s, the measured copy rate).
//
// A row is loaded once, normed and rotated in registers and leaves either as
// a row of the output tensor or as codes in its page (or both), so that
// nothing between the projection and the cache passes through memory twice.
// All rows of a token turn by the same angles: a warp computes its lanes'
// sines and cosines once and reuses them for its rows.  The angle of pair i
// at position p is p times the table's 64-bit fraction of a turn, modulo 2^64
// (whole turns drop out exactly), and its top 32 bits, as half-turns in
// [-1, 1), go to sincospif: off by at most 2^-25 half-turns at any position,
// as close as fp32 sines can use.
//
// Bound by HBM for a prompt's rotation; by instruction issue with a norm (16K
// tokens of 48 heads, 403 MB: 76 us, issue 71% active) or the coding of keys
// and values (32K tokens into 8-bit pages, 874 MB: 175 us, issue 82%); by launch
// latency for decode steps (2.3 us a launch for one token, 5.8 us for a step of
// 64 into 4-bit pages).
#include "paged.cuh"
#include "quantize_row.cuh"

namespace kvq {

namespace {

constexpr int kRowWarps = 8;    // warps per CTA
constexpr int kRowUnroll = 4;   // rows a warp loads before it uses the first

template <int BYTES> struct VecOf;
template <> struct VecOf<2> { using type = unsigned short; };
template <> struct VecOf<4> { using type = unsigned; };
template <> struct VecOf<8> { using type = uint2; };
template <> struct VecOf<16> { using type = uint4; };

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// A lane's E elements, in vectors of at most 16 bytes.
template <typename T, int E> struct Lane {
  static constexpr int kBytes = E * (int)sizeof(T);
  static constexpr int kVec = kBytes > 16 ? 16 : kBytes;
  static constexpr int N = kBytes / kVec;
  using V = typename VecOf<kVec>::type;
  union {
    V v[N];
    T t[E];
  };
  __device__ __forceinline__ Lane() {}
  __device__ __forceinline__ void load(const T* p, int vec) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = reinterpret_cast<const V*>(p)[i];
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) t[i] = p[i];
    }
  }
  __device__ __forceinline__ void store(T* p, int vec) const {
    if (vec) {
#pragma unroll
      for (int i = 0; i < N; ++i) reinterpret_cast<V*>(p)[i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) p[i] = t[i];
    }
  }
};

// How a lane finds the other channel of each of its pairs.
enum Pairing : int {
  kNone = 0,     // no rotation
  kOwn = 1,      // in the lane itself: interleaved pairs, E >= 2
  kLane = 2,     // the same register of another lane
  kAny = 3,      // any register of any lane (half layout with rot / 2 not a multiple of E)
};

template <int E>
__device__ __forceinline__ void rotate(float (&x)[E], const float (&cs)[E], const float (&sn)[E], const int (&src)[E],
                                       int pairing) {
  float o[E];
  if (pairing == kOwn) {
    if constexpr (E > 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = x[e ^ 1];
    }
  } else if (pairing == kLane) {
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = __shfl_sync(0xffffffffu, x[e], src[0]);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[e] = 0.0f;
#pragma unroll
      for (int f = 0; f < E; ++f) {
        const float v = __shfl_sync(0xffffffffu, x[f], src[e] / E);
        if (src[e] % E == f) o[e] = v;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = fmaf(o[e], sn[e], x[e] * cs[e]);
}

// Stores the lane's channels of one row in the pool by the append's rules
// (quantize_row.cuh) and leaves in x the values the row stands for.
template <int E>
__device__ __forceinline__ void store_row(const PoolSide& s, size_t row, int lane, bool live, float (&x)[E]) {
  uint8_t* codes = s.codes + row * s.row_bytes;
  if (s.bits == 16) {
    Lane<__half, E> h;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      h.t[e] = __float2half_rn(x[e]);
      x[e] = __half2float(h.t[e]);
    }
    if (live) h.store(reinterpret_cast<__half*>(codes) + lane * E, 1);
    return;
  }
  const float levels = s.bits == 8 ? 255.0f : 15.0f;
  const int width = s.group / E;   // lanes per group
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int e = 1; e < E; ++e) {
    mn = fminf(mn, x[e]);
    mx = fmaxf(mx, x[e]);
  }
  mn = group_min(mn, width);
  mx = group_max(mx, width);
  const float sc = affine_scale(mn, mx, levels);
  const float inv = __frcp_rn(sc);
  const __half s16 = __float2half_rn(sc), z16 = __float2half_rn(mn);
  int u[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    u[e] = affine_code_inv(x[e], sc, inv, mn, levels);
    x[e] = fmaf((float)u[e], __half2float(s16), __half2float(z16));
  }
  if (live) {
    store_codes<E>(codes, lane, s.bits, u);
    if (lane % width == 0) s.meta[row * s.n_groups + lane / width] = __halves2half2(s16, z16);
  }
}

// Sequence of token t: the last b with cu[b] <= t, or -1 (32 probes a step).
__device__ __forceinline__ int sequence_of(const int* cu, int n_seqs, int t, int lane) {
  if (t < cu[0] || t >= cu[n_seqs]) return -1;
  int lo = 0, n = n_seqs;   // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const unsigned below = __ballot_sync(0xffffffffu, at < n && cu[lo + at] <= t);
    const int k = below ? 31 - __clz(below) : 0;
    lo += k * step;
    n = min(step, n - k * step);
    if (n < 1) n = 1;
  }
  return lo;
}

template <int E, typename T, bool PAGED>
__global__ void __launch_bounds__(32 * kRowWarps) token_rows_kernel(const __grid_constant__ TokenArgs a) {
  constexpr int D = 32 * E;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long job = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int tok = (int)(job / a.slices);
  if (tok >= a.n_tokens) return;
  const int total = a.q.heads + a.k.heads + (PAGED ? a.v.heads : 0);
  const int r0 = (int)(job % a.slices) * a.rows_per_warp;
  const int r1 = min(r0 + a.rows_per_warp, total);
  if (r0 >= r1) return;

  // where the token goes: its offset among its sequence's own tokens, its page
  int pos = 0;
  long long page_row = -1;   // row of kv head 0, or -1: not stored
  if constexpr (PAGED) {
    int b = tok, j = 0, n = 1;
    if (a.cu) {
      b = sequence_of(a.cu, a.batch.n_seqs, tok, lane);
      if (b < 0) return;
      j = tok - a.cu[b];
      n = a.cu[b + 1] - a.cu[b];
    }
    const long long at = (long long)a.batch.lens[b] - n + j;
    if (at < 0) return;
    pos = (int)at + (a.batch.prefix_len ? max(a.batch.prefix_len[0], 0) : 0);
    if (r1 > a.q.heads) {
      const long long col = at >> a.page_log2;
      const int id = col < a.batch.max_pages ? a.batch.table[(long long)b * a.batch.max_pages + col] : -1;
      if ((unsigned)id < (unsigned)a.n_pages)
        page_row = (((long long)id * a.Hkv) << a.page_log2) + (at & ((1 << a.page_log2) - 1));
      else if (lane == 0)
        set_pool_status(a.status, KVQ_DEV_BAD_PAGE);
    }
  }
  if (a.positions) pos = a.positions[tok];

  // the lane's sines and cosines
  float cs[E], sn[E];
  int src[E];
  int pairing = kNone;
  if (a.rope.freqs && (!PAGED || r0 < a.q.heads + a.k.heads)) {
    const int half = a.rope.rot >> 1;
    const bool inter = a.rope.interleaved != 0;
    pairing = inter ? (E > 1 ? kOwn : kLane) : (half % E == 0 ? kLane : kAny);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = lane * E + e;
      cs[e] = 1.0f;
      sn[e] = 0.0f;
      src[e] = c;
      if (c < a.rope.rot) {
        const bool first = inter ? (c & 1) == 0 : c < half;
        src[e] = inter ? c ^ 1 : (first ? c + half : c - half);
        if (E > 1 && inter && (e & 1)) {   // the pair's first channel is this lane's previous one
          cs[e] = cs[e > 0 ? e - 1 : 0];
          sn[e] = -sn[e > 0 ? e - 1 : 0];
          continue;
        }
        const unsigned long long f = a.rope.freqs[inter ? c >> 1 : (first ? c : c - half)];
        const long long turn = (long long)((unsigned long long)(long long)pos * f);
        float s, co;
        sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &co);
        cs[e] = co * a.rope.mag;
        sn[e] = (first ? -s : s) * a.rope.mag;
      }
    }
    if (pairing == kLane) src[0] = E == 1 ? src[0] : src[0] / E;
  }

  for (int r = r0; r < r1; r += kRowUnroll) {
    Lane<T, E> in[kRowUnroll];
#pragma unroll
    for (int i = 0; i < kRowUnroll; ++i) {
      const int rr = r + i;
      if (rr < r1) {
        int h = rr;
        const RowsView* w = &a.q;
        if (h >= a.q.heads) {
          h -= a.q.heads;
          w = &a.k;
          if (PAGED && h >= a.k.heads) {
            h -= a.k.heads;
            w = &a.v;
          }
        }
        in[i].load(static_cast<const T*>(w->in) + tok * w->in_tok + h * w->in_head + lane * E, a.vec);
      }
    }
#pragma unroll
    for (int i = 0; i < kRowUnroll; ++i) {
      const int rr = r + i;
      if (rr < r1) {
        int h = rr, kind = 0;
        const RowsView* w = &a.q;
        if (h >= a.q.heads) {
          h -= a.q.heads;
          w = &a.k;
          kind = 1;
          if (PAGED && h >= a.k.heads) {
            h -= a.k.heads;
            w = &a.v;
            kind = 2;
          }
        }
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = In<T>::ld(&in[i].t[e]);
        if (!PAGED || kind < 2) {
          if (w->weight) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
            const T* wt = static_cast<const T*>(w->weight) + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = x[e] * inv * In<T>::ld(wt + e);
          }
          if (pairing != kNone) rotate<E>(x, cs, sn, src, pairing);
        }
        if (PAGED && kind > 0)
          store_row<E>(kind == 1 ? a.ks : a.vs, (size_t)(page_row < 0 ? 0 : page_row + ((long long)h << a.page_log2)),
                       lane, page_row >= 0, x);
        if (!PAGED || kind == 0 || w->out) {
          Lane<T, E> o;
#pragma unroll
          for (int e = 0; e < E; ++e) o.t[e] = from_f32<T>(x[e]);
          o.store(static_cast<T*>(w->out) + tok * w->out_tok + h * w->out_head + lane * E, a.vec);
        }
      }
    }
  }
}

// ------------------------------------------------- sixteen channels a lane --

// Eight consecutive elements, 16-byte aligned.
template <typename T> struct Eight {
  static constexpr int N = 8 * (int)sizeof(T) / 16;
  uint4 v[N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  }
};
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b, const __nv_bfloat16*) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b, const __half*) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  a = f.x;
  b = f.y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __nv_bfloat16*) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __half*) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void unpack8(const Eight<T>& e, float* x) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = __uint_as_float(e.v[i].x);
      x[4 * i + 1] = __uint_as_float(e.v[i].y);
      x[4 * i + 2] = __uint_as_float(e.v[i].z);
      x[4 * i + 3] = __uint_as_float(e.v[i].w);
    }
  } else {
    const T* t = nullptr;
    unpack2(e.v[0].x, x[0], x[1], t);
    unpack2(e.v[0].y, x[2], x[3], t);
    unpack2(e.v[0].z, x[4], x[5], t);
    unpack2(e.v[0].w, x[6], x[7], t);
  }
}
template <typename T>
__device__ __forceinline__ Eight<T> pack8(const float* x) {
  Eight<T> e;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      e.v[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                          __float_as_uint(x[4 * i + 3]));
  } else {
    const T* t = nullptr;
    e.v[0] = make_uint4(pack2(x[0], x[1], t), pack2(x[2], x[3], t), pack2(x[4], x[5], t), pack2(x[6], x[7], t));
  }
  return e;
}

// How the pairs of a lane's channels x[0..8) = c .. c + 7 and x[8..16) = D / 2 + c .. lie.
enum ChunkPairing : int {
  kStraight = 0,      // no rotation
  kHalves = 1,        // half layout over the whole head: x[i] with x[8 + i]
  kNeighbours = 2,    // interleaved: x[2i] with x[2i + 1]
  kQuarter = 3,       // half layout over the first D / 2 channels: x[i], i < 8, with another lane's
};

// Codes eight channels by affine_code_inv's rule, stores them and leaves the
// values they stand for.  A quotient clamped to [0, levels] plus 1.5 * 2^23
// is rounded to the nearest integer (ties to even) in the sum's low bits; only
// where some quotient lies within 2^-12 of a half do the exact divisions decide.
__device__ __forceinline__ void code_eight(uint8_t* dst, int bits, float* x, float sc, float inv, float mn, float s,
                                           float z, bool live) {
  const float levels = bits == 8 ? 255.0f : 15.0f;
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23, bits 0x4B400000
  float u[8];
  bool near_half = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = fminf(fmaxf(__fmul_rn(__fsub_rn(x[i], mn), inv), 0.0f), levels);
    u[i] = __fadd_rn(t, kMagic);
    near_half |= fabsf(__fsub_rn(t, __fsub_rn(u[i], kMagic))) > 0.5f - 0x1p-12f;
  }
  if (near_half) {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = (float)affine_code(x[i], sc, mn, levels) + kMagic;
  }
  uint32_t w0, w1 = 0;
  if (bits == 8) {
    w0 = w1 = 0u - 0x4B400000u * 0x01010101u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w0 += __float_as_uint(u[i]) << (8 * i);
      w1 += __float_as_uint(u[4 + i]) << (8 * i);
    }
  } else {
    w0 = 0u - 0x4B400000u * 0x11111111u;
#pragma unroll
    for (int i = 0; i < 8; ++i) w0 += __float_as_uint(u[i]) << (4 * i);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf(u[i] - kMagic, s, z);
  if (!live) return;
  if (bits == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w0 ^ 0x80808080u, w1 ^ 0x80808080u);
  else *reinterpret_cast<uint32_t*>(dst) = w0;
}

// store_row for a lane's two runs of eight channels; l: the lane's place in its row.
template <int D>
__device__ __forceinline__ void store_chunks(const PoolSide& s, size_t row, int l, bool live, float (&x)[16]) {
  uint8_t* codes = s.codes + row * s.row_bytes;
  if (s.bits == 16) {
    const Eight<__half> lo = pack8<__half>(x), hi = pack8<__half>(x + 8);
    if (live) {
      lo.store(reinterpret_cast<__half*>(codes) + 8 * l);
      hi.store(reinterpret_cast<__half*>(codes) + D / 2 + 8 * l);
    }
    unpack8<__half>(lo, x);
    unpack8<__half>(hi, x + 8);
    return;
  }
  float mn[2] = {x[0], x[8]}, mx[2] = {x[0], x[8]};
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    mn[0] = fminf(mn[0], x[i]);
    mx[0] = fmaxf(mx[0], x[i]);
    mn[1] = fminf(mn[1], x[8 + i]);
    mx[1] = fmaxf(mx[1], x[8 + i]);
  }
  if (s.group == D) {   // one group: both runs
    mn[0] = mn[1] = fminf(mn[0], mn[1]);
    mx[0] = mx[1] = fmaxf(mx[0], mx[1]);
  }
  const int width = min(s.group, D / 2) / 8;   // lanes that share a group
#pragma unroll
  for (int o = 1; o < D / 16; o <<= 1) {
    if (o < width) {   // the same for every lane
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mn[i] = fminf(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], o));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
      }
    }
  }
  const float levels = s.bits == 8 ? 255.0f : 15.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float sc = affine_scale(mn[i], mx[i], levels);
    const __half s16 = __float2half_rn(sc), z16 = __float2half_rn(mn[i]);
    const int c = i * (D / 2) + 8 * l;
    code_eight(codes + c * s.bits / 8, s.bits, x + 8 * i, sc, __frcp_rn(sc), mn[i], __half2float(s16),
               __half2float(z16), live);
    if (live && l % width == 0 && !(i && s.group == D)) s.meta[row * s.n_groups + c / s.group] = __halves2half2(s16, z16);
  }
}

// Groups a lane copies ahead.  Copies held in registers instead (two groups a
// batch) took 107 us for the 32K rotation and 98 us for the 16K norm against 100
// and 76.
template <typename T> constexpr int kDepth = sizeof(T) == 4 ? 2 : 4;
template <typename T> constexpr int kRingBytes = kRowWarps * kDepth<T> * 2 * Eight<T>::N * 32 * 16;

__device__ __forceinline__ void copy16(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

// A warp takes one token and `rows_per_warp` groups of 32 / (D / 16) head rows;
// groups never mix queries, keys and values.  Its rows are on their way before
// the token's page and angles are looked up, and four CTAs to an SM cover the
// issue slots (32K tokens into 8-bit pages 175 us, 9 prompts of 9K tokens into
// fp16 pages of 16 36 us; with three CTAs 181 and 39); 32-bit rows need the
// registers of three.
template <int D, typename T, bool PAGED>
__global__ void __launch_bounds__(32 * kRowWarps, sizeof(T) == 4 ? 3 : 4)
    token_chunks_kernel(const __grid_constant__ TokenArgs a) {
  constexpr int L = D / 16;     // lanes per row
  constexpr int R = 32 / L;     // rows per group
  constexpr int N = Eight<T>::N;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, l = lane % L, rg = lane / L;
  // the warp's number from one lane, so that all that follows from it is known to be uniform
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const long long job = (long long)blockIdx.x * kRowWarps + warp;
  const int tok = (int)(job / a.slices);
  if (tok >= a.n_tokens) return;
  const int gq = (a.q.heads + R - 1) / R, gk = (a.k.heads + R - 1) / R;
  const int total = gq + gk + (PAGED ? gk : 0);
  const int g0 = (int)(job % a.slices) * a.rows_per_warp;
  const int g1 = min(g0 + a.rows_per_warp, total);
  if (g0 >= g1) return;

  // Each lane copies its own channels ahead into its own slots of a ring, so
  // the copies in flight cost no registers and wait for no other lane.
  extern __shared__ __align__(16) uint4 ring[];
  uint4* mine_ring = ring + warp * (kDepth<T> * 2 * N * 32) + lane;
  auto row_of = [&](int g, int& kind) {   // head row of this lane in group g
    kind = g < gq ? 0 : (g < gq + gk ? 1 : 2);
    return (g - (kind == 0 ? 0 : kind == 1 ? gq : gq + gk)) * R + rg;
  };
  auto fetch = [&](int g) {
    if (g < g1) {
      int kind;
      const int h = row_of(g, kind);
      const RowsView& w = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
      // a group's spare lanes repeat the last row and store nothing
      const T* src = static_cast<const T*>(w.in) + tok * w.in_tok + min(h, w.heads - 1) * w.in_head + 8 * l;
      uint4* dst = mine_ring + (g - g0) % kDepth<T> * (2 * N * 32);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        copy16(dst + i * 32, reinterpret_cast<const uint4*>(src) + i);
        copy16(dst + (N + i) * 32, reinterpret_cast<const uint4*>(src + D / 2) + i);
      }
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kDepth<T>; ++i) fetch(g0 + i);
  auto leave = [] { asm volatile("cp.async.wait_all;\n" ::: "memory"); };   // nothing in flight at the end

  int pos = 0;
  long long page_row = -1;
  if constexpr (PAGED) {
    int b = tok, j = 0, n = 1;
    if (a.cu) {
      b = sequence_of(a.cu, a.batch.n_seqs, tok, lane);
      if (b < 0) return leave();
      j = tok - a.cu[b];
      n = a.cu[b + 1] - a.cu[b];
    }
    const long long at = (long long)a.batch.lens[b] - n + j;
    if (at < 0) return leave();
    pos = (int)at + (a.batch.prefix_len ? max(a.batch.prefix_len[0], 0) : 0);
    if (g1 > gq) {
      const long long col = at >> a.page_log2;
      const int id = col < a.batch.max_pages ? a.batch.table[(long long)b * a.batch.max_pages + col] : -1;
      if ((unsigned)id < (unsigned)a.n_pages)
        page_row = (((long long)id * a.Hkv) << a.page_log2) + (at & ((1 << a.page_log2) - 1));
      else if (lane == 0)
        set_pool_status(a.status, KVQ_DEV_BAD_PAGE);
    }
  }
  if (a.positions) pos = a.positions[tok];

  // Sines (of each pair's first channel) and cosines of the lane's eight pairs.
  // The lanes of the R rows at the same place turn by the same angles: each
  // works out 8 / R of them and they trade.
  float cs[8], sn[8];
  int pairing = kStraight;
  if (a.rope.freqs && g0 < gq + gk) {
    const bool inter = a.rope.interleaved != 0;
    pairing = inter ? kNeighbours : (a.rope.rot == D ? kHalves : kQuarter);
    constexpr int M = 8 / R;
    float mc[M], ms[M];
#pragma unroll
    for (int k = 0; k < M; ++k) {
      const int i = rg * M + k;
      // the pair's first channel and its index
      const int c = inter ? (i < 4 ? 0 : D / 2) + 8 * l + 2 * (i & 3) : 8 * l + i;
      const int p = inter ? c >> 1 : (pairing == kQuarter && c >= D / 4 ? c - D / 4 : c);
      mc[k] = 1.0f;
      ms[k] = 0.0f;
      if (!inter || c < a.rope.rot) {
        const long long turn = (long long)((unsigned long long)(long long)pos * a.rope.freqs[p]);
        float s, co;
        sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &co);
        mc[k] = co * a.rope.mag;
        ms[k] = (pairing == kQuarter && c >= D / 4 ? s : -s) * a.rope.mag;   // kQuarter: the lane's own sign
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = __shfl_sync(0xffffffffu, mc[i % M], (i / M) * L + l);
      sn[i] = __shfl_sync(0xffffffffu, ms[i % M], (i / M) * L + l);
    }
  }

  int last_kind = -1;
  Eight<T> wl, wh;
  bool normed = false;
#pragma unroll 1
  for (int g = g0; g < g1; ++g) {
    int kind;
    const int h = row_of(g, kind);
    const RowsView& w = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const bool mine = h < w.heads;
    if (kind != last_kind) {
      last_kind = kind;
      normed = (!PAGED || kind < 2) && w.weight != nullptr;
      if (normed) {
        wl.load(static_cast<const T*>(w.weight) + 8 * l);
        wh.load(static_cast<const T*>(w.weight) + D / 2 + 8 * l);
      }
    }
    asm volatile("cp.async.wait_group %0;\n" ::"n"(kDepth<T> - 1) : "memory");
    float x[16];
    {
      const uint4* src = mine_ring + (g - g0) % kDepth<T> * (2 * N * 32);
      Eight<T> lo, hi;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        lo.v[i] = src[i * 32];
        hi.v[i] = src[(N + i) * 32];
      }
      unpack8<T>(lo, x);
      unpack8<T>(hi, x + 8);
    }
    fetch(g + kDepth<T>);
    if (normed) {
      float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float2 v = make_float2(x[e], x[e + 1]);
        sq = fma2(v, v, sq);
      }
      float s0 = sq.x + sq.y;
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
      const float inv = rsqrtf(s0 * (1.0f / D) + a.eps);
      const float2 inv2 = make_float2(inv, inv);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float f[8];
        unpack8<T>(half ? wh : wl, f);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 v = mul2(mul2(make_float2(x[8 * half + e], x[8 * half + e + 1]), inv2), make_float2(f[e], f[e + 1]));
          x[8 * half + e] = v.x;
          x[8 * half + e + 1] = v.y;
        }
      }
    }
    if (!PAGED || kind < 2) {
      if (pairing == kHalves) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 p = make_float2(x[e], x[e + 1]), q = make_float2(x[8 + e], x[9 + e]);
          const float2 c2 = make_float2(cs[e], cs[e + 1]), s2 = make_float2(sn[e], sn[e + 1]);
          const float2 y = fma2(q, s2, mul2(p, c2)), z = fma2(p, make_float2(-s2.x, -s2.y), mul2(q, c2));
          x[e] = y.x;
          x[e + 1] = y.y;
          x[8 + e] = z.x;
          x[9 + e] = z.y;
        }
      } else if (pairing == kNeighbours) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float p = x[2 * e], q = x[2 * e + 1];
          x[2 * e] = fmaf(q, sn[e], p * cs[e]);
          x[2 * e + 1] = fmaf(p, -sn[e], q * cs[e]);
        }
      } else if (pairing == kQuarter) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float o = __shfl_xor_sync(0xffffffffu, x[e], L / 2);
          x[e] = fmaf(o, sn[e], x[e] * cs[e]);
        }
      }
    }
    if (PAGED && kind > 0)
      store_chunks<D>(kind == 1 ? a.ks : a.vs,
                      (size_t)(page_row < 0 ? 0 : page_row + ((long long)min(h, w.heads - 1) << a.page_log2)), l,
                      mine && page_row >= 0, x);
    if (mine && (!PAGED || w.out)) {
      T* o = static_cast<T*>(w.out) + tok * w.out_tok + h * w.out_head + 8 * l;
      pack8<T>(x).store(o);
      pack8<T>(x + 8).store(o + D / 2);
    }
  }
}

template <typename K>
cudaError_t launch_rows(K kernel, const TokenArgs& a, unsigned grid, int smem, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(32 * kRowWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int E, typename T>
cudaError_t launch_typed(const TokenArgs& a, bool paged, bool chunks, unsigned grid, cudaStream_t st) {
  constexpr int D = 32 * E;
  if constexpr (E == 2 || E == 4) {
    if (paged) return chunks ? launch_rows(token_chunks_kernel<D, T, true>, a, grid, kRingBytes<T>, st)
                             : launch_rows(token_rows_kernel<E, T, true>, a, grid, 0, st);
  }
  if constexpr (E > 1) {
    if (chunks) return launch_rows(token_chunks_kernel<D, T, false>, a, grid, kRingBytes<T>, st);
  }
  return launch_rows(token_rows_kernel<E, T, false>, a, grid, 0, st);
}

template <int E>
cudaError_t launch_dim(const TokenArgs& a, int dtype, bool paged, bool chunks, unsigned grid, cudaStream_t st) {
  if (dtype == KVQ_DTYPE_F32) return launch_typed<E, float>(a, paged, chunks, grid, st);
  if (dtype == KVQ_DTYPE_BF16) return launch_typed<E, __nv_bfloat16>(a, paged, chunks, grid, st);
  return launch_typed<E, __half>(a, paged, chunks, grid, st);
}

// Vector accesses of vec_bytes need every row start of `w` (and its weights) on that boundary.
bool rows_aligned(const RowsView& w, int elem, int vec_bytes) {
  if (!w.heads) return true;
  const int n = vec_bytes / elem;   // elements per vector
  auto ok = [&](const void* p, long long ts, long long hs) {
    return !p || ((reinterpret_cast<uintptr_t>(p) % vec_bytes) == 0 && ts % n == 0 && hs % n == 0);
  };
  return ok(w.in, w.in_tok, w.in_head) && ok(w.out, w.out_tok, w.out_head) && ok(w.weight, 0, 0);
}

}  // namespace

cudaError_t launch_token_rows(const TokenArgs& args, int D, int dtype, bool paged, int sms, cudaStream_t st) {
  TokenArgs a = args;
  const int elem = dtype == KVQ_DTYPE_F32 ? 4 : 2;
  auto all_aligned = [&](int bytes) {
    return rows_aligned(a.q, elem, bytes) && rows_aligned(a.k, elem, bytes) && rows_aligned(a.v, elem, bytes);
  };
  // sixteen channels a lane: whole heads, half heads of the half layout, or any interleaved run
  const bool chunks = D >= 64 && all_aligned(16) &&
                      (!a.rope.freqs || a.rope.interleaved || a.rope.rot == D || a.rope.rot == D / 2);
  const int lane_bytes = D / 32 * elem;
  a.vec = all_aligned(lane_bytes > 16 ? 16 : lane_bytes);
  // units of work of a token: rows, or groups of rows
  const int R = chunks ? 512 / D : 1;
  auto units = [&](int heads) { return (heads + R - 1) / R; };
  const int total = units(a.q.heads) + units(a.k.heads) + (paged ? units(a.v.heads) : 0);
  // Few tokens: two groups of rows a warp (four rows in the general kernel), for
  // the most warps.  Once 16 units a warp still give every SM its 64 warps twice
  // over, a warp takes 16, so that the sines are computed once for more rows.
  const int few = chunks ? 2 : kRowUnroll, many = 16;
  a.rows_per_warp = (long long)a.n_tokens * ((total + many - 1) / many) >= 128LL * sms ? many : few;
  if (a.rows_per_warp > total) a.rows_per_warp = total;
  a.slices = (total + a.rows_per_warp - 1) / a.rows_per_warp;
  const long long jobs = (long long)a.n_tokens * a.slices;
  const long long grid = (jobs + kRowWarps - 1) / kRowWarps;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  switch (D) {
    case 32: return launch_dim<1>(a, dtype, paged, chunks, (unsigned)grid, st);
    case 64: return launch_dim<2>(a, dtype, paged, chunks, (unsigned)grid, st);
    case 128: return launch_dim<4>(a, dtype, paged, chunks, (unsigned)grid, st);
    default: return launch_dim<8>(a, dtype, paged, chunks, (unsigned)grid, st);
  }
}

}  // namespace kvq

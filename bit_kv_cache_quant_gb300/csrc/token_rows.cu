// Rotary positions, per-head norms and the paged append: one warp takes one
// token and a run of its head rows, lane l the channels [l E, l E + E) with
// E = head_dim / 32.
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
// Bound by HBM for prompts and by launch latency for decode steps.
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
            const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
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

template <int E, typename T>
cudaError_t launch_typed(const TokenArgs& a, bool paged, unsigned grid, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(32 * kRowWarps);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  note_launch();
  if constexpr (E == 2 || E == 4) {
    if (paged) return cudaLaunchKernelEx(&cfg, token_rows_kernel<E, T, true>, a);
  }
  return cudaLaunchKernelEx(&cfg, token_rows_kernel<E, T, false>, a);
}

template <int E>
cudaError_t launch_dim(const TokenArgs& a, int dtype, bool paged, unsigned grid, cudaStream_t st) {
  if (dtype == KVQ_DTYPE_F32) return launch_typed<E, float>(a, paged, grid, st);
  if (dtype == KVQ_DTYPE_BF16) return launch_typed<E, __nv_bfloat16>(a, paged, grid, st);
  return launch_typed<E, __half>(a, paged, grid, st);
}

// Whole-lane vector accesses need every row start of `w` on the lane's vector size.
bool rows_aligned(const RowsView& w, int elem, int vec_bytes) {
  if (!w.heads) return true;
  const int n = vec_bytes / elem;   // elements per vector
  auto ok = [&](const void* p, long long ts, long long hs) {
    return !p || ((reinterpret_cast<uintptr_t>(p) % vec_bytes) == 0 && ts % n == 0 && hs % n == 0);
  };
  return ok(w.in, w.in_tok, w.in_head) && ok(w.out, w.out_tok, w.out_head);
}

}  // namespace

cudaError_t launch_token_rows(const TokenArgs& args, int D, int dtype, bool paged, int sms, cudaStream_t st) {
  TokenArgs a = args;
  const int elem = dtype == KVQ_DTYPE_F32 ? 4 : 2;
  const int lane_bytes = D / 32 * elem;
  const int vb = lane_bytes > 16 ? 16 : lane_bytes;
  a.vec = rows_aligned(a.q, elem, vb) && rows_aligned(a.k, elem, vb) && rows_aligned(a.v, elem, vb);
  const int total = a.q.heads + a.k.heads + (paged ? a.v.heads : 0);
  // Few tokens: one load batch a warp, for the most warps.  Once the tokens
  // alone give every SM its 64 warps twice over, a warp takes 16 rows, so that
  // the sines are computed once for more rows.
  a.rows_per_warp = (long long)a.n_tokens * ((total + 15) / 16) >= 128LL * sms ? 16 : kRowUnroll;
  if (a.rows_per_warp > total) a.rows_per_warp = total;
  a.slices = (total + a.rows_per_warp - 1) / a.rows_per_warp;
  const long long jobs = (long long)a.n_tokens * a.slices;
  const long long grid = (jobs + kRowWarps - 1) / kRowWarps;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  switch (D) {
    case 32: return launch_dim<1>(a, dtype, paged, (unsigned)grid, st);
    case 64: return launch_dim<2>(a, dtype, paged, (unsigned)grid, st);
    case 128: return launch_dim<4>(a, dtype, paged, (unsigned)grid, st);
    default: return launch_dim<8>(a, dtype, paged, (unsigned)grid, st);
  }
}

}  // namespace kvq

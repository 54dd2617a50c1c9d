// Decode attention over a page pool: one query token per sequence, over a
// prefix shared by the batch and each sequence's own pages.
//
// One CTA per (sequence, query head); its warps take rows in turn, lane l the
// channels [l E, l E + E), and keep their own online-softmax state, merged at
// the end.  Every sequence reads the prefix for itself.
#include "paged.cuh"

namespace kvq {

namespace {

constexpr int kWarps = 4;

template <int E>
__device__ __forceinline__ void load_values(const PoolSide& s, size_t row, int lane, float (&x)[E]) {
  const uint8_t* p = s.codes + row * s.row_bytes;
  if (s.bits == 16) {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = __half2float(reinterpret_cast<const __half*>(p)[lane * E + e]);
    return;
  }
  const float2 m = __half22float2(s.meta[row * s.n_groups + lane * E / s.group]);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = lane * E + e;
    const int u = s.bits == 8 ? p[c] ^ 0x80 : (p[c >> 1] >> (4 * (c & 1))) & 15;
    x[e] = fmaf((float)u, m.x, m.y);
  }
}

template <int E>
__global__ void __launch_bounds__(32 * kWarps) paged_decode_kernel(const __grid_constant__ PoolView p,
                                                                   const PagedDecodeArgs a) {
  constexpr int D = 32 * E;
  __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x, b = blockIdx.y;
  const int kvh = h / (a.Hq / p.Hkv);
  const size_t qo = ((size_t)b * a.Hq + h) * D + lane * E;
  float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = load_io(a.q, qo + e, a.io_dtype) * a.qscale;
    o[e] = 0.0f;
  }
  for (int part = 0; part < 2; ++part) {
    const int* pages = part ? a.batch.table + (size_t)b * a.batch.max_pages : a.batch.prefix_pages;
    const int cols = part ? a.batch.max_pages : a.batch.max_prefix_pages;
    long long n = part ? a.batch.lens[b] : (a.batch.max_prefix_pages ? a.batch.prefix_len[0] : 0);
    if (n > ((long long)cols << p.page_log2)) {
      n = (long long)cols << p.page_log2;
      if (threadIdx.x == 0) set_pool_status(p.status, KVQ_DEV_BAD_PAGE);
    }
    for (int j = warp; j < n; j += kWarps) {
      const int id = pages[j >> p.page_log2];
      if ((unsigned)id >= (unsigned)p.n_pages) {
        if (lane == 0) set_pool_status(p.status, KVQ_DEV_BAD_PAGE);
        continue;
      }
      const size_t row = ((((size_t)id * p.Hkv) + kvh) << p.page_log2) + (j & (p.page - 1));
      float k[E], v[E], s = 0.0f;
      load_values<E>(p.k, row, lane, k);
      load_values<E>(p.v, row, lane, v);
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
      const float mn = fmaxf(m, s);
      const float al = exp2f(m - mn), pr = exp2f(s - mn);
      l = l * al + pr;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(pr, v[e], o[e] * al);
      m = mn;
    }
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = o[e];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
    float mm = -INFINITY, ll = 0.0f, oo = 0.0f;
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w]);
    for (int w = 0; w < kWarps; ++w) {
      if (sm_l[w] == 0.0f) continue;
      const float f = exp2f(sm_m[w] - mm);
      ll = fmaf(sm_l[w], f, ll);
      oo = fmaf(sm_o[w][d], f, oo);
    }
    store_io(a.out, ((size_t)b * a.Hq + h) * D + d, a.io_dtype, ll > 0.0f ? oo / ll : 0.0f);
  }
}

}  // namespace

size_t paged_workspace_bytes(const PoolView& p, int n_seqs, int Hq, int max_prefix_pages) { return 16; }

cudaError_t launch_paged_decode(const PoolView& p, const PagedDecodeArgs& a, cudaStream_t st) {
  const dim3 grid(a.Hq, a.batch.n_seqs);
  note_launch();
  if (p.D == 64) paged_decode_kernel<2><<<grid, 32 * kWarps, 0, st>>>(p, a);
  else paged_decode_kernel<4><<<grid, 32 * kWarps, 0, st>>>(p, a);
  return cudaGetLastError();
}

}  // namespace kvq

// Launch of paged decode attention: the streaming kernel (paged_own.cuh) and
// the merge of the states of units that span CTAs.
#include "paged_own.cuh"

namespace kvq {

namespace {

// Joins a unit's states with the online-softmax rule, one warp per query
// head.  A unit that one CTA finished is left alone; one without rows gets
// zeros.
template <int D>
__global__ void __launch_bounds__(256) paged_merge_kernel(const OwnArgs a, int Hkv, int grid) {
  constexpr int C = D / 32;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, h = threadIdx.x >> 5;
  const int unit = blockIdx.x, b = unit / Hkv, kvh = unit - b * Hkv;
  const long long total = (long long)a.starts[a.batch.n_seqs] * Hkv;
  const int tiles = a.starts[b + 1] - a.starts[b];
  const long long x0 = (long long)a.starts[b] * Hkv + (long long)kvh * tiles, x1 = x0 + tiles - 1;
  const int ctas = busy_ctas(total, grid);
  int c0 = 0, n = 0;
  if (tiles > 0) {   // CTA c takes the tiles from total * c / ctas on
    c0 = (int)(((x0 + 1) * ctas + total - 1) / total) - 1;
    n = (int)(((x1 + 1) * ctas + total - 1) / total) - c0;
  }
  if (n == 1 && !a.joined) return;
  const float* own = a.parts + ((size_t)(c0 + unit) * a.G + h) * (D + kPartPad);
  const size_t stride = (size_t)a.G * (D + kPartPad);
  float m = neg_inf();
  for (int i = lane; i < n; i += 32) m = fmaxf(m, own[i * stride + D]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.0f, acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.0f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* s = own + i * stride;
    const float li = s[D + 1];
    const float w = li == 0.0f ? 0.0f : fast_exp2(s[D] - m);
    float x[C];
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = s[lane * C + c];
    l = fmaf(li, w, l);
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = fmaf(w, x[c], acc[c]);
  }
  const float r = l == 0.0f ? 0.0f : 1.0f / l;
  const size_t at = ((size_t)b * a.Hq + (size_t)kvh * a.G + h) * D + lane * C;
#pragma unroll
  for (int c = 0; c < C; ++c) store_io(a.out, at + c, a.io_dtype, acc[c] * r);
}

size_t starts_bytes(int n_seqs) { return ((size_t)(n_seqs + 1) * 4 + 255) / 256 * 256; }

template <int D, int F, int HG>
cudaError_t launch_own(const PoolView& p, OwnArgs a, int max_tiles_per_seq, cudaStream_t st) {
  using S = OwnShape<D, F, HG>;
  auto kern = paged_own_kernel<D, F, HG>;
  const int base = S::kStages * S::kStage + S::kAcc + 1024;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = once_per_device(configured, [&]() {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, base + 4097 * 4);
  });
  if (e != cudaSuccess) return e;
  const long long most = (long long)a.batch.n_seqs * p.Hkv * max_tiles_per_seq;   // tiles, at most
  long long ctas = (long long)S::kCtas * p.sms;
  if (ctas > most) ctas = most < 1 ? 1 : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = base + (a.batch.n_seqs + 1) * 4;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p, a);
  if (e != cudaSuccess) return e;
  note_launch();
  cfg.gridDim = dim3(a.batch.n_seqs * p.Hkv);
  cfg.blockDim = dim3(32 * a.G);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, paged_merge_kernel<D>, (const OwnArgs)a, p.Hkv, (int)ctas);
  note_launch();
  return e;
}

template <int D, int F>
cudaError_t launch_heads(const PoolView& p, const OwnArgs& a, int max_tiles, cudaStream_t st) {
  return a.G <= 4 ? launch_own<D, F, 1>(p, a, max_tiles, st) : launch_own<D, F, 2>(p, a, max_tiles, st);
}

template <int D>
cudaError_t launch_format(const PoolView& p, const OwnArgs& a, int max_tiles, cudaStream_t st) {
  if (p.k.bits == 16) return launch_heads<D, F_FP16>(p, a, max_tiles, st);
  if (p.k.bits == 8) return launch_heads<D, F_AFF8>(p, a, max_tiles, st);
  return launch_heads<D, F_AFF4>(p, a, max_tiles, st);
}

}  // namespace

size_t paged_workspace_bytes(const PoolView& p, int n_seqs, int Hq, int max_prefix_pages) {
  (void)max_prefix_pages;
  const size_t states = (size_t)4 * p.sms + (size_t)n_seqs * p.Hkv;
  return starts_bytes(n_seqs) + states * (Hq / p.Hkv) * (p.D + kPartPad) * sizeof(float);
}

cudaError_t launch_paged_decode(const PoolView& p, const PagedDecodeArgs& d, cudaStream_t st) {
  OwnArgs a{};
  a.batch = d.batch;
  a.q = d.q;
  a.out = d.out;
  a.starts = reinterpret_cast<int*>(d.ws);
  a.parts = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(d.ws) + starts_bytes(d.batch.n_seqs));
  a.io_dtype = d.io_dtype;
  a.Hq = d.Hq;
  a.G = d.Hq / p.Hkv;
  a.qscale = d.qscale;
  a.with_prefix = d.batch.max_prefix_pages > 0;
  a.joined = 0;
  a.stall_tx = test_stall_bytes();
  auto tiles = [&](int pages) { return (int)((((long long)pages << p.page_log2) + 63) >> 6); };
  const int max_tiles = tiles(d.batch.max_pages) + tiles(d.batch.max_prefix_pages);
  return p.D == 64 ? launch_format<64>(p, a, max_tiles, st) : launch_format<128>(p, a, max_tiles, st);
}

}  // namespace kvq

// Launch of paged decode attention: the shared prefix (paged_prefix.cuh), the
// streaming kernel (paged_own.cuh) and the merge of their states.
#include "paged_prefix.cuh"

namespace kvq {

namespace {

// Joins a unit's states with the online-softmax rule, two warps per query
// head, each half of the states: those of the CTAs that had tiles of it and,
// where the prefix was taken for the whole batch, those of the prefix's
// streams.  A unit that one CTA finished is left alone; one without rows gets
// zeros.  Bound by the latency of its few dependent loads: 11 us for 64
// sequences of 32 heads with 19 states each (20 MB from L2); one warp a head, with
// the weights in the chain of the loads, took 16.
template <int D>
__global__ void __launch_bounds__(512) paged_merge_kernel(const OwnArgs a, const PrefixArgs f, int Hkv, int grid,
                                                          int page_log2) {
  constexpr int C = D / 32;
  __shared__ float sm_l[8], sm_acc[8][D];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp >= a.G, h = part ? warp - a.G : warp;
  const int unit = blockIdx.x, b = unit / Hkv, kvh = unit - b * Hkv;
  const int start = a.starts[b], tiles = a.starts[b + 1] - start;
  const long long total = (long long)a.starts[a.batch.n_seqs] * Hkv;
  int runs = 0;
  if (a.joined) {
    const Part pre = part_of(a.batch.prefix_len[0], a.batch.max_prefix_pages, page_log2, nullptr);
    runs = prefix_runs((pre.len + 127) >> 7, f.nsplit) * f.streams;
  }
  int c0 = 0, n = 0;
  if (tiles > 0) {   // CTA c takes the tiles from total * c / ctas on
    const int ctas = busy_ctas(total, grid);
    const long long x0 = (long long)start * Hkv + (long long)kvh * tiles, x1 = x0 + tiles - 1;
    if (total * ctas < (1ll << 32)) {
      c0 = (int)(((uint32_t)(x0 + 1) * ctas + (uint32_t)total - 1) / (uint32_t)total) - 1;
      n = (int)(((uint32_t)(x1 + 1) * ctas + (uint32_t)total - 1) / (uint32_t)total) - c0;
    } else {
      c0 = (int)(((x0 + 1) * ctas + total - 1) / total) - 1;
      n = (int)(((x1 + 1) * ctas + total - 1) / total) - c0;
    }
  }
  if (n == 1 && !a.joined) return;   // (the whole block)
  const float* own = a.parts + ((size_t)(c0 + unit) * a.G + h) * (D + kPartPad);
  const size_t stride = (size_t)a.G * (D + kPartPad);
  const size_t run0 = (size_t)kvh * f.nsplit * f.streams * f.rows + (size_t)b * a.G + h;   // + run * f.rows
  // state i: an own one, or a prefix stream's; this warp's are part, part + 2, ...
  const int count = n + runs;
  auto state = [&](int i) {
    return i < n ? make_float2(own[i * stride + D], own[i * stride + D + 1]) : f.part_ml[run0 + (size_t)(i - n) * f.rows];
  };
  auto rows_of = [&](int i) { return i < n ? own + i * stride : f.part_o + (run0 + (size_t)(i - n) * f.rows) * D; };
  float m = neg_inf();
  for (int i = lane; i < count; i += 32) m = fmaxf(m, state(i).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  // Weights first, a lane a state; then the states' rows, several in flight.
  float l = 0.0f, acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.0f;
  for (int i0 = part; i0 < count; i0 += 64) {
    float wi = 0.0f;
    if (i0 + 2 * lane < count) {
      const float2 ml = state(i0 + 2 * lane);
      if (ml.y != 0.0f) {   // sum 0: no live row
        wi = fast_exp2(ml.x - m);
        l = fmaf(ml.y, wi, l);
      }
    }
    const int cnt = min(32, (count - i0 + 1) >> 1);
#pragma unroll 10
    for (int i = 0; i < cnt; ++i) {
      const float* s = rows_of(i0 + 2 * i) + lane * C;
      float x[C];
      if constexpr (C == 4) *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(s);
      else *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(s);
      const float w = __shfl_sync(0xffffffffu, wi, i);
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = w == 0.0f ? acc[c] : fmaf(w, x[c], acc[c]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (part) {
#pragma unroll
    for (int c = 0; c < C; ++c) sm_acc[h][lane * C + c] = acc[c];
    if (lane == 0) sm_l[h] = l;
  }
  __syncthreads();
  if (part) return;
  l += sm_l[h];
  const float r = l == 0.0f ? 0.0f : 1.0f / l;
  const size_t at = ((size_t)b * a.Hq + (size_t)kvh * a.G + h) * D + lane * C;
#pragma unroll
  for (int c = 0; c < C; ++c) store_io(a.out, at + c, a.io_dtype, (acc[c] + sm_acc[h][lane * C + c]) * r);
}

size_t starts_bytes(int n_seqs) { return ((size_t)(n_seqs + 1) * 4 + 255) / 256 * 256; }

struct Plan {
  int shared;     // the prefix once for the batch
  int nq;         // row tiles of 128 per CTA of the prefix kernel
  int nsplit;     // CTAs per (kv head, row tiles)
  int streams;    // states each leaves per row
  int row_ctas;   // CTAs along the query rows
};

Plan make_plan(const PoolView& p, int n_seqs, int G, int max_prefix_pages) {
  Plan r{};
  const long long rows = (long long)n_seqs * G;
  // Taking the prefix once costs a launch and a longer merge; taking it with
  // every sequence costs its tiles n_seqs times, from L2 after the first.
  // Measured at 8 kv heads of 128, four query heads each, 64 own rows, 4-bit
  // (once / with each, us): 4 sequences behind 4K 25 / 19, behind 16K 32 / 38;
  // 8 behind 4K 26 / 25; 16 behind 1K 16 / 18, behind 4K 29 / 38; 64 behind 256
  // rows 22 / 24, behind 16K 44 / 422.
  r.shared = n_seqs > 1 &&
             (long long)n_seqs * p.Hkv * ((((long long)max_prefix_pages << p.page_log2) + 63) >> 6) > 27LL * p.sms;
  if (!r.shared) return r;
  r.nq = rows > 128 ? 2 : 1;
  r.streams = r.nq == 2 ? 1 : 2;
  r.row_ctas = (int)((rows + 128 * r.nq - 1) / (128 * r.nq));
  const long long units = (long long)p.Hkv * r.row_ctas;
  const long long tiles = (((long long)max_prefix_pages << p.page_log2) + 127) >> 7;
  long long ns = p.sms / units;
  if (ns > tiles) ns = tiles;
  r.nsplit = ns < 1 ? 1 : (int)ns;
  return r;
}

size_t prefix_o_bytes(const PoolView& p, const Plan& r, int rows) {
  return r.shared ? (size_t)p.Hkv * r.nsplit * r.streams * rows * p.D * sizeof(float) : 0;
}
size_t prefix_ml_bytes(const PoolView& p, const Plan& r, int rows) {
  return r.shared ? ((size_t)p.Hkv * r.nsplit * r.streams * rows * sizeof(float2) + 255) / 256 * 256 : 0;
}

cudaLaunchConfig_t dependent_launch(dim3 grid, int threads, int smem, cudaStream_t st, cudaLaunchAttribute* at) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

template <int D, int F, int NQ>
cudaError_t launch_prefix(const PoolView& p, const PrefixArgs& f, const Plan& r, cudaStream_t st) {
  using S = PrefixShape<D, F, NQ>;
  auto kern = paged_prefix_kernel<D, F, NQ>;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = once_per_device(configured, [&]() {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = dependent_launch(dim3(r.nsplit, p.Hkv, r.row_ctas), S::kThreads, S::kSmem, st, &at);
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, p, f);
}

template <int D, int F, int M>
cudaError_t launch_own(const PoolView& p, const OwnArgs& a, const PrefixArgs& f, int max_tiles, cudaStream_t st) {
  using S = OwnShape<D, F, M>;
  auto kern = paged_own_kernel<D, F, M>;
  const int base = S::kStages * S::kStage + S::kAcc + 1024;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = once_per_device(configured, [&]() {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, base + 4097 * 4);
  });
  if (e != cudaSuccess) return e;
  const long long most = (long long)a.batch.n_seqs * p.Hkv * max_tiles;   // tiles, at most
  long long ctas = (long long)S::kCtas * p.sms;
  if (ctas > most) ctas = most < 1 ? 1 : most;
  cudaLaunchAttribute at;
  cudaLaunchConfig_t cfg =
      dependent_launch(dim3((unsigned)ctas), S::kThreads, base + (a.batch.n_seqs + 1) * 4, st, &at);
  e = cudaLaunchKernelEx(&cfg, kern, p, a);
  if (e != cudaSuccess) return e;
  note_launch();
  cfg = dependent_launch(dim3(a.batch.n_seqs * p.Hkv), 64 * a.G, 0, st, &at);
  e = cudaLaunchKernelEx(&cfg, paged_merge_kernel<D>, a, f, p.Hkv, (int)ctas, p.page_log2);
  note_launch();
  return e;
}

template <int D, int F>
cudaError_t launch_heads(const PoolView& p, const OwnArgs& a, const PrefixArgs& f, const Plan& r, int max_tiles,
                         cudaStream_t st) {
  if (r.shared) {
    const cudaError_t e = r.nq == 1 ? launch_prefix<D, F, 1>(p, f, r, st) : launch_prefix<D, F, 2>(p, f, r, st);
    if (e != cudaSuccess) return e;
  }
  if (a.G <= 4) return launch_own<D, F, kPairs>(p, a, f, max_tiles, st);
  return a.io_dtype == KVQ_DTYPE_BF16 ? launch_own<D, F, kSingles>(p, a, f, max_tiles, st)
                                      : launch_own<D, F, kTwoTiles>(p, a, f, max_tiles, st);
}

template <int D>
cudaError_t launch_format(const PoolView& p, const OwnArgs& a, const PrefixArgs& f, const Plan& r, int max_tiles,
                          cudaStream_t st) {
  if (p.k.bits == 16) return launch_heads<D, F_FP16>(p, a, f, r, max_tiles, st);
  if (p.k.bits == 8) return launch_heads<D, F_AFF8>(p, a, f, r, max_tiles, st);
  return launch_heads<D, F_AFF4>(p, a, f, r, max_tiles, st);
}

}  // namespace

size_t paged_workspace_bytes(const PoolView& p, int n_seqs, int Hq, int max_prefix_pages) {
  const int G = Hq / p.Hkv;
  const size_t states = (size_t)4 * p.sms + (size_t)n_seqs * p.Hkv;
  // A smaller batch may be cut into more runs: the prefix's states are bounded
  // by what fills the device once (256 rows a CTA) or by one run of every row.
  const Plan r = make_plan(p, n_seqs, G, max_prefix_pages);
  size_t prefix = 0;
  if (r.shared) {
    const size_t rows = (size_t)n_seqs * G > 256 ? (size_t)n_seqs * G : 256;
    const size_t most = rows * p.Hkv > (size_t)256 * p.sms ? rows * p.Hkv : (size_t)256 * p.sms;
    prefix = most * (p.D * sizeof(float) + sizeof(float2)) + 256;
  }
  return starts_bytes(n_seqs) + prefix + states * G * (p.D + kPartPad) * sizeof(float);
}

cudaError_t launch_paged_decode(const PoolView& p, const PagedDecodeArgs& d, cudaStream_t st) {
  const int G = d.Hq / p.Hkv, rows = d.batch.n_seqs * G;
  const Plan r = make_plan(p, d.batch.n_seqs, G, d.batch.max_prefix_pages);
  uint8_t* ws = reinterpret_cast<uint8_t*>(d.ws);
  OwnArgs a{};
  PrefixArgs f{};
  a.batch = f.batch = d.batch;
  a.q = f.q = d.q;
  a.io_dtype = f.io_dtype = d.io_dtype;
  a.Hq = f.Hq = d.Hq;
  a.G = f.G = G;
  a.qscale = f.qscale = d.qscale;
  a.out = d.out;
  a.starts = reinterpret_cast<int*>(ws);
  ws += starts_bytes(d.batch.n_seqs);
  f.part_ml = reinterpret_cast<float2*>(ws);
  ws += prefix_ml_bytes(p, r, rows);
  f.part_o = reinterpret_cast<float*>(ws);
  ws += prefix_o_bytes(p, r, rows);
  a.parts = reinterpret_cast<float*>(ws);
  f.rows = rows;
  f.nsplit = r.nsplit;
  f.streams = r.streams;
  a.with_prefix = d.batch.max_prefix_pages > 0 && !r.shared;
  a.joined = r.shared;
  a.stall_tx = f.stall_tx = test_stall_bytes();
  auto tiles = [&](int pages) { return (int)((((long long)pages << p.page_log2) + 63) >> 6); };
  const int max_tiles = tiles(d.batch.max_pages) + (a.with_prefix ? tiles(d.batch.max_prefix_pages) : 0);
  return p.D == 64 ? launch_format<64>(p, a, f, r, max_tiles, st) : launch_format<128>(p, a, f, r, max_tiles, st);
}

}  // namespace kvq

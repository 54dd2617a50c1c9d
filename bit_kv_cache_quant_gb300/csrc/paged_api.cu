// The extern "C" entry points of the rotary and paged-cache calls declared in
// include/kvq.h: argument checks, the frequency table, the pool's plane
// layout and handle, and kernel dispatch.  No device memory is allocated here.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <new>

#include "paged.cuh"

struct kvq_paged_s {
  kvq_paged_config cfg;
  kvq_paged_layout lay;
  uint8_t* base;
  kvq::PoolView view;
};

namespace {

constexpr int kMaxSeqs = 4096;
constexpr double kTwoPi = 6.28318530717958647692528676655900577;

kvq_status fail(kvq_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return kvq::report_error(s, buf);
}

void begin_call() { kvq::report_error(KVQ_OK, ""); }

kvq_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return KVQ_OK;
  if (e == cudaErrorNotSupported) return fail(KVQ_ERR_UNSUPPORTED, "%s: shape not instantiated", what);
  return fail(KVQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int elem_bytes(int dtype) { return dtype == KVQ_DTYPE_F32 ? 4 : 2; }

bool valid_dtype(int d) { return d == KVQ_DTYPE_F32 || d == KVQ_DTYPE_BF16 || d == KVQ_DTYPE_F16; }

bool finite_positive(double x) { return isfinite(x) && x > 0.0; }

// The number of whole turns a pair makes within the trained length decides its scaling.
double ramp(double x, double lo, double hi) {
  const double r = (x - lo) / (hi - lo);
  return r < 0.0 ? 0.0 : (r > 1.0 ? 1.0 : r);
}

kvq_status check_rope(const kvq_rope* rope, int head_dim) {
  if (!rope) return KVQ_OK;
  if (!rope->freqs) return fail(KVQ_ERR_INVALID_ARG, "null rope frequency table");
  if (!aligned(rope->freqs, 8)) return fail(KVQ_ERR_INVALID_ARG, "the rope frequency table must be 8-byte aligned");
  if (rope->rot_dim < 2 || rope->rot_dim > head_dim || rope->rot_dim % 2)
    return fail(KVQ_ERR_INVALID_ARG, "rot_dim must be even, in 2 .. head_dim");
  if (rope->interleaved != 0 && rope->interleaved != 1)
    return fail(KVQ_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (!isfinite(rope->attn_factor)) return fail(KVQ_ERR_INVALID_ARG, "attn_factor must be finite");
  return KVQ_OK;
}

kvq_status check_rows(const kvq_rows* r, const char* name, int dtype, int n_tokens, bool need_out) {
  if (!r || r->heads == 0) return KVQ_OK;
  if (r->heads < 0) return fail(KVQ_ERR_INVALID_ARG, "%s: negative head count", name);
  if (n_tokens > 0 && !r->in) return fail(KVQ_ERR_INVALID_ARG, "%s: null input", name);
  if (n_tokens > 0 && need_out && !r->out) return fail(KVQ_ERR_INVALID_ARG, "%s: null output", name);
  const size_t e = elem_bytes(dtype);
  if (!aligned(r->in, e) || !aligned(r->out, e) || !aligned(r->norm_weight, e))
    return fail(KVQ_ERR_INVALID_ARG, "%s: pointers must be aligned to their element", name);
  return KVQ_OK;
}

kvq::RowsView rows_view(const kvq_rows* r) {
  kvq::RowsView v{};
  if (!r || r->heads == 0) return v;
  v.in = r->in;
  v.out = r->out;
  v.weight = r->norm_weight;
  v.in_tok = r->in_tok_stride;
  v.in_head = r->in_head_stride;
  v.out_tok = r->out_tok_stride;
  v.out_head = r->out_head_stride;
  v.heads = r->heads;
  return v;
}

kvq::RopeView rope_view(const kvq_rope* rope) {
  kvq::RopeView v{};
  if (!rope) return v;
  v.freqs = reinterpret_cast<const unsigned long long*>(rope->freqs);
  v.rot = rope->rot_dim;
  v.interleaved = rope->interleaved;
  v.mag = rope->attn_factor;
  return v;
}

kvq_status compute_layout(const kvq_paged_config* c, kvq_paged_layout* L) {
  if (!c || !L) return fail(KVQ_ERR_INVALID_ARG, "null paged config or layout");
  if (c->n_kv_heads < 1 || c->n_pages < 1) return fail(KVQ_ERR_INVALID_ARG, "n_kv_heads and n_pages must be >= 1");
  if (c->n_kv_heads > 65535) return fail(KVQ_ERR_UNSUPPORTED, "more than 65535 kv heads");
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(KVQ_ERR_UNSUPPORTED, "paged head_dim %d not supported (64, 128)", c->head_dim);
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return fail(KVQ_ERR_UNSUPPORTED, "page_size %d not supported (16, 32, 64, 128)", c->page_size);
  const int fmt[2] = {c->k_format, c->v_format}, bits[2] = {c->k_bits, c->v_bits}, group[2] = {c->k_group, c->v_group};
  const int D = c->head_dim;
  for (int i = 0; i < 2; ++i) {
    if (fmt[i] == KVQ_FMT_FP16) {
      if (bits[i] != 16) return fail(KVQ_ERR_INVALID_ARG, "fp16 format needs bits = 16");
    } else if (fmt[i] == KVQ_FMT_AFFINE_TOKEN) {
      if (bits[i] != 8 && bits[i] != 4) return fail(KVQ_ERR_INVALID_ARG, "AFFINE_TOKEN bits must be 8 or 4");
      if ((group[i] != 32 && group[i] != 64 && group[i] != 128) || group[i] > D)
        return fail(KVQ_ERR_INVALID_ARG, "a paged AFFINE_TOKEN group must be 32, 64 or 128 and at most head_dim");
    } else {
      return fail(KVQ_ERR_UNSUPPORTED, "paged pools hold FP16 or AFFINE_TOKEN rows");
    }
  }
  if (fmt[0] != fmt[1] || bits[0] != bits[1])
    return fail(KVQ_ERR_UNSUPPORTED, "K and V of a paged pool have the same format and bits");
  const unsigned __int128 wide = (unsigned __int128)c->n_kv_heads * c->page_size * (unsigned)c->n_pages;
  if (wide >= ((unsigned __int128)1 << 31) - 128)
    return fail(KVQ_ERR_UNSUPPORTED, "n_kv_heads * page_size * n_pages must stay below 2^31 - 128 rows");
  const size_t rows = (size_t)wide;
  *L = kvq_paged_layout{};
  L->k_row_bytes = L->v_row_bytes = D * bits[0] / 8;
  L->k_n_groups = fmt[0] == KVQ_FMT_FP16 ? 0 : D / group[0];
  L->v_n_groups = fmt[1] == KVQ_FMT_FP16 ? 0 : D / group[1];
  size_t off = 256;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, kvq::kPlaneAlign);
    return bytes ? o : 0;
  };
  L->k_codes = take(rows * L->k_row_bytes);
  L->k_meta = take(rows * L->k_n_groups * 4);
  L->v_codes = take(rows * L->v_row_bytes);
  L->v_meta = take(rows * L->v_n_groups * 4);
  L->total_bytes = off;
  return KVQ_OK;
}

kvq_status check_batch(const kvq_paged_batch* b, bool prefix, kvq::BatchView* v) {
  if (!b) return fail(KVQ_ERR_INVALID_ARG, "null batch");
  if (b->n_seqs < 1 || b->n_seqs > kMaxSeqs)
    return fail(KVQ_ERR_INVALID_ARG, "n_seqs must be in 1 .. %d", kMaxSeqs);
  if (b->max_pages < 0 || b->max_prefix_pages < 0) return fail(KVQ_ERR_INVALID_ARG, "negative page counts");
  if (!b->seq_lens || (b->max_pages > 0 && !b->page_table))
    return fail(KVQ_ERR_INVALID_ARG, "null seq_lens or page_table");
  if (prefix && b->max_prefix_pages > 0 && (!b->prefix_pages || !b->prefix_len))
    return fail(KVQ_ERR_INVALID_ARG, "prefix pages need prefix_pages and prefix_len");
  v->table = b->page_table;
  v->lens = b->seq_lens;
  v->prefix_pages = prefix ? b->prefix_pages : nullptr;
  v->prefix_len = b->prefix_len;
  v->n_seqs = b->n_seqs;
  v->max_pages = b->max_pages;
  v->max_prefix_pages = prefix ? b->max_prefix_pages : 0;
  if (!aligned(v->table, 4) || !aligned(v->lens, 4) || !aligned(v->prefix_pages, 4) || !aligned(v->prefix_len, 4))
    return fail(KVQ_ERR_INVALID_ARG, "the batch's arrays must be 4-byte aligned");
  return KVQ_OK;
}

// SMs of the current device (asked for once per device), 0 on failure.
int device_sms() {
  static std::atomic<int> known[64];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

}  // namespace

extern "C" {

kvq_status kvq_rope_table(const kvq_rope_config* cfg, uint64_t* freqs, float* attn_factor) {
  begin_call();
  if (!cfg || !freqs || !attn_factor) return fail(KVQ_ERR_INVALID_ARG, "null rope config or output");
  const int rot = cfg->rot_dim;
  if (rot < 2 || rot % 2 || rot > 256) return fail(KVQ_ERR_INVALID_ARG, "rot_dim must be even, in 2 .. 256");
  if (!isfinite(cfg->base) || cfg->base <= 1.0) return fail(KVQ_ERR_INVALID_ARG, "base must be above 1");
  const int sc = cfg->scaling;
  if (sc < KVQ_ROPE_NONE || sc > KVQ_ROPE_FACTORS) return fail(KVQ_ERR_INVALID_ARG, "unknown rope scaling %d", sc);
  if (!isfinite(cfg->attn_factor) || cfg->attn_factor < 0.0)
    return fail(KVQ_ERR_INVALID_ARG, "attn_factor must be 0 or positive");
  if (sc != KVQ_ROPE_NONE && sc != KVQ_ROPE_FACTORS && !(isfinite(cfg->factor) && cfg->factor >= 1.0))
    return fail(KVQ_ERR_INVALID_ARG, "factor must be >= 1");
  if ((sc == KVQ_ROPE_YARN || sc == KVQ_ROPE_LLAMA3) && !finite_positive(cfg->original_max_position))
    return fail(KVQ_ERR_INVALID_ARG, "original_max_position must be positive");
  if (sc == KVQ_ROPE_YARN && !(finite_positive(cfg->beta_slow) && isfinite(cfg->beta_fast) &&
                               cfg->beta_fast > cfg->beta_slow))
    return fail(KVQ_ERR_INVALID_ARG, "YaRN needs beta_fast > beta_slow > 0");
  if (sc == KVQ_ROPE_LLAMA3 && !(finite_positive(cfg->low_freq_factor) && isfinite(cfg->high_freq_factor) &&
                                 cfg->high_freq_factor > cfg->low_freq_factor))
    return fail(KVQ_ERR_INVALID_ARG, "high_freq_factor > low_freq_factor > 0 required");
  if (sc == KVQ_ROPE_NTK && rot < 4) return fail(KVQ_ERR_INVALID_ARG, "NTK scaling needs rot_dim >= 4");
  if (sc == KVQ_ROPE_FACTORS) {
    if (!cfg->factors) return fail(KVQ_ERR_INVALID_ARG, "null factors");
    for (int i = 0; i < rot / 2; ++i)
      if (!finite_positive(cfg->factors[i])) return fail(KVQ_ERR_INVALID_ARG, "factor %d must be positive", i);
  }
  const double base = sc == KVQ_ROPE_NTK ? cfg->base * pow(cfg->factor, (double)rot / (rot - 2)) : cfg->base;
  // YaRN's ramp runs over pair indices: the (fractional) pair that turns beta times
  // within the trained length, rounded outwards
  double y0 = 0.0, y1 = 0.0;
  if (sc == KVQ_ROPE_YARN) {
    auto pair_of = [&](double turns) {
      return rot * log(cfg->original_max_position / (turns * kTwoPi)) / (2.0 * log(base));
    };
    y0 = fmax(floor(pair_of(cfg->beta_fast)), 0.0);
    y1 = fmin(ceil(pair_of(cfg->beta_slow)), (double)(rot - 1));
    if (y1 - y0 < 1e-3) y1 = y0 + 1e-3;
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = pow(base, -2.0 * i / rot);
    if (sc == KVQ_ROPE_LINEAR) {
      f /= cfg->factor;
    } else if (sc == KVQ_ROPE_FACTORS) {
      f /= cfg->factors[i];
    } else if (sc == KVQ_ROPE_YARN) {
      const double r = ramp((double)i, y0, y1);
      f = f * (1.0 - r) + f / cfg->factor * r;
    } else if (sc == KVQ_ROPE_LLAMA3) {
      const double turns = cfg->original_max_position * f / kTwoPi;
      const double keep = ramp(turns, cfg->low_freq_factor, cfg->high_freq_factor);
      f = f * keep + f / cfg->factor * (1.0 - keep);
    }
    double turn = f / kTwoPi;
    turn -= floor(turn);   // whole turns per position change nothing
    const double scaled = rint(turn * 0x1p64);
    freqs[i] = scaled >= 0x1p64 ? 0ull : (uint64_t)scaled;
  }
  double mag = 1.0;
  if (cfg->attn_factor > 0.0) mag = cfg->attn_factor;
  else if (sc == KVQ_ROPE_YARN) mag = 0.1 * log(cfg->factor) + 1.0;
  *attn_factor = (float)mag;
  return KVQ_OK;
}

kvq_status kvq_rope_qk(const kvq_rows* q, const kvq_rows* k, int32_t n_tokens, int32_t head_dim, int32_t dtype,
                       const int32_t* positions, const kvq_rope* rope, float eps, cudaStream_t stream) {
  begin_call();
  if (n_tokens < 0) return fail(KVQ_ERR_INVALID_ARG, "negative n_tokens");
  if (head_dim != 32 && head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(KVQ_ERR_UNSUPPORTED, "head_dim %d not supported (32, 64, 128, 256)", head_dim);
  if (!valid_dtype(dtype)) return fail(KVQ_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  kvq_status s = check_rope(rope, head_dim);
  if (s == KVQ_OK) s = check_rows(q, "q", dtype, n_tokens, true);
  if (s == KVQ_OK) s = check_rows(k, "k", dtype, n_tokens, true);
  if (s != KVQ_OK) return s;
  if (rope && n_tokens > 0 && !positions) return fail(KVQ_ERR_INVALID_ARG, "a rotation needs positions");
  if (!aligned(positions, 4)) return fail(KVQ_ERR_INVALID_ARG, "positions must be 4-byte aligned");
  if (!(eps >= 0.0f) || !isfinite(eps)) return fail(KVQ_ERR_INVALID_ARG, "eps must be 0 or positive");
  kvq::TokenArgs a{};
  a.q = rows_view(q);
  a.k = rows_view(k);
  if (a.q.heads == 0 && a.k.heads == 0) return fail(KVQ_ERR_INVALID_ARG, "neither q nor k given");
  if ((long long)a.q.heads + a.k.heads > INT32_MAX / 2) return fail(KVQ_ERR_INVALID_ARG, "too many heads");
  if (n_tokens == 0) return KVQ_OK;
  a.rope = rope_view(rope);
  a.positions = rope ? positions : nullptr;
  a.eps = eps;
  a.n_tokens = n_tokens;
  const int sms = device_sms();
  if (sms <= 0) return fail(KVQ_ERR_CUDA, "device query failed");
  return launched(kvq::launch_token_rows(a, head_dim, dtype, false, sms, stream), "kvq_rope_qk");
}

kvq_status kvq_paged_layout_query(const kvq_paged_config* cfg, kvq_paged_layout* out) {
  begin_call();
  return compute_layout(cfg, out);
}

kvq_status kvq_paged_init(const kvq_paged_config* cfg, void* dev_mem, size_t bytes, cudaStream_t stream,
                          kvq_paged* out) {
  begin_call();
  if (!out) return fail(KVQ_ERR_INVALID_ARG, "null output handle");
  *out = nullptr;
  kvq_paged_layout lay;
  const kvq_status s = compute_layout(cfg, &lay);
  if (s != KVQ_OK) return s;
  if (!dev_mem) return fail(KVQ_ERR_INVALID_ARG, "null pool buffer");
  if (!aligned(dev_mem, kvq::kPlaneAlign)) return fail(KVQ_ERR_INVALID_ARG, "pool buffer must be 256-byte aligned");
  if (bytes < lay.total_bytes)
    return fail(KVQ_ERR_CAPACITY, "pool buffer holds %zu bytes, layout needs %zu", bytes, lay.total_bytes);
  const int sms = device_sms();
  if (sms <= 0) return fail(KVQ_ERR_CUDA, "device query failed");
  kvq_paged_s* p = new (std::nothrow) kvq_paged_s();
  if (!p) return fail(KVQ_ERR_CAPACITY, "host allocation of the pool handle failed");
  p->cfg = *cfg;
  p->lay = lay;
  p->base = static_cast<uint8_t*>(dev_mem);
  kvq::PoolView& v = p->view;
  auto side = [&](size_t codes, size_t meta, int bits, int group, int rb, int ng) {
    kvq::PoolSide x{};
    x.codes = p->base + codes;
    x.meta = meta ? reinterpret_cast<__half2*>(p->base + meta) : nullptr;
    x.bits = bits;
    x.group = group;
    x.row_bytes = rb;
    x.n_groups = ng;
    return x;
  };
  v.k = side(lay.k_codes, lay.k_meta, cfg->k_bits, cfg->k_group, lay.k_row_bytes, lay.k_n_groups);
  v.v = side(lay.v_codes, lay.v_meta, cfg->v_bits, cfg->v_group, lay.v_row_bytes, lay.v_n_groups);
  v.status = reinterpret_cast<int*>(p->base);
  v.Hkv = cfg->n_kv_heads;
  v.D = cfg->head_dim;
  v.page = cfg->page_size;
  v.page_log2 = cfg->page_size == 16 ? 4 : cfg->page_size == 32 ? 5 : cfg->page_size == 64 ? 6 : 7;
  v.n_pages = cfg->n_pages;
  v.sms = sms;
  const size_t rows = (size_t)v.Hkv * v.page * v.n_pages;
  const int box = v.page < kvq::kTmaRows ? v.page : kvq::kTmaRows;
  if (!kvq::encode_rows_map(&v.kmap, v.k.codes, rows, lay.k_row_bytes, box) ||
      !kvq::encode_rows_map(&v.vmap, v.v.codes, rows, lay.v_row_bytes, box) ||
      (cfg->k_format == KVQ_FMT_FP16 &&
       (!kvq::encode_columns_map(&v.kcols, v.k.codes, rows, lay.k_row_bytes, v.page < 32 ? v.page : 32) ||
        !kvq::encode_columns_map(&v.vcols, v.v.codes, rows, lay.v_row_bytes, v.page < 32 ? v.page : 32)))) {
    delete p;
    return fail(KVQ_ERR_CUDA, "the driver could not encode the pool's tensor maps");
  }
  const cudaError_t e = cudaMemsetAsync(p->base, 0, 256, stream);
  if (e != cudaSuccess) {
    delete p;
    return fail(KVQ_ERR_CUDA, "paged init: %s", cudaGetErrorString(e));
  }
  *out = p;
  return KVQ_OK;
}

void kvq_paged_release(kvq_paged pool) { delete pool; }

kvq_status kvq_paged_append(kvq_paged pool, const kvq_paged_batch* batch, int32_t n_tokens, const int32_t* cu_tokens,
                            const kvq_rows* q, const kvq_rows* k, const kvq_rows* v, int32_t dtype,
                            const kvq_rope* rope, const int32_t* positions, float eps, cudaStream_t stream) {
  begin_call();
  if (!valid_dtype(dtype)) return fail(KVQ_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (n_tokens < 0) return fail(KVQ_ERR_INVALID_ARG, "negative n_tokens");
  kvq::TokenArgs a{};
  kvq_status s = check_batch(batch, false, &a.batch);
  if (s == KVQ_OK) s = check_rope(rope, pool ? pool->cfg.head_dim : 128);
  if (s == KVQ_OK) s = check_rows(q, "q", dtype, n_tokens, true);
  if (s == KVQ_OK) s = check_rows(k, "k", dtype, n_tokens, false);
  if (s == KVQ_OK) s = check_rows(v, "v", dtype, n_tokens, false);
  if (s != KVQ_OK) return s;
  if (!k || !v || k->heads < 1 || v->heads < 1) return fail(KVQ_ERR_INVALID_ARG, "k and v are required");
  if (v->norm_weight) return fail(KVQ_ERR_INVALID_ARG, "v takes no norm");
  if (!cu_tokens && n_tokens != batch->n_seqs)
    return fail(KVQ_ERR_INVALID_ARG, "without cu_tokens a call takes one token per sequence");
  if (!aligned(cu_tokens, 4) || !aligned(positions, 4))
    return fail(KVQ_ERR_INVALID_ARG, "cu_tokens and positions must be 4-byte aligned");
  if (!(eps >= 0.0f) || !isfinite(eps)) return fail(KVQ_ERR_INVALID_ARG, "eps must be 0 or positive");
  if (!pool) return fail(KVQ_ERR_INVALID_ARG, "null pool");
  if (k->heads != pool->cfg.n_kv_heads || v->heads != pool->cfg.n_kv_heads)
    return fail(KVQ_ERR_INVALID_ARG, "k and v must have the pool's %d heads", pool->cfg.n_kv_heads);
  a.q = rows_view(q);
  a.k = rows_view(k);
  a.v = rows_view(v);
  if ((long long)a.q.heads + 2LL * a.k.heads > INT32_MAX / 2) return fail(KVQ_ERR_INVALID_ARG, "too many heads");
  if (n_tokens == 0) return KVQ_OK;
  a.rope = rope_view(rope);
  a.positions = positions;
  a.eps = eps;
  a.n_tokens = n_tokens;
  a.cu = cu_tokens;
  const kvq::PoolView& p = pool->view;
  a.ks = p.k;
  a.vs = p.v;
  a.status = p.status;
  a.Hkv = p.Hkv;
  a.page_log2 = p.page_log2;
  a.n_pages = p.n_pages;
  return launched(kvq::launch_token_rows(a, p.D, dtype, true, p.sms, stream), "kvq_paged_append");
}

size_t kvq_paged_workspace_bytes(kvq_paged pool, int32_t n_seqs, int32_t n_q_heads, int32_t max_prefix_pages) {
  if (!pool || n_seqs < 1 || n_seqs > kMaxSeqs || n_q_heads < 1 || n_q_heads % pool->cfg.n_kv_heads ||
      max_prefix_pages < 0)
    return 0;
  return kvq::paged_workspace_bytes(pool->view, n_seqs, n_q_heads, max_prefix_pages);
}

kvq_status kvq_paged_decode_attn(kvq_paged pool, const kvq_paged_batch* batch, const void* q, void* out,
                                 int32_t n_q_heads, int32_t io_dtype, float softmax_scale, void* workspace,
                                 size_t ws_bytes, cudaStream_t stream) {
  begin_call();
  if (!q || !out) return fail(KVQ_ERR_INVALID_ARG, "null q or out");
  if (io_dtype == KVQ_DTYPE_F32)
    return fail(KVQ_ERR_UNSUPPORTED, "paged decode attention takes bf16 or fp16 queries");
  if (!valid_dtype(io_dtype)) return fail(KVQ_ERR_INVALID_ARG, "unknown dtype %d", io_dtype);
  if (!aligned(q, 16) || !aligned(out, 16)) return fail(KVQ_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if (!isfinite(softmax_scale)) return fail(KVQ_ERR_INVALID_ARG, "softmax_scale must be finite");
  kvq::PagedDecodeArgs a{};
  const kvq_status s = check_batch(batch, true, &a.batch);
  if (s != KVQ_OK) return s;
  if (!workspace || !aligned(workspace, 16))
    return fail(KVQ_ERR_INVALID_ARG, "the workspace must be 16-byte aligned device memory");
  if (!pool) return fail(KVQ_ERR_INVALID_ARG, "null pool");
  const int hkv = pool->cfg.n_kv_heads;
  if (n_q_heads < 1 || n_q_heads % hkv)
    return fail(KVQ_ERR_INVALID_ARG, "n_q_heads must be a positive multiple of n_kv_heads");
  if (n_q_heads / hkv > 8) return fail(KVQ_ERR_UNSUPPORTED, "more than 8 query heads per kv head");
  // rows, and the tiles of 64 rows of every (sequence, kv head), are counted in 32 bits
  const int64_t cols = (int64_t)batch->max_pages + batch->max_prefix_pages;
  const int64_t tiles = (cols * pool->cfg.page_size + 63) / 64 + 1;
  if (cols * pool->cfg.page_size >= INT32_MAX - 128 || tiles > INT32_MAX / batch->n_seqs / hkv)
    return fail(KVQ_ERR_UNSUPPORTED, "n_seqs * n_kv_heads * (max_pages + max_prefix_pages) * page_size / 64 must stay "
                                     "below 2^31, and a sequence's rows below 2^31 - 128");
  const size_t need = kvq::paged_workspace_bytes(pool->view, batch->n_seqs, n_q_heads, batch->max_prefix_pages);
  if (ws_bytes < need) return fail(KVQ_ERR_CAPACITY, "workspace holds %zu bytes, the call needs %zu", ws_bytes, need);
  a.q = q;
  a.out = out;
  a.ws = static_cast<float*>(workspace);
  a.io_dtype = io_dtype;
  a.Hq = n_q_heads;
  const float scale = softmax_scale > 0.0f ? softmax_scale : 1.0f / sqrtf((float)pool->cfg.head_dim);
  a.qscale = scale * 1.44269504088896340736f;
  return launched(kvq::launch_paged_decode(pool->view, a, stream), "kvq_paged_decode_attn");
}

kvq_status kvq_paged_status(kvq_paged pool, int32_t* status) {
  begin_call();
  if (!pool || !status) return fail(KVQ_ERR_INVALID_ARG, "null pool or output");
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(status, pool->view.status, sizeof(int32_t), cudaMemcpyDeviceToHost);
  return launched(e, "kvq_paged_status");
}

kvq_status kvq_paged_clear_status(kvq_paged pool, cudaStream_t stream) {
  begin_call();
  if (!pool) return fail(KVQ_ERR_INVALID_ARG, "null pool");
  return launched(cudaMemsetAsync(pool->view.status, 0, sizeof(int32_t), stream), "kvq_paged_clear_status");
}

}  // extern "C"

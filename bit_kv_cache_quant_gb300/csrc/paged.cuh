// Internal definitions of the rotary and paged-cache calls.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

// TMA map of a code plane of `rows` rows of `row_bytes` bytes, copied box_rows
// rows at a time into shared memory with the 16-byte-chunk swizzle matching
// the row length; false when the driver cannot encode it (kvq_api.cu).
bool encode_rows_map(CUtensorMap* m, void* base, size_t rows, int row_bytes, int box_rows);

// The same plane 128 bytes of box_rows rows at a time, with the 128-byte swizzle.
bool encode_columns_map(CUtensorMap* m, void* base, size_t rows, int row_bytes, int box_rows);

// The test hook of kvq_test_stall_decode_tiles: bytes a CTA's first barrier expects in excess.
unsigned test_stall_bytes();

// One tensor of a token-row launch, strides in elements.
struct RowsView {
  const void* in;
  void* out;
  const void* weight;
  long long in_tok, in_head, out_tok, out_head;
  int heads;
};

struct RopeView {
  const unsigned long long* freqs;   // turns per position times 2^64; null: no rotation
  int rot;
  int interleaved;
  float mag;
};

// One side (K or V) of a page pool: rows are numbered (page * Hkv + kv head) * page_size + row.
struct PoolSide {
  uint8_t* codes;   // [rows][row_bytes]
  __half2* meta;    // [rows][n_groups] (scale, zero); null for fp16 rows
  int bits;
  int group;
  int row_bytes;
  int n_groups;
};

struct PoolView {
  // TMA descriptors of the code planes as [rows, row_bytes], swizzled by the row length;
  // boxes of min(page_size, 64) rows (rows of 256 bytes as [rows][2][128]).
  CUtensorMap kmap;
  CUtensorMap vmap;
  // fp16 pools: the same planes 128 bytes of a row at a time, boxes of min(page_size, 32) rows.
  CUtensorMap kcols;
  CUtensorMap vcols;
  PoolSide k, v;
  int* status;
  int Hkv, D, page, page_log2, n_pages;
  int sms;
};

struct BatchView {
  const int* table;
  const int* lens;
  const int* prefix_pages;
  const int* prefix_len;
  int n_seqs, max_pages, max_prefix_pages;
};

// A token-row launch: q and k normed and rotated, and with `paged` k and v stored.
struct TokenArgs {
  RowsView q, k, v;
  RopeView rope;
  const int* positions;
  float eps;
  int n_tokens;
  int rows_per_warp, slices;   // a warp takes one token and rows_per_warp of its rows
  int vec;                     // every pointer and stride allows whole-lane vector accesses
  const int* cu;               // paged: first token of each sequence, or null
  BatchView batch;
  // the pool's side of the launch (PoolView without its tensor maps)
  PoolSide ks, vs;
  int* status;
  int Hkv, page_log2, n_pages;
};

cudaError_t launch_token_rows(const TokenArgs& a, int D, int dtype, bool paged, int sms, cudaStream_t st);

struct PagedDecodeArgs {
  BatchView batch;
  const void* q;
  void* out;
  float* ws;
  int io_dtype;
  int Hq;
  float qscale;      // softmax scale * log2(e)
};

size_t paged_workspace_bytes(const PoolView& p, int n_seqs, int Hq, int max_prefix_pages);
cudaError_t launch_paged_decode(const PoolView& p, const PagedDecodeArgs& a, cudaStream_t st);

__device__ __forceinline__ void set_pool_status(int* status, int code) { atomicCAS(status, 0, code); }

// Two fp32 operations an instruction, each rounded as its scalar form.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;\n"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;\n"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}

}  // namespace kvq

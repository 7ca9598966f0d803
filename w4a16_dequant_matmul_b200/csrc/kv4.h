// Internal launch interface of the 4-bit KV cache operators (kv4_cache.cu, kv4_decode.cu,
// kv4_prompt.cu) and the cache's layout, shared with the C ABI layer (kv4_api.cu). Launchers
// validate nothing.
//
// Cache layout. Block n, KV head h is one contiguous chunk of `block` tokens,
//     [K codes: block x D/2 B][V codes: block x D/2 B][K scales: block x G x 4 B][V scales],
// G = D / group, so that one bulk copy brings a whole block of a head (block <= 64) and every
// piece of 16 tokens starts on a 16-byte boundary. A scale word is S (low half) and Z (high
// half), both binary16. The codes of a row, two per byte in the order of its dimensions
// (byte n = q[2n] | q[2n+1] << 4), are stored transposed into the order in which lanes of the
// warp-level MMA fragments take them, so that a lane's share of a row is one shared-memory
// load and no code crosses lanes:
//     K: 32-bit word 4j + c of the row stands at word c (D/32) + j  (lane c of a quad)
//     V: byte 8i + g stands at byte g (D/16) + i                     (lane group g)
// and for D = 128 the two 32-byte halves of a V row change places on tokens t with (t & 2),
// so that the rows that a warp loads at once fall on different banks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace wq {

struct Kv4Cache {
  uint8_t* data;
  int64_t num_blocks;
  int32_t kv_heads, dim, group, block, block_log2;
  __host__ __device__ int groups() const { return dim / group; }
  __host__ __device__ int64_t chunk_bytes() const {
    return static_cast<int64_t>(block) * (dim + 8 * (dim / group));
  }
};

// Keys of a request that attention counts: positions are kept below 2^31 with room for a tile.
constexpr int kKv4MaxKeys = 1 << 30;

struct Kv4TablesArgs {
  const int32_t* ctx_lens;
  const int32_t* new_lens;
  int requests;
  const int32_t* free_blocks;
  int n_free;
  int block_log2;
  int32_t* tables;
  int width;
  int64_t ld_tables;
  int32_t* slots;
  int n_slots;
  int32_t* q_starts;
  int32_t* kv_lens;
  int32_t* taken;
  unsigned* status;
};
cudaError_t launch_kv4_block_tables(const Kv4TablesArgs& a, int sms, cudaStream_t st);

struct Kv4AppendArgs {
  const uint16_t* K;
  const uint16_t* V;
  bool bf16;
  int64_t tokens;
  int64_t k_tok, k_head, v_tok, v_head;  // strides in elements
  const int32_t* slots;
  Kv4Cache cache;
  unsigned* status;
};
cudaError_t launch_kv4_append(const Kv4AppendArgs& a, int sms, cudaStream_t st);

struct Kv4ReadArgs {
  Kv4Cache cache;
  const int32_t* slots;
  int64_t tokens;
  void* K;
  void* V;
  int out_dtype;  // WQ_F32, WQ_BF16, WQ_F16
  unsigned* status;
};
cudaError_t launch_kv4_read(const Kv4ReadArgs& a, int sms, cudaStream_t st);

struct Kv4AttnArgs {
  const uint16_t* Q;
  bool bf16;
  int tokens;  // rows of Q, out and lse
  int heads, ratio;
  int64_t q_tok, q_head, o_tok, o_head;  // strides in elements
  Kv4Cache cache;
  const int32_t* tables;
  int width;
  int64_t ld_tables;
  const int32_t* q_starts;
  const int32_t* kv_lens;
  int requests;
  float scale_log2;  // scale * log2(e)
  int causal, window;
  uint16_t* out;
  float* lse;  // [tokens, heads], or nullptr
  void* workspace;
  int most_rows;  // requests with more rows (tokens x ratio) than this go to the prompt kernel
  unsigned* status;
};
// Whether request b's rows lie in Q, behind those of the requests before it. (Rows of starts that
// do not ascend could be more than Q has, and than the grid of the prompt kernel is made for.)
__device__ __forceinline__ bool kv4_starts_ok(const Kv4AttnArgs& a, int64_t b) {
  const int lo = a.q_starts[b], hi = a.q_starts[b + 1];
  return lo >= 0 && hi >= lo && hi <= a.tokens;
}

size_t kv4_decode_workspace_bytes(int sms);
cudaError_t launch_kv4_decode(const Kv4AttnArgs& a, int max_q, int sms, cudaStream_t st);

// Requests with more rows than a.most_rows, on tcgen05.
constexpr int kKv4DecodeRows = 16;
size_t kv4_prompt_workspace_bytes(int sms);
// An upper bound of its (256 rows, KV head) units: the lengths are on the device, and CTAs without
// a unit return. It is the kernel's grid, so at most 2^31 - 1.
int64_t kv4_prompt_units(int64_t tokens, int64_t ratio, int64_t requests, int64_t kv_heads);
cudaError_t launch_kv4_prompt(const Kv4AttnArgs& a, int sms, cudaStream_t st);

}  // namespace wq

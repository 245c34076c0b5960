// ibp_kv_internal.cuh - shared internals of the paged key/value cache
// operators (not part of the ABI).
#pragma once

#include "ibp_internal.cuh"

namespace ibp {

// Every kernel of these operators is launched as a programmatic dependent: it
// reads or writes no memory before the previous kernel of the stream has
// completed, and lets the next one be placed only then.  In the other order the
// kernel after next could begin while this kernel's predecessor still writes: the
// kernels here would wait for it all the same, but a decoder with
// IBP_HINT_EARLY_FETCH reads its inputs before it waits.
__device__ __forceinline__ void pdl_begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
int kv_launch(const char* name, void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster,
              cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
  if (e != cudaSuccess) {
    set_cuda_error(e, name);
    cudaGetLastError();
    return IBP_ECUDA;
  }
  return IBP_OK;
}

__device__ __forceinline__ void kv_status(uint32_t* status, uint32_t code) {
  if (status) atomicCAS(status, 0u, code);
}

__device__ __forceinline__ uint32_t ceil_div(uint32_t a, uint32_t b) { return (a + b - 1) / b; }

// Pages of a sequence of `len` tokens, kept within its table row.
__device__ __forceinline__ uint32_t held_pages(int32_t len, uint32_t page_tokens, uint32_t max_pages) {
  if (len <= 0) return 0;
  const uint32_t n = (static_cast<uint32_t>(len) - 1) / page_tokens + 1;
  return n < max_pages ? n : max_pages;
}

// A length outside its table row is cut to it (and reported by the caller).
__device__ __forceinline__ int32_t clamp_len(int32_t len, uint32_t page_tokens, uint32_t max_pages) {
  const int64_t cap = static_cast<int64_t>(page_tokens) * max_pages;
  return len < 0 ? 0 : (len > cap ? static_cast<int32_t>(cap) : len);
}

// Half precision ends at 2^-25, so with the largest probability at 1 a row's keys
// below that would leave the product and stay in the sum: with one key that
// outweighs the rest, 65536 others of 2^-25 are 0.2 % of the output.  Their powers
// are taken against a reference kLift below the maximum, the same in product and sum,
// so the largest is 2^15 and the smallest that counts 2^-40 of it.  The reference
// is rounded up: no power is above 2^15.  bfloat16 has the exponents of a float.
template <bool F16>
constexpr float kLift = F16 ? 15.f : 0.f;

// Natural logarithm of a row's sum of exponentials from its reference and sum;
// the lift leaves the sum first, exactly, so that it costs the logarithm nothing.
template <bool F16>
__device__ __forceinline__ float row_lse(float top, float sum) {
  return (F16 ? top + kLift<F16> + log2f(sum * (1.f / 32768.f)) : top + log2f(sum)) * 0.6931471805599453f;
}

struct KvMeta {  // arguments of the page bookkeeping kernels
  const int32_t* table;
  const int32_t* lens;
  const int32_t* refs;
  uint32_t n_seqs, max_pages, page_tokens, n_pages;
  int32_t* table_out;
  int32_t* lens_out;
  int32_t* refs_out;
  int32_t* moves;
  int32_t* count;
  int32_t* ws;
  uint32_t* status;
};

// Pages as the copying kernels see them: runs of `row_bytes` rows.
struct KvRuns {
  char* data;
  uint64_t n_pools;
  int64_t pool_stride, page_stride, outer_stride, row_stride;  // bytes
  uint32_t n_pages, page_tokens;
  uint32_t outer;      // runs per page
  uint32_t row_bytes;  // bytes of a token in a run
  uint32_t vec;        // bytes per access: 16, 8, 4, 2 or 1
};

int launch_kv_fork(const KvMeta& m, const int32_t* parents, uint32_t n_out, cudaStream_t stream);
int launch_kv_free(const KvMeta& m, const int32_t* rows, uint32_t n_rows, cudaStream_t stream);
int launch_kv_compact(const KvMeta& m, cudaStream_t stream);
int launch_kv_copy(const KvRuns& r, const int32_t* moves, const int32_t* count, uint32_t max_moves,
                   uint32_t* status, int device, cudaStream_t stream);
int launch_kv_accept(const KvRuns& r, const KvMeta& m, const int32_t* n_draft, const int32_t* path,
                     const int32_t* n_accept, uint32_t max_accept, int device, cudaStream_t stream);

struct KvView {  // K or V pages of one layer; strides in bytes
  const char* data;
  int64_t page_stride, head_stride, token_stride;
};

struct AttendArgs {
  KvView k, v;
  const char* q;
  int64_t q_seq, q_token, q_head;  // bytes
  const int32_t* table;
  const int32_t* lens;
  const int32_t* n_live;    // drafted tokens / queries per sequence, or nullptr: T
  const uint32_t* mask;     // tree attention: words per query, or nullptr: a chain
  const int32_t* picks;     // sparse attention: selected pages, or nullptr
  uint32_t budget;          // entries of a list of picks
  uint32_t n_seqs, max_pages, n_pages, page_tokens;
  uint32_t T, kv_heads, group, dim, mask_words;
  float scale_log2;         // scale * log2(e)
  void* out;                // n_seqs x T x heads x dim
  float* lse;               // n_seqs x T x heads, or nullptr
  float* part;              // partial sums of split items (workspace)
  uint32_t splits;
  uint32_t cluster;         // the splits of an item are a cluster
  uint32_t* status;
  uint32_t f16;
};

// Tree attention by rows of at most 16 queries per CTA, and sparse attention
// (ibp_kv_attend.cu).
int launch_kv_attend(AttendArgs& a, int device, size_t ws_bytes, cudaStream_t stream);
// Scratch of launch_kv_attend: `items` (sequence, kv head) pairs, or (sequence,
// query, kv head) triples with `pick`, of `rows` rows and at most `tokens` tokens.
size_t kv_attend_workspace(uint64_t items, uint64_t rows, uint32_t dim, uint64_t tokens, bool pick, int device);

// Tree attention on the tensor cores (ibp_kv_tree.cu); *done is set when the
// call's shape is one it takes.
int launch_kv_tree(const AttendArgs& a, int device, size_t ws_bytes, cudaStream_t stream, bool* done);
size_t kv_tree_workspace(uint32_t n_seqs, uint32_t kv_heads, uint64_t rows, uint32_t dim, uint32_t page_tokens,
                         uint64_t tokens, int device);

uint64_t kv_tree_wait_limit(uint64_t cycles);  // sets it, returns the one before
long long kv_tree_limit();

struct SelectArgs {
  const char* q;
  int64_t q_seq, q_token, q_head;  // bytes
  const int32_t* table;
  const int32_t* lens;
  const int32_t* n_live;
  const int8_t* codes;
  const float* scales;
  uint32_t n_seqs, max_pages, n_pages, page_tokens;
  uint32_t T, kv_heads, group, dim;
  uint32_t budget, keep_first, keep_last;
  float* scores;   // n_seqs x T x kv_heads x max_pages (workspace)
  int32_t* picks;  // n_seqs x T x kv_heads x budget
  uint32_t* status;
  uint32_t f16;
};

int launch_kv_select(const SelectArgs& a, int device, cudaStream_t stream);
int launch_kv_summarize(const KvView& k, const int32_t* table, const int32_t* lens, const int32_t* first,
                        uint32_t n_seqs, uint32_t max_pages, uint32_t n_pages, uint32_t page_tokens, uint32_t heads,
                        uint32_t dim, uint32_t f16, int8_t* codes, float* scales, uint32_t* status, int device,
                        cudaStream_t stream);

}  // namespace ibp

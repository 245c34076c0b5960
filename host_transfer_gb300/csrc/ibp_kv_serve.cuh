// ibp_kv_serve.cuh - arguments of the verification of drafted tokens and of the
// eviction of cached ones.
#pragma once

#include "ibp_kv4.cuh"

namespace ibp {

struct VerifyArgs {
  const float* p;
  int64_t p_seq, p_row;  // elements
  const float* q;        // nullptr: every drafted token was certain
  int64_t q_seq, q_row;
  const int32_t* tokens;
  const int32_t* parents;  // nullptr: a chain
  const int32_t* n_draft;  // nullptr: T
  const float* u;
  uint32_t n_seqs, T, vocab;
  int32_t* path;
  int32_t* n_accept;
  int32_t* token;
  uint32_t* status;
};

int launch_kv_verify(const VerifyArgs& a, cudaStream_t stream);

struct WeighArgs {
  AttendArgs a;       // k: pages of 16 bits; v, out and part are not used
  Kv4View k4;         // pages of 4 bits, where codes is not nullptr
  const float* lse;   // n_seqs x T x heads
  const float* w;     // n_seqs x width
  float* w_out;
  uint32_t width;
  float decay;
  uint32_t q16;       // queries may be read 16 bytes at a time
};

int launch_kv_weigh(const WeighArgs& x, int device, cudaStream_t stream);
// Many rows, on the tensor cores (ibp_kv_weigh_tc.cu): dim <= 128.
int launch_kv_weigh_tc(const WeighArgs& x, int device, cudaStream_t stream);

struct EvictArgs {
  const float* w;
  float* w_out;
  const int32_t* lens;
  uint32_t n_seqs, width, budget, keep_first, keep_last;
  int32_t* path;
  int32_t* n_draft;
  int32_t* n_keep;
  uint32_t* status;
};

int launch_kv_evict(const EvictArgs& a, cudaStream_t stream);

}  // namespace ibp

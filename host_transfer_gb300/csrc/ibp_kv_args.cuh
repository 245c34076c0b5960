// ibp_kv_args.cuh - argument checks that the paged cache entry points share.
#pragma once

#include <cuda_runtime.h>

#include <type_traits>

#include "ibp_kv_internal.cuh"

namespace ibp {
namespace {

// Refuses a call with a text for ibp_last_error_detail.
int refuse(const char* text) {
  set_detail(text);
  return IBP_EINVAL;
}

int current_device(int* device) {
  const cudaError_t e = cudaGetDevice(device);
  if (e != cudaSuccess) {
    set_cuda_error(e, "cudaGetDevice");
    cudaGetLastError();
    return IBP_ECUDA;
  }
  return IBP_OK;
}

// Replaces p by the address kernels use; NULL stays NULL when `optional`.  An
// address that is not a multiple of its type's size would be a fault on the GPU.
template <typename T>
bool resolve(T*& p, int device, bool optional = false) {
  if (!p) return optional;
  if constexpr (!std::is_void_v<T>)
    if (reinterpret_cast<uintptr_t>(p) % alignof(T)) return false;
  const void* d;
  if (resolve_ptr(p, device, &d)) return false;
  p = static_cast<T*>(const_cast<void*>(d));
  return true;
}

constexpr uint64_t kMaxPages = 0x7FFFFFFFull;

int check_seqs(const ibp_kv_seqs* s, uint32_t page_tokens, bool lens_read = true) {
  if (!s) return refuse("seqs is NULL");
  if (page_tokens == 0 || page_tokens > 65536) return refuse("page_tokens outside [1, 65536]");
  if (s->n_seqs > 65535) return refuse("more than 65535 sequences");
  if (static_cast<uint64_t>(s->max_pages) * page_tokens > 0x7FFFFF00ull)
    return refuse("max_pages * page_tokens is 2^31 or more");
  if (s->n_seqs && ((lens_read && !s->lens) || (s->max_pages && !s->table))) return refuse("table or lens is NULL");
  return IBP_OK;
}

int view_of(KvView* v, const ibp_kv_pages* p, int device) {
  if (!p || !p->data) return refuse("pages is NULL");
  if (p->elem_bytes != 2) return refuse("keys and values are 16-bit");
  if (p->n_pages == 0 || p->n_pages > kMaxPages || p->heads == 0) return refuse("a page dimension is 0 or too large");
  if (p->dim == 0 || p->dim % 8 || p->dim > IBP_KV_MAX_DIM) return refuse("dim is not a multiple of 8 up to 256");
  if (p->page_stride < 0 || p->head_stride < 0 || p->token_stride < 0) return refuse("a stride is negative");
  const void* d;
  if (resolve_ptr(p->data, device, &d)) return refuse("pages are not device-accessible");
  v->data = static_cast<const char*>(d);
  v->page_stride = p->page_stride * 2;
  v->head_stride = p->heads == 1 ? 0 : p->head_stride * 2;
  v->token_stride = p->page_tokens == 1 ? 0 : p->token_stride * 2;
  if ((reinterpret_cast<uintptr_t>(d) | static_cast<uint64_t>(v->page_stride) | static_cast<uint64_t>(v->head_stride) |
       static_cast<uint64_t>(v->token_stride)) % 16)
    return refuse("pages are not 16-byte aligned in base and strides");
  return IBP_OK;
}

}  // namespace
}  // namespace ibp

// ibp_kv_serve_api.cu - C ABI of the caches in 4 bits, the verification of drafted
// tokens and the eviction of cached ones: argument checks and pointer resolution.
#include <cmath>

#include "ibp_kv_args.cuh"
#include "ibp_kv_serve.cuh"

using namespace ibp;

namespace {

int view4_of(Kv4View* v, const ibp_kv4_pages* p, int device) {
  if (!p || !p->codes || !p->scales) return refuse("4-bit pages are NULL");
  if (p->n_pages == 0 || p->n_pages > kMaxPages || p->heads == 0 || p->heads > 65535)
    return refuse("a page dimension is 0 or too large");
  if (p->dim == 0 || p->dim % IBP_KV4_GROUP || p->dim > IBP_KV_MAX_DIM) return refuse("dim is not a multiple of 32 up to 256");
  if (p->page_stride < 0 || p->head_stride < 0 || p->token_stride < 0 || p->scale_page_stride < 0 || p->scale_head_stride < 0 ||
      p->scale_token_stride < 0)
    return refuse("a stride is negative");
  const void *c, *s;
  if (resolve_ptr(p->codes, device, &c) || resolve_ptr(p->scales, device, &s)) return refuse("4-bit pages are not device-accessible");
  v->codes = static_cast<const char*>(c);
  v->page_stride = p->page_stride;
  v->head_stride = p->heads == 1 ? 0 : p->head_stride;
  v->token_stride = p->page_tokens == 1 ? 0 : p->token_stride;
  v->scales = static_cast<const char*>(s);
  v->s_page = p->scale_page_stride * 2;
  v->s_head = p->heads == 1 ? 0 : p->scale_head_stride * 2;
  v->s_token = p->page_tokens == 1 ? 0 : p->scale_token_stride * 2;
  if ((reinterpret_cast<uintptr_t>(c) | static_cast<uint64_t>(v->page_stride) | static_cast<uint64_t>(v->head_stride) |
       static_cast<uint64_t>(v->token_stride)) % 16)
    return refuse("codes are not 16-byte aligned in base and strides");
  if (reinterpret_cast<uintptr_t>(s) % 2) return refuse("scales are not 2-byte aligned");
  return IBP_OK;
}

bool alike(const ibp_kv4_pages* k, const ibp_kv4_pages* v) {
  return k->n_pages == v->n_pages && k->heads == v->heads && k->page_tokens == v->page_tokens && k->dim == v->dim;
}

int rows4_of(Kv4Rows* r, const ibp_kv4_pages* k, const ibp_kv4_pages* v, uint32_t dtype, const ibp_kv_seqs* seqs, uint32_t T,
             const int32_t* n_rows, uint32_t* status, int device) {
  *r = {};
  int rc = view4_of(&r->p[0], k, device);
  if (rc == IBP_OK) rc = view4_of(&r->p[1], v, device);
  if (rc == IBP_OK) rc = check_seqs(seqs, k->page_tokens);
  if (rc != IBP_OK) return rc;
  if (dtype > IBP_KV_F16) return refuse("dtype is neither IBP_KV_BF16 nor IBP_KV_F16");
  if (!alike(k, v)) return refuse("k and v pages differ in shape");
  if (T == 0 || T > (1u << 30)) return refuse("T outside [1, 2^30]");
  r->table = seqs->table, r->lens = seqs->lens, r->n_rows = n_rows, r->status = status;
  if (!resolve(r->table, device, seqs->max_pages == 0) || !resolve(r->lens, device) ||
      !resolve(r->n_rows, device, true) || !resolve(r->status, device, true))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  r->n_seqs = seqs->n_seqs, r->max_pages = seqs->max_pages, r->n_pages = static_cast<uint32_t>(k->n_pages);
  r->page_tokens = k->page_tokens, r->T = T, r->heads = k->heads, r->dim = k->dim;
  r->f16 = dtype == IBP_KV_F16;
  return IBP_OK;
}

// Queries, lengths and masks, as ibp_tree_attention has them; pages are the caller's matter.
int queries_of(AttendArgs* a, uint32_t heads, uint32_t page_tokens, uint64_t n_pages, uint32_t dim, uint32_t dtype,
               const ibp_kv_seqs* seqs, const void* q, int64_t qs, int64_t qt, int64_t qh, uint32_t T, uint32_t q_heads,
               const int32_t* n_draft, const uint32_t* mask, float scale, uint32_t* status, int device) {
  const int rc = check_seqs(seqs, page_tokens);
  if (rc) return rc;
  if (dtype > IBP_KV_F16) return refuse("dtype is neither IBP_KV_BF16 nor IBP_KV_F16");
  if (T == 0 || T > 65535) return refuse("T outside [1, 65535]");
  if (q_heads == 0 || q_heads % heads || q_heads > 65535) return refuse("q_heads is not a multiple of the kv heads");
  if (!std::isfinite(scale)) return refuse("scale is not finite");
  if (static_cast<uint64_t>(seqs->n_seqs) * T * q_heads > 0x7FFFFFFFull) return refuse("2^31 query rows or more");
  a->q = static_cast<const char*>(q);
  a->table = seqs->table, a->lens = seqs->lens, a->n_live = n_draft, a->mask = mask, a->status = status;
  if (!resolve(a->q, device) || !resolve(a->table, device, seqs->max_pages == 0) || !resolve(a->lens, device) ||
      !resolve(a->n_live, device, true) || !resolve(a->mask, device, true) || !resolve(a->status, device, true))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  if (reinterpret_cast<uintptr_t>(a->q) % 4 || (static_cast<uint64_t>(qs) | static_cast<uint64_t>(qt) | static_cast<uint64_t>(qh)) % 2)
    return refuse("q is not 4-byte aligned in base and strides");
  a->q_seq = qs * 2, a->q_token = qt * 2, a->q_head = qh * 2;
  a->n_seqs = seqs->n_seqs, a->max_pages = seqs->max_pages;
  a->n_pages = static_cast<uint32_t>(n_pages);
  a->page_tokens = page_tokens;
  a->T = T, a->kv_heads = heads, a->group = q_heads / heads, a->dim = dim;
  a->mask_words = (T + 31) / 32;
  a->scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a->f16 = dtype == IBP_KV_F16;
  return IBP_OK;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Which kernel takes a call.  Rows: drafted tokens times query heads of a kv head.
// Measured (us, cold; few rows / tensor cores on codes / decoded once, then tensor cores),
// 8 ragged caches of up to 16384 tokens, 8 kv heads of 128: 16 rows 58 / 83 / 195, 24 rows
// 89 / 83 / 195, 64 rows 159 / 85 / 194, 128 rows 294 / 87 / 196, 256 rows - / 149 / 218, 512
// rows - / 263 / 298, 1024 rows - / 527 / 456; one cache of 65536 tokens: 16 rows 52 / 67, 24
// rows 71 / 67, 64 rows 116 / 67; 64 of up to 1024: 16 rows 59 / 95, 24 rows 97 / 97, 48 rows
// 136 / 95; one of 777: 64 rows 22 / 28.
// Decoding once wants scratch for the whole batch in 16 bits: not beyond 4 GB.
enum Path { kFew, kCodes, kDecoded };
constexpr uint64_t kFewRows = 16, kCodesRows = 512, kDecodedBytes = 4ull << 30;

Path path_of(uint32_t n_seqs, uint32_t kv_heads, uint64_t rows, uint32_t dim, uint64_t tokens, int device) {
  if (rows <= kFewRows || !kv4_tree_takes(n_seqs, kv_heads, rows, dim, tokens, device)) return kFew;
  return rows <= kCodesRows || kv4_expand_workspace(n_seqs, tokens, kv_heads, dim) > kDecodedBytes ? kCodes : kDecoded;
}

}  // namespace

extern "C" {

int ibp_kv4_store(const ibp_kv4_pages* k_pages, const ibp_kv4_pages* v_pages, uint32_t dtype, const ibp_kv_seqs* seqs,
                  const void* k, int64_t k_seq_stride, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                  int64_t v_seq_stride, int64_t v_token_stride, int64_t v_head_stride, uint32_t T, const int32_t* n_new,
                  uint32_t* status, void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  if (seqs && seqs->n_seqs == 0) return IBP_OK;
  Kv4Rows r;
  rc = rows4_of(&r, k_pages, v_pages, dtype, seqs, T, n_new, status, device);
  if (rc) return rc;
  const uint16_t *kk = static_cast<const uint16_t*>(k), *vv = static_cast<const uint16_t*>(v);
  if (!resolve(kk, device) || !resolve(vv, device)) return refuse("k or v is NULL, misaligned or not device-accessible");
  r.x[0] = reinterpret_cast<const char*>(kk), r.x[1] = reinterpret_cast<const char*>(vv);
  r.x_seq[0] = k_seq_stride * 2, r.x_token[0] = k_token_stride * 2, r.x_head[0] = k_head_stride * 2;
  r.x_seq[1] = v_seq_stride * 2, r.x_token[1] = v_token_stride * 2, r.x_head[1] = v_head_stride * 2;
  uint64_t all = 0;
  for (int i = 0; i < 2; ++i)
    all |= reinterpret_cast<uintptr_t>(r.x[i]) | static_cast<uint64_t>(r.x_seq[i]) | static_cast<uint64_t>(r.x_token[i]) |
           static_cast<uint64_t>(r.x_head[i]);
  r.vec = all % 16 == 0;
  return launch_kv4_store(r, device, static_cast<cudaStream_t>(stream));
}

int ibp_kv4_load(const ibp_kv4_pages* k_pages, const ibp_kv4_pages* v_pages, uint32_t dtype, const ibp_kv_seqs* seqs, uint32_t T,
                 const int32_t* n_load, void* k, void* v, uint32_t* status, void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  if (seqs && seqs->n_seqs == 0) return IBP_OK;
  Kv4Rows r;
  rc = rows4_of(&r, k_pages, v_pages, dtype, seqs, T, n_load, status, device);
  if (rc) return rc;
  char *kk = static_cast<char*>(k), *vv = static_cast<char*>(v);
  if (!resolve(kk, device) || !resolve(vv, device)) return refuse("k or v is NULL or not device-accessible");
  if ((reinterpret_cast<uintptr_t>(kk) | reinterpret_cast<uintptr_t>(vv)) % 16) return refuse("k or v is not 16-byte aligned");
  r.x[0] = kk, r.x[1] = vv;
  for (int i = 0; i < 2; ++i) {
    r.x_head[i] = static_cast<int64_t>(r.dim) * 2;
    r.x_token[i] = r.x_head[i] * r.heads;
    r.x_seq[i] = r.x_token[i] * T;
  }
  r.vec = 1;
  return launch_kv4_load(r, device, static_cast<cudaStream_t>(stream));
}

size_t ibp_kv4_attention_workspace(uint32_t n_seqs, uint32_t max_pages, uint32_t page_tokens, uint32_t T, uint32_t q_heads,
                                   uint32_t kv_heads, uint32_t dim) {
  if (kv_heads == 0 || q_heads % kv_heads || dim == 0 || dim > IBP_KV_MAX_DIM || page_tokens == 0) return 0;
  const uint64_t rows = static_cast<uint64_t>(T) * (q_heads / kv_heads), tokens = static_cast<uint64_t>(max_pages) * page_tokens;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) cudaGetLastError();
  const size_t few = kv4_attend_workspace(n_seqs, kv_heads, rows, dim, tokens, device);  // for scales below 0, too
  size_t many = 0;
  switch (path_of(n_seqs, kv_heads, rows, dim, tokens, device)) {
    case kFew: break;
    case kCodes: many = kv4_tree_workspace(dim, device); break;
    case kDecoded:
      many = kv4_expand_workspace(n_seqs, tokens, kv_heads, dim) +
             kv_tree_workspace(n_seqs, kv_heads, rows, dim, kExpand, (tokens + kExpand - 1) / kExpand * kExpand, device);
  }
  return few > many ? few : many;
}

int ibp_kv4_attention(const ibp_kv4_pages* k, const ibp_kv4_pages* v, uint32_t dtype, const ibp_kv_seqs* seqs, const void* q,
                      int64_t q_seq_stride, int64_t q_token_stride, int64_t q_head_stride, uint32_t T, uint32_t q_heads,
                      const int32_t* n_draft, const uint32_t* mask, float scale, void* out, float* lse, void* ws, size_t ws_bytes,
                      uint32_t* status, void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  if (seqs && seqs->n_seqs == 0) return IBP_OK;
  Attend4Args x = {};
  AttendArgs& a = x.a;
  rc = view4_of(&x.k, k, device);
  if (rc == IBP_OK) rc = view4_of(&x.v, v, device);
  if (rc) return rc;
  if (!alike(k, v)) return refuse("k and v pages differ in shape");
  rc = queries_of(&a, k->heads, k->page_tokens, k->n_pages, k->dim, dtype, seqs, q, q_seq_stride, q_token_stride, q_head_stride, T,
                  q_heads, n_draft, mask, scale, status, device);
  if (rc) return rc;
  a.out = out, a.lse = lse, a.part = static_cast<float*>(ws);
  if (!resolve(a.out, device) || !resolve(a.lse, device, true) || !resolve(a.part, device, true))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  if (reinterpret_cast<uintptr_t>(a.out) % 4) return refuse("out is not 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(a.part) % 16) return refuse("ws is not 16-byte aligned");
  const size_t need = ibp_kv4_attention_workspace(seqs->n_seqs, seqs->max_pages, k->page_tokens, T, q_heads, k->heads, k->dim);
  if (need && (ws_bytes < need || !ws)) return refuse("ws is smaller than ibp_kv4_attention_workspace");
  const uint64_t rows = static_cast<uint64_t>(T) * a.group, tokens = static_cast<uint64_t>(a.max_pages) * a.page_tokens;
  // The tensor-core kernel takes positive scales only.
  const Path path = a.scale_log2 > 0.f ? path_of(a.n_seqs, a.kv_heads, rows, a.dim, tokens, device) : kFew;
  if (path == kFew) return launch_kv4_attend(x, device, ws_bytes, static_cast<cudaStream_t>(stream));
  if (path == kCodes) return launch_kv4_tree(x, device, ws_bytes, static_cast<cudaStream_t>(stream));
  const uint64_t tiles = (tokens + kExpand - 1) / kExpand;
  const size_t pool = align256(a.n_seqs * tiles * kExpand * a.kv_heads * a.dim * 2);
  char* w = reinterpret_cast<char*>(a.part);
  Kv4Expanded e;
  e.table = reinterpret_cast<int32_t*>(w);
  w += align256(4 * a.n_seqs * tiles);
  e.lens = reinterpret_cast<int32_t*>(w);
  w += align256(4ull * a.n_seqs);
  e.k = w;
  w += pool;
  e.v = w;
  w += pool;
  rc = launch_kv4_expand(x, e, device, static_cast<cudaStream_t>(stream));
  if (rc) return rc;
  AttendArgs wide = a;
  const int64_t head = static_cast<int64_t>(kExpand) * a.dim * 2;
  wide.k = {e.k, head * a.kv_heads, a.kv_heads == 1 ? 0 : head, static_cast<int64_t>(a.dim) * 2};
  wide.v = {e.v, head * a.kv_heads, a.kv_heads == 1 ? 0 : head, static_cast<int64_t>(a.dim) * 2};
  wide.table = e.table, wide.lens = e.lens;
  wide.max_pages = static_cast<uint32_t>(tiles), wide.n_pages = static_cast<uint32_t>(a.n_seqs * tiles), wide.page_tokens = kExpand;
  wide.part = reinterpret_cast<float*>(w);
  bool done = false;
  rc = launch_kv_tree(wide, device, ws_bytes - (w - reinterpret_cast<char*>(a.part)), static_cast<cudaStream_t>(stream), &done);
  if (rc || done) return rc;
  set_detail("the tensor-core kernel refused decoded pages");
  return IBP_ECUDA;
}

int ibp_kv_verify(const float* p, int64_t p_seq_stride, int64_t p_row_stride, const float* q, int64_t q_seq_stride,
                  int64_t q_row_stride, uint32_t vocab, const int32_t* tokens, const int32_t* parents, const int32_t* n_draft,
                  uint32_t n_seqs, uint32_t T, const float* u, int32_t* path, int32_t* n_accept, int32_t* token, uint32_t* status,
                  void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  if (vocab == 0 || vocab > IBP_VERIFY_MAX_VOCAB) return refuse("vocab outside [1, IBP_VERIFY_MAX_VOCAB]");
  if (T > IBP_VERIFY_MAX_DRAFT) return refuse("T above IBP_VERIFY_MAX_DRAFT");
  if (n_seqs > 65535) return refuse("more than 65535 sequences");
  if (n_seqs == 0) return IBP_OK;
  VerifyArgs a = {};
  a.p = p, a.q = q, a.tokens = tokens, a.parents = parents, a.n_draft = n_draft, a.u = u;
  a.p_seq = p_seq_stride, a.p_row = p_row_stride, a.q_seq = q_seq_stride, a.q_row = q_row_stride;
  a.n_seqs = n_seqs, a.T = T, a.vocab = vocab;
  a.path = path, a.n_accept = n_accept, a.token = token, a.status = status;
  if (!resolve(a.p, device) || !resolve(a.q, device, true) || !resolve(a.tokens, device, T == 0) || !resolve(a.parents, device, true) ||
      !resolve(a.n_draft, device, true) || !resolve(a.u, device) || !resolve(a.path, device, T == 0) || !resolve(a.n_accept, device) ||
      !resolve(a.token, device) || !resolve(a.status, device, true))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  return launch_kv_verify(a, static_cast<cudaStream_t>(stream));
}

static int weigh(WeighArgs& x, const float* lse, const float* w, float* w_out, uint32_t width, float decay, int device, void* stream) {
  if (width > 0x7FFFFFFFu) return refuse("width is 2^31 or more");
  if (!std::isfinite(decay)) return refuse("decay is not finite");
  x.lse = lse, x.w = w, x.w_out = w_out, x.width = width, x.decay = decay;
  if (!resolve(x.lse, device) || !resolve(x.w, device, width == 0) || !resolve(x.w_out, device, width == 0))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  const size_t bytes = 4ull * x.a.n_seqs * width;
  const uintptr_t from = reinterpret_cast<uintptr_t>(x.w), to = reinterpret_cast<uintptr_t>(x.w_out);
  if (from != to && from < to + bytes && to < from + bytes) return refuse("w_out overlaps w without being w");
  if (width == 0) return IBP_OK;
  x.q16 = ((reinterpret_cast<uintptr_t>(x.a.q) | static_cast<uint64_t>(x.a.q_seq) | static_cast<uint64_t>(x.a.q_token) |
            static_cast<uint64_t>(x.a.q_head)) & 15u) == 0;
  return launch_kv_weigh(x, device, static_cast<cudaStream_t>(stream));
}

int ibp_kv_weigh(const ibp_kv_pages* k, uint32_t dtype, const ibp_kv_seqs* seqs, const void* q, int64_t q_seq_stride,
                 int64_t q_token_stride, int64_t q_head_stride, uint32_t T, uint32_t q_heads, const int32_t* n_draft,
                 const uint32_t* mask, float scale, const float* lse, const float* w, float* w_out, uint32_t width, float decay,
                 uint32_t* status, void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  if (seqs && seqs->n_seqs == 0) return IBP_OK;
  WeighArgs x = {};
  rc = view_of(&x.a.k, k, device);
  if (rc == IBP_OK)
    rc = queries_of(&x.a, k->heads, k->page_tokens, k->n_pages, k->dim, dtype, seqs, q, q_seq_stride, q_token_stride, q_head_stride,
                    T, q_heads, n_draft, mask, scale, status, device);
  if (rc) return rc;
  return weigh(x, lse, w, w_out, width, decay, device, stream);
}

int ibp_kv4_weigh(const ibp_kv4_pages* k, uint32_t dtype, const ibp_kv_seqs* seqs, const void* q, int64_t q_seq_stride,
                  int64_t q_token_stride, int64_t q_head_stride, uint32_t T, uint32_t q_heads, const int32_t* n_draft,
                  const uint32_t* mask, float scale, const float* lse, const float* w, float* w_out, uint32_t width, float decay,
                  uint32_t* status, void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  if (seqs && seqs->n_seqs == 0) return IBP_OK;
  WeighArgs x = {};
  rc = view4_of(&x.k4, k, device);
  if (rc == IBP_OK)
    rc = queries_of(&x.a, k->heads, k->page_tokens, k->n_pages, k->dim, dtype, seqs, q, q_seq_stride, q_token_stride, q_head_stride,
                    T, q_heads, n_draft, mask, scale, status, device);
  if (rc) return rc;
  return weigh(x, lse, w, w_out, width, decay, device, stream);
}

int ibp_kv_evict(const float* w, uint32_t width, const int32_t* lens, uint32_t n_seqs, uint32_t budget, uint32_t keep_first,
                 uint32_t keep_last, int32_t* path, int32_t* n_draft, int32_t* n_keep, float* w_out, uint32_t* status, void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  if (n_seqs > 65535) return refuse("more than 65535 sequences");
  if (width > 0x7FFFFF00u) return refuse("width above 2^31 - 256");
  if (budget == 0 || budget > 0x7FFFFFFFu || static_cast<uint64_t>(keep_first) + keep_last > budget)
    return refuse("budget is 0, or keep_first + keep_last is above it");
  if (n_seqs == 0) return IBP_OK;
  EvictArgs a = {};
  a.w = w, a.w_out = w_out, a.lens = lens, a.n_seqs = n_seqs, a.width = width, a.budget = budget;
  a.keep_first = keep_first, a.keep_last = keep_last, a.path = path, a.n_draft = n_draft, a.n_keep = n_keep, a.status = status;
  if (!resolve(a.w, device, width == 0) || !resolve(a.w_out, device, width == 0) || !resolve(a.lens, device) || !resolve(a.path, device) ||
      !resolve(a.n_draft, device) || !resolve(a.n_keep, device) || !resolve(a.status, device, true))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  const size_t bytes = 4ull * n_seqs * width;
  const uintptr_t from = reinterpret_cast<uintptr_t>(a.w), to = reinterpret_cast<uintptr_t>(a.w_out);
  if (bytes && from < to + bytes && to < from + bytes) return refuse("w_out overlaps w");
  return launch_kv_evict(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

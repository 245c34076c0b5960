// ibp_kv_api.cu - C ABI of the paged key/value cache operators: argument
// checks and pointer resolution.  Kernels live in the other ibp_kv_*.cu files.
#include <cuda_runtime.h>
#include <stdio.h>

#include <cmath>

#include "ibp_kv_args.cuh"

using namespace ibp;

namespace {

int meta_of(KvMeta* m, const ibp_kv_seqs* s, uint32_t page_tokens, const int32_t* refs, uint64_t n_pages,
            int32_t* table_out, int32_t* lens_out, int32_t* refs_out, uint32_t* status, int device,
            bool lens_read = true) {
  const int rc = check_seqs(s, page_tokens, lens_read);
  if (rc) return rc;
  if (n_pages == 0 || n_pages > kMaxPages) return refuse("n_pages outside [1, 2^31)");
  *m = {};
  m->table = s->table, m->lens = s->lens, m->refs = refs;
  m->n_seqs = s->n_seqs, m->max_pages = s->max_pages, m->page_tokens = page_tokens;
  m->n_pages = static_cast<uint32_t>(n_pages);
  m->table_out = table_out, m->lens_out = lens_out, m->refs_out = refs_out, m->status = status;
  const bool rows = s->n_seqs > 0, entries = rows && s->max_pages > 0;
  if (!resolve(m->table, device, !entries) || !resolve(m->lens, device, !rows || !lens_read) || !resolve(m->refs, device) ||
      !resolve(m->refs_out, device) || !resolve(m->status, device, true))
    return refuse("a table, length, reference or status pointer is misaligned or not device-accessible");
  return IBP_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && x < y + nb && y < x + na;
}

// Runs of the copying kernels: heads that lie next to one another in a token
// make one row, tokens that lie next to one another one run.
int runs_of(KvRuns* r, const ibp_kv_pages* p, int device) {
  if (!p || !p->data) return refuse("pages is NULL");
  const uint32_t es = p->elem_bytes;
  if (es != 1 && es != 2 && es != 4 && es != 8) return refuse("elem_bytes is not 1, 2, 4 or 8");
  if (p->n_pools == 0 || p->n_pages == 0 || p->n_pages > kMaxPages || p->heads == 0 || p->page_tokens == 0 ||
      p->page_tokens > 65536 || p->dim == 0)
    return refuse("a page dimension is 0 or too large");
  if (static_cast<uint64_t>(p->heads) * p->dim * es > (1u << 30)) return refuse("a token is larger than 2^30 bytes");
  if (p->page_stride < 0 || p->pool_stride < 0 || p->head_stride < 0 || p->token_stride < 0)
    return refuse("a stride is negative");
  char* data = static_cast<char*>(p->data);
  if (!resolve(data, device)) return refuse("pages are not device-accessible");
  *r = {};
  r->data = data;
  r->n_pools = p->n_pools;
  r->pool_stride = p->pool_stride * es;
  r->page_stride = p->page_stride * es;
  r->n_pages = static_cast<uint32_t>(p->n_pages);
  r->page_tokens = p->page_tokens;
  r->row_stride = p->token_stride * es;
  if (p->heads == 1 || p->head_stride == static_cast<int64_t>(p->dim)) {
    r->outer = 1;
    r->outer_stride = 0;
    r->row_bytes = p->heads * p->dim * es;
  } else {
    r->outer = p->heads;
    r->outer_stride = p->head_stride * es;
    r->row_bytes = p->dim * es;
  }
  if (p->page_tokens == 1) r->row_stride = r->row_bytes;
  uint64_t all = reinterpret_cast<uintptr_t>(data) | r->row_bytes | static_cast<uint64_t>(r->page_stride) |
                 static_cast<uint64_t>(r->row_stride) | static_cast<uint64_t>(r->outer_stride);
  if (p->n_pools > 1) all |= static_cast<uint64_t>(r->pool_stride);
  r->vec = all % 16 == 0 ? 16 : (all % 8 == 0 ? 8 : (all % 4 == 0 ? 4 : (all % 2 == 0 ? 2 : 1)));
  if (static_cast<uint64_t>(r->page_tokens) * (r->row_bytes / r->vec) > 0xFFFFFFFFull)
    return refuse("a page is too large");
  return IBP_OK;
}

int attend_of(AttendArgs* a, const ibp_kv_pages* k, const ibp_kv_pages* v, uint32_t dtype, const ibp_kv_seqs* seqs,
              const void* q, int64_t qs, int64_t qt, int64_t qh, uint32_t T, uint32_t q_heads, const int32_t* n_live,
              float scale, void* out, float* lse, void* ws, uint32_t* status, int device) {
  *a = {};
  int rc = view_of(&a->k, k, device);
  if (rc == IBP_OK) rc = view_of(&a->v, v, device);
  if (rc == IBP_OK) rc = check_seqs(seqs, k->page_tokens);
  if (rc != IBP_OK) return rc;
  if (dtype > IBP_KV_F16) return refuse("dtype is neither IBP_KV_BF16 nor IBP_KV_F16");
  if (k->n_pages != v->n_pages || k->heads != v->heads || k->page_tokens != v->page_tokens || k->dim != v->dim)
    return refuse("k and v pages differ in shape");
  if (T == 0 || T > 65535) return refuse("T outside [1, 65535]");
  if (q_heads == 0 || q_heads % k->heads || q_heads > 65535) return refuse("q_heads is not a multiple of the kv heads");
  if (!std::isfinite(scale)) return refuse("scale is not finite");
  if (static_cast<uint64_t>(seqs->n_seqs) * T * q_heads > 0x7FFFFFFFull) return refuse("2^31 query rows or more");
  a->q = static_cast<const char*>(q);
  a->out = out, a->lse = lse, a->part = static_cast<float*>(ws);
  a->table = seqs->table, a->lens = seqs->lens, a->n_live = n_live, a->status = status;
  if (!resolve(a->q, device) || !resolve(a->out, device) || !resolve(a->lse, device, true) ||
      !resolve(a->part, device, true) || !resolve(a->table, device, seqs->max_pages == 0) ||
      !resolve(a->lens, device) || !resolve(a->n_live, device, true) || !resolve(a->status, device, true))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  if ((reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->out)) % 4 ||
      (static_cast<uint64_t>(qs) | static_cast<uint64_t>(qt) | static_cast<uint64_t>(qh)) % 2)
    return refuse("q is not 4-byte aligned in base and strides, or out in base");
  if (reinterpret_cast<uintptr_t>(a->part) % 16) return refuse("ws is not 16-byte aligned");
  a->q_seq = qs * 2, a->q_token = qt * 2, a->q_head = qh * 2;
  a->n_seqs = seqs->n_seqs, a->max_pages = seqs->max_pages;
  a->n_pages = static_cast<uint32_t>(k->n_pages);
  a->page_tokens = k->page_tokens;
  a->T = T, a->kv_heads = k->heads, a->group = q_heads / k->heads, a->dim = k->dim;
  a->mask_words = (T + 31) / 32;
  a->scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a->f16 = dtype == IBP_KV_F16;
  return IBP_OK;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

extern "C" {

size_t ibp_kv_pages_workspace(uint64_t n_pages, uint32_t n_out) {
  return 4ull * (3 * n_pages + 2ull * n_out + 1);
}

int ibp_kv_fork(const ibp_kv_seqs* seqs, uint32_t page_tokens, const int32_t* refs, uint64_t n_pages,
                const int32_t* parents, uint32_t n_out, int32_t* table_out, int32_t* lens_out, int32_t* refs_out,
                int32_t* moves, int32_t* count, void* ws, size_t ws_bytes, uint32_t* status, void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  KvMeta m;
  rc = meta_of(&m, seqs, page_tokens, refs, n_pages, table_out, lens_out, refs_out, status, device);
  if (rc) return rc;
  if (n_out > 65535) return refuse("more than 65535 result rows");
  m.moves = moves, m.count = count, m.ws = static_cast<int32_t*>(ws);
  const bool rows = n_out > 0;
  if (!resolve(parents, device, !rows) || !resolve(m.table_out, device, !rows || !m.max_pages) ||
      !resolve(m.lens_out, device, !rows) || !resolve(m.moves, device, !rows) || !resolve(m.count, device) ||
      !resolve(m.ws, device))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  if (ws_bytes < ibp_kv_pages_workspace(n_pages, n_out)) return refuse("ws is smaller than ibp_kv_pages_workspace");
  const size_t row = 4ull * m.max_pages;
  if (overlap(m.table, row * m.n_seqs, m.table_out, row * n_out) ||
      overlap(m.lens, 4ull * m.n_seqs, m.lens_out, 4ull * n_out))
    return refuse("table_out or lens_out overlaps the present rows");
  return launch_kv_fork(m, parents, n_out, static_cast<cudaStream_t>(stream));
}

int ibp_kv_free(const ibp_kv_seqs* seqs, uint32_t page_tokens, const int32_t* refs, uint64_t n_pages,
                const int32_t* rows, uint32_t n_rows, int32_t* table_out, int32_t* lens_out, int32_t* refs_out,
                uint32_t* status, void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  KvMeta m;
  rc = meta_of(&m, seqs, page_tokens, refs, n_pages, table_out, lens_out, refs_out, status, device);
  if (rc) return rc;
  if (!resolve(rows, device, n_rows == 0) || !resolve(m.table_out, device, !m.n_seqs || !m.max_pages) ||
      !resolve(m.lens_out, device, !m.n_seqs))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  return launch_kv_free(m, rows, n_rows, static_cast<cudaStream_t>(stream));
}

int ibp_kv_compact(const ibp_kv_seqs* seqs, uint32_t page_tokens, const int32_t* refs, uint64_t n_pages,
                   int32_t* table_out, int32_t* refs_out, int32_t* moves, int32_t* count, void* ws, size_t ws_bytes,
                   uint32_t* status, void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  KvMeta m;
  // the references say which pages live
  rc = meta_of(&m, seqs, page_tokens, refs, n_pages, table_out, nullptr, refs_out, status, device, false);
  if (rc) return rc;
  m.moves = moves, m.count = count, m.ws = static_cast<int32_t*>(ws);
  if (!resolve(m.table_out, device, !m.n_seqs || !m.max_pages) || !resolve(m.moves, device) ||
      !resolve(m.count, device) || !resolve(m.ws, device))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  if (ws_bytes < ibp_kv_pages_workspace(n_pages, 0)) return refuse("ws is smaller than ibp_kv_pages_workspace");
  return launch_kv_compact(m, static_cast<cudaStream_t>(stream));
}

int ibp_kv_copy(const ibp_kv_pages* pages, const int32_t* moves, const int32_t* count, uint32_t max_moves,
                uint32_t* status, void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  KvRuns r;
  rc = runs_of(&r, pages, device);
  if (rc) return rc;
  if (max_moves == 0) return IBP_OK;
  if (!resolve(moves, device) || !resolve(count, device) || !resolve(status, device, true))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  return launch_kv_copy(r, moves, count, max_moves, status, device, static_cast<cudaStream_t>(stream));
}

int ibp_kv_accept(const ibp_kv_pages* pages, const ibp_kv_seqs* seqs, const int32_t* refs, const int32_t* n_draft,
                  const int32_t* path, const int32_t* n_accept, uint32_t max_accept, int32_t* table_out,
                  int32_t* lens_out, int32_t* refs_out, uint32_t* status, void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  KvRuns r;
  rc = runs_of(&r, pages, device);
  if (rc) return rc;
  KvMeta m;
  rc = meta_of(&m, seqs, pages->page_tokens, refs, pages->n_pages, table_out, lens_out, refs_out, status, device);
  if (rc) return rc;
  if (m.n_seqs == 0) {
    if (m.refs_out != m.refs) return refuse("no sequences: refs_out has to be refs");
    return IBP_OK;
  }
  if (!resolve(n_draft, device) || !resolve(path, device, max_accept == 0) || !resolve(n_accept, device) ||
      !resolve(m.table_out, device, !m.max_pages) || !resolve(m.lens_out, device))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  return launch_kv_accept(r, m, n_draft, path, n_accept, max_accept, device, static_cast<cudaStream_t>(stream));
}

size_t ibp_tree_attention_workspace(uint32_t n_seqs, uint32_t max_pages, uint32_t page_tokens, uint32_t T,
                                    uint32_t q_heads, uint32_t kv_heads, uint32_t dim) {
  if (kv_heads == 0 || q_heads % kv_heads || dim == 0 || dim > IBP_KV_MAX_DIM || page_tokens == 0) return 0;
  const uint64_t rows = static_cast<uint64_t>(T) * (q_heads / kv_heads), tokens = static_cast<uint64_t>(max_pages) * page_tokens;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) cudaGetLastError();
  const size_t few = kv_attend_workspace(static_cast<uint64_t>(n_seqs) * kv_heads, rows, dim, tokens, false, device);
  const size_t many = kv_tree_workspace(n_seqs, kv_heads, rows, dim, page_tokens, tokens, device);
  return few > many ? few : many;
}

int ibp_tree_attention(const ibp_kv_pages* k, const ibp_kv_pages* v, uint32_t dtype, const ibp_kv_seqs* seqs,
                       const void* q, int64_t q_seq_stride, int64_t q_token_stride, int64_t q_head_stride, uint32_t T,
                       uint32_t q_heads, const int32_t* n_draft, const uint32_t* mask, float scale, void* out,
                       float* lse, void* ws, size_t ws_bytes, uint32_t* status, void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  if (seqs && seqs->n_seqs == 0) return IBP_OK;
  AttendArgs a;
  rc = attend_of(&a, k, v, dtype, seqs, q, q_seq_stride, q_token_stride, q_head_stride, T, q_heads, n_draft, scale,
                 out, lse, ws, status, device);
  if (rc) return rc;
  a.mask = mask;
  if (!resolve(a.mask, device, true)) return refuse("mask is misaligned or not device-accessible");
  const size_t need = ibp_tree_attention_workspace(seqs->n_seqs, seqs->max_pages, k->page_tokens, T, q_heads, k->heads, k->dim);
  if (need && (ws_bytes < need || !ws))
    return refuse("ws is smaller than ibp_tree_attention_workspace");
  bool done = false;
  rc = launch_kv_tree(a, device, ws_bytes, static_cast<cudaStream_t>(stream), &done);
  if (rc || done) return rc;
  return launch_kv_attend(a, device, ws_bytes, static_cast<cudaStream_t>(stream));
}

uint64_t ibp_kv_set_wait_limit(uint64_t cycles) {
  return kv_tree_wait_limit(cycles < IBP_KV_WAIT_CYCLES ? cycles : IBP_KV_WAIT_CYCLES);
}

int ibp_kv_summarize(const ibp_kv_pages* k, uint32_t dtype, const ibp_kv_seqs* seqs, const int32_t* first,
                     int8_t* codes, float* scales, uint32_t* status, void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  KvView kv;
  rc = view_of(&kv, k, device);
  if (rc == IBP_OK) rc = check_seqs(seqs, k->page_tokens);
  if (rc) return rc;
  if (dtype > IBP_KV_F16) return refuse("dtype is neither IBP_KV_BF16 nor IBP_KV_F16");
  if (seqs->n_seqs == 0 || seqs->max_pages == 0) return IBP_OK;
  const int32_t *table = seqs->table, *lens = seqs->lens;
  if (!resolve(table, device) || !resolve(lens, device) || !resolve(first, device, true) || !resolve(codes, device) ||
      !resolve(scales, device) || !resolve(status, device, true))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  if (reinterpret_cast<uintptr_t>(codes) % 4) return refuse("codes is not 4-byte aligned");
  return launch_kv_summarize(kv, table, lens, first, seqs->n_seqs, seqs->max_pages, static_cast<uint32_t>(k->n_pages),
                             k->page_tokens, k->heads, k->dim, dtype == IBP_KV_F16, codes, scales, status, device,
                             static_cast<cudaStream_t>(stream));
}

size_t ibp_sparse_attention_workspace(uint32_t n_seqs, uint32_t max_pages, uint32_t page_tokens, uint32_t T,
                                      uint32_t q_heads, uint32_t kv_heads, uint32_t dim, uint32_t budget) {
  if (kv_heads == 0 || q_heads % kv_heads || dim == 0 || dim > IBP_KV_MAX_DIM) return 0;
  const uint64_t rows = static_cast<uint64_t>(n_seqs) * T * kv_heads;
  const uint64_t tokens = static_cast<uint64_t>(budget < max_pages ? budget : max_pages) * page_tokens;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) cudaGetLastError();
  const size_t scores = max_pages > budget ? align256(4 * rows * max_pages) : 0;
  return scores + align256(4 * rows * budget) + kv_attend_workspace(rows, q_heads / kv_heads, dim, tokens, true, device);
}

int ibp_sparse_attention(const ibp_kv_pages* k, const ibp_kv_pages* v, uint32_t dtype, const ibp_kv_seqs* seqs,
                         const int8_t* codes, const float* scales, const void* q, int64_t q_seq_stride,
                         int64_t q_token_stride, int64_t q_head_stride, uint32_t T, uint32_t q_heads,
                         const int32_t* n_query, uint32_t budget, uint32_t keep_first, uint32_t keep_last, float scale,
                         void* out, float* lse, int32_t* pages_out, void* ws, size_t ws_bytes, uint32_t* status,
                         void* stream) {
  clear_error_detail();
  int device;
  int rc = current_device(&device);
  if (rc) return rc;
  if (seqs && seqs->n_seqs == 0) return IBP_OK;
  AttendArgs a;
  rc = attend_of(&a, k, v, dtype, seqs, q, q_seq_stride, q_token_stride, q_head_stride, T, q_heads, n_query, scale,
                 out, lse, ws, status, device);
  if (rc) return rc;
  if (budget == 0 || budget > IBP_SPARSE_MAX_BUDGET) return refuse("budget outside [1, IBP_SPARSE_MAX_BUDGET]");
  if (keep_last == 0 || static_cast<uint64_t>(keep_first) + keep_last > budget)
    return refuse("keep_last is 0, or keep_first + keep_last is above the budget");
  if (static_cast<uint64_t>(a.group) * a.dim > 65536 || a.group > 256)
    return refuse("a group of more than 256 heads or 65536 elements");
  if (!resolve(codes, device) || !resolve(scales, device) || !resolve(pages_out, device, true))
    return refuse("a pointer is NULL, misaligned or not device-accessible");
  if (reinterpret_cast<uintptr_t>(codes) % 4) return refuse("codes is not 4-byte aligned");
  if (!ws || ws_bytes < ibp_sparse_attention_workspace(seqs->n_seqs, seqs->max_pages, k->page_tokens, T, q_heads,
                                                        k->heads, k->dim, budget))
    return refuse("ws is smaller than ibp_sparse_attention_workspace");
  const uint64_t rows = static_cast<uint64_t>(seqs->n_seqs) * T * k->heads;
  const size_t scores = seqs->max_pages > budget ? align256(4 * rows * seqs->max_pages) : 0;
  const size_t picks = align256(4 * rows * budget);
  char* w = reinterpret_cast<char*>(a.part);
  SelectArgs s = {};
  s.q = a.q, s.q_seq = a.q_seq, s.q_token = a.q_token, s.q_head = a.q_head;
  s.table = a.table, s.lens = a.lens, s.n_live = a.n_live, s.codes = codes, s.scales = scales;
  s.n_seqs = a.n_seqs, s.max_pages = a.max_pages, s.n_pages = a.n_pages, s.page_tokens = a.page_tokens;
  s.T = T, s.kv_heads = a.kv_heads, s.group = a.group, s.dim = a.dim;
  s.budget = budget, s.keep_first = keep_first, s.keep_last = keep_last;
  s.scores = reinterpret_cast<float*>(w);
  s.picks = pages_out ? pages_out : reinterpret_cast<int32_t*>(w + scores);
  s.status = a.status, s.f16 = a.f16;
  rc = launch_kv_select(s, device, static_cast<cudaStream_t>(stream));
  if (rc) return rc;
  a.picks = s.picks;
  a.budget = budget;
  a.part = reinterpret_cast<float*>(w + scores + picks);
  return launch_kv_attend(a, device, ws_bytes - scores - picks, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

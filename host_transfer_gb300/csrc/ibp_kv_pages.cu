// ibp_kv_pages.cu - forking, freeing, compacting and copying pages of a paged
// key/value cache, and keeping the accepted tokens of a draft.
//
// Bookkeeping (tables, lengths, reference counts) is a few kilobytes to a few
// megabytes of integers: each call is one CTA, or one cluster of eight for the
// larger ones, whose phases are separated by barriers instead of launches.  It is
// bound by the latency of its four or five dependent phases, not by bytes (a fork
// of 24 sequences in a pool of 128 pages 9.9 us, 12.5 in a cluster; a compaction
// 6.1, 9.0 in a cluster).  The copies that follow from it move gigabytes and
// fill the GPU: they are a kernel of their own, driven by a list in device memory,
// so nothing returns to the host in between.
#include <cuda_runtime.h>

#include "ibp_kv_internal.cuh"

namespace ibp {

constexpr uint32_t kClusterMax = 8;  // CTAs of a bookkeeping cluster (the portable size)
constexpr uint32_t kMt = 512;        // threads of each
constexpr uint64_t kOneCta = 16384;  // integers that one CTA handles by itself

__device__ __forceinline__ uint32_t cl_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// All threads of the cluster; global and shared writes before it are visible
// to the cluster after it.
template <uint32_t kCl>
__device__ __forceinline__ void cl_sync() {
  if (kCl == 1) {
    __syncthreads();
    return;
  }
  __threadfence();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// *p of CTA `rank` of the cluster, p in shared memory.
template <uint32_t kCl>
__device__ __forceinline__ uint32_t cl_read(const uint32_t* p, uint32_t rank) {
  if (kCl == 1) return *p;
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), v;
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Exclusive prefix count of `flag` over the CTA, and the CTA's total.
__device__ uint32_t block_rank(bool flag, uint32_t* warp_sums, uint32_t* total) {
  const uint32_t lane = threadIdx.x & 31u, w = threadIdx.x >> 5;
  const uint32_t b = __ballot_sync(0xFFFFFFFFu, flag);
  __syncthreads();
  if (lane == 0) warp_sums[w] = __popc(b);
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (uint32_t i = 0; i < kMt / 32; ++i) {
    const uint32_t s = warp_sums[i];
    before += i < w ? s : 0;
    all += s;
  }
  *total = all;
  return before + __popc(b & lanemask_lt());
}

// Pages [lo, hi) of this CTA's share of n, ascending with the rank.
template <uint32_t kCl>
__device__ __forceinline__ void slice(uint32_t n, uint32_t rank, uint32_t* lo, uint32_t* hi) {
  const uint32_t per = ceil_div(n, kCl);
  const uint64_t a = static_cast<uint64_t>(per) * rank;
  *lo = a < n ? static_cast<uint32_t>(a) : n;
  *hi = n - *lo > per ? *lo + per : n;
}

__device__ __forceinline__ int32_t ld_cg(const int32_t* p) { return __ldcg(p); }

struct MetaShared {
  uint32_t sums[kMt / 32];
  uint32_t count, count2;
};

// Copies what the outputs start from; nothing to do where they are the inputs.
template <uint32_t kCl>
__device__ void carry(int32_t* out, const int32_t* in, uint64_t n, uint32_t gt) {
  if (out == in) return;
  for (uint64_t i = gt; i < n; i += kCl * kMt) out[i] = in[i];
}

// ws: owner[n_pages] (lowest result row whose last, partly filled page it is),
// wants[n_out] (1: the row wants a copy), list[n_out] (rows that want one, in
// order), n_want.
template <uint32_t kCl>
__global__ void __launch_bounds__(kMt) k_kv_fork(const KvMeta m, const int32_t* __restrict__ parents,
                                                 uint32_t n_out) {
  __shared__ MetaShared sh;
  pdl_begin();
  const uint32_t rank = kCl == 1 ? 0 : cl_rank(), t = threadIdx.x, gt = rank * kMt + t, lane = t & 31u;
  const uint32_t gw = gt >> 5, n_warps = kCl * kMt / 32, P = m.max_pages;
  int32_t *owner = m.ws, *wants = owner + m.n_pages, *list = wants + n_out, *n_want = list + n_out;

  carry<kCl>(m.refs_out, m.refs, m.n_pages, gt);
  for (uint32_t i = gt; i < m.n_pages; i += kCl * kMt) owner[i] = 0x7FFFFFFF;
  for (uint64_t i = gt; i < 3ull * n_out; i += kCl * kMt) m.moves[i] = -1;
  cl_sync<kCl>();

  // The present rows give up their references; each last page finds its owner.
  for (uint32_t r = gw; r < m.n_seqs; r += n_warps) {
    const int32_t len = m.lens[r];
    if (len != clamp_len(len, m.page_tokens, P) && lane == 0) kv_status(m.status, IBP_ERANGE);
    const uint32_t np = held_pages(len, m.page_tokens, P);
    for (uint32_t p = lane; p < np; p += 32) {
      const uint32_t pg = static_cast<uint32_t>(m.table[static_cast<uint64_t>(r) * P + p]);
      if (pg >= m.n_pages)
        kv_status(m.status, IBP_ERANGE);
      else if (atomicSub(&m.refs_out[pg], 1) <= 0) {
        atomicAdd(&m.refs_out[pg], 1);
        kv_status(m.status, IBP_ECORRUPT);
      }
    }
  }
  for (uint32_t i = gt; i < n_out; i += kCl * kMt) {
    const uint32_t par = static_cast<uint32_t>(parents[i]);
    if (par >= m.n_seqs) {
      kv_status(m.status, IBP_ERANGE);
      continue;
    }
    const int32_t len = clamp_len(m.lens[par], m.page_tokens, P);
    if (len % m.page_tokens == 0) continue;
    const uint32_t pg = static_cast<uint32_t>(m.table[static_cast<uint64_t>(par) * P + len / m.page_tokens]);
    if (pg < m.n_pages) atomicMin(&owner[pg], static_cast<int32_t>(i));
  }
  cl_sync<kCl>();

  // The result rows take theirs.
  for (uint32_t i = gw; i < n_out; i += n_warps) {
    const uint32_t par = static_cast<uint32_t>(parents[i]);
    const int32_t len = par < m.n_seqs ? clamp_len(m.lens[par], m.page_tokens, P) : 0;
    const uint32_t np = held_pages(len, m.page_tokens, P), full = len / m.page_tokens;
    const int32_t* row = m.table + static_cast<uint64_t>(par < m.n_seqs ? par : 0) * P;
    bool want = false;
    if (full < np) {
      const uint32_t pg = static_cast<uint32_t>(row[full]);
      want = pg < m.n_pages && ld_cg(&owner[pg]) != static_cast<int32_t>(i);
    }
    for (uint32_t p = lane; p < P; p += 32) {
      int32_t pg = -1;
      if (p < np && !(want && p == full)) {
        pg = row[p];
        if (static_cast<uint32_t>(pg) < m.n_pages)
          atomicAdd(&m.refs_out[pg], 1);
        else
          pg = -1;
      }
      m.table_out[static_cast<uint64_t>(i) * P + p] = pg;
    }
    if (lane == 0) {
      m.lens_out[i] = len;
      wants[i] = want;
    }
  }
  cl_sync<kCl>();

  // Free pages of each CTA's share; the rows that want one, in order.
  uint32_t lo, hi;
  slice<kCl>(m.n_pages, rank, &lo, &hi);
  uint32_t mine = 0, total;
  for (uint32_t a = lo; a < hi; a += kMt) {
    block_rank(a + t < hi && ld_cg(&m.refs_out[a + t < hi ? a + t : lo]) == 0, sh.sums, &total);
    mine += total;
  }
  if (t == 0) sh.count = mine;
  if (rank == 0) {
    uint32_t n = 0;
    for (uint32_t a = 0; a < n_out; a += kMt) {
      const bool w = a + t < n_out && ld_cg(&wants[a + t < n_out ? a + t : 0]) != 0;
      const uint32_t at = block_rank(w, sh.sums, &total);
      if (w) list[n + at] = static_cast<int32_t>(a + t);
      n += total;
    }
    if (t == 0) *n_want = static_cast<int32_t>(n);
  }
  cl_sync<kCl>();

  // The r-th free page goes to the r-th of them.
  uint32_t base = 0, n_free = 0;
  for (uint32_t c = 0; c < kCl; ++c) {
    const uint32_t v = cl_read<kCl>(&sh.count, c);
    base += c < rank ? v : 0;
    n_free += v;
  }
  const uint32_t want_n = static_cast<uint32_t>(ld_cg(n_want));
  for (uint32_t a = lo; a < hi && base < want_n; a += kMt) {
    const uint32_t pg = a + t;
    const bool fr = pg < hi && ld_cg(&m.refs_out[pg < hi ? pg : lo]) == 0;
    const uint32_t at = base + block_rank(fr, sh.sums, &total);
    if (fr && at < want_n) {
      const uint32_t i = static_cast<uint32_t>(ld_cg(&list[at])), par = static_cast<uint32_t>(parents[i]);
      const int32_t len = clamp_len(m.lens[par], m.page_tokens, P);
      const uint32_t full = len / m.page_tokens;
      m.table_out[static_cast<uint64_t>(i) * P + full] = static_cast<int32_t>(pg);
      m.refs_out[pg] = 1;
      m.moves[3ull * at] = m.table[static_cast<uint64_t>(par) * P + full];
      m.moves[3ull * at + 1] = static_cast<int32_t>(pg);
      m.moves[3ull * at + 2] = len % m.page_tokens;
    }
    base += total;
  }
  if (rank == 0) {
    for (uint32_t at = n_free + t; at < want_n; at += kMt) {
      const int32_t i = ld_cg(&list[at]);
      m.lens_out[i] = ld_cg(&m.lens_out[i]) / static_cast<int32_t>(m.page_tokens) * static_cast<int32_t>(m.page_tokens);
      kv_status(m.status, IBP_ENOMEM);
    }
    if (t == 0) *m.count = static_cast<int32_t>(want_n < n_free ? want_n : n_free);
  }
  cl_sync<kCl>();  // no CTA leaves while another reads its shared memory
}

template <uint32_t kCl>
__global__ void __launch_bounds__(kMt) k_kv_free(const KvMeta m, const int32_t* __restrict__ rows, uint32_t n_rows) {
  pdl_begin();
  const uint32_t t = threadIdx.x, gt = (kCl == 1 ? 0 : cl_rank()) * kMt + t, lane = t & 31u;
  const uint32_t gw = gt >> 5, n_warps = kCl * kMt / 32, P = m.max_pages;
  carry<kCl>(m.refs_out, m.refs, m.n_pages, gt);
  carry<kCl>(m.lens_out, m.lens, m.n_seqs, gt);
  carry<kCl>(m.table_out, m.table, static_cast<uint64_t>(m.n_seqs) * P, gt);
  cl_sync<kCl>();
  for (uint32_t i = gw; i < n_rows; i += n_warps) {
    const uint32_t s = static_cast<uint32_t>(rows[i]);
    if (s >= m.n_seqs) {
      if (lane == 0) kv_status(m.status, IBP_ERANGE);
      continue;
    }
    // The first warp to take the length frees the row; a second listing finds 0.
    int32_t len = lane == 0 ? atomicExch(&m.lens_out[s], 0) : 0;
    len = __shfl_sync(0xFFFFFFFFu, len, 0);
    if (len == 0) continue;
    if (len != clamp_len(len, m.page_tokens, P) && lane == 0) kv_status(m.status, IBP_ERANGE);
    const uint32_t np = held_pages(len, m.page_tokens, P);
    int32_t* row = m.table_out + static_cast<uint64_t>(s) * P;
    for (uint32_t p = lane; p < P; p += 32) {
      const uint32_t pg = static_cast<uint32_t>(ld_cg(&row[p]));
      if (p < np) {
        if (pg >= m.n_pages)
          kv_status(m.status, IBP_ERANGE);
        else if (atomicSub(&m.refs_out[pg], 1) <= 0) {
          atomicAdd(&m.refs_out[pg], 1);
          kv_status(m.status, IBP_ECORRUPT);
        }
      }
      row[p] = -1;
    }
  }
}

// ws: to[n_pages] (new place of each page), from[n_pages] and into[n_pages]
// (moving pages and holes, in order).
template <uint32_t kCl>
__global__ void __launch_bounds__(kMt) k_kv_compact(const KvMeta m) {
  __shared__ MetaShared sh;
  pdl_begin();
  const uint32_t rank = kCl == 1 ? 0 : cl_rank(), t = threadIdx.x, gt = rank * kMt + t;
  int32_t *to = m.ws, *from = to + m.n_pages, *into = from + m.n_pages;
  uint32_t lo, hi, total;
  slice<kCl>(m.n_pages, rank, &lo, &hi);

  uint32_t mine = 0;
  for (uint32_t a = lo; a < hi; a += kMt) {
    block_rank(a + t < hi && m.refs[a + t < hi ? a + t : lo] > 0, sh.sums, &total);
    mine += total;
  }
  if (t == 0) sh.count = mine;
  for (uint64_t i = gt; i < 3ull * m.n_pages; i += kCl * kMt) m.moves[i] = -1;
  cl_sync<kCl>();
  uint32_t base = 0, n_live = 0;
  for (uint32_t c = 0; c < kCl; ++c) {
    const uint32_t v = cl_read<kCl>(&sh.count, c);
    base += c < rank ? v : 0;
    n_live += v;
  }
  // Ranks: a hole's is the number of free pages below it; a moving page's is
  // the number of live pages from n_live up to it, counted per share.
  uint32_t above = 0, seen = base;
  for (uint32_t a = lo; a < hi; a += kMt) {
    const uint32_t pg = a + t;
    const bool live = pg < hi && m.refs[pg < hi ? pg : lo] > 0;
    const uint32_t at = seen + block_rank(live, sh.sums, &total);
    if (pg < hi && !live && pg < n_live) into[pg - at] = static_cast<int32_t>(pg);
    seen += total;
    block_rank(live && pg >= n_live, sh.sums, &total);
    above += total;
  }
  if (t == 0) sh.count2 = above;
  cl_sync<kCl>();
  uint32_t mbase = 0, n_moves = 0;
  for (uint32_t c = 0; c < kCl; ++c) {
    const uint32_t v = cl_read<kCl>(&sh.count2, c);
    mbase += c < rank ? v : 0;
    n_moves += v;
  }
  for (uint32_t a = lo; a < hi; a += kMt) {
    const uint32_t pg = a + t;
    const int32_t refs = pg < hi ? m.refs[pg] : 0;
    const bool mv = refs > 0 && pg >= n_live;
    const uint32_t at = mbase + block_rank(mv, sh.sums, &total);
    if (pg < hi) to[pg] = mv ? ld_cg(&into[at]) : static_cast<int32_t>(pg);
    if (mv) from[at] = static_cast<int32_t>(pg);
    mbase += total;
  }
  cl_sync<kCl>();
  for (uint32_t i = gt; i < n_moves; i += kCl * kMt) {
    m.moves[3ull * i] = ld_cg(&from[i]);
    m.moves[3ull * i + 1] = ld_cg(&into[i]);
    m.moves[3ull * i + 2] = static_cast<int32_t>(m.page_tokens);
  }
  if (gt == 0) *m.count = static_cast<int32_t>(n_moves);
  // References follow: a moving page's own count is written by whoever holds
  // the pair, so that refs_out may be refs.
  for (uint32_t i = gt; i < n_moves; i += kCl * kMt) {
    const int32_t src = ld_cg(&from[i]), dst = ld_cg(&into[i]);
    m.refs_out[dst] = m.refs[src];
    m.refs_out[src] = 0;
  }
  if (m.refs_out != m.refs)
    for (uint32_t pg = gt; pg < m.n_pages; pg += kCl * kMt) {
      const int32_t v = m.refs[pg];
      const bool hole = v <= 0 && pg < n_live, mover = v > 0 && pg >= n_live;
      if (!hole && !mover) m.refs_out[pg] = v;
    }
  for (uint64_t i = gt; i < static_cast<uint64_t>(m.n_seqs) * m.max_pages; i += kCl * kMt) {
    const int32_t v = m.table[i];
    int32_t w = -1;
    if (v >= 0) {
      if (static_cast<uint32_t>(v) < m.n_pages)
        w = ld_cg(&to[v]);
      else
        kv_status(m.status, IBP_ERANGE);
    }
    m.table_out[i] = w;
  }
  cl_sync<kCl>();
}

// ---------------------------------------------------------------------------
// Copies

constexpr int kCpThreads = 256;
constexpr uint32_t kCpFly = 8;  // accesses a thread has in flight
constexpr uint32_t kAcFly = 4;  // the same where accepted tokens move: paths are short, threads many

// A run (one head's tokens of a page, or all heads' where they are
// contiguous) is copied in pieces of 8 accesses per lane by one warp; every
// lane loads its eight before it stores any, so a full SM keeps 64 KB and more
// in flight.  Bound by DRAM: each byte is read once and written once (2.5 GB of page
// moves: 337 us, 7.3 TB/s).
template <typename V>
__global__ void __launch_bounds__(kCpThreads) k_kv_copy(const KvRuns r, const int32_t* __restrict__ moves,
                                                        const int32_t* __restrict__ count, uint32_t max_moves,
                                                        uint32_t pieces, uint32_t* status) {
  pdl_begin();
  const uint32_t lane = threadIdx.x & 31u;
  const uint64_t gw = (static_cast<uint64_t>(blockIdx.x) * kCpThreads + threadIdx.x) >> 5;
  const uint64_t n_warps = (static_cast<uint64_t>(gridDim.x) * kCpThreads) >> 5;
  const int32_t c = *count;
  const uint32_t n = c < 0 ? 0 : (static_cast<uint32_t>(c) < max_moves ? c : max_moves);
  const uint64_t units = static_cast<uint64_t>(n) * r.n_pools * r.outer * pieces;
  const uint32_t vr = r.row_bytes / sizeof(V);  // accesses per token
  const bool packed = r.row_stride == r.row_bytes;
  for (uint64_t u = gw; u < units; u += n_warps) {
    const uint32_t piece = static_cast<uint32_t>(u % pieces);
    uint64_t x = u / pieces;
    const uint32_t o = static_cast<uint32_t>(x % r.outer);
    x /= r.outer;
    const uint64_t pool = x % r.n_pools;
    const uint32_t k = static_cast<uint32_t>(x / r.n_pools);
    const uint32_t src = static_cast<uint32_t>(moves[3ull * k]), dst = static_cast<uint32_t>(moves[3ull * k + 1]);
    const int32_t tk = moves[3ull * k + 2];
    if (src >= r.n_pages || dst >= r.n_pages) {
      if (lane == 0) kv_status(status, IBP_ERANGE);
      continue;
    }
    const uint32_t tokens = tk < 0 ? 0 : (static_cast<uint32_t>(tk) < r.page_tokens ? tk : r.page_tokens);
    const uint64_t total = static_cast<uint64_t>(tokens) * vr;
    const int64_t off = static_cast<int64_t>(pool) * r.pool_stride + static_cast<int64_t>(o) * r.outer_stride;
    const char* s = r.data + off + static_cast<int64_t>(src) * r.page_stride;
    char* d = r.data + off + static_cast<int64_t>(dst) * r.page_stride;
    const uint64_t at = static_cast<uint64_t>(piece) * (32 * kCpFly) + lane;
    if (packed) {
      V v[kCpFly];
#pragma unroll
      for (uint32_t i = 0; i < kCpFly; ++i)
        if (at + 32 * i < total) v[i] = __ldcs(reinterpret_cast<const V*>(s) + at + 32 * i);
#pragma unroll
      for (uint32_t i = 0; i < kCpFly; ++i)
        if (at + 32 * i < total) __stcs(reinterpret_cast<V*>(d) + at + 32 * i, v[i]);
    } else {
      V v[kCpFly];
      int64_t w[kCpFly];
#pragma unroll
      for (uint32_t i = 0; i < kCpFly; ++i) {
        const uint32_t e = static_cast<uint32_t>(at + 32 * i), row = e / vr;
        w[i] = static_cast<int64_t>(row) * r.row_stride + static_cast<int64_t>(e - row * vr) * sizeof(V);
        if (at + 32 * i < total) v[i] = __ldcs(reinterpret_cast<const V*>(s + w[i]));
      }
#pragma unroll
      for (uint32_t i = 0; i < kCpFly; ++i)
        if (at + 32 * i < total) __stcs(reinterpret_cast<V*>(d + w[i]), v[i]);
    }
  }
}

// Number of entries of path[b] that count: up to n_accept, ascending and below
// n_draft; *still: how many of them, from the first on, stay where they are.  One warp.
__device__ uint32_t valid_path(const int32_t* path, int32_t n_accept, uint32_t max_accept, int32_t n_draft,
                               bool* bad, uint32_t* still) {
  const uint32_t lane = threadIdx.x & 31u;
  uint32_t n = n_accept < 0 ? 0 : (static_cast<uint32_t>(n_accept) < max_accept ? n_accept : max_accept);
  *bad = n_accept < 0 || static_cast<uint32_t>(n_accept) > max_accept;
  *still = 0xFFFFFFFFu;
  for (uint32_t a = 0; a < n; a += 32) {
    const uint32_t j = a + lane;
    const int32_t x = j < n ? path[j] : 0;
    const bool wrong = j < n && (x < 0 || x >= n_draft || (j > 0 && x <= path[j - 1]));
    const uint32_t w = __ballot_sync(0xFFFFFFFFu, wrong), moved = __ballot_sync(0xFFFFFFFFu, j < n && x != static_cast<int32_t>(j));
    if (moved && *still == 0xFFFFFFFFu) *still = a + __ffs(moved) - 1;
    if (w) {
      *bad = true;
      n = a + __ffs(w) - 1;
    }
  }
  if (*still > n) *still = n;
  return n;
}

// Whether a page onto which a token of a draft moves is another sequence's, too.  Thread
// `nth` of `step` looks at every step-th page of the draft; the first is on its way while the
// path is read.
struct DraftPages {
  const KvMeta& m;
  uint64_t row;
  uint32_t page, step, id;
  __device__ __forceinline__ DraftPages(const KvMeta& m_, uint32_t b, int64_t ctx, int32_t len, uint32_t nth, uint32_t step_)
      : m(m_), row(static_cast<uint64_t>(b) * m_.max_pages), step(step_), id(0xFFFFFFFFu) {
    page = ctx < 0 ? 0xFFFFFFFFu : static_cast<uint32_t>(ctx) / m.page_tokens + nth;
    if (ctx >= 0 && static_cast<uint64_t>(page) * m.page_tokens < static_cast<uint64_t>(len)) id = static_cast<uint32_t>(m.table[row + page]);
  }
  __device__ __forceinline__ bool shared() const { return id < m.n_pages && m.refs[id] > 1; }
  // Of the pages of tokens from to `to` - 1 of the sequence; `one`: shared() of the first.
  __device__ __forceinline__ bool written(int64_t from, int64_t to, bool one) {
    if (from < 0 || from >= to) return false;
    const uint32_t lo = static_cast<uint32_t>(from) / m.page_tokens, hi = static_cast<uint32_t>(to - 1) / m.page_tokens;
    bool r = one && page >= lo && page <= hi;
    for (uint32_t p = page + step; p <= hi && p > page; p += step) {
      id = static_cast<uint32_t>(m.table[row + p]);
      r = r || (p >= lo && shared());
    }
    return r;
  }
};

// The CTAs of a sequence move the rows of its accepted tokens.  A thread takes
// one access-wide column of one run in one pool after another, four
// tokens of it at a time: it loads them all before it stores any.  Sources ascend and
// never lie below their targets, so a row is always read before it is
// overwritten, and only by the thread that overwrites it.  A sequence that would write a page
// which another holds as well is left alone; for 61 drafts of 24 finding out costs nothing that
// can be measured (33 us with and without).  Bound by the latency
// of two dependent accesses for short paths, by DRAM sectors for long ones.
template <typename V>
__global__ void __launch_bounds__(kCpThreads, 6) k_kv_accept_move(const KvRuns r, const KvMeta m,
                                                               const int32_t* __restrict__ n_draft,
                                                               const int32_t* __restrict__ path,
                                                               const int32_t* __restrict__ n_accept,
                                                               uint32_t max_accept) {
  __shared__ int64_t from[32], into[32];
  __shared__ uint32_t n_sh, still_sh;
  pdl_begin();
  const uint32_t b = blockIdx.y, t = threadIdx.x;
  const int32_t len = clamp_len(m.lens[b], m.page_tokens, m.max_pages), nd = n_draft[b];
  const int64_t ctx = static_cast<int64_t>(len) - nd;
  const int32_t* pb = path + static_cast<uint64_t>(b) * max_accept;
  DraftPages pages(m, b, t < 32 ? -1 : ctx, len, t - 32, kCpThreads - 32);  // by the warps that do not read the path
  bool one = false;
  if (t < 32) {
    bool bad;
    uint32_t still, n = valid_path(pb, n_accept[b], max_accept, nd, &bad, &still);
    if (nd < 0 || ctx < 0) n = 0;
    if (t == 0) n_sh = n, still_sh = still;
  } else {
    one = pages.shared();
  }
  __syncthreads();
  const uint32_t n = n_sh;
  // every CTA of the sequence, and the bookkeeping, come to the same answer from the same counts
  if (__syncthreads_or(t >= 32 && pages.written(ctx + still_sh, ctx + n, one))) return;
  const uint32_t cols = r.row_bytes / sizeof(V);
  const uint64_t columns = r.n_pools * r.outer * cols;
  for (uint32_t a = 0; a < n; a += 32) {
    __syncthreads();
    if (t < 32 && a + t < n) {
      const uint64_t row = static_cast<uint64_t>(b) * m.max_pages;
      const uint32_t p = static_cast<uint32_t>(ctx + pb[a + t]), q = static_cast<uint32_t>(ctx + a + t);
      const uint32_t ps = static_cast<uint32_t>(m.table[row + p / m.page_tokens]);
      const uint32_t qs = static_cast<uint32_t>(m.table[row + q / m.page_tokens]);
      const bool ok = ps < r.n_pages && qs < r.n_pages;
      if (!ok) kv_status(m.status, IBP_ERANGE);
      from[t] = ok && p != q ? ps * r.page_stride + static_cast<int64_t>(p % m.page_tokens) * r.row_stride : -1;
      into[t] = qs * r.page_stride + static_cast<int64_t>(q % m.page_tokens) * r.row_stride;
    }
    __syncthreads();
    const uint32_t e = n - a < 32 ? n - a : 32;
    for (uint64_t x = static_cast<uint64_t>(blockIdx.x) * kCpThreads + t; x < columns;
         x += static_cast<uint64_t>(gridDim.x) * kCpThreads) {
      const uint64_t y = x / cols;
      const uint32_t col = static_cast<uint32_t>(x - y * cols), o = static_cast<uint32_t>(y % r.outer);
      char* base = r.data + static_cast<int64_t>(y / r.outer) * r.pool_stride + static_cast<int64_t>(o) * r.outer_stride +
                   static_cast<int64_t>(col) * sizeof(V);
      for (uint32_t j = 0; j < e; j += kAcFly) {
        V v[kAcFly];
#pragma unroll
        for (uint32_t i = 0; i < kAcFly; ++i)
          if (j + i < e && from[j + i] >= 0) v[i] = *reinterpret_cast<const V*>(base + from[j + i]);
#pragma unroll
        for (uint32_t i = 0; i < kAcFly; ++i)
          if (j + i < e && from[j + i] >= 0) *reinterpret_cast<V*>(base + into[j + i]) = v[i];
      }
    }
  }
}

template <uint32_t kCl>
__global__ void __launch_bounds__(kMt) k_kv_accept_meta(const KvMeta m, const int32_t* __restrict__ n_draft,
                                                        const int32_t* __restrict__ path,
                                                        const int32_t* __restrict__ n_accept, uint32_t max_accept) {
  pdl_begin();
  // What is left of each of a warp's sequences, found before any reference is given up:
  // the counts that say whether a page is shared may be the ones that are changed.
  constexpr uint32_t kWarps = kMt / 32, kEach = kCl == 1 ? 1 : (65535 + kCl * kWarps - 1) / (kCl * kWarps);
  __shared__ int32_t left[kWarps][kEach];
  const uint32_t t = threadIdx.x, gt = (kCl == 1 ? 0 : cl_rank()) * kMt + t, lane = t & 31u;
  const uint32_t gw = gt >> 5, n_warps = kCl * kWarps, P = m.max_pages;
  carry<kCl>(m.refs_out, m.refs, m.n_pages, gt);
  for (uint32_t b = gw, i = 0; b < m.n_seqs; b += n_warps, ++i) {
    const int32_t raw = m.lens[b], len = clamp_len(raw, m.page_tokens, P), nd = n_draft[b];
    DraftPages pages(m, b, static_cast<int64_t>(len) - nd, len, lane, 32);
    bool bad;
    uint32_t still, n = valid_path(path + static_cast<uint64_t>(b) * max_accept, n_accept[b], max_accept, nd, &bad, &still);
    int32_t kept = len - nd + static_cast<int32_t>(n);
    if (nd < 0 || nd > len) {
      bad = true;
      kept = len;
    } else if (__any_sync(0xFFFFFFFFu, pages.written(static_cast<int64_t>(len) - nd + still, kept, pages.shared()))) {
      if (lane == 0) kv_status(m.status, IBP_EINVAL);
      kept = len;
    }
    if ((bad || raw != len) && lane == 0) kv_status(m.status, IBP_ERANGE);
    if (lane == 0) left[t >> 5][i] = kept;
  }
  cl_sync<kCl>();
  for (uint32_t b = gw, i = 0; b < m.n_seqs; b += n_warps, ++i) {
    const int32_t len = clamp_len(m.lens[b], m.page_tokens, P);
    // Lane 0 reads what it has written.  With the whole warp reading it the others got 0 (code of
    // nvcc 13.0.88, behind any barrier).
    const int32_t kept = __shfl_sync(0xFFFFFFFFu, lane == 0 ? left[t >> 5][i] : 0, 0);
    const uint32_t was = held_pages(len, m.page_tokens, P), now = held_pages(kept, m.page_tokens, P);
    for (uint32_t p = lane; p < P; p += 32) {
      const uint64_t at = static_cast<uint64_t>(b) * P + p;
      const int32_t pg = m.table[at];
      if (p >= now && p < was) {
        if (static_cast<uint32_t>(pg) >= m.n_pages)
          kv_status(m.status, IBP_ERANGE);
        else if (atomicSub(&m.refs_out[pg], 1) <= 0) {
          atomicAdd(&m.refs_out[pg], 1);
          kv_status(m.status, IBP_ECORRUPT);
        }
      }
      m.table_out[at] = p < now ? pg : -1;
    }
    if (lane == 0) m.lens_out[b] = kept;
  }
}

// ---------------------------------------------------------------------------

// One CTA's barriers cost less than a cluster's; past some ten thousand integers
// the work of one CTA costs more.
static bool one_cta(const KvMeta& m, uint32_t n_out) {
  return (static_cast<uint64_t>(m.n_seqs) + n_out) * m.max_pages + m.n_pages <= kOneCta;
}

int launch_kv_fork(const KvMeta& m, const int32_t* parents, uint32_t n_out, cudaStream_t stream) {
  if (one_cta(m, n_out))
    return kv_launch("k_kv_fork", k_kv_fork<1>, dim3(1), kMt, 0, 1, stream, m, parents, n_out);
  return kv_launch("k_kv_fork", k_kv_fork<kClusterMax>, dim3(kClusterMax), kMt, 0, kClusterMax, stream, m, parents, n_out);
}

int launch_kv_free(const KvMeta& m, const int32_t* rows, uint32_t n_rows, cudaStream_t stream) {
  if (one_cta(m, n_rows)) return kv_launch("k_kv_free", k_kv_free<1>, dim3(1), kMt, 0, 1, stream, m, rows, n_rows);
  return kv_launch("k_kv_free", k_kv_free<kClusterMax>, dim3(kClusterMax), kMt, 0, kClusterMax, stream, m, rows, n_rows);
}

int launch_kv_compact(const KvMeta& m, cudaStream_t stream) {
  if (one_cta(m, 0)) return kv_launch("k_kv_compact", k_kv_compact<1>, dim3(1), kMt, 0, 1, stream, m);
  return kv_launch("k_kv_compact", k_kv_compact<kClusterMax>, dim3(kClusterMax), kMt, 0, kClusterMax, stream, m);
}

int launch_kv_copy(const KvRuns& r, const int32_t* moves, const int32_t* count, uint32_t max_moves,
                   uint32_t* status, int device, cudaStream_t stream) {
  const uint64_t per_run = static_cast<uint64_t>(r.page_tokens) * (r.row_bytes / r.vec);
  const uint32_t pieces = static_cast<uint32_t>((per_run + 32 * kCpFly - 1) / (32 * kCpFly));
  const uint64_t warps = static_cast<uint64_t>(max_moves) * r.n_pools * r.outer * pieces;
  const uint64_t need = (warps * 32 + kCpThreads - 1) / kCpThreads, cap = 8ull * sm_count(device);
  const dim3 grid(static_cast<unsigned>(need < cap ? need : cap));
  auto go = [&](auto kern) {
    return kv_launch("k_kv_copy", kern, grid, kCpThreads, 0, 1, stream, r, moves, count, max_moves, pieces, status);
  };
  switch (r.vec) {
    case 16: return go(k_kv_copy<uint4>);
    case 8: return go(k_kv_copy<uint2>);
    case 4: return go(k_kv_copy<uint32_t>);
    case 2: return go(k_kv_copy<uint16_t>);
    default: return go(k_kv_copy<uint8_t>);
  }
}

int launch_kv_accept(const KvRuns& r, const KvMeta& m, const int32_t* n_draft, const int32_t* path,
                     const int32_t* n_accept, uint32_t max_accept, int device, cudaStream_t stream) {
  // Three rounds of CTAs: the lookups that a CTA begins with are four dependent
  // loads, so not many; but sequences keep from none to all of their draft, so more
  // than one.
  const uint64_t cols = r.n_pools * r.outer * (r.row_bytes / r.vec), want = (cols + kCpThreads - 1) / kCpThreads;
  const uint64_t cap = (24ull * sm_count(device) + m.n_seqs - 1) / m.n_seqs;
  const dim3 grid(static_cast<unsigned>(want < cap ? want : cap), m.n_seqs);
  int rc = IBP_OK;
  if (max_accept > 0) {
    auto go = [&](auto kern) {
      return kv_launch("k_kv_accept_move", kern, grid, kCpThreads, 0, 1, stream, r, m, n_draft, path, n_accept,
                       max_accept);
    };
    switch (r.vec) {
      case 16: rc = go(k_kv_accept_move<uint4>); break;
      case 8: rc = go(k_kv_accept_move<uint2>); break;
      case 4: rc = go(k_kv_accept_move<uint32_t>); break;
      case 2: rc = go(k_kv_accept_move<uint16_t>); break;
      default: rc = go(k_kv_accept_move<uint8_t>); break;
    }
  }
  if (rc != IBP_OK) return rc;
  if (one_cta(m, 0) && m.n_seqs <= kMt / 32)  // a warp a sequence
    return kv_launch("k_kv_accept_meta", k_kv_accept_meta<1>, dim3(1), kMt, 0, 1, stream, m, n_draft, path, n_accept,
                     max_accept);
  return kv_launch("k_kv_accept_meta", k_kv_accept_meta<kClusterMax>, dim3(kClusterMax), kMt, 0, kClusterMax, stream, m,
                   n_draft, path, n_accept, max_accept);
}

}  // namespace ibp

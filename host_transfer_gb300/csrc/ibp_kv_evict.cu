// ibp_kv_evict.cu - the tokens of a cache that stay when a budget is exceeded.
//
// A cluster takes a sequence, each CTA a stretch of its positions.  The weight at
// which the budget is full is found digit by digit from the top (three digits of 11,
// 11 and 10 bits of an order-preserving code): a histogram in shared memory, added up
// in the cluster's first CTA.  Positions with that very weight stay from the lowest on.  A second
// walk writes the kept positions and their weights at places known from the counts of
// the warps before.  Nothing depends on the order in which threads run.
//
// Measured on one GB300: 8 sequences of 2063 positions 17 us, 32 of 65521 down to 8192 36 us
// with cold caches (12.7 MB, 2 us at the copy rate).  Bound by latency: three digits of a
// histogram, its joining and two cluster barriers each, then the placing.  A CTA's lanes hold
// up to 8192 positions in registers, a cluster of eight 65536; what is longer is read again for
// every digit.  One CTA or eight, us: 8192 positions 32 sequences 24 / 22, 256 30 / 93;
// 16384 positions 32 sequences 46 / 24, 256 65 / 106; 32768 positions 32 sequences 85 / 28,
// 256 124 / 126.
//
// The move of what stays is ibp_kv_accept's (ibp_kv_pages.cu), which was made for drafts and
// walks a path 32 tokens at a time: 4 calls (codes and scales of K and V, 8 heads of 128) take
// 1.1 ms for the 8 sequences above and 8.0 ms for the 32 (604 MB, 89 us at the copy rate).
#include "ibp_kv_serve.cuh"

namespace ibp {

constexpr int kEvThreads = 512;
constexpr uint32_t kEvWarps = kEvThreads / 32;
constexpr uint32_t kEvBins = 2048;

// Larger weights have larger codes; both zeros are alike, and NaN is below all.
__device__ __forceinline__ uint32_t weight_code(float w) {
  if (w != w) return 0u;
  uint32_t b = __float_as_uint(w);
  if (b == 0x80000000u) b = 0u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct EvictShared {
  uint32_t hist[kEvBins];     // of this CTA
  uint32_t all[kEvBins];      // of the cluster, in its first CTA
  uint32_t digit, above;      // the bin found, and how many lie above it
  uint32_t run[kEvWarps];
  uint32_t n_more[kEvWarps], n_equal[kEvWarps];
  uint32_t cta_more, cta_equal;
};

constexpr uint32_t kEvHold = 16;  // codes of a lane: sequences of up to 8192 positions a CTA are read once

__device__ __forceinline__ uint32_t remote_u32(const uint32_t* p, uint32_t rank) {
  uint32_t addr = smem_u32(p), v;
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(addr) : "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void remote_store(uint32_t* p, uint32_t rank, uint32_t x) {
  uint32_t addr = smem_u32(p);
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(addr) : "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ void remote_add(uint32_t* p, uint32_t rank, uint32_t x) {
  uint32_t addr = smem_u32(p);
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(addr) : "r"(rank));
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}

template <uint32_t C>
__device__ __forceinline__ void ev_sync() {
  if (C == 1)
    __syncthreads();
  else
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <uint32_t C>
__global__ void __launch_bounds__(kEvThreads) k_kv_evict(const EvictArgs a) {
  __shared__ EvictShared sh;
  pdl_begin();
  const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
  const uint32_t rank = C == 1 ? 0 : blockIdx.x % C, b = blockIdx.x / C;
  const int32_t raw = a.lens[b];
  const uint32_t len = raw < 0 ? 0u : (static_cast<uint32_t>(raw) < a.width ? static_cast<uint32_t>(raw) : a.width);
  if (static_cast<int64_t>(raw) != static_cast<int64_t>(len) && rank == 0 && tid == 0) kv_status(a.status, IBP_ERANGE);
  const float* w = a.w + static_cast<uint64_t>(b) * a.width;
  float* out = a.w_out + static_cast<uint64_t>(b) * a.width;
  int32_t* path = a.path + static_cast<uint64_t>(b) * a.budget;
  // A sequence longer than its weights is left alone: the path would name positions of the
  // part that has weights, and ibp_kv_accept goes by the whole length.
  const bool over = len > a.budget && raw == static_cast<int32_t>(len);
  if (rank == 0 && tid == 0) {
    a.n_draft[b] = over ? static_cast<int32_t>(len) : 0;
    a.n_keep[b] = over ? static_cast<int32_t>(a.budget) : 0;
  }
  const uint32_t me = rank * kEvThreads + tid;
  if (!over) {  // the same for the whole cluster
    for (uint32_t i = me; i < a.width; i += C * kEvThreads) out[i] = i < len ? w[i] : 0.f;
    for (uint32_t i = me; i < a.budget; i += C * kEvThreads) path[i] = -1;
    return;
  }
  for (uint32_t i = a.budget + me; i < a.width; i += C * kEvThreads) out[i] = 0.f;
  // Positions that do not stay in any case: [lo, hi); keep_first + keep_last <= budget < len.
  const uint32_t lo = a.keep_first, hi = len - a.keep_last, want = a.budget - a.keep_first - a.keep_last;
  const uint32_t part = (len + C * kEvWarps * 32 - 1) / (C * kEvWarps * 32) * 32;  // of a warp
  auto clip = [&](uint32_t x) { return x < len ? x : len; };
  const uint32_t from = clip((rank * kEvWarps + warp) * part), to = clip(from + part);

  // Codes of 16 positions a lane at a time: kind() of 0 goes for positions outside the walk.
  uint32_t held[kEvHold];
  const bool once = part <= 32 * kEvHold;
  auto read = [&](uint32_t at) {
#pragma unroll
    for (uint32_t u = 0; u < kEvHold; ++u) {
      const uint32_t i = at + 32 * u + lane;
      held[u] = i < to ? weight_code(__ldg(w + i)) : 0u;
    }
  };
  if (once) read(from);
  for (uint32_t i = tid; i < kEvBins; i += kEvThreads) sh.hist[i] = sh.all[i] = 0;
  ev_sync<C>();

  // The code at which `want` are reached, and how many above it.
  uint32_t prefix = 0, left = want;
  if (want) {
#pragma unroll 1
    for (uint32_t d = 0; d < 3; ++d) {
      const uint32_t shift = d == 0 ? 21 : (d == 1 ? 10 : 0), bins = d == 2 ? 1024 : 2048;
      const uint32_t known = d == 0 ? 0u : 0xFFFFFFFFu << (d == 1 ? 21 : 10);
      for (uint32_t at = from; at < to; at += 32 * kEvHold) {
        if (!once) read(at);
#pragma unroll
        for (uint32_t u = 0; u < kEvHold; ++u) {
          const uint32_t i = at + 32 * u + lane;
          if (i >= lo && i < hi && i < to && (held[u] & known) == prefix) atomicAdd(&sh.hist[(held[u] >> shift) & (bins - 1)], 1u);
        }
      }
      __syncthreads();
      // counts come together in the first CTA; most bins are empty
      for (uint32_t i = tid; i < bins; i += kEvThreads) {
        const uint32_t n = sh.hist[i];
        if (n) {
          if (C == 1)
            sh.all[i] = n;
          else
            remote_add(&sh.all[i], 0, n);
          sh.hist[i] = 0;
        }
      }
      ev_sync<C>();
      if (rank == 0) {
        // from the highest bin down: a thread has bins / kEvThreads of them
        const uint32_t per = bins / kEvThreads, top = bins - tid * per;
        uint32_t n[4], sum = 0;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          n[i] = i < per ? sh.all[top - 1 - i] : 0u;
          sum += n[i];
        }
        uint32_t run = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, run, o);
          if (static_cast<int>(lane) >= o) run += y;
        }
        if (lane == 31) sh.run[warp] = run;
        __syncthreads();
        for (uint32_t x = 0; x < warp; ++x) run += sh.run[x];
        uint32_t above = run - sum;
        if (above < left && left <= run) {  // one thread
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) {
            if (above < left && left <= above + n[i]) {
              for (uint32_t r = 0; r < C; ++r) {
                if (C == 1) {
                  sh.digit = top - 1 - i, sh.above = above;
                } else {
                  remote_store(&sh.digit, r, top - 1 - i);
                  remote_store(&sh.above, r, above);
                }
              }
            }
            above += n[i];
          }
        }
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
          if (i < per) sh.all[top - 1 - i] = 0;
      }
      ev_sync<C>();
      prefix |= sh.digit << shift;
      left -= sh.above;
    }
  }
  // left: how many of the positions with the code `prefix` stay
  auto kind = [&](uint32_t i, uint32_t c) -> uint32_t {  // 2 stays, 1 has the last weight, 0 goes
    if (i >= to) return 0u;
    if (i < lo || i >= hi) return 2u;
    if (!want) return 0u;
    return c > prefix ? 2u : (c == prefix ? 1u : 0u);
  };
  uint32_t more = 0, equal = 0;
  for (uint32_t at = from; at < to; at += 32 * kEvHold) {
    if (!once) read(at);
#pragma unroll
    for (uint32_t u = 0; u < kEvHold; ++u) {
      const uint32_t k = kind(at + 32 * u + lane, held[u]);
      more += __popc(__ballot_sync(0xFFFFFFFFu, k == 2u));
      equal += __popc(__ballot_sync(0xFFFFFFFFu, k == 1u));
    }
  }
  if (lane == 0) sh.n_more[warp] = more, sh.n_equal[warp] = equal;
  __syncthreads();
  if (tid == 0) {
    uint32_t m = 0, e = 0;
    for (uint32_t x = 0; x < kEvWarps; ++x) m += sh.n_more[x], e += sh.n_equal[x];
    sh.cta_more = m, sh.cta_equal = e;
  }
  ev_sync<C>();
  uint32_t before_more = 0, before_equal = 0;
  if constexpr (C > 1)
    for (uint32_t r = 0; r < rank; ++r) before_more += remote_u32(&sh.cta_more, r), before_equal += remote_u32(&sh.cta_equal, r);
  for (uint32_t x = 0; x < warp; ++x) before_more += sh.n_more[x], before_equal += sh.n_equal[x];
  const uint32_t lt = lanemask_lt();
  for (uint32_t at = from; at < to; at += 32 * kEvHold) {
    if (!once) read(at);
#pragma unroll
    for (uint32_t u = 0; u < kEvHold; ++u) {
      const uint32_t i = at + 32 * u + lane, k = kind(i, held[u]);
      const uint32_t eq = __ballot_sync(0xFFFFFFFFu, k == 1u), mo = __ballot_sync(0xFFFFFFFFu, k == 2u);
      const uint32_t e = before_equal + __popc(eq & lt), m = before_more + __popc(mo & lt);
      if (k == 2u || (k == 1u && e < left)) {
        const uint32_t to_place = m + (e < left ? e : left);
        path[to_place] = static_cast<int32_t>(i);
        out[to_place] = __ldg(w + i);
      }
      before_equal += __popc(eq);
      before_more += __popc(mo);
    }
  }
  if (C > 1) ev_sync<C>();  // no CTA leaves while another reads its counts
}

int launch_kv_evict(const EvictArgs& a, cudaStream_t stream) {
  if (a.width <= (a.n_seqs > 128 ? 16384u : 8192u)) return kv_launch("k_kv_evict", k_kv_evict<1>, dim3(a.n_seqs), kEvThreads, 0, 1, stream, a);
  return kv_launch("k_kv_evict", k_kv_evict<8>, dim3(a.n_seqs * 8), kEvThreads, 0, 8, stream, a);
}

}  // namespace ibp

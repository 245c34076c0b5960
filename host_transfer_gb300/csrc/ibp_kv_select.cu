// ibp_kv_select.cu - 8-bit bounds of a page's keys, and the selection of pages
// by the score of those bounds for each query.
//
// The score is an upper estimate of q . k over the page: each dimension takes
// the bound that its query's sign asks for.  With codes of 8 bits on both
// sides the sum is whole-number arithmetic, so every split, order and GPU
// selects the same pages.  The sum over a group's heads needs no loop over
// them: total = (sum_g max(c, 0)) . max + (sum_g min(c, 0)) . min, so one pair
// of 16-bit vectors per query and kv head meets the page's 8-bit codes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "ibp_kv_internal.cuh"

namespace ibp {

constexpr int kSumThreads = 256;
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ float2 pair_f32(uint32_t v, bool f16) {
  return f16 ? __half22float2(*reinterpret_cast<__half2*>(&v))
             : __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&v));
}

// NaN if either is, so that a page with one shows it.
template <bool F16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (F16)
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (F16)
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 127 * (1 / a), each operation rounded: the codes are the same wherever they
// are computed in this order.
__device__ __forceinline__ float code_factor(float a) { return __fmul_rn(__frcp_rn(a), 127.f); }

__device__ __forceinline__ bool finite_f(float x) { return fabsf(x) <= 3.402823466e38f; }

// A warp takes one head of one page: each lane holds the minima and maxima of
// eight dimensions over every (32 / (dim / 8))-th token and the lanes of a
// dimension meet at the end.  Bound by DRAM: the keys are read once, 16 bytes a
// lane with eight loads in flight (737 MB: 117 us, 6.3 TB/s).
template <bool F16>
__global__ void __launch_bounds__(kSumThreads)
    k_kv_summarize(const KvView k, const int32_t* __restrict__ table, const int32_t* __restrict__ lens,
                   const int32_t* __restrict__ first, uint32_t max_pages, uint32_t n_pages, uint32_t page_tokens,
                   uint32_t heads, uint32_t dim, int8_t* __restrict__ codes, float* __restrict__ scales,
                   uint32_t* status) {
  pdl_begin();
  const uint32_t b = blockIdx.y, lane = threadIdx.x & 31u;
  const int32_t raw = lens[b], len = clamp_len(raw, page_tokens, max_pages);
  if (raw != len && blockIdx.x == 0 && threadIdx.x == 0) kv_status(status, IBP_ERANGE);
  int32_t f = first ? first[b] : 0;
  f = f < 0 ? 0 : f;
  const uint32_t p0 = static_cast<uint32_t>(f) / page_tokens, p1 = held_pages(len, page_tokens, max_pages);
  if (f >= len || p0 >= p1) return;
  const uint64_t units = static_cast<uint64_t>(p1 - p0) * heads;
  const uint32_t cpr = dim / 8, rows = 32 / cpr;
  const uint32_t col = lane % cpr, row0 = lane / cpr;
  constexpr uint32_t kFly = 8;
  for (uint64_t u = static_cast<uint64_t>(blockIdx.x) * (kSumThreads / 32) + (threadIdx.x >> 5); u < units;
       u += static_cast<uint64_t>(gridDim.x) * (kSumThreads / 32)) {
    const uint32_t h = static_cast<uint32_t>(u % heads), p = p0 + static_cast<uint32_t>(u / heads);
    const uint32_t pg = static_cast<uint32_t>(table[static_cast<uint64_t>(b) * max_pages + p]);
    if (pg >= n_pages) {
      if (lane == 0) kv_status(status, IBP_ERANGE);
      continue;
    }
    const uint32_t left = static_cast<uint32_t>(len) - p * page_tokens;
    const uint32_t n = left < page_tokens ? left : page_tokens;
    const char* src = k.data + static_cast<int64_t>(pg) * k.page_stride + static_cast<int64_t>(h) * k.head_stride +
                      col * 16;
    const uint32_t pinf = F16 ? 0x7C007C00u : 0x7F807F80u, ninf = pinf | 0x80008000u;
    uint4 lo = make_uint4(pinf, pinf, pinf, pinf), hi = make_uint4(ninf, ninf, ninf, ninf);
    if (row0 < rows) {
      for (uint32_t r = row0; r < n; r += rows * kFly) {
        uint4 x[kFly];
#pragma unroll
        for (uint32_t i = 0; i < kFly; ++i) {
          // a row past the end repeats the first one: it changes no bound
          const uint32_t rr = r + i * rows < n ? r + i * rows : r;
          x[i] = __ldcs(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(rr) * k.token_stride));
        }
#pragma unroll
        for (uint32_t i = 0; i < kFly; ++i) {
          lo.x = min2<F16>(lo.x, x[i].x), lo.y = min2<F16>(lo.y, x[i].y);
          lo.z = min2<F16>(lo.z, x[i].z), lo.w = min2<F16>(lo.w, x[i].w);
          hi.x = max2<F16>(hi.x, x[i].x), hi.y = max2<F16>(hi.y, x[i].y);
          hi.z = max2<F16>(hi.z, x[i].z), hi.w = max2<F16>(hi.w, x[i].w);
        }
      }
    }
    for (uint32_t i = 1; i < rows; ++i) {  // lanes of row group 0 collect the others
      const uint32_t from = col + i * cpr;
      uint4 a, c;
      a.x = __shfl_sync(0xFFFFFFFFu, lo.x, from), a.y = __shfl_sync(0xFFFFFFFFu, lo.y, from);
      a.z = __shfl_sync(0xFFFFFFFFu, lo.z, from), a.w = __shfl_sync(0xFFFFFFFFu, lo.w, from);
      c.x = __shfl_sync(0xFFFFFFFFu, hi.x, from), c.y = __shfl_sync(0xFFFFFFFFu, hi.y, from);
      c.z = __shfl_sync(0xFFFFFFFFu, hi.z, from), c.w = __shfl_sync(0xFFFFFFFFu, hi.w, from);
      if (row0 == 0) {
        lo.x = min2<F16>(lo.x, a.x), lo.y = min2<F16>(lo.y, a.y), lo.z = min2<F16>(lo.z, a.z);
        lo.w = min2<F16>(lo.w, a.w);
        hi.x = max2<F16>(hi.x, c.x), hi.y = max2<F16>(hi.y, c.y), hi.z = max2<F16>(hi.z, c.z);
        hi.w = max2<F16>(hi.w, c.w);
      }
    }
    float l8[8], h8[8], amax = 0.f;
    bool bad = false;
    const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = pair_f32(lw[i], F16), c = pair_f32(hw[i], F16);
      l8[2 * i] = a.x, l8[2 * i + 1] = a.y, h8[2 * i] = c.x, h8[2 * i + 1] = c.y;
    }
    if (row0 == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        bad = bad || !finite_f(l8[i]) || !finite_f(h8[i]);
        amax = fmaxf(amax, fmaxf(fabsf(l8[i]), fabsf(h8[i])));
      }
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    const bool fine = !bad && amax >= kTiny;
    const float inv = fine ? code_factor(amax) : 0.f;
    const uint64_t at = static_cast<uint64_t>(pg) * heads + h;
    if (row0 == 0) {
      uint32_t w[4] = {0, 0, 0, 0};  // minima then maxima, four codes a word
      if (fine) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int cl = max(-127, min(127, __float2int_rn(__fmul_rn(l8[i], inv))));
          const int ch = max(-127, min(127, __float2int_rn(__fmul_rn(h8[i], inv))));
          w[i / 4] |= static_cast<uint32_t>(cl & 0xFF) << (8 * (i % 4));
          w[2 + i / 4] |= static_cast<uint32_t>(ch & 0xFF) << (8 * (i % 4));
        }
      }
      uint32_t* dst = reinterpret_cast<uint32_t*>(codes + at * 2 * dim);
      dst[2 * col] = w[0], dst[2 * col + 1] = w[1];
      dst[dim / 4 + 2 * col] = w[2], dst[dim / 4 + 2 * col + 1] = w[3];
    }
    if (lane == 0) scales[at] = bad ? __int_as_float(0x7F800000) : (fine ? __fmul_rn(amax, 1.f / 127.f) : 0.f);
  }
}

int launch_kv_summarize(const KvView& k, const int32_t* table, const int32_t* lens, const int32_t* first,
                        uint32_t n_seqs, uint32_t max_pages, uint32_t n_pages, uint32_t page_tokens, uint32_t heads,
                        uint32_t dim, uint32_t f16, int8_t* codes, float* scales, uint32_t* status, int device,
                        cudaStream_t stream) {
  // Two units a warp fill the longest sequence; at most 32 CTAs per SM in all,
  // so that a step that touches one page each does not launch empty CTAs by the
  // ten thousand.
  const uint64_t units = static_cast<uint64_t>(max_pages) * heads;
  const uint64_t want = (units + 2 * (kSumThreads / 32) - 1) / (2 * (kSumThreads / 32));
  const uint64_t cap = (32ull * sm_count(device) + n_seqs - 1) / n_seqs;
  const dim3 grid(static_cast<unsigned>(want < cap ? want : cap), n_seqs);
  auto go = [&](auto kern) {
    return kv_launch("k_kv_summarize", kern, grid, kSumThreads, 0, 1, stream, k, table, lens, first, max_pages,
                     n_pages, page_tokens, heads, dim, codes, scales, status);
  };
  return f16 ? go(k_kv_summarize<true>) : go(k_kv_summarize<false>);
}

// ---------------------------------------------------------------------------
// Scores

constexpr int kScThreads = 256;

__device__ __forceinline__ int dp2a(uint32_t a16, uint32_t b8, int c, bool high) {
  int d;
  if (high)
    asm("dp2a.hi.s32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a16), "r"(b8), "r"(c));
  else
    asm("dp2a.lo.s32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a16), "r"(b8), "r"(c));
  return d;
}

// Position of query t of sequence b, or -1 where there is no such query.  A count
// above T is cut to it, as the attention does: both have to place a query alike,
// for the attention reads as many entries of its list as its place calls for.
__device__ __forceinline__ int32_t query_place(const SelectArgs& a, uint32_t b, uint32_t t, int32_t len) {
  const int32_t T = static_cast<int32_t>(a.T), raw = a.n_live ? a.n_live[b] : T, n = raw < T ? raw : T;
  if (static_cast<int32_t>(t) >= n) return -1;
  const int32_t p = len - n + static_cast<int32_t>(t);
  return p < 0 ? -1 : p;
}

// CTA (sequence, block of NQ queries and share of the pages; kv head):
// quantises its queries into shared memory, then scores its share of the pages.
// LPP lanes hold a page's codes, 16 each (minima in the lower lanes, maxima in
// the upper), four or eight pages a lane group in flight, and the queries' 16 sums for the
// same dimensions stay in registers.  One query is summed over its lanes by a
// butterfly; eight are by a halving exchange that leaves each lane one query's
// total, 7 to 9 shuffles for the eight.  Bound by the latency of two dependent
// loads and the start of each CTA: 32 tokens over up to 1024 pages and 8 heads
// (45 MB of codes) 18 us, 1022 tokens over up to 512 pages and 4 heads 23 us.
// pages a lane group has in flight
template <int NQ>
constexpr uint32_t kScFly = NQ == 1 ? 8 : 4;

template <int NQ, int LPP>
__global__ void __launch_bounds__(kScThreads, NQ == 1 ? 4 : 2) k_kv_score(const SelectArgs a, uint32_t q_blocks, uint32_t shares) {
  extern __shared__ uint32_t sq[];  // NQ x dim words of two 16-bit sums: min part, max part
  __shared__ int32_t place[NQ];
  __shared__ uint32_t most;
  __shared__ float tops[kScThreads / 32];
  pdl_begin();
  const uint32_t h = blockIdx.y, share = blockIdx.x % shares, bq = blockIdx.x / shares;
  const uint32_t b = bq / q_blocks, t0 = bq % q_blocks * NQ;
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const int32_t len = clamp_len(a.lens[b], a.page_tokens, a.max_pages);
  if (threadIdx.x == 0) most = 0;
  __syncthreads();
  if (threadIdx.x < NQ) {
    const uint32_t t = t0 + threadIdx.x;
    const int32_t p = t < a.T ? query_place(a, b, t, len) : -1;
    // a query that sees no more pages than its budget takes them all unscored
    const uint32_t n = p < 0 ? 0 : static_cast<uint32_t>(p) / a.page_tokens + 1;
    place[threadIdx.x] = n > a.budget ? p : -1;
    if (n > a.budget) atomicMax(&most, n);
  }
  __syncthreads();
  const uint32_t n_pages = most;
  if (n_pages == 0) return;
  constexpr uint32_t kPer = 32 / LPP, kFly = kScFly<NQ>;  // pages a warp instruction, and in flight
  const uint32_t sub = lane % LPP;
  const bool on = sub * 8 < a.dim;  // lanes past a dimension that is no power of two idle
  const bool wide = (reinterpret_cast<uintptr_t>(a.codes) & 15u) == 0;
  const int32_t* row = a.table + static_cast<uint64_t>(b) * a.max_pages;
  uint4 c[kFly];
  float scale[kFly];
  auto fetch = [&](uint32_t p0) {
    uint32_t pg[kFly];
#pragma unroll
    for (uint32_t u = 0; u < kFly; ++u) {
      const uint32_t p = p0 + u * kPer + lane / LPP;
      pg[u] = p < n_pages ? static_cast<uint32_t>(row[p]) : 0u;
    }
#pragma unroll
    for (uint32_t u = 0; u < kFly; ++u) {
      const uint32_t p = p0 + u * kPer + lane / LPP;
      c[u] = make_uint4(0, 0, 0, 0);
      scale[u] = 0.f;
      if (p < n_pages && pg[u] < a.n_pages) {
        const uint64_t at = static_cast<uint64_t>(pg[u]) * a.kv_heads + h;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(a.codes + at * 2 * a.dim) + sub * 4;
        if (on) c[u] = wide ? *reinterpret_cast<const uint4*>(src) : make_uint4(src[0], src[1], src[2], src[3]);
        scale[u] = a.scales[at];
      } else if (p < n_pages && sub == 0) {
        kv_status(a.status, IBP_ERANGE);
      }
    }
  };
  const uint32_t step = kScThreads / 32 * kPer * kFly * shares;
  const uint32_t start = (share * (kScThreads / 32) + warp) * kPer * kFly;
  if (start < n_pages) fetch(start);  // on their way while the queries are quantised
  const uint32_t nd = a.dim / 2;  // words of two elements
  // kTeam threads a query: its largest element, then the sums of its codes.
  constexpr uint32_t kTeam = kScThreads / NQ;
  {
    const uint32_t i = threadIdx.x / kTeam, me = threadIdx.x % kTeam, words = a.group * nd;
    const char* q = a.q + static_cast<int64_t>(b) * a.q_seq + static_cast<int64_t>(t0 + i) * a.q_token +
                    static_cast<int64_t>(h) * a.group * a.q_head;
    const bool is = place[i] >= 0;
    float amax = 0.f;
    bool bad = false;
    if (is)
#pragma unroll 4
      for (uint32_t x = me; x < words; x += kTeam) {
        const uint32_t g = x / nd;
        const float2 v = pair_f32(*reinterpret_cast<const uint32_t*>(q + static_cast<int64_t>(g) * a.q_head + 4 * (x - g * nd)), a.f16);
        bad = bad || !finite_f(v.x) || !finite_f(v.y);
        amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
      }
    if (bad) amax = __int_as_float(0x7F800000);
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if (kTeam > 32) {
      if (lane == 0) tops[warp] = amax;
      __syncthreads();
#pragma unroll
      for (uint32_t w = 0; w < kScThreads / 32; ++w) amax = fmaxf(amax, tops[w]);
    }
    const float inv = finite_f(amax) && amax >= kTiny ? code_factor(amax) : 0.f;
    for (uint32_t w = me; w < nd; w += kTeam) {
      int lx = 0, ly = 0, hx = 0, hy = 0;
      if (inv != 0.f)
#pragma unroll 4
        for (uint32_t g = 0; g < a.group; ++g) {
          const float2 v = pair_f32(*reinterpret_cast<const uint32_t*>(q + static_cast<int64_t>(g) * a.q_head + 4 * w), a.f16);
          const int x = max(-127, min(127, __float2int_rn(__fmul_rn(v.x, inv))));
          const int y = max(-127, min(127, __float2int_rn(__fmul_rn(v.y, inv))));
          lx += min(x, 0), ly += min(y, 0), hx += max(x, 0), hy += max(y, 0);
        }
      sq[i * a.dim + w] = (lx & 0xFFFF) | (static_cast<uint32_t>(ly) << 16);
      sq[i * a.dim + nd + w] = (hx & 0xFFFF) | (static_cast<uint32_t>(hy) << 16);
    }
  }
  __syncthreads();
  uint32_t qw[NQ][8];
#pragma unroll
  for (int i = 0; i < NQ; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) qw[i][e] = on ? sq[i * a.dim + sub * 8 + e] : 0u;
  for (uint32_t p0 = start; p0 < n_pages; p0 += step) {
    if (p0 != start) fetch(p0);
#pragma unroll
    for (uint32_t u = 0; u < kFly; ++u) {
      const uint32_t p = p0 + u * kPer + lane / LPP;
      int s[NQ];
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        int x = 0;
        x = dp2a(qw[i][0], c[u].x, x, false), x = dp2a(qw[i][1], c[u].x, x, true);
        x = dp2a(qw[i][2], c[u].y, x, false), x = dp2a(qw[i][3], c[u].y, x, true);
        x = dp2a(qw[i][4], c[u].z, x, false), x = dp2a(qw[i][5], c[u].z, x, true);
        x = dp2a(qw[i][6], c[u].w, x, false), x = dp2a(qw[i][7], c[u].w, x, true);
        s[i] = x;
      }
      // After the exchanges over lane bits LPP/2, LPP/4, ... a lane holds the
      // query whose number its bits spell (as many bits as queries need).
      uint32_t mine = 0;
      int left = NQ;
#pragma unroll
      for (uint32_t o = LPP / 2; o; o >>= 1) {
        if (left > 1) {
          const bool up = lane & o;
#pragma unroll
          for (int i = 0; i < NQ / 2; ++i)
            if (i < left / 2) {
              const int give = up ? s[i] : s[i + left / 2], keep = up ? s[i + left / 2] : s[i];
              s[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
            }
          left /= 2;
          mine += up ? left : 0;
        } else {
          s[0] += __shfl_xor_sync(0xFFFFFFFFu, s[0], o);
        }
      }
      // lanes that still hold `left` queries each (fewer lanes than queries), and
      // one lane of those that hold the same
      const bool writes = LPP >= NQ ? (sub % (LPP / (LPP < NQ ? LPP : NQ))) == 0 : true;
      if (writes && p < n_pages)
#pragma unroll
        for (int i = 0; i < NQ; ++i)
          if (i < left && place[mine + i] >= 0)
            a.scores[((static_cast<uint64_t>(b) * a.T + t0 + mine + i) * a.kv_heads + h) * a.max_pages + p] =
                finite_f(scale[u]) ? __fmul_rn(__int2float_rn(s[i]), scale[u]) : __int_as_float(0x7F800000);
    }
  }
}

// ---------------------------------------------------------------------------
// Selection

constexpr uint32_t kSelShared = 8192;  // scores held in shared memory; more are read from L2 on every pass

// Whole-number key in the order of the score; +0 and -0 are equal.
__device__ __forceinline__ uint32_t order_key(float s) {
  const uint32_t u = __float_as_uint(s == 0.f ? 0.f : s);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One CTA per query and kv head.  The threshold key comes from passes of an
// 8-bit histogram over the scores that are neither forced nor hidden, and ends
// early when a digit's keys are all wanted (two passes, as a rule); then each
// warp counts what it takes in its own stretch of pages and writes it, ascending,
// behind the warps before it.  Bound by the latency of its passes (256 rows of up
// to 1024 pages 9 us, 4088 rows of up to 512 19 us).
template <int NT>
__global__ void __launch_bounds__(NT) k_kv_select(const SelectArgs a, uint32_t key_cap) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[256], sums[2][NT / 32], sh_digit, sh_left, sh_all;
  pdl_begin();
  const uint64_t row = blockIdx.x;
  const uint64_t bt = row / a.kv_heads;
  const uint32_t t = static_cast<uint32_t>(bt % a.T), b = static_cast<uint32_t>(bt / a.T), tid = threadIdx.x;
  const uint32_t lane = tid & 31u, warp = tid >> 5;
  const int32_t raw = a.lens[b], len = clamp_len(raw, a.page_tokens, a.max_pages);
  const int32_t place = query_place(a, b, t, len);
  if (tid == 0) {
    const int32_t nl = a.n_live ? a.n_live[b] : static_cast<int32_t>(a.T);
    if (raw != len || nl > len || nl < 0 || nl > static_cast<int32_t>(a.T)) kv_status(a.status, IBP_ERANGE);
  }
  int32_t* out = a.picks + row * a.budget;
  const uint32_t n = place < 0 ? 0 : static_cast<uint32_t>(place) / a.page_tokens + 1;
  if (n <= a.budget) {
    for (uint32_t i = tid; i < a.budget; i += NT) out[i] = i < n ? static_cast<int32_t>(i) : -1;
    return;
  }
  // here keep_first + keep_last <= budget < n: the two forced ranges are apart
  const uint32_t f0 = a.keep_first, f1 = n - a.keep_last;
  const float* scores = a.scores + row * a.max_pages;
  const bool held = n <= key_cap;
  for (uint32_t i = tid; i < 256; i += NT) hist[i] = 0;
  __syncthreads();
  uint32_t left = a.budget - a.keep_first - a.keep_last;  // to be taken by score
  const bool any = left > 0;
  // keys at or above `prefix` with its low bits clear: `left` of those equal in
  // the high bits `high`
  uint32_t prefix = 0, high = 0;
  bool all = false;  // every key equal in the high bits is taken
  if (any) {
    for (int shift = 24; shift >= 0 && !all; shift -= 8) {
      for (uint32_t i = f0 + tid; i < f1; i += NT) {
        uint32_t k;
        if (shift == 24) {
          k = order_key(scores[i]);
          if (held) keys[i] = k;
        } else {
          k = held ? keys[i] : order_key(scores[i]);
        }
        if ((k & high) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (warp == 0) {  // lane l holds the digits 8l .. 8l+7; counts from the top
        uint32_t d8[8], mine = 0;
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
          d8[i] = hist[8 * lane + i];
          hist[8 * lane + i] = 0;
          mine += d8[i];
        }
        uint32_t above = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_down_sync(0xFFFFFFFFu, above, o);
          if (lane + o < 32) above += v;
        }
        above -= mine;  // keys of higher lanes
        if (above < left && above + mine >= left) {
          uint32_t acc = above;
          bool found = false;
#pragma unroll
          for (int d = 7; d >= 0; --d) {
            if (!found && acc + d8[d] >= left) {
              found = true;
              sh_digit = 8 * lane + d;
              sh_left = left - acc;
              sh_all = left - acc == d8[d];
            }
            acc += d8[d];
          }
        }
      }
      __syncthreads();
      prefix |= sh_digit << shift;
      high |= 255u << shift;
      left = sh_left;
      all = sh_all != 0;
    }
  }
  // Each warp's stretch: counts of taken pages and of ties, then their places.
  const uint32_t per = ceil_div(ceil_div(n, NT / 32), 32) * 32;
  const uint32_t w0 = warp * per < n ? warp * per : n, w1 = n - w0 < per ? n : w0 + per;
  auto kind = [&](uint32_t i, bool* take, bool* tie) {
    *take = *tie = false;
    if (i >= w1) return;
    if (i < f0 || i >= f1) {
      *take = true;
    } else if (any) {
      const uint32_t k = held ? keys[i] : order_key(scores[i]);
      const uint32_t kh = k & high;
      *take = kh > prefix || (all && kh == prefix);
      *tie = !all && kh == prefix;
    }
  };
  uint32_t n_take = 0, n_tie = 0;
  for (uint32_t i = w0; i < w1; i += 32) {
    bool take, tie;
    kind(i + lane, &take, &tie);
    n_take += __popc(__ballot_sync(0xFFFFFFFFu, take));
    n_tie += __popc(__ballot_sync(0xFFFFFFFFu, tie));
  }
  if (lane == 0) sums[0][warp] = n_take, sums[1][warp] = n_tie;
  __syncthreads();
  uint32_t at = 0, ties = 0;
  for (uint32_t w = 0; w < warp; ++w) at += sums[0][w], ties += sums[1][w];
  at += ties < left ? ties : left;
  for (uint32_t i = w0; i < w1; i += 32) {
    bool take, tie;
    kind(i + lane, &take, &tie);
    const uint32_t tm = __ballot_sync(0xFFFFFFFFu, tie);
    take = take || (tie && ties + __popc(tm & lanemask_lt()) < left);
    ties += __popc(tm);
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, take);
    const uint32_t to = at + __popc(m & lanemask_lt());
    if (take && to < a.budget) out[to] = static_cast<int32_t>(i + lane);
    at += __popc(m);
  }
}

template <int NQ>
static int launch_score(const SelectArgs& a, int device, cudaStream_t stream) {
  const uint32_t q_blocks = (a.T + NQ - 1) / NQ;
  uint32_t lpp = 1;
  while (lpp * 8 < a.dim) lpp <<= 1;
  // Shares of at least one step, as many as the GPU holds at once.
  const uint32_t per_cta = kScThreads / 32 * (32 / lpp) * kScFly<NQ>;
  const uint64_t want = (a.max_pages + per_cta - 1) / per_cta;
  const uint64_t rows = static_cast<uint64_t>(a.kv_heads) * a.n_seqs * q_blocks;
  const uint64_t cap = (NQ == 1 ? 4ull : 2ull) * sm_count(device) / rows;
  const uint32_t shares = static_cast<uint32_t>(cap < 1 ? 1 : (want < cap ? want : cap));
  const dim3 grid(a.n_seqs * q_blocks * shares, a.kv_heads);
  auto go = [&](auto kern) {
    return kv_launch("k_kv_score", kern, grid, kScThreads, NQ * a.dim * 4, 1, stream, a, q_blocks, shares);
  };
  switch (lpp) {
    case 1: return go(k_kv_score<NQ, 1>);
    case 2: return go(k_kv_score<NQ, 2>);
    case 4: return go(k_kv_score<NQ, 4>);
    case 8: return go(k_kv_score<NQ, 8>);
    case 16: return go(k_kv_score<NQ, 16>);
    default: return go(k_kv_score<NQ, 32>);
  }
}

int launch_kv_select(const SelectArgs& a, int device, cudaStream_t stream) {
  int rc = IBP_OK;
  // Eight queries share a CTA's reading of the codes; a single token would leave
  // seven of the eight sums idle.
  if (a.max_pages > a.budget) rc = a.T == 1 ? launch_score<1>(a, device, stream) : launch_score<8>(a, device, stream);
  if (rc != IBP_OK) return rc;
  const uint32_t cap = a.max_pages < kSelShared ? a.max_pages : kSelShared;
  const dim3 grid(a.n_seqs * a.T * a.kv_heads);
  // A wide CTA shortens the passes over many pages.  Rows by the thousand finish
  // sooner a warp each, without barriers between warps.
  const uint32_t sms = sm_count(device);
  if (a.max_pages > 512 && grid.x <= 4 * sms)
    return kv_launch("k_kv_select", k_kv_select<512>, grid, 512, 4ull * cap, 1, stream, a, cap);
  if (a.max_pages <= 1024 && grid.x >= 16 * sms)
    return kv_launch("k_kv_select", k_kv_select<32>, grid, 32, 4ull * cap, 1, stream, a, cap);
  return kv_launch("k_kv_select", k_kv_select<128>, grid, 128, 4ull * cap, 1, stream, a, cap);
}

}  // namespace ibp

// ibp_kv4.cu - tokens into and out of paged caches held in 4 bits.
//
// A thread takes 8 elements (16 bytes) and four threads a group of 32, so that
// the largest magnitude is two exchanges and every access of a warp is a run of
// whole sectors.  Bound by DRAM for prompts (2 bytes read and 9/16 written an
// element, or the other way), by latency for single tokens.
#include "ibp_kv4.cuh"

namespace ibp {

constexpr int kRowThreads = 256;

struct Row8 {  // eight elements of a row: which tensor, sequence, token, head, chunk
  uint32_t b, t, h, c, which;
};

__device__ __forceinline__ Row8 row8_of(const Kv4Rows& r, uint64_t x) {
  Row8 e;
  const uint32_t chunks = r.dim / 8;
  e.c = static_cast<uint32_t>(x % chunks);
  x /= chunks;
  e.h = static_cast<uint32_t>(x % r.heads);
  x /= r.heads;
  e.t = static_cast<uint32_t>(x % r.T);
  x /= r.T;
  e.b = static_cast<uint32_t>(x % r.n_seqs);
  e.which = static_cast<uint32_t>(x / r.n_seqs);
  return e;
}

// The page and slot of row t of a sequence; page 2^32 - 1 where there is none.
struct Spot {
  uint32_t page, slot;
};
__device__ __forceinline__ Spot spot_of(const Kv4Rows& r, uint32_t b, uint32_t t) {
  Spot s = {0xFFFFFFFFu, 0u};
  const int32_t raw = r.lens[b], len = clamp_len(raw, r.page_tokens, r.max_pages);
  const int32_t want = r.n_rows ? r.n_rows[b] : static_cast<int32_t>(r.T);
  const int32_t n = want < 0 ? 0 : (want > static_cast<int32_t>(r.T) ? static_cast<int32_t>(r.T) : want);
  if (raw != len || want != n || n > len) kv_status(r.status, IBP_ERANGE);
  const int32_t pos = len - n + static_cast<int32_t>(t);
  if (static_cast<int32_t>(t) >= n || pos < 0) return s;
  const uint32_t nth = static_cast<uint32_t>(pos) / r.page_tokens;
  const uint32_t page = static_cast<uint32_t>(r.table[static_cast<uint64_t>(b) * r.max_pages + nth]);
  if (page >= r.n_pages) {
    kv_status(r.status, IBP_ERANGE);
    return s;
  }
  s.page = page;
  s.slot = static_cast<uint32_t>(pos) - nth * r.page_tokens;
  return s;
}

__device__ __forceinline__ char* codes_at(const Kv4View& v, const Spot& s, uint32_t h, uint32_t c) {
  return const_cast<char*>(v.codes) + static_cast<int64_t>(s.page) * v.page_stride + static_cast<int64_t>(h) * v.head_stride +
         static_cast<int64_t>(s.slot) * v.token_stride + c * 4;
}
__device__ __forceinline__ char* scale_at(const Kv4View& v, const Spot& s, uint32_t h, uint32_t c) {
  return const_cast<char*>(v.scales) + static_cast<int64_t>(s.page) * v.s_page + static_cast<int64_t>(h) * v.s_head +
         static_cast<int64_t>(s.slot) * v.s_token + c / 4 * 2;
}

// Scale of a group from its largest magnitude: a / 7 to 5 significant bits, ties to
// even, as bits of the type.  The division and the rounding are exact roundings, so the
// result does not depend on who computes it.
template <bool F16>
__device__ __forceinline__ uint32_t scale_of(float a) {
  uint32_t b = __float_as_uint(__fdiv_rn(a, 7.f));
  b = (b + 0x3FFFFu + ((b >> 19) & 1u)) & 0xFFF80000u;
  if (F16) return pack2<true>(__uint_as_float(b), 0.f) & 0xFFFFu;
  const float s = __uint_as_float(b);
  if (s < 0x1p-100f) return 0;
  return __float_as_uint(fminf(s, 0x1p121f)) >> 16;
}

// rint(x / s) for whole x / s + 1/2 too.  x times the rounded reciprocal is off by
// 2^-23 of itself at most, while x / s (11 bits by 5) is a tie or 2^-16 away from one:
// only at a tie may the product round to the wrong side, which the remainder shows.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  float r = rintf(__fmul_rn(x, inv));
  const float e = __fmaf_rn(-r, s, x);                      // exact
  const bool tie = __fmul_rn(2.f, fabsf(e)) == s;
  const bool uneven = (static_cast<int>(fmaxf(fminf(r, 8.f), -8.f)) & 1) != 0;
  if (tie && uneven) r += e > 0.f ? 1.f : -1.f;
  return fmaxf(fminf(r, 7.f), -7.f);
}

template <bool F16>
__global__ void __launch_bounds__(kRowThreads) k_kv4_store(const Kv4Rows r, uint64_t total) {
  pdl_begin();
  // whole groups of four threads run alike, since total is a multiple of four
  for (uint64_t x = static_cast<uint64_t>(blockIdx.x) * kRowThreads + threadIdx.x; x < total;
       x += static_cast<uint64_t>(gridDim.x) * kRowThreads) {
    const uint32_t quad = 0xFu << (threadIdx.x & 28u);
    const Row8 e = row8_of(r, x);
    const Spot s = spot_of(r, e.b, e.t);
    const bool live = s.page != 0xFFFFFFFFu;
    const char* src = r.x[e.which] + static_cast<int64_t>(e.b) * r.x_seq[e.which] + static_cast<int64_t>(e.t) * r.x_token[e.which] +
                      static_cast<int64_t>(e.h) * r.x_head[e.which] + e.c * 16;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (live) {
      if (r.vec) {
        const uint4 u = *reinterpret_cast<const uint4*>(src);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = *reinterpret_cast<const uint16_t*>(src + 4 * i) | (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(src + 4 * i + 2)) << 16);
      }
    }
    float v[8], a = 0.f;
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = quad::to_float<F16>(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu);
      fine = fine && isfinite(v[i]);
      a = fmaxf(a, fabsf(v[i]));
    }
    a = fmaxf(a, __shfl_xor_sync(quad, a, 1));
    a = fmaxf(a, __shfl_xor_sync(quad, a, 2));
    fine = __ballot_sync(quad, fine) == quad;
    uint32_t sb = fine ? scale_of<F16>(a) : 0u;
    const float sc = quad::to_float<F16>(sb), inv = sc > 0.f ? __fdiv_rn(1.f, sc) : 0.f;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = sc > 0.f ? quotient(v[i], sc, inv) : 0.f;
      word |= static_cast<uint32_t>(static_cast<int>(c) + 8) << (4 * i);
    }
    if (!fine) sb = F16 ? 0x7E00u : 0x7FC0u;
    if (live) {
      *reinterpret_cast<uint32_t*>(codes_at(r.p[e.which], s, e.h, e.c)) = word;
      if ((e.c & 3u) == 0) *reinterpret_cast<uint16_t*>(scale_at(r.p[e.which], s, e.h, e.c)) = static_cast<uint16_t>(sb);
    }
  }
}

// Eight elements as the type holds them.
template <bool F16>
__device__ __forceinline__ uint4 decode8(uint32_t word, uint32_t scale) {
  const quad::Pair<F16> p(scale * 0x10001u);
  const quad::Magic<F16> m;
  const uint32_t a = quad::decode<F16, 0>(word, p, m), b = quad::decode<F16, 1>(word, p, m);  // elements (0, 4), (1, 5)
  const uint32_t c = quad::decode<F16, 2>(word, p, m), d = quad::decode<F16, 3>(word, p, m);
  return make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(c, d, 0x7632));
}

template <bool F16>
__global__ void __launch_bounds__(kRowThreads) k_kv4_load(const Kv4Rows r, uint64_t total) {
  pdl_begin();
  for (uint64_t x = static_cast<uint64_t>(blockIdx.x) * kRowThreads + threadIdx.x; x < total;
       x += static_cast<uint64_t>(gridDim.x) * kRowThreads) {
    const Row8 e = row8_of(r, x);
    const Spot s = spot_of(r, e.b, e.t);
    char* dst = const_cast<char*>(r.x[e.which]) + static_cast<int64_t>(e.b) * r.x_seq[e.which] +
                static_cast<int64_t>(e.t) * r.x_token[e.which] + static_cast<int64_t>(e.h) * r.x_head[e.which] + e.c * 16;
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (s.page != 0xFFFFFFFFu) {
      const uint32_t word = *reinterpret_cast<const uint32_t*>(codes_at(r.p[e.which], s, e.h, e.c));
      u = decode8<F16>(word, *reinterpret_cast<const uint16_t*>(scale_at(r.p[e.which], s, e.h, e.c)));
    }
    *reinterpret_cast<uint4*>(dst) = u;
  }
}

static uint64_t row_grid(uint64_t total, int device) {
  const uint64_t want = (total + kRowThreads - 1) / kRowThreads, most = 16ull * sm_count(device);
  return want < most ? want : most;
}

int launch_kv4_store(const Kv4Rows& r, int device, cudaStream_t stream) {
  const uint64_t total = 2ull * r.n_seqs * r.T * r.heads * (r.dim / 8);
  return kv_launch("k_kv4_store", r.f16 ? k_kv4_store<true> : k_kv4_store<false>, dim3(static_cast<unsigned>(row_grid(total, device))),
                   kRowThreads, 0, 1, stream, r, total);
}

int launch_kv4_load(const Kv4Rows& r, int device, cudaStream_t stream) {
  const uint64_t total = 2ull * r.n_seqs * r.T * r.heads * (r.dim / 8);
  return kv_launch("k_kv4_load", r.f16 ? k_kv4_load<true> : k_kv4_load<false>, dim3(static_cast<unsigned>(row_grid(total, device))),
                   kRowThreads, 0, 1, stream, r, total);
}

// ---------------------------------------------------------------------------
// The whole cache in 16 bits, for the tensor-core kernel

// CTA (tile, sequence): kExpand tokens of every head.
template <bool F16>
__global__ void __launch_bounds__(kRowThreads) k_kv4_expand(const Attend4Args x, const Kv4Expanded o, uint32_t tiles) {
  pdl_begin();
  const AttendArgs& a = x.a;
  const uint32_t b = blockIdx.y, chunks = a.dim / 8;
  const int32_t raw = a.lens[b], len = clamp_len(raw, a.page_tokens, a.max_pages);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (raw != len) kv_status(a.status, IBP_ERANGE);
    o.lens[b] = len;
  }
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    if (threadIdx.x == 0) o.table[static_cast<uint64_t>(b) * tiles + tile] = static_cast<int32_t>(b * tiles + tile);
    const int32_t first = static_cast<int32_t>(tile * kExpand);
    if (first >= len) continue;
    const uint32_t n = static_cast<uint32_t>(len - first) < kExpand ? static_cast<uint32_t>(len - first) : kExpand;
    for (uint32_t i = threadIdx.x; i < a.kv_heads * n * chunks; i += kRowThreads) {
      const uint32_t c = i % chunks, tok = i / chunks % n, h = i / chunks / n;
      const uint32_t pos = static_cast<uint32_t>(first) + tok, nth = pos / a.page_tokens;
      Spot s;
      s.page = static_cast<uint32_t>(a.table[static_cast<uint64_t>(b) * a.max_pages + nth]);
      s.slot = pos - nth * a.page_tokens;
      uint4 uk = make_uint4(0u, 0u, 0u, 0u), uv = uk;
      if (s.page < a.n_pages) {
        const uint32_t kw = *reinterpret_cast<const uint32_t*>(codes_at(x.k, s, h, c)), vw = *reinterpret_cast<const uint32_t*>(codes_at(x.v, s, h, c));
        const uint32_t ks = *reinterpret_cast<const uint16_t*>(scale_at(x.k, s, h, c)), vs = *reinterpret_cast<const uint16_t*>(scale_at(x.v, s, h, c));
        uk = decode8<F16>(kw, ks);
        uv = decode8<F16>(vw, vs);
      } else {
        kv_status(a.status, IBP_ERANGE);
      }
      const uint64_t at = (((static_cast<uint64_t>(b) * tiles + tile) * a.kv_heads + h) * kExpand + tok) * a.dim * 2 + c * 16;
      *reinterpret_cast<uint4*>(o.k + at) = uk;
      *reinterpret_cast<uint4*>(o.v + at) = uv;
    }
  }
}

static size_t align256(size_t x) { return (x + 255) / 256 * 256; }

size_t kv4_expand_workspace(uint32_t n_seqs, uint64_t tokens, uint32_t heads, uint32_t dim) {
  const uint64_t tiles = (tokens + kExpand - 1) / kExpand;
  return align256(4 * n_seqs * tiles) + align256(4ull * n_seqs) + 2 * align256(n_seqs * tiles * kExpand * heads * dim * 2);
}

int launch_kv4_expand(const Attend4Args& x, const Kv4Expanded& e, int device, cudaStream_t stream) {
  const uint64_t tokens = static_cast<uint64_t>(x.a.max_pages) * x.a.page_tokens;
  const uint32_t tiles = static_cast<uint32_t>((tokens + kExpand - 1) / kExpand);
  const uint32_t most = 65535u < tiles ? 65535u : tiles;
  return kv_launch("k_kv4_expand", x.a.f16 ? k_kv4_expand<true> : k_kv4_expand<false>, dim3(most, x.a.n_seqs), kRowThreads, 0, 1,
                   stream, x, e, tiles);
}

}  // namespace ibp

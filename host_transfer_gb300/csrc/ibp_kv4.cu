// ibp_kv4.cu - tokens into and out of paged caches held in 4 bits.
//
// A thread takes 8 elements (16 bytes) of four tokens and four threads a group of 32, so
// that the largest magnitude is two exchanges and every access of a warp is a run of
// whole sectors.  What a prompt cannot do without is 2 bytes read and 9/16 written an
// element, or the other way; a single token is latency.
//
// Measured on one GB300, 4 prompts of 8191 tokens, 8 kv heads of 128, K and V stored and
// read back (306 MB): 91 us for both calls (55 to 60 the store, 35 to 37 the load), 3.4 TB/s,
// with cold caches.  Issue bounds both: 74 and 76 % of the slots are used, DRAM for 35 and 41 %.
// A token at a time with a division an element took 245 us, four in flight 142 us, magnitudes
// as whole numbers and codes packed by bytes 105 us.  32 sequences of one token: 11 us, two launches' latency.
#include "ibp_kv4.cuh"

namespace ibp {

constexpr int kRowThreads = 256;
constexpr uint32_t kRowFly = 4;  // tokens of a thread, all of them read before any is written
constexpr uint32_t kRowLoops = 4;  // rounds of them a block, where there are blocks enough: 1 takes 104 us for the prompts above, 2 93, 4 91, 8 95

// The page and slot of a row; page 2^32 - 1 where there is none.
struct Spot {
  uint32_t page, slot;
};

// The rows of block (tokens, sequence, K or V): threads take neighbouring pieces of eight
// elements of a token, as many tokens at a time as fit.
struct Rows {
  uint32_t pieces;      // of a token
  uint32_t width;       // of them at a time
  uint32_t at_once;     // tokens at a time
  uint32_t first;       // this block's first token
  uint32_t b, which;
  int32_t n, base;      // rows of the sequence, position of row 0
  __device__ __forceinline__ explicit Rows(const Kv4Rows& r) {
    pieces = r.heads * (r.dim / 8);
    width = pieces < kRowThreads ? pieces : kRowThreads;
    at_once = kRowThreads / width;
    first = blockIdx.x * at_once * kRowFly * r.loops;
    b = blockIdx.y, which = blockIdx.z;
    const int32_t raw = r.lens[b], len = clamp_len(raw, r.page_tokens, r.max_pages);
    const int32_t want = r.n_rows ? r.n_rows[b] : static_cast<int32_t>(r.T);
    n = want < 0 ? 0 : (want > static_cast<int32_t>(r.T) ? static_cast<int32_t>(r.T) : want);
    base = len - n;
    if (blockIdx.x == 0 && threadIdx.x == 0 && (raw != len || want != n || base < 0)) kv_status(r.status, IBP_ERANGE);
  }
  __device__ __forceinline__ Spot spot(const Kv4Rows& r, uint32_t t) const {
    Spot s = {0xFFFFFFFFu, 0u};
    const int32_t pos = base + static_cast<int32_t>(t);
    if (static_cast<int32_t>(t) >= n || pos < 0) return s;
    const uint32_t p = static_cast<uint32_t>(pos), nth = r.shift >= 0 ? p >> r.shift : p / r.page_tokens;
    s.page = static_cast<uint32_t>(__ldg(r.table + static_cast<uint64_t>(b) * r.max_pages + nth));
    s.slot = r.shift >= 0 ? p & ((1u << r.shift) - 1u) : p - nth * r.page_tokens;
    if (s.page >= r.n_pages) {
      kv_status(r.status, IBP_ERANGE);
      s.page = 0xFFFFFFFFu;
    }
    return s;
  }
};

// A thread's piece of token slot 0 of page 0; from there by page and slot.  NARROW:
// strides of 32 bits.
template <bool NARROW>
struct Piece {
  char *codes, *scale;
  const Kv4View& v;
  __device__ __forceinline__ Piece(const Kv4View& v_, uint32_t h, uint32_t c) : v(v_) {
    codes = const_cast<char*>(v.codes) + static_cast<int64_t>(h) * v.head_stride + c * 4;
    scale = const_cast<char*>(v.scales) + static_cast<int64_t>(h) * v.s_head + c / 4 * 2;
  }
  static __device__ __forceinline__ uint64_t times(uint32_t x, int64_t stride) {
    return NARROW ? static_cast<uint64_t>(x) * static_cast<uint32_t>(stride) : static_cast<uint64_t>(x) * static_cast<uint64_t>(stride);
  }
  __device__ __forceinline__ char* codes_of(const Spot& s) const { return codes + times(s.page, v.page_stride) + times(s.slot, v.token_stride); }
  __device__ __forceinline__ char* scale_of(const Spot& s) const { return scale + times(s.page, v.s_page) + times(s.slot, v.s_token); }
};

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

// 8 + rint(x / s) in the lowest byte, with `edge` kept within 1 to 15.  x times the reciprocal
// (within 2^-22 of itself) is off by 2^-19 at most, while x / s (11 bits by 5) is a tie
// k + 1/2 or 2^-12 away from one: rounded to multiples of 2^-16 first, ties are exact again
// and go to even like the quotient's own.
__device__ __forceinline__ uint32_t code_of(float x, float inv, bool edge) {
  float y = __fadd_rn(__fmaf_rn(x, inv, 192.f), -192.f);
  if (edge) y = fmaxf(fminf(y, 7.f), -7.f);
  return __float_as_uint(__fadd_rn(y, 12582920.f));  // 1.5 2^23 + 8
}

// FAST: rows that may be read 16 bytes at a time, and narrow strides.
template <bool F16, bool FAST>
__global__ void __launch_bounds__(kRowThreads) k_kv4_store(const Kv4Rows r) {
  pdl_begin();
  const Rows o(r);
  const uint32_t mine = threadIdx.x / o.width, chunks = r.dim / 8;
  // whole warps go round alike: the four threads of a group exchange their maxima
  for (uint32_t p0 = 0; p0 < o.pieces; p0 += o.width) {
    const uint32_t piece = p0 + threadIdx.x - mine * o.width;
    const bool on = mine < o.at_once && piece < o.pieces;
    const uint32_t h = on ? piece / chunks : 0, c = on ? piece - h * chunks : 0;
    const Piece<FAST> to(r.p[o.which], h, c);
    const char* src = r.x[o.which] + static_cast<int64_t>(o.b) * r.x_seq[o.which] + static_cast<int64_t>(h) * r.x_head[o.which] + c * 16 +
                      static_cast<int64_t>(o.first + mine) * r.x_token[o.which];
    const int64_t next = static_cast<int64_t>(o.at_once) * r.x_token[o.which];
    uint32_t t0 = on ? o.first + mine : 0x40000000u;
#pragma unroll 1
    for (uint32_t l = 0; l < r.loops; ++l, t0 += kRowFly * o.at_once, src += kRowFly * next) {
      if (o.first + l * kRowFly * o.at_once >= static_cast<uint32_t>(o.n)) break;  // the same for the block
      Spot at[kRowFly];
      uint32_t w[kRowFly][4];
#pragma unroll
      for (uint32_t i = 0; i < kRowFly; ++i) {
        at[i] = o.spot(r, t0 + i * o.at_once);
        w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0u;
        if (static_cast<int32_t>(t0 + i * o.at_once) < o.n) {
          const char* x = src + i * next;
          if (FAST) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(x));
            w[i][0] = u.x, w[i][1] = u.y, w[i][2] = u.z, w[i][3] = u.w;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w[i][j] = *reinterpret_cast<const uint16_t*>(x + 4 * j) | (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(x + 4 * j + 2)) << 16);
          }
        }
      }
#pragma unroll
      for (uint32_t i = 0; i < kRowFly; ++i) {
        // magnitudes are ordered as whole numbers are, infinities and NaN above all
        uint32_t top = __vmaxu2(__vmaxu2(w[i][0] & 0x7FFF7FFFu, w[i][1] & 0x7FFF7FFFu), __vmaxu2(w[i][2] & 0x7FFF7FFFu, w[i][3] & 0x7FFF7FFFu));
        top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        top = max(top & 0xFFFFu, top >> 16);
        const bool fine = top < (F16 ? 0x7C00u : 0x7F80u);
        uint32_t sb = fine ? scale_of<F16>(quad::to_float<F16>(top)) : 0u;
        const float sc = quad::to_float<F16>(sb);
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(sc));
        uint32_t word = 0x88888888u;
        if (sb) {
          // only the type's smallest and largest scales leave quotients above 7 1/2
          const bool edge = F16 ? sb < 0x0400u : sb >= 0x7C00u;
          uint32_t f[8];
          auto codes = [&](bool at_edge) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = code_of(quad::to_float<F16>(j & 1 ? w[i][j / 2] >> 16 : w[i][j / 2] & 0xFFFFu), inv, at_edge);
          };
          if (edge)
            codes(true);
          else
            codes(false);
          const uint32_t low = __byte_perm(__byte_perm(f[0], f[2], 0x0040), __byte_perm(f[4], f[6], 0x0040), 0x5410);
          const uint32_t high = __byte_perm(__byte_perm(f[1], f[3], 0x0040), __byte_perm(f[5], f[7], 0x0040), 0x5410);
          word = low | high << 4;
        }
        if (!fine) sb = F16 ? 0x7E00u : 0x7FC0u;
        if (at[i].page == 0xFFFFFFFFu) continue;
        *reinterpret_cast<uint32_t*>(to.codes_of(at[i])) = word;
        if ((c & 3u) == 0) *reinterpret_cast<uint16_t*>(to.scale_of(at[i])) = static_cast<uint16_t>(sb);
      }
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

template <bool F16, bool FAST>
__global__ void __launch_bounds__(kRowThreads) k_kv4_load(const Kv4Rows r) {
  pdl_begin();
  const Rows o(r);
  const uint32_t mine = threadIdx.x / o.width, chunks = r.dim / 8;
  if (mine >= o.at_once) return;
  for (uint32_t piece = threadIdx.x - mine * o.width; piece < o.pieces; piece += o.width) {
    const uint32_t h = piece / chunks, c = piece - h * chunks;
    const Piece<FAST> from(r.p[o.which], h, c);
    char* dst = const_cast<char*>(r.x[o.which]) + static_cast<int64_t>(o.b) * r.x_seq[o.which] + static_cast<int64_t>(h) * r.x_head[o.which] + c * 16 +
                static_cast<int64_t>(o.first + mine) * r.x_token[o.which];
    const int64_t next = static_cast<int64_t>(o.at_once) * r.x_token[o.which];
    uint32_t t0 = o.first + mine;
#pragma unroll 1
    for (uint32_t l = 0; l < r.loops && t0 < r.T; ++l, t0 += kRowFly * o.at_once, dst += kRowFly * next) {
      uint32_t word[kRowFly], scale[kRowFly];
#pragma unroll
      for (uint32_t i = 0; i < kRowFly; ++i) {
        const Spot s = o.spot(r, t0 + i * o.at_once);
        word[i] = scale[i] = 0u;  // code 0 times 0
        if (s.page != 0xFFFFFFFFu) {
          word[i] = __ldg(reinterpret_cast<const uint32_t*>(from.codes_of(s)));
          scale[i] = __ldg(reinterpret_cast<const uint16_t*>(from.scale_of(s)));
        }
      }
#pragma unroll
      for (uint32_t i = 0; i < kRowFly; ++i) {
        if (t0 + i * o.at_once >= r.T) continue;
        uint4 u = decode8<F16>(word[i], scale[i]);
        if (F16 && scale[i] == 0u) u = make_uint4(0u, 0u, 0u, 0u);  // not -0
        *reinterpret_cast<uint4*>(dst + i * next) = u;
      }
    }
  }
}

static dim3 row_grid(const Kv4Rows& r) {
  const uint64_t pieces = r.heads * (r.dim / 8), at_once = pieces < kRowThreads ? kRowThreads / pieces : 1, each = at_once * kRowFly * r.loops;
  return dim3(static_cast<unsigned>((r.T + each - 1) / each), r.n_seqs, 2);
}

static bool narrow(const Kv4Rows& r) {
  uint64_t all = 0;
  for (int i = 0; i < 2; ++i)
    all |= static_cast<uint64_t>(r.p[i].page_stride) | static_cast<uint64_t>(r.p[i].token_stride) | static_cast<uint64_t>(r.p[i].s_page) |
           static_cast<uint64_t>(r.p[i].s_token);
  return all <= 0xFFFFFFFFull;
}

// What the kernels go by besides: pages of 2^shift tokens; and several rounds of tokens a
// block, so that what it begins with counts less, where there are blocks enough.
static Kv4Rows planned(Kv4Rows r, int device) {
  r.shift = -1;
  if ((r.page_tokens & (r.page_tokens - 1)) == 0)
    for (r.shift = 0; (1u << r.shift) < r.page_tokens;) ++r.shift;
  r.loops = 1;
  const dim3 g = row_grid(r);
  if (static_cast<uint64_t>(g.x) * g.y * 2 >= 32ull * sm_count(device)) r.loops = kRowLoops;
  return r;
}

int launch_kv4_store(const Kv4Rows& rows, int device, cudaStream_t stream) {
  const Kv4Rows r = planned(rows, device);
  const bool fast = r.vec && narrow(r);
  auto kern = r.f16 ? (fast ? k_kv4_store<true, true> : k_kv4_store<true, false>) : (fast ? k_kv4_store<false, true> : k_kv4_store<false, false>);
  return kv_launch("k_kv4_store", kern, row_grid(r), kRowThreads, 0, 1, stream, r);
}

int launch_kv4_load(const Kv4Rows& rows, int device, cudaStream_t stream) {
  const Kv4Rows r = planned(rows, device);
  const bool fast = narrow(r);
  auto kern = r.f16 ? (fast ? k_kv4_load<true, true> : k_kv4_load<true, false>) : (fast ? k_kv4_load<false, true> : k_kv4_load<false, false>);
  return kv_launch("k_kv4_load", kern, row_grid(r), kRowThreads, 0, 1, stream, r);
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

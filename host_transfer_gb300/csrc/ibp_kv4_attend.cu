// ibp_kv4_attend.cu - attention of few queries over a paged cache held in 4 bits.
//
// A CTA holds 8 or 16 query rows of one sequence and kv head (drafted tokens times
// the group's heads) and walks a share of the tokens, 16 to a warp's step, each warp
// with its own running maximum and sum.  The products are taken transposed, S^T = K Q^T
// and O^T = V^T P^T, so that tokens and dimensions fill the 16-row side of
// mma.m16n8k16 and queries the 8-wide side.
//
// A dot product may add its dimensions in any order, so a lane takes for its part of
// a K row the codes that lie next to one another, up to 32 of one group: one 16-byte
// load, one scale, and the queries are laid out to match.  The same holds for the rows
// of O^T: a lane takes neighbouring dimensions of V for the four tokens that are its
// part of the product, and pairs of tokens are made by byte permutations.  So codes go
// from global memory to registers, are decoded there and are the operands: nothing
// passes through shared memory until the warps are joined.
//
// Decoding is what counts beside the cache's bytes: 12 instructions for 8 elements
// (a shift, a mask with the exponent put in, one fused multiply-add a pair).
#include <type_traits>

#include "ibp_kv4.cuh"

namespace ibp {

constexpr uint32_t kQdWarps = 4;

// What a lane holds of a step's 16 tokens.
template <uint32_t DP>
struct QuadStep {
  uint32_t kw[2][DP / 32];               // K codes of tokens g and g + 8
  uint32_t ks[2][DP == 256 ? 2 : 1];     // their scales
  uint32_t vw[4][DP / 64];               // V codes of tokens 2t, 2t + 1, 2t + 8, 2t + 9
  uint32_t vs[4];
};

template <uint32_t N>
__device__ __forceinline__ void ld_words(uint32_t (&w)[N], const char* p, bool on) {
  static_assert(N == 1 || N == 2 || N == 4, "");
#pragma unroll
  for (uint32_t i = 0; i < N; ++i) w[i] = 0u;
  if (!on) return;
  if constexpr (N == 4)
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
  else if constexpr (N == 2)
    asm("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  else
    asm("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
}
__device__ __forceinline__ uint32_t ld_scale(const char* p, bool on) {
  return on ? static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(p))) : 0u;
}

template <uint32_t DP, uint32_t NT, bool F16>
struct Quad {
  static constexpr uint32_t kRows = 8 * NT;
  // the join: [warp][row][DP] and [warp][row][2], then a cluster's part [row][2 + DP]
  static constexpr uint32_t kBytes = (kQdWarps * kRows * (DP + 2) + kRows * (DP + 2)) * 4;

  static __device__ __forceinline__ bool sees(const AttendArgs& a, uint32_t b, int32_t ctx, int32_t len, uint32_t r, int32_t pos) {
    if (pos >= len) return false;
    if (pos < ctx) return true;
    const uint32_t t = r / a.group, i = static_cast<uint32_t>(pos - ctx);
    if (!a.mask) return i <= t;
    return (a.mask[(static_cast<uint64_t>(b) * a.T + t) * a.mask_words + (i >> 5)] >> (i & 31u)) & 1u;
  }
};

// Where a lane's parts of a step lie.
struct QuadLane {
  const char *kc, *ks, *vc, *vs;  // this lane's part of token 0 of slot 0 of page 0
  const int32_t* row;
  int32_t shift;                  // pages hold 2^shift steps; -1: another whole number; -2: steps cross pages
  bool k_on[2], v_on;             // the dim reaches this lane's groups
};

__device__ __forceinline__ uint32_t quad_page(const AttendArgs& a, const QuadLane& ln, uint32_t step, uint32_t steps) {
  if (ln.shift < -1 || step >= steps) return 0xFFFFFFFFu;
  return static_cast<uint32_t>(__ldg(ln.row + (ln.shift >= 0 ? step >> ln.shift : step * 16 / a.page_tokens)));
}

template <uint32_t DP>
__device__ __forceinline__ void quad_load(const Attend4Args& x, const QuadLane& ln, uint32_t step, uint32_t n_tok, uint32_t page,
                                          QuadStep<DP>& s) {
  const AttendArgs& a = x.a;
  const uint32_t lane = threadIdx.x & 31u, g = lane >> 2, t = lane & 3u;
  constexpr uint32_t kK = DP / 32;  // words of K a lane and token
  auto load_k = [&](uint32_t i, const char* codes, const char* scales, bool on) {
    if constexpr (kK == 8) {
      uint32_t lo[4], hi[4];
      ld_words<4>(lo, codes, on && ln.k_on[0]);
      ld_words<4>(hi, codes + 16, on && ln.k_on[1]);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) s.kw[i][j] = lo[j], s.kw[i][4 + j] = hi[j];
      s.ks[i][0] = ld_scale(scales, on && ln.k_on[0]);
      s.ks[i][DP == 256 ? 1 : 0] = ld_scale(scales + 2, on && ln.k_on[1]);
    } else {
      ld_words<kK>(s.kw[i], codes, on && ln.k_on[0]);
      s.ks[i][0] = ld_scale(scales, on && ln.k_on[0]);
    }
  };
  if (ln.shift >= -1) {
    const uint32_t at = ln.shift >= 0 ? step >> ln.shift : step * 16 / a.page_tokens;
    const uint32_t s0 = step * 16 - at * a.page_tokens, left = n_tok - step * 16;
    const bool good = page < a.n_pages;
    if (!good) kv_status(a.status, IBP_ERANGE);
    const int64_t pg = good ? page : 0;
    const char* kc = ln.kc + pg * x.k.page_stride + static_cast<int64_t>(s0 + g) * x.k.token_stride;
    const char* ks = ln.ks + pg * x.k.s_page + static_cast<int64_t>(s0 + g) * x.k.s_token;
    load_k(0, kc, ks, good && g < left);
    load_k(1, kc + 8 * x.k.token_stride, ks + 8 * x.k.s_token, good && g + 8 < left);
    const char* vc = ln.vc + pg * x.v.page_stride + static_cast<int64_t>(s0 + 2 * t) * x.v.token_stride;
    const char* vs = ln.vs + pg * x.v.s_page + static_cast<int64_t>(s0 + 2 * t) * x.v.s_token;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t off = (i & 1u) + (i >> 1) * 8;
      const bool on = good && 2 * t + off < left && ln.v_on;
      ld_words<DP / 64>(s.vw[i], vc + off * x.v.token_stride, on);
      s.vs[i] = ld_scale(vs + off * x.v.s_token, on);
    }
    return;
  }
  // Steps cross pages: lane i finds token i and tells the others.
  const uint32_t tok = step * 16 + (lane & 15u);
  uint32_t pg = 0xFFFFFFFFu, slot = 0;
  if (tok < n_tok) {
    const uint32_t nth = tok / a.page_tokens;
    slot = tok - nth * a.page_tokens;
    pg = static_cast<uint32_t>(ln.row[nth]);
    if (pg >= a.n_pages) {
      kv_status(a.status, IBP_ERANGE);
      pg = 0xFFFFFFFFu;
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < 2; ++i) {
    const uint32_t p = __shfl_sync(0xFFFFFFFFu, pg, g + 8 * i), sl = __shfl_sync(0xFFFFFFFFu, slot, g + 8 * i);
    const bool on = p != 0xFFFFFFFFu;
    const int64_t q = on ? p : 0;
    load_k(i, ln.kc + q * x.k.page_stride + static_cast<int64_t>(sl) * x.k.token_stride,
           ln.ks + q * x.k.s_page + static_cast<int64_t>(sl) * x.k.s_token, on);
  }
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    const uint32_t from = 2 * t + (i & 1u) + (i >> 1) * 8;
    const uint32_t p = __shfl_sync(0xFFFFFFFFu, pg, from), sl = __shfl_sync(0xFFFFFFFFu, slot, from);
    const bool on = p != 0xFFFFFFFFu && ln.v_on;
    const int64_t q = on ? p : 0;
    ld_words<DP / 64>(s.vw[i], ln.vc + q * x.v.page_stride + static_cast<int64_t>(sl) * x.v.token_stride, on);
    s.vs[i] = ld_scale(ln.vs + q * x.v.s_page + static_cast<int64_t>(sl) * x.v.s_token, on);
  }
}

// A warp's running softmax of its rows.
template <uint32_t DP, uint32_t NT>
struct QuadAcc {
  float o[DP / 16][NT][4];  // rows: dimensions 2j and 2j + 1 of the lane's; columns: queries 2t, 2t + 1
  float m[NT][2], l[NT][2];
};

template <uint32_t DP, uint32_t NT, bool F16>
__device__ __forceinline__ void quad_step(const AttendArgs& a, QuadStep<DP>& s, const uint32_t (&qf)[NT][DP / 16][2],
                                          QuadAcc<DP, NT>& acc, uint32_t b, int32_t ctx, int32_t len, uint32_t row0,
                                          uint32_t live_rows, int32_t first) {
  using Q = Quad<DP, NT, F16>;
  const uint32_t lane = threadIdx.x & 31u;
  float c[NT][4];
#pragma unroll
  for (uint32_t n = 0; n < NT; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
#pragma unroll
  for (uint32_t w = 0; w < DP / 32; ++w) {
    const uint32_t gi = DP == 256 ? w / 4 : 0;
    const quad::Pair<F16> p0(quad::scale_bits<F16>(s.ks[0][gi]) * 0x10001u), p1(quad::scale_bits<F16>(s.ks[1][gi]) * 0x10001u);
    const uint32_t x = s.kw[0][w], y = s.kw[1][w];
    const uint32_t lo[4] = {quad::decode<F16, 0>(x, p0), quad::decode<F16, 0>(y, p1), quad::decode<F16, 1>(x, p0), quad::decode<F16, 1>(y, p1)};
    const uint32_t hi[4] = {quad::decode<F16, 2>(x, p0), quad::decode<F16, 2>(y, p1), quad::decode<F16, 3>(x, p0), quad::decode<F16, 3>(y, p1)};
#pragma unroll
    for (uint32_t n = 0; n < NT; ++n) {
      mma16816<F16>(c[n], lo, qf[n][2 * w][0], qf[n][2 * w][1]);
      mma16816<F16>(c[n], hi, qf[n][2 * w + 1][0], qf[n][2 * w + 1][1]);
    }
  }
  // Scores in powers of two; what a row does not see is -infinity.
  const bool open = first + 16 <= (ctx < len ? ctx : len);
#pragma unroll
  for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) c[n][e] *= a.scale_log2;
  if (!open) {
#pragma unroll
    for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) {
        const uint32_t r = n * 8 + (lane & 3u) * 2 + (e & 1u);
        const int32_t pos = first + static_cast<int32_t>(lane / 4 + (e < 2 ? 0 : 8));
        if (r >= live_rows || !Q::sees(a, b, ctx, len, row0 + r, pos)) c[n][e] = -INFINITY;
      }
  }
  float cm[NT][2];
  bool grow = false;
#pragma unroll
  for (uint32_t n = 0; n < NT; ++n) {
    cm[n][0] = fmaxf(c[n][0], c[n][2]);
    cm[n][1] = fmaxf(c[n][1], c[n][3]);
#pragma unroll
    for (uint32_t w = 4; w < 32; w <<= 1) {
      cm[n][0] = fmaxf(cm[n][0], __shfl_xor_sync(0xFFFFFFFFu, cm[n][0], w));
      cm[n][1] = fmaxf(cm[n][1], __shfl_xor_sync(0xFFFFFFFFu, cm[n][1], w));
    }
    if (F16) cm[n][0] = __fadd_ru(cm[n][0], -kLift<F16>), cm[n][1] = __fadd_ru(cm[n][1], -kLift<F16>);
    grow = grow || cm[n][0] > acc.m[n][0] || cm[n][1] > acc.m[n][1];
  }
  if (__any_sync(0xFFFFFFFFu, grow)) {
    // Rescaled at once, so that a row's largest probability is a power of two and its
    // rounding to the cache's type costs nothing.
#pragma unroll
    for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
      for (uint32_t e = 0; e < 2; ++e)
        if (cm[n][e] > acc.m[n][e]) {
          const float f = ex2(acc.m[n][e] - cm[n][e]);
          acc.m[n][e] = cm[n][e];
          acc.l[n][e] *= f;
#pragma unroll
          for (uint32_t d = 0; d < DP / 16; ++d) acc.o[d][n][e] *= f, acc.o[d][n][2 + e] *= f;
        }
  }
  uint32_t pf[NT][2];
#pragma unroll
  for (uint32_t n = 0; n < NT; ++n) {
    const float m0 = acc.m[n][0] == -INFINITY ? 0.f : acc.m[n][0], m1 = acc.m[n][1] == -INFINITY ? 0.f : acc.m[n][1];
    c[n][0] = ex2(c[n][0] - m0), c[n][1] = ex2(c[n][1] - m1);
    c[n][2] = ex2(c[n][2] - m0), c[n][3] = ex2(c[n][3] - m1);
    acc.l[n][0] += c[n][0] + c[n][2];
    acc.l[n][1] += c[n][1] + c[n][3];
    pf[n][0] = transpose8(pack2<F16>(c[n][0], c[n][1]));
    pf[n][1] = transpose8(pack2<F16>(c[n][2], c[n][3]));
  }
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) s.vs[i] = quad::scale_bits<F16>(s.vs[i]);
  if (!open) {
    // Groups of V that may hold infinities or NaN: a row that does not see them must
    // not meet them, even with probability zero.  They leave the product and are
    // added to the rows that see them.
    bool bad = false;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) bad = bad || quad::odd<F16>(s.vs[i]);
    if (__any_sync(0xFFFFFFFFu, bad)) {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
#pragma unroll 1
        for (uint32_t tt = 0; tt < 4; ++tt) {
          const uint32_t tok = 2 * tt + (i & 1u) + (i >> 1) * 8;  // its row in S^T
          const uint32_t sc = __shfl_sync(0xFFFFFFFFu, s.vs[i], (lane & 28u) | tt);
          uint32_t words[DP / 64];
#pragma unroll
          for (uint32_t w = 0; w < DP / 64; ++w) words[w] = __shfl_sync(0xFFFFFFFFu, s.vw[i][w], (lane & 28u) | tt);
#pragma unroll
          for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
            for (uint32_t e = 0; e < 2; ++e) {
              const float p = __shfl_sync(0xFFFFFFFFu, c[n][(i >> 1) * 2 + e], ((tok & 7u) << 2) | (lane & 3u));
              const uint32_t r = n * 8 + (lane & 3u) * 2 + e;
              if (quad::odd<F16>(sc) && r < live_rows &&
                  Q::sees(a, b, ctx, len, row0 + r, first + static_cast<int32_t>(tok))) {
#pragma unroll
                for (uint32_t d = 0; d < DP / 16; ++d) {
                  acc.o[d][n][e] += p * quad::value<F16>(words[d / 4], (2 * d) & 7u, sc);
                  acc.o[d][n][2 + e] += p * quad::value<F16>(words[d / 4], (2 * d + 1) & 7u, sc);
                }
              }
            }
        }
        if (quad::odd<F16>(s.vs[i])) s.vs[i] = 0u;
      }
    }
  }
  const quad::Pair<F16> pa(s.vs[0] | s.vs[1] << 16), pb(s.vs[2] | s.vs[3] << 16);
#pragma unroll
  for (uint32_t w = 0; w < DP / 64; ++w) {
    // elements 0 - 3 and 4 - 7 of a word for a pair of tokens
    const uint32_t a0 = __byte_perm(s.vw[0][w], s.vw[1][w], 0x5410), a1 = __byte_perm(s.vw[0][w], s.vw[1][w], 0x7632);
    const uint32_t b0 = __byte_perm(s.vw[2][w], s.vw[3][w], 0x5410), b1 = __byte_perm(s.vw[2][w], s.vw[3][w], 0x7632);
    const uint32_t f[4][4] = {
        {quad::decode<F16, 0>(a0, pa), quad::decode<F16, 1>(a0, pa), quad::decode<F16, 0>(b0, pb), quad::decode<F16, 1>(b0, pb)},
        {quad::decode<F16, 2>(a0, pa), quad::decode<F16, 3>(a0, pa), quad::decode<F16, 2>(b0, pb), quad::decode<F16, 3>(b0, pb)},
        {quad::decode<F16, 0>(a1, pa), quad::decode<F16, 1>(a1, pa), quad::decode<F16, 0>(b1, pb), quad::decode<F16, 1>(b1, pb)},
        {quad::decode<F16, 2>(a1, pa), quad::decode<F16, 3>(a1, pa), quad::decode<F16, 2>(b1, pb), quad::decode<F16, 3>(b1, pb)}};
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
#pragma unroll
      for (uint32_t n = 0; n < NT; ++n) mma16816<F16>(acc.o[4 * w + j][n], f[j], pf[n][0], pf[n][1]);
  }
}

template <uint32_t DP, uint32_t NT, bool F16>
__global__ void __launch_bounds__(kQdWarps * 32, DP == 256 || NT == 2 ? 2 : 4)
    k_kv4_attend(const Attend4Args x, uint32_t row_tiles, int32_t shift, uint32_t chunk) {
  using Q = Quad<DP, NT, F16>;
  const AttendArgs& a = x.a;
  extern __shared__ __align__(16) unsigned char sm[];
  pdl_begin();
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3u;
  const uint32_t split = blockIdx.x % a.splits, item = blockIdx.x / a.splits;
  const uint32_t tile = item % row_tiles, h = item / row_tiles % a.kv_heads, b = item / row_tiles / a.kv_heads;
  const uint32_t row0 = tile * Q::kRows;
  const int32_t raw = a.lens[b], len = clamp_len(raw, a.page_tokens, a.max_pages);
  const int32_t live = a.n_live ? a.n_live[b] : static_cast<int32_t>(a.T);
  if ((raw != len || live > len || live < 0 || live > static_cast<int32_t>(a.T)) && threadIdx.x == 0)
    kv_status(a.status, IBP_ERANGE);
  const int32_t n_live = live < 0 ? 0 : (live > static_cast<int32_t>(a.T) ? static_cast<int32_t>(a.T) : live);
  const int32_t ctx = len - n_live;  // below 0: the draft's first tokens do not exist
  const uint32_t all_rows = a.T * a.group;
  const uint32_t rows = all_rows - row0 < Q::kRows ? all_rows - row0 : Q::kRows;
  const uint32_t lr = static_cast<uint32_t>(n_live) * a.group;
  const uint32_t live_rows = lr > row0 ? (lr - row0 < rows ? lr - row0 : rows) : 0;
  const uint32_t n_tok = live_rows ? static_cast<uint32_t>(len) : 0;
  const uint32_t steps = ceil_div(n_tok, 16);
  // This CTA's share: an even one in a cluster, a chunk otherwise.
  const uint32_t per = a.cluster ? ceil_div(steps, a.splits) : chunk;
  const uint32_t s0 = split * per < steps ? split * per : steps, s1 = steps - s0 < per ? steps : s0 + per;
  if (!a.cluster && split && s0 == s1) return;  // the join does not look at it

  // Q^T as B operands, dimensions in the order in which a lane decodes K.
  uint32_t qf[NT][DP / 16][2];
#pragma unroll
  for (uint32_t n = 0; n < NT; ++n) {
    const bool on = n * 8 + g < live_rows;
    const uint32_t r = on ? row0 + n * 8 + g : 0;
    const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q + static_cast<int64_t>(b) * a.q_seq + static_cast<int64_t>(r / a.group) * a.q_token +
                                                          static_cast<int64_t>(h * a.group + r % a.group) * a.q_head);
#pragma unroll
    for (uint32_t kk = 0; kk < DP / 16; ++kk)
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        const uint32_t d = t * (DP / 4) + kk / 2 * 8 + (kk & 1u) * 2 + i;  // and d + 4
        qf[n][kk][i] = on && d < a.dim ? q[d] | static_cast<uint32_t>(q[d + 4]) << 16 : 0u;
      }
  }

  QuadAcc<DP, NT> acc;
#pragma unroll
  for (uint32_t n = 0; n < NT; ++n) {
    acc.m[n][0] = acc.m[n][1] = -INFINITY;
    acc.l[n][0] = acc.l[n][1] = 0.f;
#pragma unroll
    for (uint32_t d = 0; d < DP / 16; ++d) acc.o[d][n][0] = acc.o[d][n][1] = acc.o[d][n][2] = acc.o[d][n][3] = 0.f;
  }

  QuadLane ln;
  ln.kc = x.k.codes + static_cast<int64_t>(h) * x.k.head_stride + t * (DP / 8);
  ln.ks = x.k.scales + static_cast<int64_t>(h) * x.k.s_head + t * (DP / 4) / kQuadGroup * 2;
  ln.vc = x.v.codes + static_cast<int64_t>(h) * x.v.head_stride + g * (DP / 16);
  ln.vs = x.v.scales + static_cast<int64_t>(h) * x.v.s_head + g * (DP / 8) / kQuadGroup * 2;
  ln.row = a.table + static_cast<uint64_t>(b) * a.max_pages;
  ln.shift = shift;
  ln.k_on[0] = t * (DP / 4) < a.dim;
  ln.k_on[1] = DP == 256 && t * (DP / 4) + 32 < a.dim;
  ln.v_on = g * (DP / 8) < a.dim;

  // One step ahead of the one that is computed.
  QuadStep<DP> st[2];
  uint32_t s = s0 + warp;
  uint32_t page = quad_page(a, ln, s, s1);
  if (s < s1) quad_load<DP>(x, ln, s, n_tok, page, st[0]);
  page = quad_page(a, ln, s + kQdWarps, s1);
  while (s < s1) {
#pragma unroll
    for (uint32_t u = 0; u < 2; ++u) {
      if (s >= s1) break;
      if (s + kQdWarps < s1) quad_load<DP>(x, ln, s + kQdWarps, n_tok, page, st[u ^ 1]);
      page = quad_page(a, ln, s + 2 * kQdWarps, s1);
      quad_step<DP, NT, F16>(a, st[u], qf, acc, b, ctx, len, row0, live_rows, static_cast<int32_t>(s * 16));
      s += kQdWarps;
    }
  }

  // Join the warps: sums of a lane's tokens first.
#pragma unroll
  for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
    for (uint32_t e = 0; e < 2; ++e)
#pragma unroll
      for (uint32_t w = 4; w < 32; w <<= 1) acc.l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, acc.l[n][e], w);
  float* so = reinterpret_cast<float*>(sm);           // [warp][row][DP]
  float* sml = so + kQdWarps * Q::kRows * DP;         // [warp][row][2]
  float* sp = sml + kQdWarps * Q::kRows * 2;          // [row][2 + DP]
#pragma unroll
  for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
    for (uint32_t e = 0; e < 2; ++e) {
      const uint32_t r = n * 8 + t * 2 + e;
      float* dst = so + (warp * Q::kRows + r) * DP + g * (DP / 8);
#pragma unroll
      for (uint32_t d = 0; d < DP / 16; ++d) *reinterpret_cast<float2*>(dst + 2 * d) = make_float2(acc.o[d][n][e], acc.o[d][n][2 + e]);
      if (g == 0) {
        sml[(warp * Q::kRows + r) * 2] = acc.m[n][e];
        sml[(warp * Q::kRows + r) * 2 + 1] = acc.l[n][e];
      }
    }
  __syncthreads();
  for (uint32_t r = warp; r < rows; r += kQdWarps) {
    float mw[kQdWarps], top = -INFINITY, sum = 0.f;
    const bool live_row = r < live_rows;
#pragma unroll
    for (uint32_t w = 0; w < kQdWarps; ++w) {
      mw[w] = live_row ? sml[(w * Q::kRows + r) * 2] : -INFINITY;
      top = fmaxf(top, mw[w]);
    }
#pragma unroll
    for (uint32_t w = 0; w < kQdWarps; ++w) {
      const float ls = live_row ? sml[(w * Q::kRows + r) * 2 + 1] : 0.f;
      // a NaN sum stays one: only an empty warp is left out
      mw[w] = mw[w] == -INFINITY ? (ls == 0.f ? 0.f : 1.f) : exp2f(mw[w] - top);
      sum += mw[w] * ls;
    }
    const uint32_t gr = row0 + r;
    const uint64_t orow = (static_cast<uint64_t>(b) * a.T + gr / a.group) * a.kv_heads * a.group + h * a.group + gr % a.group;
    const bool whole = a.splits == 1;
    const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
    float* part = a.cluster ? sp + r * (DP + 2)
                            : a.part + (static_cast<uint64_t>(item) * a.splits + split) * Q::kRows * (DP + 2) + r * (DP + 2);
    for (uint32_t d = lane * 2; d < a.dim; d += 64) {
      float v0 = 0.f, v1 = 0.f;
#pragma unroll
      for (uint32_t w = 0; w < kQdWarps; ++w) {
        const float2 y = *reinterpret_cast<const float2*>(so + (w * Q::kRows + r) * DP + d);
        if (live_row) v0 += mw[w] * y.x, v1 += mw[w] * y.y;
      }
      if (whole)
        *reinterpret_cast<uint32_t*>(static_cast<char*>(a.out) + (orow * a.dim + d) * 2) = pack2<F16>(v0 * inv, v1 * inv);
      else
        *reinterpret_cast<float2*>(part + 2 + d) = make_float2(v0, v1);
    }
    if (lane == 0) {
      if (whole) {
        if (a.lse) a.lse[orow] = row_lse<F16>(top, sum);
      } else {
        part[0] = top;
        part[1] = sum;
      }
    }
  }
  if (!a.cluster) return;
  // The splits of an item are a cluster: each CTA joins every a.splits-th row out
  // of the others' shared memory.
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (uint32_t r = split + a.splits * warp; r < rows; r += a.splits * kQdWarps) {
    auto remote = [&](uint32_t rank, uint32_t at) {
      uint32_t addr = smem_u32(sp + r * (DP + 2) + at);
      asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(addr) : "r"(rank));
      return addr;
    };
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < a.splits)
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(ml.x), "=f"(ml.y) : "r"(remote(lane, 0)) : "memory");
    float top = ml.x;
#pragma unroll
    for (int w = 4; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, w));
    top = __shfl_sync(0xFFFFFFFFu, top, 0);
    const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2f(ml.x - top);
    float sum = 0.f;
    float2 o[DP / 64];
#pragma unroll
    for (uint32_t i = 0; i < DP / 64; ++i) o[i] = make_float2(0.f, 0.f);
    for (uint32_t c = 0; c < a.splits; ++c) {
      const float fc = __shfl_sync(0xFFFFFFFFu, f, c);
      sum += fc * __shfl_sync(0xFFFFFFFFu, ml.y, c);
#pragma unroll
      for (uint32_t i = 0; i < DP / 64; ++i) {
        if (lane * 2 + i * 64 >= a.dim) continue;
        float2 y;
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(y.x), "=f"(y.y) : "r"(remote(c, 2 + lane * 2 + i * 64)) : "memory");
        o[i].x += fc * y.x, o[i].y += fc * y.y;
      }
    }
    const uint32_t gr = row0 + r;
    const uint64_t orow = (static_cast<uint64_t>(b) * a.T + gr / a.group) * a.kv_heads * a.group + h * a.group + gr % a.group;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (uint32_t i = 0; i < DP / 64; ++i) {
      const uint32_t d = lane * 2 + i * 64;
      if (d < a.dim)
        *reinterpret_cast<uint32_t*>(static_cast<char*>(a.out) + (orow * a.dim + d) * 2) = pack2<F16>(o[i].x * inv, o[i].y * inv);
    }
    if (lane == 0 && a.lse) a.lse[orow] = row_lse<F16>(top, sum);
  }
  // no CTA leaves while another reads its shared memory
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Joins the chunks of items: a warp per row, in the chunks' order.
template <uint32_t DP, bool F16>
__global__ void __launch_bounds__(128) k_kv4_join(const AttendArgs a, uint32_t row_tiles, uint32_t tile_rows, uint32_t n_rows,
                                                  uint32_t chunk) {
  pdl_begin();
  const uint32_t lane = threadIdx.x & 31u;
  const uint64_t w = static_cast<uint64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const uint64_t item = w / tile_rows;
  const uint32_t r = static_cast<uint32_t>(w % tile_rows), tile = static_cast<uint32_t>(item % row_tiles);
  const uint32_t h = static_cast<uint32_t>(item / row_tiles % a.kv_heads);
  const uint64_t b = item / row_tiles / a.kv_heads;
  const uint32_t gr = tile * tile_rows + r;
  if (b >= a.n_seqs || gr >= n_rows) return;
  // the chunks that the item's CTAs have walked
  const int32_t len = clamp_len(a.lens[b], a.page_tokens, a.max_pages);
  const int32_t live = a.n_live ? a.n_live[b] : static_cast<int32_t>(a.T);
  const int32_t n_live = live < 0 ? 0 : (live > static_cast<int32_t>(a.T) ? static_cast<int32_t>(a.T) : live);
  const bool any = static_cast<uint32_t>(n_live) * a.group > tile * tile_rows;
  uint32_t parts = any ? ceil_div(ceil_div(static_cast<uint32_t>(len), 16), chunk) : 1u;
  if (parts == 0) parts = 1;
  const float* part = a.part + (item * a.splits * tile_rows + r) * (DP + 2);
  const uint64_t stride = static_cast<uint64_t>(tile_rows) * (DP + 2);
  float top = -INFINITY;
  for (uint32_t s = lane; s < parts; s += 32) top = fmaxf(top, part[s * stride]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  float sum = 0.f;
  float2 acc[DP / 64];
#pragma unroll
  for (uint32_t i = 0; i < DP / 64; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (uint32_t s = 0; s < parts; ++s) {
    const float2 ml = *reinterpret_cast<const float2*>(part + s * stride);
    const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2f(ml.x - top);
    sum += f * ml.y;
#pragma unroll
    for (uint32_t i = 0; i < DP / 64; ++i) {
      const uint32_t d = lane * 2 + i * 64;
      if (d < a.dim) {
        const float2 y = *reinterpret_cast<const float2*>(part + s * stride + 2 + d);
        acc[i].x += f * y.x, acc[i].y += f * y.y;
      }
    }
  }
  const uint64_t orow = (b * a.T + gr / a.group) * a.kv_heads * a.group + h * a.group + gr % a.group;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (uint32_t i = 0; i < DP / 64; ++i) {
    const uint32_t d = lane * 2 + i * 64;
    if (d < a.dim)
      *reinterpret_cast<uint32_t*>(static_cast<char*>(a.out) + (orow * a.dim + d) * 2) = pack2<F16>(acc[i].x * inv, acc[i].y * inv);
  }
  if (lane == 0 && a.lse) a.lse[orow] = row_lse<F16>(top, sum);
}

// ---------------------------------------------------------------------------

struct QuadPlan {
  uint32_t dp, rows_per, tiles, splits, cluster, chunk;  // chunk: steps of a CTA where splits are not a cluster
  uint64_t items;
};

static QuadPlan quad_plan(uint32_t n_seqs, uint32_t kv_heads, uint64_t rows, uint32_t dim, uint64_t tokens, int device) {
  QuadPlan p = {};
  p.dp = dim <= 64 ? 64 : (dim <= 128 ? 128 : 256);
  p.rows_per = rows > 8 && p.dp < 256 ? 16 : 8;
  p.tiles = static_cast<uint32_t>((rows + p.rows_per - 1) / p.rows_per);
  p.items = static_cast<uint64_t>(n_seqs) * kv_heads * p.tiles;
  const uint64_t resident = static_cast<uint64_t>(sm_count(device)) * (p.dp == 256 || p.rows_per == 16 ? 2 : 4);
  const uint64_t steps = (tokens + 15) / 16;
  uint64_t s = 1;
  while (s < 8 && 2 * s * p.items <= resident && steps >= 2 * s * 2 * kQdWarps) s *= 2;
  p.splits = static_cast<uint32_t>(s);
  p.cluster = s > 1;
  // Chunks of 64 steps, where they are more than a cluster's worth: units enough that
  // ragged lengths even out over the SMs.
  const uint64_t chunk = 64, parts = (steps + chunk - 1) / chunk;
  if (parts > p.splits && parts * p.items > resident) {
    p.splits = static_cast<uint32_t>(parts);
    p.cluster = 0;
    p.chunk = static_cast<uint32_t>(chunk);
  } else {
    p.chunk = static_cast<uint32_t>(steps);
  }
  return p;
}

size_t kv4_attend_workspace(uint32_t n_seqs, uint32_t kv_heads, uint64_t rows, uint32_t dim, uint64_t tokens, int device) {
  const QuadPlan p = quad_plan(n_seqs, kv_heads, rows, dim, tokens, device);
  return p.cluster || p.splits == 1 ? 0 : p.items * p.splits * p.rows_per * (p.dp + 2) * 4;
}

template <uint32_t DP, uint32_t NT, bool F16>
static int launch_quad(Attend4Args& x, const QuadPlan& p, cudaStream_t stream) {
  using Q = Quad<DP, NT, F16>;
  static_assert(Q::kBytes <= 48 * 1024, "no attribute is set for the shared memory");
  int32_t shift = -2;
  if (x.a.page_tokens % 16 == 0) {
    const uint32_t steps = x.a.page_tokens / 16;
    shift = steps & (steps - 1) ? -1 : 0;
    while (shift >= 0 && (1u << shift) < steps) ++shift;
  }
  const int rc = kv_launch("k_kv4_attend", k_kv4_attend<DP, NT, F16>, dim3(static_cast<unsigned>(p.items * p.splits)), kQdWarps * 32,
                           Q::kBytes, p.cluster ? p.splits : 1, stream, x, p.tiles, shift, p.chunk);
  if (rc != IBP_OK || p.cluster || p.splits == 1) return rc;
  const uint64_t warps = p.items * Q::kRows;
  return kv_launch("k_kv4_join", k_kv4_join<DP, F16>, dim3(static_cast<unsigned>((warps + 3) / 4)), 128, 0, 1, stream, x.a, p.tiles,
                   Q::kRows, x.a.T * x.a.group, p.chunk);
}

int launch_kv4_attend(Attend4Args& x, int device, size_t ws_bytes, cudaStream_t stream) {
  AttendArgs& a = x.a;
  const uint64_t tokens = static_cast<uint64_t>(a.max_pages) * a.page_tokens;
  const QuadPlan p = quad_plan(a.n_seqs, a.kv_heads, static_cast<uint64_t>(a.T) * a.group, a.dim, tokens, device);
  if (p.items * p.splits > 0x7FFFFFFFull) {
    set_detail("more than 2^31 blocks");
    return IBP_EINVAL;
  }
  if (!p.cluster && p.splits > 1 && (!a.part || ws_bytes < p.items * p.splits * p.rows_per * (p.dp + 2) * 4)) return IBP_EINVAL;
  a.splits = p.splits;
  a.cluster = p.cluster;
  auto go = [&](auto f16) {
    constexpr bool F = decltype(f16)::value;
    if (p.dp == 64) return p.rows_per == 16 ? launch_quad<64, 2, F>(x, p, stream) : launch_quad<64, 1, F>(x, p, stream);
    if (p.dp == 128) return p.rows_per == 16 ? launch_quad<128, 2, F>(x, p, stream) : launch_quad<128, 1, F>(x, p, stream);
    return launch_quad<256, 1, F>(x, p, stream);
  };
  return a.f16 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace ibp

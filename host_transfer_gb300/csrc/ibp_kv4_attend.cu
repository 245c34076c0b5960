// ibp_kv4_attend.cu - attention of few queries over a paged cache held in 4 bits.
//
// A CTA holds 8 or 16 query rows of one sequence and kv head (drafted tokens times
// the group's heads) and walks a share of the tokens; its four warps take a step of 16
// or 32 tokens in turn, each with a ring of stages that asynchronous copies fill and a
// running maximum and sum of its own.  The products are taken transposed, S^T = K Q^T and
// O^T = V^T P^T, so that tokens and dimensions fill the 16-row side of mma.m16n8k16
// and queries the 8-wide side.
//
// A dot product may add its dimensions in any order, so a lane takes for its part of
// a K row the codes that lie next to one another, up to 32 of one group: one 16-byte
// read, one scale, and the queries are laid out to match.  The same holds for the rows of
// O^T: a lane takes neighbouring dimensions of V for the four tokens that are its part
// of the product, and pairs of tokens are made by byte permutations.  Codes are
// decoded in registers and are the operands.
//
// Probabilities are rounded to the cache's type, as the product with V needs them (by half a
// step at most); their sum is of those not rounded, in 32 bits like scores, maxima and
// outputs.  Against 64 bits the outputs of the timed cases are off by 0.0018 to 0.0019 of their
// size in bfloat16, where rounding the exact ones gives 0.0017, and by 0.00024 against 0.00021 in
// half precision.
//
// Work is split evenly over the CTAs that the GPU holds at once, by tiles of all items
// in a row, as in the tensor-core kernel (ibp_kv_tree.cuh), whose walk and join serve
// here too: ragged lengths cost nothing.
//
// Decoding is what counts beside the cache's bytes: 12 instructions for 8 elements
// (a shift, a mask with the exponent put in, one fused multiply-add a pair).
//
// Measured on one GB300: 32 ragged caches of up to 32768 tokens, 8 kv heads of 8 query
// heads of 128, one token each (798 MB): 200 us with cold caches, 4.0 TB/s; the same
// caches in 16 bits, 3.5 times the bytes, take 422 us.  16 tokens of K and V cost about 440
// warp instructions, of which 192 decode, 32 are products and most others move operands
// and find maxima.  Issue slots are 61 % used, the pipe of shifts and masks 53 %, DRAM 52 %: with
// 2.7 warps a scheduler no more of the steps' latencies (the decoding, the products into one
// accumulator, the maxima over the lanes) is covered.  A single cache of 777 tokens: 15 us
// cold, 9 us warm, the latency of table, codes and a second launch for the join.
// Stages by bulk copies instead of 16-byte ones were 2 % faster for 8 rows and 6 % slower
// for 16, and were not kept.
#include <type_traits>

#include "ibp_kv_tree.cuh"

namespace ibp {

constexpr uint32_t kQdWarps = 4;
// CTAs of a SM for 8 rows: at 168 registers a thread the decoding has the independent
// instructions that four CTAs at 128 lack (32 ragged caches of up to 32768 tokens, 8 kv
// heads of 8 query heads: 199 us against 216 us).
constexpr uint32_t kQdCtas = 3;

template <uint32_t DP, uint32_t NT>
struct Quad {
  // Tokens of a step: what a step costs besides decoding and products (maxima over the
  // lanes, bookkeeping) is shared by two blocks of 16 where the registers allow it.
  static constexpr uint32_t kMma = DP == 256 ? 1 : 2;
  static constexpr uint32_t kSub = 16 * kMma;
  static constexpr uint32_t kTile = kSub * kQdWarps;       // a step of every warp
  static constexpr uint32_t kRows = 8 * NT;
  static constexpr uint32_t kCodes = kSub * DP / 2;        // bytes of K's or V's codes in a stage
  static constexpr uint32_t kScale = DP / 16;              // bytes of a token's scales
  static constexpr uint32_t kStage = 2 * kCodes + 2 * kSub * kScale;
  static constexpr uint32_t kStages = 3;
  static constexpr uint32_t kRing = kQdWarps * kStages * kStage;
  static constexpr uint32_t kJoin = kQdWarps * kRows * (DP + 2) * 4;
  static constexpr uint32_t kBytes = kRing > kJoin ? kRing : kJoin;

  static __device__ __forceinline__ bool sees(const AttendArgs& a, uint32_t b, int32_t ctx, int32_t len, uint32_t r, int32_t pos) {
    if (pos >= len) return false;
    if (pos < ctx) return true;
    const uint32_t t = r / a.group, i = static_cast<uint32_t>(pos - ctx);
    if (!a.mask) return i <= t;
    return (a.mask[(static_cast<uint64_t>(b) * a.T + t) * a.mask_words + (i >> 5)] >> (i & 31u)) & 1u;
  }

  // Place of 16 bytes of a token's codes: a line of 128 bytes holds 4, 2 or 1 tokens,
  // its pieces in an order that differs from line to line, so that neither the reads of K
  // (eight lanes on neighbouring rows) nor those of V (lanes on rows two apart) meet in a
  // bank.  Eight tokens on, the order is the same.
  static __device__ __forceinline__ uint32_t at(uint32_t tok, uint32_t c) {
    const uint32_t piece = tok * (DP / 32) + c, line = piece >> 3;
    const uint32_t turn = DP == 64 ? (line & 1u) * 2 : (DP == 128 ? (line & 3u) * 2 : line & 7u);
    return (piece ^ turn) * 16;
  }
};

// A copy of N bytes into shared memory, or zeros.
template <uint32_t N>
__device__ __forceinline__ void quad_copy(uint32_t dst, const void* src, bool on) {
  if constexpr (N == 16)
    cp16(dst, src, on);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(on ? N : 0u) : "memory");
}

// How the cache is laid out: pages of whole blocks of 16 tokens, a token's scales all of
// DP's and aligned (kEven); anything else (kAny).
enum QuadForm { kEven, kAny };

// Pages of a step's blocks of 16 (kEven), or the page and slot of the lane's token
// (kAny), still on their way.
struct QuadSpot {
  uint32_t page[2];
  bool there;
};

template <QuadForm FORM, uint32_t KM>
__device__ __forceinline__ QuadSpot quad_spot(const AttendArgs& a, int32_t shift, const int32_t* row, uint32_t tok, uint32_t n_tok) {
  QuadSpot s;
  s.page[0] = s.page[1] = 0xFFFFFFFFu;
  auto page_of = [&](uint32_t x) { return static_cast<uint32_t>(__ldg(row + (shift >= 0 ? x >> shift : x / a.page_tokens))); };
  if (FORM == kEven) {
    s.there = tok < n_tok;
    if (s.there) s.page[0] = page_of(tok);
    if (KM == 2 && tok + 16 < n_tok) s.page[1] = page_of(tok + 16);
  } else {
    const uint32_t mine = tok + (threadIdx.x & 31u);
    s.there = (threadIdx.x & 31u) < 16 * KM && mine < n_tok;
    if (s.there) s.page[0] = page_of(mine);
  }
  return s;
}

// Asks for the codes and scales of the step at token tok.  Tokens past the last, pages
// that are not there and dimensions that do not exist become zeros.  base: K's codes and
// scales, V's codes and scales of this head; with kEven of this lane's chunk and first
// token (codes) and of this lane's token modulo 16 (scales).
template <uint32_t DP, uint32_t NT, QuadForm FORM>
__device__ __forceinline__ void quad_fill(const TcArgs& t, const QuadSpot& sp, int32_t shift, uint32_t tok, uint32_t n_tok,
                                          const char* const (&base)[4], uint32_t stage, unsigned char* stage_p) {
  using Q = Quad<DP, NT>;
  const AttendArgs& a = t.a;
  const uint32_t lane = threadIdx.x & 31u;
  constexpr uint32_t kChunks = DP / 32, kPer = 32 / kChunks;  // 16-byte chunks of a token, tokens an instruction
  constexpr uint32_t kTurns = kPer < 8 ? 8 / kPer : 1;        // instructions after which the order repeats
  const uint32_t c = lane % kChunks, r0 = lane / kChunks;
  uint32_t dst[kTurns];
#pragma unroll
  for (uint32_t i = 0; i < kTurns; ++i) dst[i] = stage + Q::at(r0 + i * kPer, c) - i * kPer * (DP / 2);
  if (FORM == kEven) {
    // strides of 32 bits, and a page's tokens within 32 bits
    auto small = [](int64_t x) { return static_cast<uint32_t>(x); };
    auto at_page = [&](uint32_t page, int64_t stride) { return static_cast<uint64_t>(page) * small(stride); };
    const uint32_t left = n_tok - tok;
    const char *k[Q::kMma], *v[Q::kMma];
    bool good[Q::kMma];
    uint32_t slot[Q::kMma];
#pragma unroll
    for (uint32_t x = 0; x < Q::kMma; ++x) {
      const uint32_t first = tok + 16 * x;
      slot[x] = shift >= 0 ? first & ((1u << shift) - 1u) : first % a.page_tokens;
      good[x] = sp.page[x] < a.n_pages;
      if (!good[x] && first < n_tok) kv_status(a.status, IBP_ERANGE);
      const uint32_t page = good[x] ? sp.page[x] : 0;
      k[x] = base[0] + at_page(page, t.four[0].page_stride) + slot[x] * small(t.four[0].token_stride);
      v[x] = base[2] + at_page(page, t.four[1].page_stride) + slot[x] * small(t.four[1].token_stride);
    }
    const bool all = left >= Q::kSub && good[0] && good[Q::kMma - 1];
    const uint32_t mine = lane / 16 % Q::kMma;  // the block of this lane's token
    const uint32_t page = (mine ? good[Q::kMma - 1] : good[0]) ? (mine ? sp.page[Q::kMma - 1] : sp.page[0]) : 0;
    const uint32_t sl = mine ? slot[Q::kMma - 1] : slot[0];
    const uint32_t to = stage + 2 * Q::kCodes + lane * Q::kScale;
    const char* ks = base[1] + at_page(page, t.four[0].s_page) + sl * small(t.four[0].s_token);
    const char* vs = base[3] + at_page(page, t.four[1].s_page) + sl * small(t.four[1].s_token);
    constexpr uint32_t kEach = 16 / kPer;  // instructions a block
    if (all) {
#pragma unroll
      for (uint32_t i = 0; i < Q::kSub / kPer; ++i) {
        quad_copy<16>(dst[i % kTurns] + i * kPer * (DP / 2), k[i / kEach] + i % kEach * kPer * small(t.four[0].token_stride), true);
        quad_copy<16>(dst[i % kTurns] + i * kPer * (DP / 2) + Q::kCodes, v[i / kEach] + i % kEach * kPer * small(t.four[1].token_stride), true);
      }
      if (Q::kSub == 32 || lane < Q::kSub) {
        quad_copy<Q::kScale>(to, ks, true);
        quad_copy<Q::kScale>(to + Q::kSub * Q::kScale, vs, true);
      }
    } else {
#pragma unroll
      for (uint32_t i = 0; i < Q::kSub / kPer; ++i) {
        const bool on = good[i / kEach] && r0 + i * kPer < left;
        quad_copy<16>(dst[i % kTurns] + i * kPer * (DP / 2), on ? k[i / kEach] + i % kEach * kPer * small(t.four[0].token_stride) : base[0], on);
        quad_copy<16>(dst[i % kTurns] + i * kPer * (DP / 2) + Q::kCodes, on ? v[i / kEach] + i % kEach * kPer * small(t.four[1].token_stride) : base[2], on);
      }
      if (lane < Q::kSub) {
        const bool on = (mine ? good[Q::kMma - 1] : good[0]) && lane < left;
        quad_copy<Q::kScale>(to, on ? ks : base[1], on);
        quad_copy<Q::kScale>(to + Q::kSub * Q::kScale, on ? vs : base[3], on);
      }
    }
    return;
  }
  const bool good = sp.there && sp.page[0] < a.n_pages;
  if (sp.there && !good) kv_status(a.status, IBP_ERANGE);
  const bool col = c * 32 < a.dim;
  const uint32_t page = good ? sp.page[0] : 0xFFFFFFFFu, own = tok + lane;
  const uint32_t slot_of_mine = shift >= 0 ? own & ((1u << shift) - 1u) : own % a.page_tokens;
#pragma unroll
  for (uint32_t i = 0; i < Q::kSub / kPer; ++i) {
    const uint32_t r = r0 + i * kPer;
    const uint32_t pg = __shfl_sync(0xFFFFFFFFu, page, r), slot = __shfl_sync(0xFFFFFFFFu, slot_of_mine, r);
    const bool on = pg != 0xFFFFFFFFu && col;
    const int64_t p = on ? pg : 0, sl = on ? slot : 0;
    quad_copy<16>(dst[i % kTurns] + i * kPer * (DP / 2), base[0] + p * t.four[0].page_stride + sl * t.four[0].token_stride + (on ? c * 16 : 0), on);
    quad_copy<16>(dst[i % kTurns] + i * kPer * (DP / 2) + Q::kCodes, base[2] + p * t.four[1].page_stride + sl * t.four[1].token_stride + (on ? c * 16 : 0), on);
  }
  if (lane < Q::kSub) {
    const int64_t p = good ? page : 0, sl = good ? slot_of_mine : 0;
#pragma unroll
    for (uint32_t kv = 0; kv < 2; ++kv) {
      const char* src = base[2 * kv + 1] + p * t.four[kv].s_page + sl * t.four[kv].s_token;
#pragma unroll
      for (uint32_t g = 0; g < DP / 32; ++g)
        *reinterpret_cast<uint16_t*>(stage_p + 2 * Q::kCodes + (kv * Q::kSub + lane) * Q::kScale + 2 * g) =
            good && g * 32 < a.dim ? __ldg(reinterpret_cast<const uint16_t*>(src) + g) : uint16_t(0);
    }
  }
}

template <uint32_t DP, uint32_t NT, bool F16, QuadForm FORM>
__global__ void __launch_bounds__(kQdWarps * 32, DP == 256 || NT == 2 ? 2 : kQdCtas) k_kv4_attend(const __grid_constant__ TcArgs t, int32_t shift) {
  using Q = Quad<DP, NT>;
  constexpr uint32_t kM = Q::kMma, kSub = Q::kSub;
  const AttendArgs& a = t.a;
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ struct {
    uint32_t pair0, b0, sums[kQdWarps];
    uint64_t in0;
  } sh;
  pdl_begin();
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, g = lane >> 2, tq = lane & 3u;

  // Where this CTA's range begins, as in k_kv_tree.
  {
    uint32_t n = 0;
    for (uint32_t b = threadIdx.x; b < a.n_seqs; b += kQdWarps * 32) n += tiles_of<Q::kTile>(a, b);
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    if (lane == 0) sh.sums[warp] = n;
    __syncthreads();
  }
  uint64_t total = 0;
#pragma unroll
  for (uint32_t i = 0; i < kQdWarps; ++i) total += sh.sums[i];
  const uint64_t block = total * a.kv_heads;  // tiles of a row block
  total = block * t.row_pairs;
  const uint64_t share = (total + t.n_ctas - 1) / t.n_ctas;
  const uint64_t at = blockIdx.x * share < total ? blockIdx.x * share : total;
  const uint64_t end = total - at < share ? total : at + share;
  if (warp == 0 && at < end) {
    const uint32_t pair = static_cast<uint32_t>(at / block);
    const uint64_t in = at - pair * block;
    uint64_t seen = 0;
    for (uint32_t c = 0; c < a.n_seqs; c += 32) {
      const uint32_t b = c + lane;
      uint64_t n = b < a.n_seqs ? static_cast<uint64_t>(tiles_of<Q::kTile>(a, b)) * a.kv_heads : 0, incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= static_cast<uint32_t>(o)) incl += v;
      }
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, seen + incl > in);
      if (hit) {
        if (lane == static_cast<uint32_t>(__ffs(hit) - 1)) {
          sh.pair0 = pair;
          sh.b0 = b;
          sh.in0 = in - (seen + incl - n);
        }
        break;
      }
      seen += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
  }
  __syncthreads();
  TcWalkOf<Q::kTile> walk(t, sh.pair0, sh.b0, sh.in0, at, end);
  TcSeg s;
  bool first_seg = true;
  const quad::Magic<F16> magic;
  unsigned char* const ring_p = sm + warp * Q::kStages * Q::kStage;
  const uint32_t ring = smem_u32(ring_p);
  if (threadIdx.x == 0 && blockIdx.x == 0)
    t.first[t.n_ctas] = make_int4(static_cast<int>(share & 0xFFFFFFFFu), static_cast<int>(share >> 32), 0, 0);
  if (threadIdx.x == 0 && at >= end) t.first[blockIdx.x] = make_int4(-1, 0, 0, 0);

  while (walk.next(&s)) {
    const uint32_t row0 = s.pair * Q::kRows, b = s.b, h = s.h;
    const int32_t len = s.len, ctx = s.ctx;
    if (threadIdx.x == 0) {
      const int32_t raw = a.lens[b], n = a.n_live ? a.n_live[b] : static_cast<int32_t>(a.T);
      if (raw != len || n != s.n_live || n > len) kv_status(a.status, IBP_ERANGE);
      if (first_seg) t.first[blockIdx.x] = make_int4(b, h, s.pair, s.tile0);
    }
    first_seg = false;
    const uint32_t all_rows = a.T * a.group;
    const uint32_t rows = all_rows - row0 < Q::kRows ? all_rows - row0 : Q::kRows;
    const uint32_t lr = static_cast<uint32_t>(s.n_live) * a.group;
    const uint32_t live_rows = lr > row0 ? (lr - row0 < rows ? lr - row0 : rows) : 0;
    const uint32_t n_tok = live_rows && len > 0 ? static_cast<uint32_t>(len) : 0;

    const int32_t* row = a.table + static_cast<uint64_t>(b) * a.max_pages;
    constexpr uint32_t kChunks = DP / 32;
    const uint32_t ahead_c = FORM == kEven ? lane % kChunks * 16 : 0, ahead_r = FORM == kEven ? lane / kChunks : 0;
    const uint32_t ahead_t = FORM == kEven ? lane % 16 : 0;
    const char* const base[4] = {
        t.four[0].codes + static_cast<int64_t>(h) * t.four[0].head_stride + ahead_c + static_cast<int64_t>(ahead_r) * t.four[0].token_stride,
        t.four[0].scales + static_cast<int64_t>(h) * t.four[0].s_head + static_cast<int64_t>(ahead_t) * t.four[0].s_token,
        t.four[1].codes + static_cast<int64_t>(h) * t.four[1].head_stride + ahead_c + static_cast<int64_t>(ahead_r) * t.four[1].token_stride,
        t.four[1].scales + static_cast<int64_t>(h) * t.four[1].s_head + static_cast<int64_t>(ahead_t) * t.four[1].s_token};
    // Step j of this warp: tokens of tile tile0 + j; without live rows there is none.
    const uint32_t steps = n_tok ? s.tiles : 0;
    auto token = [&](uint32_t j) { return (s.tile0 + j) * Q::kTile + warp * kSub; };
    auto spot = [&](uint32_t j) { return quad_spot<FORM, kM>(a, shift, row, token(j), j < steps ? n_tok : 0); };
    auto fill = [&](uint32_t j, const QuadSpot& sp, uint32_t stage) {
      if (token(j) < n_tok) {
        quad_fill<DP, NT, FORM>(t, sp, shift, token(j), n_tok, base, ring + stage * Q::kStage, ring_p + stage * Q::kStage);
      } else {  // the item's last tile, past its last token
        for (uint32_t i = lane * 16; i < Q::kStage; i += 512)
          *reinterpret_cast<uint4*>(ring_p + stage * Q::kStage + i) = make_uint4(0u, 0u, 0u, 0u);
      }
    };
    constexpr uint32_t kAhead = Q::kStages - 1;
    QuadSpot sp[kAhead];
#pragma unroll
    for (uint32_t i = 0; i < kAhead; ++i) sp[i] = spot(i);
    QuadSpot next = spot(kAhead);

    // Q^T as B operands, dimensions in the order in which a lane decodes K.
    uint32_t qf[NT][DP / 16][2];
#pragma unroll
    for (uint32_t n = 0; n < NT; ++n) {
      const bool on = n * 8 + g < live_rows;
      const uint32_t r = on ? row0 + n * 8 + g : 0;
      const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q + static_cast<int64_t>(b) * a.q_seq + static_cast<int64_t>(r / a.group) * a.q_token +
                                                            static_cast<int64_t>(h * a.group + r % a.group) * a.q_head);
#pragma unroll
      for (uint32_t w = 0; w < DP / 32; ++w) {  // eight dimensions
        const uint32_t d = tq * (DP / 4) + 8 * w;
        const bool in = on && d < a.dim;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (in) {
          if (t.q16)
            x = *reinterpret_cast<const uint4*>(q + d);
          else
            x = make_uint4(q[d] | static_cast<uint32_t>(q[d + 1]) << 16, q[d + 2] | static_cast<uint32_t>(q[d + 3]) << 16,
                           q[d + 4] | static_cast<uint32_t>(q[d + 5]) << 16, q[d + 6] | static_cast<uint32_t>(q[d + 7]) << 16);
        }
        qf[n][2 * w][0] = __byte_perm(x.x, x.z, 0x5410), qf[n][2 * w][1] = __byte_perm(x.x, x.z, 0x7632);
        qf[n][2 * w + 1][0] = __byte_perm(x.y, x.w, 0x5410), qf[n][2 * w + 1][1] = __byte_perm(x.y, x.w, 0x7632);
      }
    }
#pragma unroll
    for (uint32_t i = 0; i < kAhead; ++i) {
      if (i < steps) fill(i, sp[i], i);
      cp_commit();
    }

    float o[DP / 16][NT][4];  // rows: dimensions 2j and 2j + 1 of the lane's; columns: queries 2t, 2t + 1
    float m[NT][2], l[NT][2];
#pragma unroll
    for (uint32_t n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (uint32_t d = 0; d < DP / 16; ++d) o[d][n][0] = o[d][n][1] = o[d][n][2] = o[d][n][3] = 0.f;
    }

    // This lane's places in a stage, for the first of the tokens eight apart.
    const uint32_t k_at = DP == 64 ? Q::at(g, tq / 2) + (tq & 1u) * 8 : Q::at(g, tq * (DP == 256 ? 2 : 1));
    const uint32_t k_two = DP == 256 ? Q::at(g, tq * 2 + 1) : 0;
    const uint32_t v_at[2] = {Q::at(2 * tq, g * (DP / 16) / 16) + g * (DP / 16) % 16, Q::at(2 * tq + 1, g * (DP / 16) / 16) + g * (DP / 16) % 16};
    uint32_t slot = 0;  // of step j
#pragma unroll 1
    for (uint32_t j = 0; j < steps; ++j) {
      __syncwarp();  // every lane is done with the stage that is filled next
      if (j + kAhead < steps) {
        fill(j + kAhead, next, slot == 0 ? kAhead : slot - 1);
      }
      next = spot(j + kAhead + 1);
      cp_commit();
      cp_wait<kAhead>();
      __syncwarp();
      const unsigned char* st = ring_p + slot * Q::kStage;
      const unsigned char *ksc = st + 2 * Q::kCodes, *vsc = ksc + kSub * Q::kScale;
      slot = slot == kAhead ? 0 : slot + 1;
      const int32_t first = static_cast<int32_t>(token(j));
      float c[kM][NT][4];
#pragma unroll
      for (uint32_t x = 0; x < kM; ++x) {
#pragma unroll
        for (uint32_t n = 0; n < NT; ++n) c[x][n][0] = c[x][n][1] = c[x][n][2] = c[x][n][3] = 0.f;
        // this lane's dimensions: DP / 4 from tq * DP / 4 on
        constexpr uint32_t kW = DP / 32, kG = DP == 256 ? 2 : 1;
        uint32_t w[2][kW];
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
          if constexpr (kW == 2) {
            const uint2 u = *reinterpret_cast<const uint2*>(st + k_at + (16 * x + 8 * i) * (DP / 2));
            w[i][0] = u.x, w[i][1] = u.y;
          } else {
#pragma unroll
            for (uint32_t e = 0; e < kG; ++e) {
              const uint4 u = *reinterpret_cast<const uint4*>(st + (e ? k_two : k_at) + (16 * x + 8 * i) * (DP / 2));
              w[i][4 * e] = u.x, w[i][4 * e + 1] = u.y, w[i][4 * e + 2] = u.z, w[i][4 * e + 3] = u.w;
            }
          }
        }
#pragma unroll
        for (uint32_t e = 0; e < kG; ++e) {
          const uint32_t gi = DP == 64 ? tq / 2 : tq * kG + e;
          const quad::Pair<F16> p0(*reinterpret_cast<const uint16_t*>(ksc + (16 * x + g) * Q::kScale + 2 * gi) * 0x10001u);
          const quad::Pair<F16> p1(*reinterpret_cast<const uint16_t*>(ksc + (16 * x + g + 8) * Q::kScale + 2 * gi) * 0x10001u);
#pragma unroll
          for (uint32_t y = e * (kW / kG); y < (e + 1) * (kW / kG); ++y) {
            const uint32_t lo[4] = {quad::decode<F16, 0>(w[0][y], p0, magic), quad::decode<F16, 0>(w[1][y], p1, magic),
                                    quad::decode<F16, 1>(w[0][y], p0, magic), quad::decode<F16, 1>(w[1][y], p1, magic)};
            const uint32_t hi[4] = {quad::decode<F16, 2>(w[0][y], p0, magic), quad::decode<F16, 2>(w[1][y], p1, magic),
                                    quad::decode<F16, 3>(w[0][y], p0, magic), quad::decode<F16, 3>(w[1][y], p1, magic)};
#pragma unroll
            for (uint32_t n = 0; n < NT; ++n) {
              mma16816<F16>(c[x][n], lo, qf[n][2 * y][0], qf[n][2 * y][1]);
              mma16816<F16>(c[x][n], hi, qf[n][2 * y + 1][0], qf[n][2 * y + 1][1]);
            }
          }
        }
      }
      // Scores in powers of two; what a row does not see is -infinity.
      const bool open = first + static_cast<int32_t>(kSub) <= (ctx < len ? ctx : len);
#pragma unroll
      for (uint32_t x = 0; x < kM; ++x)
#pragma unroll
        for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) c[x][n][e] *= a.scale_log2;
      if (!open) {
#pragma unroll
        for (uint32_t x = 0; x < kM; ++x)
#pragma unroll
          for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) {
              const uint32_t r = n * 8 + tq * 2 + (e & 1u);
              const int32_t pos = first + static_cast<int32_t>(16 * x + g + (e < 2 ? 0 : 8));
              if (r >= live_rows || !Q::sees(a, b, ctx, len, row0 + r, pos)) c[x][n][e] = -INFINITY;
            }
      }
      float cm[NT][2];
      bool grow = false;
#pragma unroll
      for (uint32_t n = 0; n < NT; ++n) {
#pragma unroll
        for (uint32_t e = 0; e < 2; ++e) {
          cm[n][e] = fmaxf(c[0][n][e], c[0][n][2 + e]);
          if (kM == 2) cm[n][e] = fmaxf(cm[n][e], fmaxf(c[kM - 1][n][e], c[kM - 1][n][2 + e]));
#pragma unroll
          for (uint32_t w = 4; w < 32; w <<= 1) cm[n][e] = fmaxf(cm[n][e], __shfl_xor_sync(0xFFFFFFFFu, cm[n][e], w));
          if (F16) cm[n][e] = __fadd_ru(cm[n][e], -kLift<F16>);
          grow = grow || cm[n][e] > m[n][e];
        }
      }
      if (__any_sync(0xFFFFFFFFu, grow)) {
        // Rescaled at once, so that a row's largest probability is a power of two and its
        // rounding to the cache's type costs nothing.
#pragma unroll
        for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
          for (uint32_t e = 0; e < 2; ++e) {
            const float top = fmaxf(m[n][e], cm[n][e]);
            const float f = top > m[n][e] ? ex2(m[n][e] - top) : 1.f;
            m[n][e] = top;
            l[n][e] *= f;
#pragma unroll
            for (uint32_t d = 0; d < DP / 16; ++d) o[d][n][e] *= f, o[d][n][2 + e] *= f;
          }
      }
      uint32_t pf[kM][NT][2];
#pragma unroll
      for (uint32_t n = 0; n < NT; ++n) {
        const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
        for (uint32_t x = 0; x < kM; ++x) {
          float(&p)[4] = c[x][n];
          p[0] = ex2(p[0] - m0), p[1] = ex2(p[1] - m1), p[2] = ex2(p[2] - m0), p[3] = ex2(p[3] - m1);
          l[n][0] += p[0] + p[2];
          l[n][1] += p[1] + p[3];
          pf[x][n][0] = transpose8(pack2<F16>(p[0], p[1]));
          pf[x][n][1] = transpose8(pack2<F16>(p[2], p[3]));
        }
      }
#pragma unroll
      for (uint32_t x = 0; x < kM; ++x) {
        constexpr uint32_t kW = DP / 64;
        // tokens 2t, 2t + 1, 2t + 8, 2t + 9; DP / 8 dimensions from g * DP / 8 on
        uint32_t w[4][kW], sc[4];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          const uint32_t tok = 16 * x + 2 * tq + (i & 1u) + (i >> 1) * 8;
          const unsigned char* src = st + Q::kCodes + v_at[i & 1u] + (16 * x + (i >> 1) * 8) * (DP / 2);
          if constexpr (kW == 4) {
            const uint4 u = *reinterpret_cast<const uint4*>(src);
            w[i][0] = u.x, w[i][1] = u.y, w[i][2] = u.z, w[i][3] = u.w;
          } else if constexpr (kW == 2) {
            const uint2 u = *reinterpret_cast<const uint2*>(src);
            w[i][0] = u.x, w[i][1] = u.y;
          } else {
            w[i][0] = *reinterpret_cast<const uint32_t*>(src);
          }
          sc[i] = *reinterpret_cast<const uint16_t*>(vsc + tok * Q::kScale + g * (DP / 8) / kQuadGroup * 2);
        }
        if (!open) {
          // Groups of V that may hold infinities or NaN: a row that does not see them must
          // not meet them, even with probability zero.  They leave the product and are
          // added to the rows that see them.
          bool bad = false;
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) bad = bad || quad::odd<F16>(quad::scale_bits<F16>(sc[i]));
          if (__any_sync(0xFFFFFFFFu, bad)) {
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
#pragma unroll 1
              for (uint32_t tt = 0; tt < 4; ++tt) {
                const uint32_t tok = 2 * tt + (i & 1u) + (i >> 1) * 8;  // its row in S^T
                const uint32_t from = (lane & 28u) | tt, sb = quad::scale_bits<F16>(__shfl_sync(0xFFFFFFFFu, sc[i], from));
                uint32_t words[kW];
#pragma unroll
                for (uint32_t y = 0; y < kW; ++y) words[y] = __shfl_sync(0xFFFFFFFFu, w[i][y], from);
#pragma unroll
                for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
                  for (uint32_t e = 0; e < 2; ++e) {
                    const float p = __shfl_sync(0xFFFFFFFFu, c[x][n][(i >> 1) * 2 + e], ((tok & 7u) << 2) | tq);
                    const uint32_t r = n * 8 + tq * 2 + e;
                    if (quad::odd<F16>(sb) && r < live_rows &&
                        Q::sees(a, b, ctx, len, row0 + r, first + static_cast<int32_t>(16 * x + tok))) {
#pragma unroll
                      for (uint32_t d = 0; d < DP / 16; ++d) {
                        o[d][n][e] += p * quad::value<F16>(words[d / 4], (2 * d) & 7u, sb);
                        o[d][n][2 + e] += p * quad::value<F16>(words[d / 4], (2 * d + 1) & 7u, sb);
                      }
                    }
                  }
              }
              if (quad::odd<F16>(quad::scale_bits<F16>(sc[i]))) sc[i] = 0u;
            }
          }
        }
        const quad::Pair<F16> pa(__byte_perm(sc[0], sc[1], 0x5410)), pb(__byte_perm(sc[2], sc[3], 0x5410));
#pragma unroll
        for (uint32_t y = 0; y < kW; ++y) {
          // elements 0 - 3 and 4 - 7 of a word for a pair of tokens
          const uint32_t a0 = __byte_perm(w[0][y], w[1][y], 0x5410), a1 = __byte_perm(w[0][y], w[1][y], 0x7632);
          const uint32_t b0 = __byte_perm(w[2][y], w[3][y], 0x5410), b1 = __byte_perm(w[2][y], w[3][y], 0x7632);
          auto product = [&](uint32_t d, const uint32_t(&f)[4]) {
#pragma unroll
            for (uint32_t n = 0; n < NT; ++n) mma16816<F16>(o[4 * y + d][n], f, pf[x][n][0], pf[x][n][1]);
          };
          product(0, {quad::decode<F16, 0>(a0, pa, magic), quad::decode<F16, 1>(a0, pa, magic),
                      quad::decode<F16, 0>(b0, pb, magic), quad::decode<F16, 1>(b0, pb, magic)});
          product(1, {quad::decode<F16, 2>(a0, pa, magic), quad::decode<F16, 3>(a0, pa, magic),
                      quad::decode<F16, 2>(b0, pb, magic), quad::decode<F16, 3>(b0, pb, magic)});
          product(2, {quad::decode<F16, 0>(a1, pa, magic), quad::decode<F16, 1>(a1, pa, magic),
                      quad::decode<F16, 0>(b1, pb, magic), quad::decode<F16, 1>(b1, pb, magic)});
          product(3, {quad::decode<F16, 2>(a1, pa, magic), quad::decode<F16, 3>(a1, pa, magic),
                      quad::decode<F16, 2>(b1, pb, magic), quad::decode<F16, 3>(b1, pb, magic)});
        }
      }
    }
    cp_wait<0>();

    // Join the warps: sums of a lane's tokens first.
#pragma unroll
    for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
      for (uint32_t e = 0; e < 2; ++e)
#pragma unroll
        for (uint32_t w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], w);
    float* so = reinterpret_cast<float*>(sm);    // [warp][row][DP]
    float* sml = so + kQdWarps * Q::kRows * DP;  // [warp][row][2]
    __syncthreads();                             // the rings are done with
#pragma unroll
    for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
      for (uint32_t e = 0; e < 2; ++e) {
        const uint32_t r = n * 8 + tq * 2 + e;
        float* dst = so + (warp * Q::kRows + r) * DP + g * (DP / 8);
#pragma unroll
        for (uint32_t d = 0; d < DP / 16; ++d) *reinterpret_cast<float2*>(dst + 2 * d) = make_float2(o[d][n][e], o[d][n][2 + e]);
        if (g == 0) {
          sml[(warp * Q::kRows + r) * 2] = m[n][e];
          sml[(warp * Q::kRows + r) * 2 + 1] = l[n][e];
        }
      }
    __syncthreads();
    const bool whole = s.tiles == s.all;
    const uint64_t part = (2ull * blockIdx.x + (s.tile0 == 0 ? 1 : 0)) * Q::kRows;  // as k_kv_tree_join reads them
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
      const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
      for (uint32_t d = lane * 2; d < DP; d += 64) {
        float v0 = 0.f, v1 = 0.f;
#pragma unroll
        for (uint32_t w = 0; w < kQdWarps; ++w) {
          const float2 y = *reinterpret_cast<const float2*>(so + (w * Q::kRows + r) * DP + d);
          if (live_row) v0 += mw[w] * y.x, v1 += mw[w] * y.y;
        }
        if (!whole)
          *reinterpret_cast<float2*>(t.o_part + (part + r) * DP + d) = make_float2(v0, v1);
        else if (d < a.dim)
          *reinterpret_cast<uint32_t*>(static_cast<char*>(a.out) + (orow * a.dim + d) * 2) = pack2<F16>(v0 * inv, v1 * inv);
      }
      if (lane == 0) {
        if (!whole)
          t.ml_part[part + r] = make_float2(top, sum);
        else if (a.lse)
          a.lse[orow] = row_lse<F16>(top, sum);
      }
    }
    __syncthreads();  // the next segment's copies may overwrite the sums
  }
}

// ---------------------------------------------------------------------------

struct QuadPlan {
  uint32_t dp, rows_per, tiles, tile, n_ctas;  // tiles: of rows
};

static QuadPlan quad_plan(uint32_t n_seqs, uint32_t kv_heads, uint64_t rows, uint32_t dim, uint64_t tokens, int device) {
  QuadPlan p = {};
  p.dp = dim <= 64 ? 64 : (dim <= 128 ? 128 : 256);
  p.rows_per = rows > 8 && p.dp < 256 ? 16 : 8;
  p.tiles = static_cast<uint32_t>((rows + p.rows_per - 1) / p.rows_per);
  p.tile = (p.dp == 256 ? 16 : 32) * kQdWarps;
  const uint64_t resident = static_cast<uint64_t>(sm_count(device)) * (p.dp == 256 || p.rows_per == 16 ? 2 : kQdCtas);
  const uint64_t longest = tokens ? (tokens + p.tile - 1) / p.tile : 1;
  const uint64_t work = longest * n_seqs * kv_heads * p.tiles;
  p.n_ctas = static_cast<uint32_t>(work < resident ? work : resident);
  return p;
}

static size_t align256(size_t x) { return (x + 255) / 256 * 256; }

size_t kv4_attend_workspace(uint32_t n_seqs, uint32_t kv_heads, uint64_t rows, uint32_t dim, uint64_t tokens, int device) {
  const QuadPlan p = quad_plan(n_seqs, kv_heads, rows, dim, tokens, device);
  return align256((p.n_ctas + 1) * sizeof(int4)) + align256(2ull * p.n_ctas * p.rows_per * sizeof(float2)) +
         2ull * p.n_ctas * p.rows_per * p.dp * 4;
}

template <uint32_t DP, uint32_t NT, bool F16>
static int launch_quad(const TcArgs& t, int device, cudaStream_t stream) {
  using Q = Quad<DP, NT>;
  int32_t shift = -1;
  if ((t.a.page_tokens & (t.a.page_tokens - 1)) == 0)
    for (shift = 0; (1u << shift) < t.a.page_tokens;) ++shift;
  uint64_t all = 0;
  for (int i = 0; i < 2; ++i)
    all |= reinterpret_cast<uintptr_t>(t.four[i].scales) | static_cast<uint64_t>(t.four[i].s_page) |
           static_cast<uint64_t>(t.four[i].s_head) | static_cast<uint64_t>(t.four[i].s_token);
  bool even = t.a.dim == DP && all % Q::kScale == 0 && t.a.page_tokens % 16 == 0;
  for (int i = 0; i < 2; ++i) {
    const uint64_t most = 0xFFFFFFFFull / t.a.page_tokens;
    even = even && static_cast<uint64_t>(t.four[i].page_stride) <= 0xFFFFFFFFull && static_cast<uint64_t>(t.four[i].s_page) <= 0xFFFFFFFFull &&
           static_cast<uint64_t>(t.four[i].token_stride) <= most && static_cast<uint64_t>(t.four[i].s_token) <= most;
  }
  auto kern = even ? k_kv4_attend<DP, NT, F16, kEven> : k_kv4_attend<DP, NT, F16, kAny>;
  static std::atomic<int> ready[2][64];
  if (device < 0 || device >= 64 || !ready[even][device].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Q::kBytes);
    if (e != cudaSuccess) {
      set_cuda_error(e, "set-up of k_kv4_attend");
      cudaGetLastError();
      return IBP_ECUDA;
    }
    if (device >= 0 && device < 64) ready[even][device].store(1, std::memory_order_release);
  }
  const int rc = kv_launch("k_kv4_attend", kern, dim3(t.n_ctas), kQdWarps * 32, Q::kBytes, 1, stream, t, shift);
  if (rc != IBP_OK || t.n_ctas == 1) return rc;
  return kv_launch("k_kv_tree_join", k_kv_tree_join<DP, Q::kRows, F16, Q::kTile>,
                   dim3(t.n_ctas - 1, (Q::kRows + kJoinRows - 1) / kJoinRows), kJoinThreads, 0, 1, stream, t);
}

int launch_kv4_attend(const Attend4Args& x, int device, size_t ws_bytes, cudaStream_t stream) {
  const AttendArgs& a = x.a;
  const uint64_t tokens = static_cast<uint64_t>(a.max_pages) * a.page_tokens;
  const QuadPlan p = quad_plan(a.n_seqs, a.kv_heads, static_cast<uint64_t>(a.T) * a.group, a.dim, tokens, device);
  if (!a.part || ws_bytes < kv4_attend_workspace(a.n_seqs, a.kv_heads, static_cast<uint64_t>(a.T) * a.group, a.dim, tokens, device))
    return IBP_EINVAL;
  TcArgs t = {};
  t.a = a;
  t.four[0] = x.k, t.four[1] = x.v;
  t.row_pairs = p.tiles;
  t.n_ctas = p.n_ctas;
  t.q16 = ((reinterpret_cast<uintptr_t>(a.q) | static_cast<uint64_t>(a.q_seq) | static_cast<uint64_t>(a.q_token) |
            static_cast<uint64_t>(a.q_head)) & 15u) == 0;
  char* w = reinterpret_cast<char*>(a.part);
  t.first = reinterpret_cast<int4*>(w);
  w += align256((p.n_ctas + 1) * sizeof(int4));
  t.ml_part = reinterpret_cast<float2*>(w);
  w += align256(2ull * p.n_ctas * p.rows_per * sizeof(float2));
  t.o_part = reinterpret_cast<float*>(w);
  auto go = [&](auto f16) {
    constexpr bool F = decltype(f16)::value;
    if (p.dp == 64) return p.rows_per == 16 ? launch_quad<64, 2, F>(t, device, stream) : launch_quad<64, 1, F>(t, device, stream);
    if (p.dp == 128) return p.rows_per == 16 ? launch_quad<128, 2, F>(t, device, stream) : launch_quad<128, 1, F>(t, device, stream);
    return launch_quad<256, 1, F>(t, device, stream);
  };
  return a.f16 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace ibp

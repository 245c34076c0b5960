// ibp_kv_attend.cu - attention of few queries over a paged cache: a tree of
// drafted tokens, and single queries over selected pages.
//
// A CTA holds 8 or 16 query rows of one sequence and kv head (the group's heads,
// and the drafted tokens) and walks a share of the tokens.  With so few rows
// the cache's bytes are what counts, so the layout serves the loads: each of
// the four warps has its own ring of stages of 16 or 32 tokens, filled by 16-byte
// asynchronous copies, and its own running maximum and sum; no barrier is met
// until the warps are joined at the end.  Where there are items enough for every
// warp (a chunk of sparse queries), each warp takes an item of its own.
//
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T, so that the
// 16-row side of mma.m16n8k16 is filled by tokens and dimensions and the 8-wide
// side by queries: eight rows cost half of what the other order would.  The
// accumulator of S^T becomes the operand P^T by one 8x8 transpose per register.
// Tensor-core work is far from the bound here: for 8 rows of 128 dimensions a
// 16-token step is 16 instructions for 8 KB of cache.
//
// Measured on one GB300: 32 queries over 64 pages of 64 tokens each, 8 kv heads of
// 4 query heads and 128 dimensions (533 MB): 84 us, 6.3 TB/s; 1022 queries of 8
// heads over 24 pages of 32 tokens of 64 dimensions (803 MB out of L2): 75 us,
// bound by issue (34 M instructions) and the few warps its stages leave room for.
//
// Softmax statistics and sums are 32-bit; the probabilities are rounded to the
// cache's type for the second product (the tensor core wants both operands
// alike), which adds an error of the size of the output's own rounding.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "ibp_kv_mma.cuh"

namespace ibp {

constexpr uint32_t kAtWarps = 4;

// One CTA's work: rows [row0, row0 + 8 NT) of a sequence and kv head, against
// tokens [first, last) of its list (all positions, or the selected pages').
struct Item {
  uint32_t b, h, t0;   // t0: the query (sparse), or 0
  uint32_t row0, rows; // rows that exist
  int32_t ctx;         // first drafted position (tree)
  int32_t seen;        // positions below this may be seen
  uint32_t n_tok;      // tokens of the list
  const int32_t* picks;  // selected pages
};

template <uint32_t DP, uint32_t NT, bool F16, bool PICK>
struct Attend {
  // Tokens of a step: what a step costs besides its products (page, maxima over
  // the lanes, bookkeeping) is halved for narrow heads, whose bytes are few.
  static constexpr uint32_t kSub = DP == 64 ? 32 : 16;
  static constexpr uint32_t kMma = kSub / 16;
  static constexpr uint32_t kPitch = DP * 2;                 // bytes of a token in a stage
  static constexpr uint32_t kTile = kSub * kPitch;           // bytes of K or V in a stage
  static constexpr uint32_t kStages = DP == 128 ? 3 : 2;
  static constexpr uint32_t kWarpBytes = kStages * 2 * kTile;
  static constexpr uint32_t kBytes = kAtWarps * kWarpBytes;
  static constexpr uint32_t kRows = 8 * NT;
  static_assert((kRows * DP + 2 * kRows) * 4 <= kWarpBytes, "the join fits the stages");
  static_assert((kAtWarps + 1) * kRows * (DP + 2) * 4 <= kBytes, "a cluster's part fits beside it");

  // Row of the flat (token, group head) order: the query token of row r.
  static __device__ __forceinline__ uint32_t token_of(const AttendArgs& a, const Item& it, uint32_t r) {
    return PICK ? it.t0 : r / a.group;
  }

  static __device__ __forceinline__ bool sees(const AttendArgs& a, const Item& it, uint32_t r, int32_t pos) {
    if (pos >= it.seen) return false;
    if (PICK || pos < it.ctx) return true;
    const uint32_t t = r / a.group, i = static_cast<uint32_t>(pos - it.ctx);
    if (!a.mask) return i <= t;
    return (a.mask[(static_cast<uint64_t>(it.b) * a.T + t) * a.mask_words + (i >> 5)] >> (i & 31u)) & 1u;
  }
};

// The page of a step, looked up one step before its tokens are asked for.
struct Ahead {
  uint32_t nth, page;
};

// What a lane's copies need in every step.
struct Lane {
  const char *k, *v;  // this lane's chunk of the first token of a step at offset 0
  const int32_t* row; // the sequence's table row
  int32_t shift;      // pages hold 2^shift steps; -1: some other whole number; -2: steps cross pages
};

template <uint32_t DP, uint32_t NT, bool F16, bool PICK>
__device__ __forceinline__ Ahead look_ahead(const AttendArgs& a, const Item& it, const Lane& ln, uint32_t sub) {
  using A = Attend<DP, NT, F16, PICK>;
  Ahead x = {0u, 0xFFFFFFFFu};
  if (ln.shift < -1 || sub * A::kSub >= it.n_tok) return x;
  const uint32_t at = ln.shift >= 0 ? sub >> ln.shift : sub * A::kSub / a.page_tokens;
  x.nth = PICK ? static_cast<uint32_t>(it.picks[at]) : at;
  // the list may lie in the caller's buffer: an entry outside the table row is a bad page
  if (!PICK || x.nth < a.max_pages) x.page = static_cast<uint32_t>(ln.row[x.nth]);
  return x;
}

// Copies the tokens of step `sub` into a stage; tokens that no row may see
// are zeros, so nothing they hold reaches a sum.  *pos_out: the position of this
// lane's token (lane modulo the step).
template <uint32_t DP, uint32_t NT, bool F16, bool PICK>
__device__ __forceinline__ void load_stage(const AttendArgs& a, const Item& it, const Lane& ln, uint32_t sub,
                                           uint32_t stage, const Ahead& ah, int32_t* pos_out) {
  using A = Attend<DP, NT, F16, PICK>;
  const uint32_t lane = threadIdx.x & 31u;
  constexpr uint32_t kSub = A::kSub;
  constexpr uint32_t kChunks = DP / 8;      // 16-byte chunks of a token
  constexpr uint32_t kPer = 32 / kChunks;   // tokens per warp instruction
  const uint32_t c = lane % kChunks, r0 = lane / kChunks;
  const bool col = c < a.dim / 8;
  const uint32_t dst0 = stage + r0 * A::kPitch;
  const uint32_t left = it.n_tok - sub * kSub;  // tokens from this step on
  if (ln.shift >= -1) {
    const uint32_t at = ln.shift >= 0 ? sub >> ln.shift : sub * kSub / a.page_tokens;
    const uint32_t s0 = sub * kSub - at * a.page_tokens;  // first token of the step in its page
    const uint32_t mine = lane % kSub;
    *pos_out = mine < left ? static_cast<int32_t>(ah.nth * a.page_tokens + s0 + mine) : 0x7FFFFFFF;
    const bool good = ah.page < a.n_pages;
    if (!good) kv_status(a.status, IBP_ERANGE);
    const char* k = ln.k + static_cast<int64_t>(ah.page) * a.k.page_stride + static_cast<int64_t>(s0) * a.k.token_stride;
    const char* v = ln.v + static_cast<int64_t>(ah.page) * a.v.page_stride + static_cast<int64_t>(s0) * a.v.token_stride;
#pragma unroll
    for (uint32_t i = 0; i < kSub / kPer; ++i) {
      const uint32_t r = r0 + i * kPer;
      const uint32_t dst = dst0 + i * kPer * A::kPitch + ((c ^ (r & 7u)) << 4);
      const bool on = good && col && r < left;
      cp16(dst, on ? k : a.k.data, on);
      cp16(dst + A::kTile, on ? v : a.v.data, on);
      k += kPer * a.k.token_stride;
      v += kPer * a.v.token_stride;
    }
    return;
  }
  // Steps cross pages: lane i finds token i and tells the others.
  const uint32_t tok = sub * kSub + lane % kSub, at = tok / a.page_tokens, slot = tok - at * a.page_tokens;
  uint32_t page = 0xFFFFFFFFu;
  int32_t pos = 0x7FFFFFFF;
  if (tok < it.n_tok) {
    const uint32_t nth = PICK ? static_cast<uint32_t>(it.picks[at]) : at;
    pos = static_cast<int32_t>(nth * a.page_tokens + slot);
    if (pos < it.seen) {
      if (!PICK || nth < a.max_pages) page = static_cast<uint32_t>(ln.row[nth]);
      if (page >= a.n_pages) {
        kv_status(a.status, IBP_ERANGE);
        page = 0xFFFFFFFFu;
      }
    }
  }
  *pos_out = pos;
  const int64_t tk = static_cast<int64_t>(page) * a.k.page_stride + static_cast<int64_t>(slot) * a.k.token_stride;
  const int64_t tv = static_cast<int64_t>(page) * a.v.page_stride + static_cast<int64_t>(slot) * a.v.token_stride;
  const int64_t bk = static_cast<int64_t>(r0) * a.k.token_stride, bv = static_cast<int64_t>(r0) * a.v.token_stride;
#pragma unroll
  for (uint32_t i = 0; i < kSub / kPer; ++i) {
    const uint32_t r = r0 + i * kPer;
    const bool on = (__shfl_sync(0xFFFFFFFFu, page, r) != 0xFFFFFFFFu) && col;
    const int64_t ok = __shfl_sync(0xFFFFFFFFu, tk, r), ov = __shfl_sync(0xFFFFFFFFu, tv, r);
    const uint32_t dst = dst0 + i * kPer * A::kPitch + ((c ^ (r & 7u)) << 4);
    cp16(dst, on ? ln.k + (ok - bk) : a.k.data, on);
    cp16(dst + A::kTile, on ? ln.v + (ov - bv) : a.v.data, on);
  }
}

template <uint32_t DP, uint32_t NT, bool F16, bool PICK, uint32_t WPI>
__global__ void __launch_bounds__(kAtWarps * 32)
    k_kv_attend(const AttendArgs a, uint32_t row_tiles, int32_t shift, uint32_t items) {
  using A = Attend<DP, NT, F16, PICK>;
  constexpr uint32_t kSub = A::kSub, kM = A::kMma;
  extern __shared__ __align__(128) unsigned char sm[];
  pdl_begin();
  // WPI warps share an item: all four of a CTA, or one each.
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x / 32 % WPI, group = threadIdx.x / 32 / WPI;
  auto sync = [] {
    if (WPI == 1)
      __syncwarp();
    else
      __syncthreads();
  };
  const uint32_t split = blockIdx.x % a.splits;
  uint32_t x = blockIdx.x / a.splits * (kAtWarps / WPI) + group;
  const uint32_t item = x;
  if (item >= items) return;
  Item it;
  const uint32_t tile = x % row_tiles;
  x /= row_tiles;
  it.h = x % a.kv_heads;
  x /= a.kv_heads;
  it.t0 = PICK ? x % a.T : 0;
  it.b = PICK ? x / a.T : x;
  it.row0 = tile * A::kRows;
  const int32_t raw = a.lens[it.b], len = clamp_len(raw, a.page_tokens, a.max_pages);
  const int32_t live = a.n_live ? a.n_live[it.b] : static_cast<int32_t>(a.T);
  if ((raw != len || live > len || live < 0 || live > static_cast<int32_t>(a.T)) && warp == 0 && lane == 0)
    kv_status(a.status, IBP_ERANGE);
  const int32_t n_live = live < 0 ? 0 : (live > static_cast<int32_t>(a.T) ? static_cast<int32_t>(a.T) : live);
  it.ctx = len - n_live;  // below 0: the draft's first tokens do not exist
  const uint32_t all_rows = (PICK ? 1u : a.T) * a.group;
  it.rows = all_rows - it.row0 < A::kRows ? all_rows - it.row0 : A::kRows;
  uint32_t live_rows = it.rows;
  if (PICK) {
    const int32_t p = static_cast<int32_t>(it.t0) < n_live ? it.ctx + static_cast<int32_t>(it.t0) : -1;
    it.seen = p + 1 > 0 ? p + 1 : 0;
    const int32_t* pk =
        a.picks + ((static_cast<uint64_t>(it.b) * a.T + it.t0) * a.kv_heads + it.h) * a.budget;
    it.picks = pk;
    // All pages the query sees, or `budget` of them; the last is the query's own
    // and ends at its position.
    if (it.seen > 0) {
      const uint32_t own = static_cast<uint32_t>(p) / a.page_tokens;
      const uint32_t n = own + 1 < a.budget ? own + 1 : a.budget;
      it.n_tok = (n - 1) * a.page_tokens + static_cast<uint32_t>(p) % a.page_tokens + 1;
    } else {
      it.n_tok = 0;
    }
  } else {
    it.seen = len;
    const uint32_t lr = static_cast<uint32_t>(n_live) * a.group;
    live_rows = lr > it.row0 ? (lr - it.row0 < it.rows ? lr - it.row0 : it.rows) : 0;
    it.n_tok = live_rows ? static_cast<uint32_t>(len) : 0;
  }
  // This CTA's share of the steps.
  const uint32_t steps = ceil_div(it.n_tok, kSub);
  const uint32_t per = ceil_div(steps, a.splits);
  const uint32_t s0 = split * per < steps ? split * per : steps, s1 = steps - s0 < per ? steps : s0 + per;

  // Q^T as B operands: columns are rows of Q.  A row past the end is zero.
  uint32_t qf[NT][DP / 16][2];
#pragma unroll
  for (uint32_t n = 0; n < NT; ++n) {
    const uint32_t r = it.row0 + n * 8 + lane / 4;
    const bool on = n * 8 + lane / 4 < live_rows;
    const uint32_t t = on ? A::token_of(a, it, r) : 0, g = on ? r % a.group : 0;
    const char* q = a.q + static_cast<int64_t>(it.b) * a.q_seq + static_cast<int64_t>(t) * a.q_token +
                    static_cast<int64_t>(it.h * a.group + g) * a.q_head;
#pragma unroll
    for (uint32_t kk = 0; kk < DP / 16; ++kk)
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        const uint32_t d = kk * 16 + i * 8 + (lane & 3u) * 2;
        qf[n][kk][i] = on && d < a.dim ? *reinterpret_cast<const uint32_t*>(q + d * 2) : 0u;
      }
  }

  float o[DP / 16][NT][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (uint32_t n = 0; n < NT; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (uint32_t d = 0; d < DP / 16; ++d) o[d][n][0] = o[d][n][1] = o[d][n][2] = o[d][n][3] = 0.f;
  }

  unsigned char* const mine = sm + group * WPI * A::kWarpBytes;
  const uint32_t ring = smem_u32(mine) + warp * A::kWarpBytes;
  Lane ln;
  {
    constexpr uint32_t kChunks = DP / 8;
    const uint32_t c = lane % kChunks, r0 = lane / kChunks;
    ln.k = a.k.data + static_cast<int64_t>(it.h) * a.k.head_stride + c * 16 + static_cast<int64_t>(r0) * a.k.token_stride;
    ln.v = a.v.data + static_cast<int64_t>(it.h) * a.v.head_stride + c * 16 + static_cast<int64_t>(r0) * a.v.token_stride;
    ln.row = a.table + static_cast<uint64_t>(it.b) * a.max_pages;
    ln.shift = shift;
  }
  int32_t pos_ring[A::kStages];  // the position of this lane's token, for each stage in flight
  Ahead ah = look_ahead<DP, NT, F16, PICK>(a, it, ln, s0 + warp);
#pragma unroll
  for (uint32_t i = 0; i < A::kStages - 1; ++i) {
    const uint32_t s = s0 + warp + i * WPI;
    if (s < s1) {
      load_stage<DP, NT, F16, PICK>(a, it, ln, s, ring + i * 2 * A::kTile, ah, &pos_ring[i]);
      ah = look_ahead<DP, NT, F16, PICK>(a, it, ln, s + WPI);
    }
    cp_commit();
  }
  for (uint32_t sb = s0 + warp; sb < s1; sb += WPI * A::kStages) {
#pragma unroll
    for (uint32_t u = 0; u < A::kStages; ++u) {
      const uint32_t s = sb + u * WPI;
      if (s >= s1) break;
      constexpr uint32_t kAhead = A::kStages - 1;
      const uint32_t un = (u + kAhead) % A::kStages;
      __syncwarp();  // every lane is done with the stage that is filled next
      if (s + kAhead * WPI < s1) {
        load_stage<DP, NT, F16, PICK>(a, it, ln, s + kAhead * WPI, ring + un * 2 * A::kTile, ah, &pos_ring[un]);
        ah = look_ahead<DP, NT, F16, PICK>(a, it, ln, s + (kAhead + 1) * WPI);
      }
      cp_commit();
      cp_wait<kAhead>();
      __syncwarp();
      const uint32_t kt = ring + u * 2 * A::kTile, vt = kt + A::kTile;
      const int32_t my_pos = pos_ring[u];

      float c[kM][NT][4];
#pragma unroll
      for (uint32_t x = 0; x < kM; ++x) {
#pragma unroll
        for (uint32_t n = 0; n < NT; ++n) c[x][n][0] = c[x][n][1] = c[x][n][2] = c[x][n][3] = 0.f;
        const uint32_t r = lane & 15u, hi = lane >> 4;
        const uint32_t base = kt + (16 * x + r) * A::kPitch;
#pragma unroll
        for (uint32_t kk = 0; kk < DP / 16; ++kk) {
          uint32_t f[4];
          ldsm4(f, base + (((kk * 2 + hi) ^ (r & 7u)) << 4));
#pragma unroll
          for (uint32_t n = 0; n < NT; ++n) mma16816<F16>(c[x][n], f, qf[n][kk][0], qf[n][kk][1]);
        }
      }
      // Scores in powers of two; what a row does not see is -infinity.
      const int32_t edge = PICK ? it.seen : (it.ctx < it.seen ? it.ctx : it.seen);
      const bool open = __all_sync(0xFFFFFFFFu, my_pos < edge);  // every row sees the whole step
      float cm[NT][2];
#pragma unroll
      for (uint32_t n = 0; n < NT; ++n) {
#pragma unroll
        for (uint32_t x = 0; x < kM; ++x) {
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) c[x][n][e] *= a.scale_log2;
        }
      }
      if (!open) {
#pragma unroll
        for (uint32_t x = 0; x < kM; ++x) {
          const int32_t p_lo = __shfl_sync(0xFFFFFFFFu, my_pos, 16 * x + lane / 4);
          const int32_t p_hi = __shfl_sync(0xFFFFFFFFu, my_pos, 16 * x + lane / 4 + 8);
#pragma unroll
          for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) {
              const uint32_t r = n * 8 + (lane & 3u) * 2 + (e & 1u);
              if (r >= live_rows || !A::sees(a, it, it.row0 + r, e < 2 ? p_lo : p_hi)) c[x][n][e] = -INFINITY;
            }
        }
      }
#pragma unroll
      for (uint32_t n = 0; n < NT; ++n) {
#pragma unroll
        for (uint32_t e = 0; e < 2; ++e) {
          cm[n][e] = fmaxf(c[0][n][e], c[0][n][2 + e]);
#pragma unroll
          for (uint32_t x = 1; x < kM; ++x) cm[n][e] = fmaxf(cm[n][e], fmaxf(c[x][n][e], c[x][n][2 + e]));
        }
#pragma unroll
        for (uint32_t w = 4; w < 32; w <<= 1) {
          cm[n][0] = fmaxf(cm[n][0], __shfl_xor_sync(0xFFFFFFFFu, cm[n][0], w));
          cm[n][1] = fmaxf(cm[n][1], __shfl_xor_sync(0xFFFFFFFFu, cm[n][1], w));
        }
        if (F16) cm[n][0] = __fadd_ru(cm[n][0], -kLift<F16>), cm[n][1] = __fadd_ru(cm[n][1], -kLift<F16>);
      }
      bool grow = false;
#pragma unroll
      for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
        for (uint32_t e = 0; e < 2; ++e) grow = grow || cm[n][e] > m[n][e];
      if (__any_sync(0xFFFFFFFFu, grow)) {
        // Rescale what was summed under the lower maximum.  At once: the largest
        // probability is then a power of two and its rounding costs nothing, where a
        // row has one key that outweighs the rest (putting it off until the
        // maximum had grown by 2^8 took the output's error from 1.1 to 1.5 of the
        // rounding of the result itself).
#pragma unroll
        for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
          for (uint32_t e = 0; e < 2; ++e)
            if (cm[n][e] > m[n][e]) {
              const float f = ex2(m[n][e] - cm[n][e]);
              m[n][e] = cm[n][e];
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
          const float p0 = ex2(c[x][n][0] - m0), p1 = ex2(c[x][n][1] - m1);
          const float p2 = ex2(c[x][n][2] - m0), p3 = ex2(c[x][n][3] - m1);
          l[n][0] += p0 + p2;
          l[n][1] += p1 + p3;
          pf[x][n][0] = transpose8(pack2<F16>(p0, p1));
          pf[x][n][1] = transpose8(pack2<F16>(p2, p3));
        }
      }
      if (!PICK && !open) {
        // Infinities and NaN among the draft's values: a row that does not see
        // them must not meet them, even with probability zero.  They leave the
        // product and are added to the rows that see them, whose outputs they
        // decide whatever their probability.
        uint32_t odd = 0;
        const uint32_t ex = F16 ? 0x7C00u : 0x7F80u;
        for (uint32_t i = lane; i < kSub * DP / 8; i += 32) {
          const uint4 w = *reinterpret_cast<const uint4*>(sm + (vt - smem_u32(sm)) + i * 16);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j)
            odd |= ((ws[j] & ex) == ex) | (((ws[j] >> 16) & ex) == ex);
        }
        if (__any_sync(0xFFFFFFFFu, odd)) {
#pragma unroll 1
          for (uint32_t tk = 0; tk < kSub; ++tk) {
            const int32_t pos = __shfl_sync(0xFFFFFFFFu, my_pos, tk);
#pragma unroll
            for (uint32_t d = 0; d < DP / 16; ++d)
#pragma unroll
              for (uint32_t half = 0; half < 2; ++half) {
                const uint32_t dd = d * 16 + half * 8 + lane / 4;
                const uint32_t off = (vt - smem_u32(sm)) + tk * A::kPitch + (((dd / 8) ^ (tk & 7u)) << 4) + (dd & 7u) * 2;
                const uint32_t raw16 = *reinterpret_cast<const uint16_t*>(sm + off);
                if ((raw16 & ex) == ex) {
                  const float val = F16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(raw16)))
                                        : __uint_as_float(raw16 << 16);
#pragma unroll
                  for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
                    for (uint32_t e = 0; e < 2; ++e) {
                      const uint32_t r = n * 8 + (lane & 3u) * 2 + e;
                      if (r < live_rows && A::sees(a, it, it.row0 + r, pos)) o[d][n][half * 2 + e] += val;
                    }
                }
              }
          }
          __syncwarp();
          for (uint32_t i = lane; i < kSub * DP; i += 32) {
            uint16_t* w = reinterpret_cast<uint16_t*>(sm + (vt - smem_u32(sm))) + i;
            if ((*w & ex) == ex) *w = 0;
          }
          __syncwarp();
        }
      }
#pragma unroll
      for (uint32_t x = 0; x < kM; ++x) {
        const uint32_t r = lane & 7u, quad = lane >> 3;
        const uint32_t tok = 16 * x + r + (quad >> 1) * 8;
        const uint32_t base = vt + tok * A::kPitch;
#pragma unroll
        for (uint32_t d = 0; d < DP / 16; ++d) {
          uint32_t f[4];
          ldsm4t(f, base + (((d * 2 + (quad & 1u)) ^ (tok & 7u)) << 4));
#pragma unroll
          for (uint32_t n = 0; n < NT; ++n) mma16816<F16>(o[d][n], f, pf[x][n][0], pf[x][n][1]);
        }
      }
    }
  }
  cp_wait<0>();

  // Join the warps: sums of a lane's tokens first, then the item's warps'.
#pragma unroll
  for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
    for (uint32_t e = 0; e < 2; ++e)
#pragma unroll
      for (uint32_t w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], w);
  sync();
  float* so = reinterpret_cast<float*>(mine);                     // [warp][row][DP]
  float* sml = so + WPI * A::kRows * DP;                          // [warp][row][2]
  float* sp = sml + WPI * A::kRows * 2;                           // [row][2 + DP]: this CTA's part in a cluster
#pragma unroll
  for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
    for (uint32_t e = 0; e < 2; ++e) {
      const uint32_t r = n * 8 + (lane & 3u) * 2 + e;
      float* dst = so + (warp * A::kRows + r) * DP + lane / 4;
#pragma unroll
      for (uint32_t d = 0; d < DP / 16; ++d) dst[d * 16] = o[d][n][e], dst[d * 16 + 8] = o[d][n][2 + e];
      if (lane < 4) {
        sml[(warp * A::kRows + r) * 2] = m[n][e];
        sml[(warp * A::kRows + r) * 2 + 1] = l[n][e];
      }
    }
  sync();
  for (uint32_t r = warp; r < it.rows; r += WPI) {
    float mw[WPI], top = -INFINITY, sum = 0.f;
    const bool live_row = r < live_rows;
#pragma unroll
    for (uint32_t w = 0; w < WPI; ++w) {
      mw[w] = live_row ? sml[(w * A::kRows + r) * 2] : -INFINITY;
      top = fmaxf(top, mw[w]);
    }
#pragma unroll
    for (uint32_t w = 0; w < WPI; ++w) {
      const float s = live_row ? sml[(w * A::kRows + r) * 2 + 1] : 0.f;
      // a NaN sum stays one: only an empty warp is left out
      mw[w] = mw[w] == -INFINITY ? (s == 0.f ? 0.f : 1.f) : exp2f(mw[w] - top);
      sum += mw[w] * s;
    }
    const uint32_t gr = it.row0 + r, t = A::token_of(a, it, gr), g = gr % a.group;
    const uint64_t orow = (static_cast<uint64_t>(it.b) * a.T + t) * a.kv_heads * a.group + it.h * a.group + g;
    const bool whole = a.splits == 1;
    const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
    float* part = a.cluster ? sp + r * (DP + 2)
                            : a.part + (static_cast<uint64_t>(item) * a.splits + split) * A::kRows * (DP + 2) + r * (DP + 2);
    for (uint32_t d = lane * 2; d < a.dim; d += 64) {
      float v0 = 0.f, v1 = 0.f;
#pragma unroll
      for (uint32_t w = 0; w < WPI; ++w) {
        const float2 y = *reinterpret_cast<const float2*>(so + (w * A::kRows + r) * DP + d);
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
  for (uint32_t r = split + a.splits * warp; r < it.rows; r += a.splits * WPI) {
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
    float2 acc[DP / 64];
#pragma unroll
    for (uint32_t i = 0; i < DP / 64; ++i) acc[i] = make_float2(0.f, 0.f);
    for (uint32_t c = 0; c < a.splits; ++c) {
      const float fc = __shfl_sync(0xFFFFFFFFu, f, c);
      sum += fc * __shfl_sync(0xFFFFFFFFu, ml.y, c);
#pragma unroll
      for (uint32_t i = 0; i < DP / 64; ++i) {
        float2 y;
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(y.x), "=f"(y.y) : "r"(remote(c, 2 + lane * 2 + i * 64)) : "memory");
        if (lane * 2 + i * 64 < a.dim) acc[i].x += fc * y.x, acc[i].y += fc * y.y;
      }
    }
    const uint32_t gr = it.row0 + r, t = A::token_of(a, it, gr), g = gr % a.group;
    const uint64_t orow = (static_cast<uint64_t>(it.b) * a.T + t) * a.kv_heads * a.group + it.h * a.group + g;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (uint32_t i = 0; i < DP / 64; ++i) {
      const uint32_t d = lane * 2 + i * 64;
      if (d < a.dim)
        *reinterpret_cast<uint32_t*>(static_cast<char*>(a.out) + (orow * a.dim + d) * 2) =
            pack2<F16>(acc[i].x * inv, acc[i].y * inv);
    }
    if (lane == 0 && a.lse) a.lse[orow] = row_lse<F16>(top, sum);
  }
  // no CTA leaves while another reads its shared memory
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Joins the partial sums of split items: a warp per row.
template <uint32_t DP, bool F16, bool PICK>
__global__ void __launch_bounds__(128) k_kv_join(const AttendArgs a, uint32_t row_tiles, uint32_t tile_rows,
                                                 uint32_t n_rows) {
  pdl_begin();
  const uint32_t lane = threadIdx.x & 31u;
  const uint64_t w = static_cast<uint64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const uint64_t items = w / tile_rows;
  const uint32_t r = static_cast<uint32_t>(w % tile_rows);
  uint64_t x = items;
  const uint32_t tile = static_cast<uint32_t>(x % row_tiles);
  x /= row_tiles;
  const uint32_t h = static_cast<uint32_t>(x % a.kv_heads);
  x /= a.kv_heads;
  const uint32_t t0 = PICK ? static_cast<uint32_t>(x % a.T) : 0;
  const uint64_t b = PICK ? x / a.T : x;
  const uint32_t gr = tile * tile_rows + r;
  if (b >= a.n_seqs || gr >= n_rows) return;
  const uint32_t t = PICK ? t0 : gr / a.group, g = gr % a.group;
  const float* part = a.part + (items * a.splits * tile_rows + r) * (DP + 2);
  const uint64_t stride = static_cast<uint64_t>(tile_rows) * (DP + 2);
  float top = -INFINITY;
  for (uint32_t s = lane; s < a.splits; s += 32) top = fmaxf(top, part[s * stride]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  float sum = 0.f;
  float2 acc[DP / 64];
#pragma unroll
  for (uint32_t i = 0; i < DP / 64; ++i) acc[i] = make_float2(0.f, 0.f);
  for (uint32_t s = 0; s < a.splits; ++s) {
    const float ms = part[s * stride], ls = part[s * stride + 1];
    const float f = ms == -INFINITY ? (ls == 0.f ? 0.f : 1.f) : exp2f(ms - top);
    sum += f * ls;
#pragma unroll
    for (uint32_t i = 0; i < DP / 64; ++i) {
      const uint32_t d = lane * 2 + i * 64;
      if (d < a.dim) {
        const float2 y = *reinterpret_cast<const float2*>(part + s * stride + 2 + d);
        acc[i].x += f * y.x, acc[i].y += f * y.y;
      }
    }
  }
  const uint64_t orow = (b * a.T + t) * a.kv_heads * a.group + h * a.group + g;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (uint32_t i = 0; i < DP / 64; ++i) {
    const uint32_t d = lane * 2 + i * 64;
    if (d < a.dim)
      *reinterpret_cast<uint32_t*>(static_cast<char*>(a.out) + (orow * a.dim + d) * 2) =
          pack2<F16>(acc[i].x * inv, acc[i].y * inv);
  }
  if (lane == 0 && a.lse) a.lse[orow] = row_lse<F16>(top, sum);
}

// ---------------------------------------------------------------------------

constexpr uint32_t kMaxUnits = 2048;  // CTAs up to which items are split
constexpr uint32_t kLeast = 128;      // tokens of a share

static uint32_t padded_dim(uint32_t dim) { return dim <= 64 ? 64 : (dim <= 128 ? 128 : 256); }
// 16 rows a CTA where there are more than 8 and the registers allow it.
static uint32_t tile_rows(uint64_t rows, uint32_t dp) { return rows > 8 && dp < 256 ? 16 : 8; }

// Splits of an item: as many CTAs as the GPU holds at once, by powers of two up
// to a cluster of eight, which joins in place, and down to two steps a warp.
// Lengths are on the device, so the longest possible counts.  One round of CTAs
// beats two: 256 items of 4096 tokens took 113 us unsplit, 126 us in quarters; 64
// items 52, 45 and 49 us in 2, 4 and 8.  Only a handful of long items is split
// further, with a second kernel for the join.
static uint32_t splits_of(uint64_t items, uint64_t tokens, uint64_t resident) {
  uint64_t s = 1;
  while (s < 8 && 2 * s * items <= resident && tokens >= 2 * s * kLeast) s *= 2;
  if (s == 8 && 4 * s * items <= resident && tokens >= 32 * s * kLeast) {
    const uint64_t most = tokens / (8 * kLeast);
    s = resident / items < most ? resident / items : most;
    if (s * items > kMaxUnits) s = kMaxUnits / items;
  }
  return static_cast<uint32_t>(s);
}

// CTAs that the GPU holds at once.
static uint64_t resident_ctas(uint32_t dp, int device) {
  const uint32_t bytes = dp == 64 ? Attend<64, 1, false, false>::kBytes
                                  : (dp == 128 ? Attend<128, 1, false, false>::kBytes : Attend<256, 1, false, false>::kBytes);
  return static_cast<uint64_t>(sm_count(device)) * (232448 / (bytes + 1024));
}

size_t kv_attend_workspace(uint64_t items, uint64_t rows, uint32_t dim, uint64_t tokens, bool pick, int device) {
  const uint32_t dp = padded_dim(dim), tr = tile_rows(rows, dp);
  const uint64_t tiles = items * ((rows + tr - 1) / tr), resident = resident_ctas(dp, device);
  if (pick && tiles >= 2 * resident * kAtWarps) return 0;
  const uint32_t splits = splits_of(tiles, tokens, resident);
  return splits <= 8 ? 0 : tiles * splits * tr * (dp + 2) * 4;
}

template <uint32_t DP, uint32_t NT, bool F16, bool PICK, uint32_t WPI>
static int launch_items(const AttendArgs& a, uint32_t tiles, uint64_t items, int device, cudaStream_t stream) {
  using A = Attend<DP, NT, F16, PICK>;
  auto kern = k_kv_attend<DP, NT, F16, PICK, WPI>;
  static std::atomic<int> ready[64];
  if (device < 0 || device >= 64 || !ready[device].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, A::kBytes);
    if (e != cudaSuccess) {
      set_cuda_error(e, "set-up of k_kv_attend");
      cudaGetLastError();
      return IBP_ECUDA;
    }
    if (device >= 0 && device < 64) ready[device].store(1, std::memory_order_release);
  }
  const uint64_t per = kAtWarps / WPI;
  int32_t shift = -2;
  if (a.page_tokens % A::kSub == 0) {
    const uint32_t steps = a.page_tokens / A::kSub;
    shift = steps & (steps - 1) ? -1 : 0;
    while (shift >= 0 && (1u << shift) < steps) ++shift;
  }
  return kv_launch("k_kv_attend", kern, dim3(static_cast<unsigned>((items + per - 1) / per * a.splits)), kAtWarps * 32,
                   A::kBytes, a.cluster ? a.splits : 1, stream, a, tiles, shift, static_cast<uint32_t>(items));
}

template <uint32_t DP, uint32_t NT, bool F16, bool PICK>
static int launch_attend(AttendArgs& a, int device, size_t ws_bytes, cudaStream_t stream) {
  using A = Attend<DP, NT, F16, PICK>;
  const uint32_t rows = (PICK ? 1u : a.T) * a.group, tiles = (rows + A::kRows - 1) / A::kRows;
  const uint64_t items = static_cast<uint64_t>(a.n_seqs) * (PICK ? a.T : 1u) * a.kv_heads * tiles;
  if (items > 0x7FFFFFFFull) return IBP_EINVAL;
  const uint64_t resident = resident_ctas(DP, device);
  a.splits = 1;
  a.cluster = 0;
  if (PICK && items >= 2 * resident * kAtWarps)
    return launch_items<DP, NT, F16, PICK, PICK ? 1 : kAtWarps>(a, tiles, items, device, stream);
  a.splits = splits_of(items, (PICK && a.budget < a.max_pages ? a.budget : a.max_pages) * static_cast<uint64_t>(a.page_tokens),
                       resident);
  a.cluster = a.splits > 1 && a.splits <= 8;
  if (a.splits > 8 && ws_bytes < items * a.splits * A::kRows * (DP + 2) * 4) return IBP_EINVAL;
  const int rc = launch_items<DP, NT, F16, PICK, kAtWarps>(a, tiles, items, device, stream);
  if (rc != IBP_OK || a.splits <= 8) return rc;
  const uint64_t warps = items * A::kRows;
  return kv_launch("k_kv_join", k_kv_join<DP, F16, PICK>, dim3(static_cast<unsigned>((warps + 3) / 4)), 128, 0, 1,
                   stream, a, tiles, A::kRows, rows);
}

template <uint32_t DP, uint32_t NT>
static int launch_attend_t(AttendArgs& a, int device, size_t ws_bytes, cudaStream_t stream) {
  if (a.picks)
    return a.f16 ? launch_attend<DP, NT, true, true>(a, device, ws_bytes, stream)
                 : launch_attend<DP, NT, false, true>(a, device, ws_bytes, stream);
  return a.f16 ? launch_attend<DP, NT, true, false>(a, device, ws_bytes, stream)
               : launch_attend<DP, NT, false, false>(a, device, ws_bytes, stream);
}

int launch_kv_attend(AttendArgs& a, int device, size_t ws_bytes, cudaStream_t stream) {
  const uint32_t dp = padded_dim(a.dim), rows = (a.picks ? 1u : a.T) * a.group;
  const bool two = tile_rows(rows, dp) == 16;
  if (dp == 64)
    return two ? launch_attend_t<64, 2>(a, device, ws_bytes, stream) : launch_attend_t<64, 1>(a, device, ws_bytes, stream);
  if (dp == 128)
    return two ? launch_attend_t<128, 2>(a, device, ws_bytes, stream)
               : launch_attend_t<128, 1>(a, device, ws_bytes, stream);
  return launch_attend_t<256, 1>(a, device, ws_bytes, stream);
}

}  // namespace ibp

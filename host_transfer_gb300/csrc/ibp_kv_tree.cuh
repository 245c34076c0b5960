// ibp_kv_tree.cuh - tree attention on the tensor cores (tcgen05), for every call
// with work enough for its set-up (tc_takes in ibp_kv_tree.cu).
//
// A CTA takes MT tiles of 128 query rows (drafted tokens times group heads) of
// one sequence and kv head and walks 128-token tiles of the cache:
//   one producer warp   TMA boxes of K and V, page by page, into a ring;
//   one MMA warp        S = Q K^T (operands in shared memory, S in TMEM), then
//                       O += P V (P in TMEM, V in shared memory, O in TMEM);
//   MT warpgroups       a thread per row: running maximum and sum in registers,
//                       P = exp2(S - m) back to TMEM in the cache's type.
// TMEM (512 columns): two S slots of 128 columns, whose first halves are
// overwritten by P, and O.  With two row tiles each owns a slot and the tensor
// core works on one while the other's softmax runs; with one tile the slots
// alternate between cache tiles.
//
// One row tile is bound by the cache's bytes (64 KB a tile against 1024 cycles
// of tensor work), two by the tensor core (2048 cycles for the same bytes), so
// two are taken wherever there are more than 128 rows.
//
// O is rescaled as soon as a row's maximum grows, so that the largest probability
// is a power of two and its rounding to the cache's type costs nothing.  Putting the
// rescaling off until the maximum has grown by 2^8 saves 2 % on two row tiles
// and takes the output's error from 1.15 to 1.3 - 1.5 of the result's own rounding.
//
// Work is split evenly over the CTAs, one per SM, by tiles of all items in a
// row: a CTA's range may end inside an item, whose parts are then joined by
// k_kv_tree_join in a fixed order.  Ragged lengths thus cost nothing and the
// scratch is two slots per CTA.  The row blocks of a kv head are furthest apart
// in that order and the number of CTAs is a multiple of theirs, so the CTAs that
// read the same cache tiles do so at about the same time: two row blocks read
// DRAM 1.5 times, not twice.
//
// The same kernel serves caches held in 4 bits (tc_load4): codes are decoded on their
// way into the ring, which the tensor core reads as before.  Eight warps do so, a thread
// for each token of K and of V, which makes thirteen in all and leaves the softmax 128
// registers a thread (more than sixteen would leave it fewer).  Measured: the drafts of 13 tokens over 8 caches named at
// tc_load4, 108 MB of codes and scales, 85 us with cold caches (1.3 TB/s; the same
// shape in 16 bits, 384 MB, 80 us).  Neither bytes nor products bound it: about 2900 cycles
// a tile, of which the tensor core works 1030, a loader warp 1500 to 2000 and a softmax
// warp 2400, each of them waiting for another at times; issue slots are 42 % used.  Two
// things that did not help: 64 of the 128 lanes of TMEM on each half of a tile's tokens
// (85 us), and O rescaled only after a growth by 2^8 (85 us, error 1.30 to 1.36 of the
// result's rounding).
//
// Measured on one GB300: 16 ragged caches of up to 32768 tokens, 8 kv heads of 128
// (1.48 GB): 64 rows a head 233 us (6.4 TB/s, 0.94 of the copy rate), 512 rows
// 600 to 640 us in replayed graphs (1.18 to 1.26 PFLOP/s, 0.62 to 0.66 of the library's
// burst product rate and 0.70 to 0.74 of its sustained one; the clock is held down by
// power, and the products alone, without any softmax work, took 502 us) and 680 us
// a pass among single calls on inputs that change.
//
// Every wait has a limit: a CTA that runs into it raises a flag all its waits heed,
// records IBP_ETIMEOUT and returns.  Whether it does or not, the producer leaves
// when its last copies have landed and the MMA warp when its last products and
// their arrivals are done, so nothing writes to a CTA that has left.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ibp_kv4.cuh"

namespace ibp {

constexpr uint32_t kTcTile = 128;      // tokens of a cache tile, rows of a query tile
constexpr uint32_t kTcMinTiles = 2;    // smallest share of a CTA
constexpr float kTcLarge = 262144.f;   // scores (in powers of two) from which the rounding of the maximum shows
constexpr long long kTcWait = IBP_KV_WAIT_CYCLES;  // clock cycles (about 2 s) after which a wait gives up

struct TcArgs {
  AttendArgs a;
  uint32_t box;       // tokens of a TMA box
  uint32_t row_pairs; // row blocks (MT tiles) of an item
  uint32_t q16;       // queries may be read 16 bytes at a time
  float* o_part;      // [2 per CTA][128 MT][DP]
  float2* ml_part;    // [2 per CTA][128 MT]
  int4* first;        // [per CTA]: sequence, kv head, row block of its first segment, its tiles before the range;
                      // then one entry: the tiles of a CTA's range, as 64 bits
  uint32_t n_ctas;
  long long limit;    // clock cycles after which a wait gives up
  Kv4View four[2];    // K and V of a cache in 4 bits
  int32_t shift;      // its pages hold 2^shift tokens; -1: another number
  uint32_t narrow;    // strides, and a page's tokens, within 32 bits
};

namespace tc {

__device__ __forceinline__ uint32_t s32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// False when the limit was met or another wait of the CTA has met it.  A limit of 0
// is met at once, done or not.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* stop, long long limit) {
  if (limit && bar_try(bar, parity)) return true;
  const long long t0 = clock64();
  while (clock64() - t0 < limit) {
    for (uint32_t i = 0; i < 16; ++i)
      if (bar_try(bar, parity)) return true;
    if (*stop) return false;
  }
  *stop = 1;
  return false;
}
// Waits for what the CTA has in flight itself, whatever the flag says.
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!bar_try(bar, parity) && clock64() - t0 < kTcWait) {
  }
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int tok, int head, int page,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(tok), "r"(head), "r"(page), "r"(bar)
      : "memory");
}

// Shared-memory operand of 128-byte swizzled rows.  lead: bytes between 64-
// element groups of the major dimension (V), stride: between groups of 8 rows.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void ld32(float* r, uint32_t addr) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(addr));
}
__device__ __forceinline__ void st32(uint32_t addr, const float* r) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
      "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
      "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
      : "memory");
}
// The loaded registers pass through the wait, so that no use of them can be
// moved before it.
__device__ __forceinline__ void ld_wait32(float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]), "+r"(u[6]), "+r"(u[7]), "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]), "+r"(u[12]), "+r"(u[13]), "+r"(u[14]), "+r"(u[15]), "+r"(u[16]), "+r"(u[17]), "+r"(u[18]), "+r"(u[19]), "+r"(u[20]), "+r"(u[21]), "+r"(u[22]), "+r"(u[23]), "+r"(u[24]), "+r"(u[25]), "+r"(u[26]), "+r"(u[27]), "+r"(u[28]), "+r"(u[29]), "+r"(u[30]), "+r"(u[31])
               :
               : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two single-precision lanes in one register pair.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace tc

// FOUR: the cache is held in 4 bits.  Instead of the warp that issues TMA boxes, eight
// warps read codes and write the tiles: a thread has one token of K or V.
template <uint32_t DP, uint32_t MT, bool FOUR = false>
struct TcShape {
  static constexpr uint32_t kHalves = DP / 64;                       // 128-byte wide panels of a tile
  static constexpr uint32_t kPanel = kTcTile * 128;                  // bytes of a panel
  static constexpr uint32_t kTileBytes = kHalves * kPanel;           // K or V of a stage, Q of a tile
  // Two tiles of Q: one for each row tile, or for one row tile the next segment's
  // beside this one's, so that its scores begin while the output is still written.
  static constexpr uint32_t kQ = 2;
  // Ring of tiles, K and V in turn.  One row tile is bound by the loads and takes
  // all that fit, two and a half cache tiles (with two, the 16 caches above take 5 %
  // more); two row tiles are bound by the products and do no better with more than
  // two (with two and a half 2 % more).
  static constexpr uint32_t kSlots = DP == 128 ? (MT == 1 ? 5 : 4) : (MT == 1 ? 11 : 8);
  static constexpr uint32_t kBytes = (kQ + kSlots) * kTileBytes;
  static constexpr uint32_t kSmem = kBytes + 1024 + 512;             // alignment, barriers
  static constexpr uint32_t kLoaders = FOUR ? 8 : 1;                 // warps
  static constexpr uint32_t kMmaWarp = MT * 4 + (FOUR ? 0 : 1);
  static constexpr uint32_t kLoadWarp = MT * 4 + (FOUR ? 1 : 0);     // the first of them
  static constexpr uint32_t kThreads = MT * 128 + 32 + kLoaders * 32;
  static constexpr uint32_t kOCol = 256;                             // first column of O
};

struct TcShared {
  uint64_t full[11], empty[11];
  uint64_t s_full[2], p_full[2][2], pv_done[2], q_full[2], done;  // p_full: per slot and half
  uint32_t tmem;
  uint32_t stop;
  uint32_t odd[2];    // even and odd segments: 1 + the last whose draft holds infinities or NaN among its values
  uint32_t pair0, b0; // row block and sequence in which this CTA's range begins
  uint64_t in0;       // tiles of that sequence before the range
  uint32_t sums[14];
};

// A part of an item inside one CTA's range.
struct TcSeg {
  uint32_t b, h, pair;
  uint32_t tile0, tiles;   // first cache tile and their number
  uint32_t all;            // cache tiles of the item
  int32_t len, n_live, ctx;
};

// Cache tiles of a sequence, at least one, so that empty items write their zeros.
template <uint32_t TILE = kTcTile>
__device__ __forceinline__ uint32_t tiles_of(const AttendArgs& a, uint32_t b) {
  const int32_t len = clamp_len(a.lens[b], a.page_tokens, a.max_pages);
  return len > 0 ? ceil_div(static_cast<uint32_t>(len), TILE) : 1u;
}

// Walks the segments of [at, end): every role of the CTA does so by itself.
template <uint32_t TILE = kTcTile>
struct TcWalkOf {
  const TcArgs& t;
  uint32_t pair, b;     // present row block and sequence
  uint32_t tiles;       // of each of its items
  uint64_t in;          // position inside the sequence's tiles
  uint64_t left;
  __device__ TcWalkOf(const TcArgs& t_, uint32_t pair0, uint32_t b0, uint64_t in0, uint64_t at, uint64_t end) : t(t_) {
    pair = pair0;
    b = b0;
    tiles = at < end ? tiles_of<TILE>(t.a, b) : 1;
    in = in0;
    left = end - at;
  }
  __device__ bool next(TcSeg* s) {
    if (left == 0) return false;
    if (in == static_cast<uint64_t>(tiles) * t.a.kv_heads) {
      if (++b == t.a.n_seqs) {
        b = 0;
        ++pair;
      }
      in = 0;
      tiles = tiles_of<TILE>(t.a, b);
    }
    const uint32_t item = static_cast<uint32_t>(in / tiles);
    s->tile0 = static_cast<uint32_t>(in - static_cast<uint64_t>(item) * tiles);
    const uint64_t rest = tiles - s->tile0;
    s->tiles = static_cast<uint32_t>(rest < left ? rest : left);
    s->all = tiles;
    s->b = b;
    s->pair = pair;
    s->h = item;
    const int32_t len = clamp_len(t.a.lens[b], t.a.page_tokens, t.a.max_pages);
    const int32_t n = t.a.n_live ? t.a.n_live[b] : static_cast<int32_t>(t.a.T);
    s->len = len;
    s->n_live = n < 0 ? 0 : (n > static_cast<int32_t>(t.a.T) ? static_cast<int32_t>(t.a.T) : n);
    s->ctx = len - s->n_live;
    in += s->tiles;
    left -= s->tiles;
    return true;
  }
};

struct TcWalk : TcWalkOf<> {
  __device__ TcWalk(const TcArgs& t_, const TcShared& sh, uint64_t at, uint64_t end)
      : TcWalkOf<>(t_, sh.pair0, sh.b0, sh.in0, at, end) {}
};

// Bit i: position p0 + i is seen by draft token t (false for rows that do not exist).
__device__ __forceinline__ uint32_t seen_bits(const AttendArgs& a, const TcSeg& s, const uint32_t* words, uint32_t t,
                                              int32_t p0) {
  uint32_t bits = 0;
  const int32_t before = s.ctx - p0;  // positions of the context in this word
  if (before >= 32)
    bits = 0xFFFFFFFFu;
  else {
    if (before > 0) bits = (1u << before) - 1u;
    // draft bits i0 .. i0 + 31, i0 = p0 - ctx
    const int32_t i0 = -before;
    uint32_t d;
    if (!a.mask) {
      const int32_t n = static_cast<int32_t>(t) + 1 - i0;  // i <= t
      d = n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u);
      if (i0 < 0) d &= ~((1u << -i0) - 1u);
    } else {
      const int32_t w = i0 >> 5;
      const uint32_t sh = static_cast<uint32_t>(i0) & 31u;
      const uint32_t lo = w >= 0 && w < static_cast<int32_t>(a.mask_words) ? words[w] : 0u;
      const uint32_t hi = w + 1 >= 0 && w + 1 < static_cast<int32_t>(a.mask_words) ? words[w + 1] : 0u;
      d = __funnelshift_r(lo, hi, sh);
    }
    bits |= d;
  }
  const int32_t room = s.len - p0;
  if (room < 32) bits &= room <= 0 ? 0u : (1u << room) - 1u;
  return bits;
}

// The tiles of a cache in 4 bits: thread r of the first half writes token r of every K
// tile, one of the second half of every V tile, in the swizzled layout that TMA boxes
// have, the elements of eight in the decoder's order.  Codes are two tiles ahead of
// the one that is decoded, pages three.
// EVEN: all of DP's dimensions, a token's scales aligned for one read.
template <uint32_t DP, uint32_t MT, bool F16, bool EVEN>
__device__ __forceinline__ void tc_load4(const TcArgs& t, TcShared& sh, uint64_t at, uint64_t end, unsigned char* ring_sm, uint32_t thread) {
  using S = TcShape<DP, MT, true>;
  const AttendArgs& a = t.a;
  const uint32_t r = thread & 127u, kv = thread >> 7, lane = thread & 31u;
  const Kv4View& v = t.four[kv];
  volatile uint32_t* stop = &sh.stop;
  struct Spot {  // nothing is done with the page here: it is still on its way
    uint32_t page, slot;
    const char *codes, *scales;  // of the head
    bool there;
  };
  struct Raw {
    uint4 w[DP / 32];
    uint32_t s[DP / 32];  // EVEN: two to a word
    bool good;
  };
  TcWalk walk(t, sh, at, end);
  TcSeg s;
  bool more = walk.next(&s);
  uint32_t j = 0;
  const char *codes = v.codes, *scales = v.scales;
  const int32_t* row = a.table;
  auto next_spot = [&](Spot& sp) {
    sp.page = sp.slot = 0;
    sp.there = false;
    if (!more) return;
    if (j == 0) {
      codes = v.codes + static_cast<int64_t>(s.h) * v.head_stride;
      scales = v.scales + static_cast<int64_t>(s.h) * v.s_head;
      row = a.table + static_cast<uint64_t>(s.b) * a.max_pages;
      if (thread == 0) {
        const int32_t raw = a.lens[s.b], n = a.n_live ? a.n_live[s.b] : static_cast<int32_t>(a.T);
        if (raw != s.len || n != s.n_live || n > s.len) kv_status(a.status, IBP_ERANGE);
      }
    }
    const uint32_t p = (s.tile0 + j) * kTcTile + r;
    sp.codes = codes, sp.scales = scales;
    if (static_cast<int32_t>(p) < s.len) {
      const uint32_t nth = t.shift >= 0 ? p >> t.shift : p / a.page_tokens;
      sp.slot = t.shift >= 0 ? p & ((1u << t.shift) - 1u) : p - nth * a.page_tokens;
      sp.there = true;
      sp.page = static_cast<uint32_t>(__ldg(row + nth));
    }
    if (++j == s.tiles) {
      more = walk.next(&s);
      j = 0;
    }
  };
  // Tokens that are not there read page 0 and become zeros when they are decoded.
  auto fetch = [&](const Spot& sp, Raw& raw) {
    raw.good = sp.there && sp.page < a.n_pages;
    if (!raw.good && sp.there) kv_status(a.status, IBP_ERANGE);
    const char *c = v.codes, *sc = v.scales;
    if (raw.good) {
      if (t.narrow) {
        c = sp.codes + static_cast<uint64_t>(sp.page) * static_cast<uint32_t>(v.page_stride) + static_cast<uint64_t>(sp.slot) * static_cast<uint32_t>(v.token_stride);
        sc = sp.scales + static_cast<uint64_t>(sp.page) * static_cast<uint32_t>(v.s_page) + static_cast<uint64_t>(sp.slot) * static_cast<uint32_t>(v.s_token);
      } else {
        c = sp.codes + static_cast<int64_t>(sp.page) * v.page_stride + static_cast<int64_t>(sp.slot) * v.token_stride;
        sc = sp.scales + static_cast<int64_t>(sp.page) * v.s_page + static_cast<int64_t>(sp.slot) * v.s_token;
      }
    }
    if constexpr (EVEN) {
#pragma unroll
      for (uint32_t g = 0; g < DP / 32; ++g) raw.w[g] = __ldg(reinterpret_cast<const uint4*>(c + g * 16));
      if constexpr (DP == 128) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(sc));
        raw.s[0] = x.x, raw.s[1] = x.y;
      } else {
        raw.s[0] = __ldg(reinterpret_cast<const uint32_t*>(sc));
      }
    } else {
#pragma unroll
      for (uint32_t g = 0; g < DP / 32; ++g) {
        const bool in = g * 32 < a.dim;
        raw.w[g] = in ? __ldg(reinterpret_cast<const uint4*>(c + g * 16)) : make_uint4(0u, 0u, 0u, 0u);
        raw.s[g] = in ? static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(sc + g * 2))) : 0u;
      }
    }
  };
  uint32_t turn[8];  // places of a row's pieces of 16 bytes
#pragma unroll
  for (uint32_t c = 0; c < 8; ++c) turn[c] = r * 128 + ((c ^ (r & 7u)) << 4);
  const quad::Magic<F16> magic;
  const uint64_t n = end - at;
  Spot spot;
  Raw raw[2];
  next_spot(spot);
  fetch(spot, raw[0]);
  next_spot(spot);
  fetch(spot, raw[1]);
  next_spot(spot);
  bool ok = true;
  // One tile a round, the next one's codes moved up: with two rounds written out the
  // loop and the softmax's do not stay in the instruction cache (104 us against 85 us for
  // drafts of 13 tokens, 8 ragged caches of up to 16384, 8 kv heads of 4 query heads of 128).
#pragma unroll 1
  for (uint64_t i = 0; i < n && ok; ++i) {
    const uint32_t f = static_cast<uint32_t>(2 * i) + kv, slot = f % S::kSlots;
    if (lane == 0) ok = tc::bar_wait(tc::s32(&sh.empty[slot]), (f / S::kSlots & 1u) ^ 1u, stop, t.limit);
    ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    if (!ok) break;
    unsigned char* dst = ring_sm + slot * S::kTileBytes;
#pragma unroll
    for (uint32_t g = 0; g < DP / 32; ++g) {
      const quad::Pair<F16> p(EVEN ? __byte_perm(raw[0].s[g / 2], 0, g & 1u ? 0x3232 : 0x1010) : __byte_perm(raw[0].s[g], 0, 0x1010), raw[0].good);
      const uint32_t w[4] = {raw[0].w[g].x, raw[0].w[g].y, raw[0].w[g].z, raw[0].w[g].w};
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) {
        const uint32_t c = g * 4 + e;
        *reinterpret_cast<uint4*>(dst + (c / 8) * S::kPanel + turn[c & 7u]) =
            make_uint4(quad::decode<F16, 0>(w[e], p, magic), quad::decode<F16, 1>(w[e], p, magic),
                       quad::decode<F16, 2>(w[e], p, magic), quad::decode<F16, 3>(w[e], p, magic));
      }
    }
    tc::fence_async();
    tc::bar_arrive(tc::s32(&sh.full[slot]));
    raw[0] = raw[1];
    // here and not at the round's end, where it would wait for the codes just asked for
#pragma unroll
    for (uint32_t g = 0; g < DP / 32; ++g)
      asm volatile("" : "+r"(raw[0].w[g].x), "+r"(raw[0].w[g].y), "+r"(raw[0].w[g].z), "+r"(raw[0].w[g].w), "+r"(raw[0].s[EVEN ? g / 2 : g]));
    fetch(spot, raw[1]);
    next_spot(spot);
  }
}

// Element of a group of eight that the decoder puts at place k, and the place of element e.
__device__ constexpr uint32_t quad_element(uint32_t k) { return (k >> 1) + (k & 1u) * 4; }
__device__ constexpr uint32_t quad_place(uint32_t e) { return (e & 3u) * 2 + (e >> 2); }

template <uint32_t DP, uint32_t MT, bool F16, bool FOUR = false, bool EVEN = false>
__global__ void __launch_bounds__(TcShape<DP, MT, FOUR>::kThreads, 1)
    k_kv_tree(const __grid_constant__ TcArgs t, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v) {
  using S = TcShape<DP, MT, FOUR>;
  const AttendArgs& a = t.a;
  extern __shared__ unsigned char raw_sm[];
  unsigned char* sm = raw_sm + ((1024 - (tc::s32(raw_sm) & 1023u)) & 1023u);
  const uint32_t base = tc::s32(sm);
  TcShared& sh = *reinterpret_cast<TcShared*>(sm + S::kBytes);
  static_assert(sizeof(TcShared) <= 512, "barriers");
  const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
  const uint32_t q_sm = base, kv_sm = base + S::kQ * S::kTileBytes;
  // Fill f of the ring is K of tile f / 2 of this CTA's range, or its V.
  auto ring = [](uint32_t f) { return f % S::kSlots; };
  auto ring_phase = [](uint32_t f) { return (f / S::kSlots) & 1u; };
  auto ring_at = [&](uint32_t f) { return kv_sm + ring(f) * S::kTileBytes; };

  if (tid == 0) {
    for (uint32_t i = 0; i < S::kSlots; ++i) {
      tc::bar_init(tc::s32(&sh.full[i]), FOUR ? 128 : 1);
      tc::bar_init(tc::s32(&sh.empty[i]), 1);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      tc::bar_init(tc::s32(&sh.s_full[i]), 1);
      tc::bar_init(tc::s32(&sh.p_full[i][0]), 128);
      tc::bar_init(tc::s32(&sh.p_full[i][1]), 128);
      tc::bar_init(tc::s32(&sh.pv_done[i]), 1);
      tc::bar_init(tc::s32(&sh.q_full[i]), 128);
    }
    tc::bar_init(tc::s32(&sh.done), 1);
    sh.stop = 0;
    sh.odd[0] = sh.odd[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if constexpr (!FOUR) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v) : "memory");
    }
  }
  if (warp == S::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::s32(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_begin();

  // Where this CTA's range begins: the tiles of all sequences, and the first
  // sequence that reaches past the start.
  {
    uint32_t n = 0;
    for (uint32_t b = tid; b < a.n_seqs; b += S::kThreads) n += tiles_of(a, b);
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    if (lane == 0) sh.sums[warp] = n;
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
  }
  uint64_t total = 0;
#pragma unroll
  for (uint32_t i = 0; i < S::kThreads / 32; ++i) total += sh.sums[i];
  const uint64_t block = total * a.kv_heads;  // tiles of a row block
  total = block * t.row_pairs;
  uint64_t share = (total + t.n_ctas - 1) / t.n_ctas;
  if (share < kTcMinTiles) share = kTcMinTiles;
  const uint64_t at = blockIdx.x * share < total ? blockIdx.x * share : total;
  const uint64_t end = total - at < share ? total : at + share;
  if (warp == 0 && at < end) {
    const uint32_t pair = static_cast<uint32_t>(at / block);
    const uint64_t in = at - pair * block;
    uint64_t seen = 0;
    for (uint32_t c = 0; c < a.n_seqs; c += 32) {
      const uint32_t b = c + lane;
      uint64_t n = b < a.n_seqs ? static_cast<uint64_t>(tiles_of(a, b)) * a.kv_heads : 0, incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
      }
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, seen + incl > in);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
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
  const uint32_t tmem = sh.tmem;
  volatile uint32_t* stop = &sh.stop;

  if (warp >= S::kLoadWarp && warp < S::kLoadWarp + S::kLoaders) {
    if constexpr (FOUR) {
      tc_load4<DP, MT, F16, EVEN>(t, sh, at, end, sm + (kv_sm - base), tid - S::kLoadWarp * 32);
    } else {
      // ---- producer: one lane issues; all follow the same path
      TcWalk walk(t, sh, at, end);
      TcSeg s;
      uint32_t f = 0;  // fills so far
      bool ok = true;
      const uint32_t boxes = kTcTile / t.box;
      while (ok && walk.next(&s)) {
        const int32_t* row = a.table + static_cast<uint64_t>(s.b) * a.max_pages;
        if (lane == 0) {
          const int32_t raw = a.lens[s.b], n = a.n_live ? a.n_live[s.b] : static_cast<int32_t>(a.T);
          if (raw != s.len || n != s.n_live || n > s.len) kv_status(a.status, IBP_ERANGE);
        }
        for (uint32_t j = 0; j < s.tiles && ok; ++j) {
          const int32_t p0 = static_cast<int32_t>((s.tile0 + j) * kTcTile);
          // lane i finds the page of box i
          const int32_t p = p0 + static_cast<int32_t>(lane * t.box);
          const bool have = lane < boxes && p < s.len;
          int32_t page = 0, slot = 0;
          if (have) {
            const uint32_t nth = static_cast<uint32_t>(p) / a.page_tokens;
            slot = p - static_cast<int32_t>(nth * a.page_tokens);
            page = row[nth];
            if (static_cast<uint32_t>(page) >= a.n_pages) {
              kv_status(a.status, IBP_ERANGE);
              page = static_cast<int32_t>(a.n_pages);  // past the last page: the box reads zeros
            }
          }
          const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, have));
          const uint32_t bytes = n * t.box * 128 * S::kHalves;
#pragma unroll
          for (uint32_t kv = 0; kv < 2; ++kv, ++f) {
            ok = tc::bar_wait(tc::s32(&sh.empty[ring(f)]), ring_phase(f) ^ 1u, stop, t.limit);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const uint32_t bar = tc::s32(&sh.full[ring(f)]), dst = ring_at(f) + lane * t.box * 128;
            if (lane == 0) tc::bar_expect(bar, bytes);
            __syncwarp();
            if (have)
#pragma unroll
              for (uint32_t hf = 0; hf < S::kHalves; ++hf)
                tc::tma_box(dst + hf * S::kPanel, kv ? &map_v : &map_k, hf * 64, slot, s.h, page, bar);
          }
        }
      }
      for (uint32_t i = 0; i < S::kSlots; ++i) {  // copies in flight land before the CTA leaves
        const uint32_t n = (f + S::kSlots - 1 - i) / S::kSlots;  // fills of slot i
        if (n) tc::bar_drain(tc::s32(&sh.full[i]), (n - 1) & 1u);
      }
    }
  } else if (warp == S::kMmaWarp) {
    // ---- MMA
    const uint32_t fmt = F16 ? 0u : 1u;
    const uint32_t id_qk = (1u << 4) | (fmt << 7) | (fmt << 10) | ((kTcTile >> 3) << 17) | ((kTcTile >> 4) << 24);
    const uint32_t id_pv = (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 16) | ((DP >> 3) << 17) | ((kTcTile >> 4) << 24);
    TcWalk walk(t, sh, at, end);
    TcSeg s;
    uint32_t g = 0, segs = 0;
    bool ok = true;
    // One elected thread issues.  The descriptors of a group differ from its
    // first by constants, so that eight products are little more than eight
    // instructions: built one by one from addresses, beside two busy softmax warps
    // on the scheduler, each took 110 cycles instead of the 64 it runs for.
    const uint64_t qd = tc::operand(q_sm, 16), kd = tc::operand(kv_sm, 16), vd = tc::operand(kv_sm, S::kPanel);
    constexpr uint32_t kTileStep = S::kTileBytes >> 4;
    auto qk = [&](uint32_t tile, uint32_t slot, uint32_t f) {
      if (tc::elect()) {
        const uint64_t qa = qd + (MT == 1 ? segs & 1u : tile) * kTileStep, ka = kd + ring(f) * kTileStep;
        const uint32_t d = tmem + slot * 128;
#pragma unroll
        for (uint32_t kk = 0; kk < DP / 16; ++kk) {
          const uint32_t off = ((kk / 4) * S::kPanel + (kk % 4) * 32) >> 4;
          tc::mma_ss(d, qa + off, ka + off, id_qk, kk > 0);
        }
        tc::commit(tc::s32(&sh.s_full[slot]));
      }
      __syncwarp();
    };
    // Half hf of P V: 64 tokens.
    auto pv = [&](uint32_t tile, uint32_t slot, uint32_t f, uint32_t hf, bool add) {
      if (tc::elect()) {
        const uint64_t va = vd + ring(f) * kTileStep + hf * (8192 >> 4);
        const uint32_t d = tmem + S::kOCol + tile * DP, p = tmem + slot * 128 + hf * 32;
        tc::mma_ts(d, p, va, id_pv, add);
#pragma unroll
        for (uint32_t kk = 1; kk < kTcTile / 32; ++kk) tc::mma_ts(d, p + kk * 8, va + kk * (2048 >> 4), id_pv, 1);
        if (hf) tc::commit(tc::s32(&sh.pv_done[slot]));
      }
      __syncwarp();
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool r = tc::bar_wait(tc::s32(bar), parity, stop, t.limit);
      return __all_sync(0xFFFFFFFFu, r) != 0;
    };
    auto release = [&](uint64_t* bar) {
      if (tc::elect()) tc::commit(tc::s32(bar));
      __syncwarp();
    };
    // V of the item's last tiles: tokens past the length become zeros (what the
    // pages hold there must not meet a zero probability), and infinities and NaN
    // of drafted tokens are taken out for the epilogue to add.
    auto clean = [&](const TcSeg& sg, uint32_t j, uint32_t f) {
      const int32_t p0 = static_cast<int32_t>((sg.tile0 + j) * kTcTile);
      const int32_t end_tok = sg.len - p0;                        // tokens of this tile
      if (end_tok >= static_cast<int32_t>(kTcTile) && p0 + static_cast<int32_t>(kTcTile) <= sg.ctx) return;
      unsigned char* v = sm + (ring_at(f) - base);
      const uint32_t valid = end_tok <= 0 ? 0u : (end_tok < static_cast<int32_t>(kTcTile) ? end_tok : kTcTile);
      for (uint32_t i = valid * 8 + lane; i < kTcTile * 8; i += 32)
#pragma unroll
        for (uint32_t hf = 0; hf < S::kHalves; ++hf)
          *reinterpret_cast<uint4*>(v + hf * S::kPanel + i * 16) = make_uint4(0, 0, 0, 0);
      const int32_t d0 = sg.ctx - p0;
      const uint32_t from = d0 <= 0 ? 0u : static_cast<uint32_t>(d0);
      const uint32_t ex = F16 ? 0x7C007C00u : 0x7F807F80u;
      uint32_t odd = 0;
      for (uint32_t hf = 0; hf < S::kHalves; ++hf)
        for (uint32_t i = from * 8 + lane; i < valid * 8; i += 32) {
          uint4* w = reinterpret_cast<uint4*>(v + hf * S::kPanel + i * 16);
          uint4 x = *w;
          uint32_t* xs = reinterpret_cast<uint32_t*>(&x);
          uint32_t hit = 0;
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) {
            const uint32_t m = xs[e] & ex;
            const uint32_t lo = (m & 0xFFFFu) == (ex & 0xFFFFu) ? 0xFFFFu : 0u;
            const uint32_t hi = (m >> 16) == (ex >> 16) ? 0xFFFF0000u : 0u;
            hit |= lo | hi;
            xs[e] &= ~(lo | hi);
          }
          if (hit) *w = x;
          odd |= hit;
        }
      if (__any_sync(0xFFFFFFFFu, odd != 0) && lane == 0) *reinterpret_cast<volatile uint32_t*>(&sh.odd[segs & 1u]) = segs + 1;
      tc::fence_async();
      __syncwarp();
    };
    while (ok && walk.next(&s)) {
#pragma unroll
      for (uint32_t m = 0; m < MT; ++m) ok = ok && wait(&sh.q_full[m], segs & 1u);
      if (!ok) break;
      tc::fence_after();
      const uint32_t n = s.tiles;
      auto kf = [&](uint32_t j) { return 2 * (g + j); };
      auto vf = [&](uint32_t j) { return 2 * (g + j) + 1; };
      auto loaded = [&](uint32_t f) { return wait(&sh.full[ring(f)], ring_phase(f)); };
      if (MT == 2) {
        if (!(ok = loaded(kf(0)))) break;
        qk(0, 0, kf(0));
        qk(1, 1, kf(0));
        release(&sh.empty[ring(kf(0))]);
        for (uint32_t j = 0; j < n; ++j) {
          if (!(ok = loaded(vf(j)))) break;
          clean(s, j, vf(j));
          if (!(ok = wait(&sh.p_full[0][0], (g + j) & 1u))) break;
          tc::fence_after();
          pv(0, 0, vf(j), 0, j > 0);
          if (!(ok = wait(&sh.p_full[0][1], (g + j) & 1u))) break;
          tc::fence_after();
          pv(0, 0, vf(j), 1, true);
          if (j + 1 < n) {
            if (!(ok = loaded(kf(j + 1)))) break;
            qk(0, 0, kf(j + 1));
          }
          if (!(ok = wait(&sh.p_full[1][0], (g + j) & 1u))) break;
          tc::fence_after();
          pv(1, 1, vf(j), 0, j > 0);
          if (!(ok = wait(&sh.p_full[1][1], (g + j) & 1u))) break;
          tc::fence_after();
          pv(1, 1, vf(j), 1, true);
          release(&sh.empty[ring(vf(j))]);
          if (j + 1 < n) {
            qk(1, 1, kf(j + 1));
            release(&sh.empty[ring(kf(j + 1))]);
          }
        }
      } else {
        for (uint32_t j = 0; j < 2 && j < n; ++j) {
          if (!(ok = loaded(kf(j)))) break;
          qk(0, (g + j) & 1u, kf(j));
          release(&sh.empty[ring(kf(j))]);
        }
        for (uint32_t j = 0; j < n && ok; ++j) {
          if (!(ok = loaded(vf(j)))) break;
          clean(s, j, vf(j));
          const uint32_t slot = (g + j) & 1u, ph = ((g + j) >> 1) & 1u;
          if (!(ok = wait(&sh.p_full[slot][0], ph))) break;
          tc::fence_after();
          pv(0, slot, vf(j), 0, j > 0);
          if (!(ok = wait(&sh.p_full[slot][1], ph))) break;
          tc::fence_after();
          pv(0, slot, vf(j), 1, true);
          release(&sh.empty[ring(vf(j))]);
          if (j + 2 < n) {
            if (!(ok = loaded(kf(j + 2)))) break;
            qk(0, (g + j) & 1u, kf(j + 2));
            release(&sh.empty[ring(kf(j + 2))]);
          }
        }
      }
      g += n;
      ++segs;
    }
    // the last products and the arrivals they cause end before the CTA leaves
    release(&sh.done);
    tc::bar_drain(tc::s32(&sh.done), 0);
    __syncwarp();
  } else if (warp < MT * 4) {
    // ---- softmax: warpgroup m, a thread per row
    const uint32_t m = warp / 4, r = tid & 127u;
    const uint32_t lanes = (warp & 3u) << 21;  // this warp's quarter of the TMEM lanes
    TcWalk walk(t, sh, at, end);
    TcSeg s, following;
    uint32_t g = 0, segs = 0;
    bool ok = true;
    // This thread's row of Q of a segment.
    auto load_q = [&](const TcSeg& sg, uint32_t nth) {
      const uint32_t gr = (sg.pair * MT + m) * kTcTile + r;
      const uint32_t tok = gr / a.group, head = gr - tok * a.group;
      const bool live = static_cast<int32_t>(tok) < sg.n_live;
      const char* q = a.q + static_cast<int64_t>(sg.b) * a.q_seq + static_cast<int64_t>(live ? tok : 0) * a.q_token +
                      static_cast<int64_t>(sg.h * a.group + (live ? head : 0)) * a.q_head;
      unsigned char* dst = sm + (MT == 1 ? nth & 1u : m) * S::kTileBytes + r * 128;
#pragma unroll
      for (uint32_t c = 0; c < DP / 8; ++c) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (live && c * 8 < a.dim) {
          if (t.q16)
            x = *reinterpret_cast<const uint4*>(q + c * 16);
          else {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(q + c * 16);
            x = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if constexpr (FOUR)  // dimensions as the decoder has them
          x = make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                         __byte_perm(x.y, x.w, 0x7632));
        *reinterpret_cast<uint4*>(dst + (c / 8) * S::kPanel + (((c & 7u) ^ (r & 7u)) << 4)) = x;
      }
      tc::fence_async();
      tc::bar_arrive(tc::s32(&sh.q_full[m]));
    };
    // Waits for P V of a tile, and so for all before it.  A wait by parity must be
    // neither a phase behind its barrier nor two ahead.  With alternating slots the
    // last two products may both be under way, or both done, so each slot has a
    // barrier: its product before was done when this tile's scores were, and its
    // next one needs this thread's P.
    auto product_done = [&](uint32_t x) {
      const bool r = tc::bar_wait(tc::s32(&sh.pv_done[MT == 2 ? m : x & 1u]), (MT == 2 ? x : x >> 1) & 1u, stop, t.limit);
      return __all_sync(0xFFFFFFFFu, r) != 0;
    };
    bool more = walk.next(&s);
    // What the join goes by is written before anything is waited for.
    if (tid == 0) {
      t.first[blockIdx.x] = more ? make_int4(s.b, s.h, s.pair, s.tile0) : make_int4(-1, 0, 0, 0);
      if (blockIdx.x == 0)
        t.first[t.n_ctas] = make_int4(static_cast<int>(share & 0xFFFFFFFFu), static_cast<int>(share >> 32), 0, 0);
    }
    if (more) load_q(s, 0);
    while (ok && more) {
      const uint32_t gr = (s.pair * MT + m) * kTcTile + r;
      const uint32_t tok = gr / a.group, head = gr - tok * a.group;
      const bool exists = tok < a.T, live = static_cast<int32_t>(tok) < s.n_live;
      const uint32_t* words =
          a.mask ? a.mask + (static_cast<uint64_t>(s.b) * a.T + (live ? tok : 0)) * a.mask_words : nullptr;
      float top = -INFINITY, sum = 0.f;  // running maximum (of score * log2 e, less the lift) and sum
      const uint32_t o_col = tmem + lanes + S::kOCol + m * DP;
      for (uint32_t j = 0; j < s.tiles; ++j) {
        const uint32_t slot = MT == 2 ? m : (g + j) & 1u;
        const uint32_t ph = MT == 2 ? (g + j) & 1u : ((g + j) >> 1) & 1u;
        ok = tc::bar_wait(tc::s32(&sh.s_full[slot]), ph, stop, t.limit);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc::fence_after();
        if constexpr (FOUR) {
          // a warp without a row: what its lanes of TMEM hold reaches no other row
          if (!__any_sync(0xFFFFFFFFu, live)) {
            tc::fence_before();
            tc::bar_arrive(tc::s32(&sh.p_full[slot][0]));
            tc::bar_arrive(tc::s32(&sh.p_full[slot][1]));
            continue;
          }
        }
        const uint32_t s_col = tmem + lanes + slot * 128;
        const int32_t p0 = static_cast<int32_t>((s.tile0 + j) * kTcTile);
        const bool partly = p0 + static_cast<int32_t>(kTcTile) > s.ctx;  // some row may not see it all
        if (partly) {  // what the row does not see becomes -infinity, in place
#pragma unroll 1
          for (uint32_t c = 0; c < 4; ++c) {
            const uint32_t bits = live ? seen_bits(a, s, words, tok, p0 + 32 * static_cast<int32_t>(c)) : 0u;
            float x[32];
            tc::ld32(x, s_col + 32 * c);
            tc::ld_wait32(x);
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i)
              if (!((bits >> i) & 1u)) x[i] = -INFINITY;
            tc::st32(s_col + 32 * c, x);
          }
          tc::st_wait();
        }
        // The scores are read twice, 32 at a time: for the maximum, and for the
        // exponentials.  All 128 in registers would spill at 168 a thread.
        float y[2][32];
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        tc::ld32(y[0], s_col);
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
          float(&x)[32] = y[c & 1u];
          tc::ld_wait32(x);
          tc::ld32(y[(c + 1) & 1u], s_col + 32 * ((c + 1) & 3u));
#pragma unroll
          for (uint32_t i = 0; i < 32; i += 8)
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], fmaxf(x[i + e], x[i + e + 4]));
        }
        float high = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // The exponent scale x - top keeps what the rounding of top lost, up to an ulp of
        // it: nothing beside the row's own roundings for ordinary scores, but powers of two
        // by the dozen for scores past 2^26.  A row with such a maximum has its scores
        // scaled first, in place, so that its largest exponent is exact again.
        const bool large = fabsf(high) * a.scale_log2 >= kTcLarge && fabsf(high) < INFINITY;
        if (__any_sync(0xFFFFFFFFu, large)) {
          const float f = large ? a.scale_log2 : 1.f;
          tc::ld_wait32(y[0]);
#pragma unroll 1
          for (uint32_t c = 0; c < 4; ++c) {
            float x[32];
            tc::ld32(x, s_col + 32 * c);
            tc::ld_wait32(x);
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i) x[i] *= f;
            tc::st32(s_col + 32 * c, x);
          }
          tc::st_wait();
          tc::ld32(y[0], s_col);
          high *= f;
        }
        const float scale = large ? 1.f : a.scale_log2;
        const float tile_top = F16 ? __fmaf_ru(high, scale, -kLift<F16>) : high * scale;
        const bool grow = tile_top > top;
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float f = grow ? tc::ex2(top - tile_top) : 1.f;
          if (grow) top = tile_top;
          sum *= f;
          if (j > 0) {
            // O holds the sums up to the tile before
            ok = product_done(g + j - 1);
            if (!ok) {
              tc::ld_wait32(y[0]);  // no load is under way into registers that are used again
              break;
            }
            tc::fence_after();
#pragma unroll
            for (uint32_t c = 0; c < DP / 32; ++c) {
              float o[32];
              tc::ld32(o, o_col + 32 * c);
              tc::ld_wait32(o);
#pragma unroll
              for (uint32_t i = 0; i < 32; ++i) o[i] *= f;
              tc::st32(o_col + 32 * c, o);
            }
          }
        }
        const float off = top == -INFINITY ? 0.f : -top;
        uint64_t part[2] = {0, 0};  // two sums of two lanes
        const uint64_t scale2 = tc::two(scale, scale), off2 = tc::two(off, off);
        float w[32];
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
          float(&x)[32] = y[c & 1u];
          tc::ld_wait32(x);
          if (c < 3) tc::ld32(y[(c + 1) & 1u], s_col + 32 * (c + 1));
#pragma unroll
          for (uint32_t i = 0; i < 16; ++i) {
            float p, q;
            tc::split(tc::fma2(tc::two(x[2 * i], x[2 * i + 1]), scale2, off2), p, q);
            p = tc::ex2(p), q = tc::ex2(q);
            part[i & 1u] = tc::add2(part[i & 1u], tc::two(p, q));
            w[(c & 1u) * 16 + i] = __uint_as_float(tc::pack2<F16>(p, q));
          }
          if (c & 1u) {  // half of P: its product may begin
            tc::st32(s_col + 32 * (c / 2), w);
            tc::st_wait();
            tc::fence_before();
            tc::bar_arrive(tc::s32(&sh.p_full[slot][c / 2]));
          }
        }
        float s0, s1;
        tc::split(tc::add2(part[0], part[1]), s0, s1);
        sum += s0 + s1;
      }
      if (!ok) break;
      // Every product of the segment before that read the other buffer has been
      // waited for.
      const bool again = walk.next(&following);
      if (MT == 1 && again) load_q(following, segs + 1);
      // ---- this segment's sums
      if (!(ok = product_done(g + s.tiles - 1))) break;
      tc::fence_after();
      const bool whole = s.tiles == s.all;
      const uint64_t slot = 2ull * blockIdx.x + (s.tile0 == 0 ? 1 : 0);  // as k_kv_tree_join reads them
      const uint64_t prow = slot * (MT * kTcTile) + m * kTcTile + r;
      const uint64_t orow = (static_cast<uint64_t>(s.b) * a.T + tok) * a.kv_heads * a.group + s.h * a.group + head;
      const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
      const bool odd = *reinterpret_cast<volatile uint32_t*>(&sh.odd[segs & 1u]) == segs + 1;
#pragma unroll
      for (uint32_t c = 0; c < DP / 32; ++c) {
        float o[32];
        tc::ld32(o, o_col + 32 * c);
        tc::ld_wait32(o);
        if (odd && live) {
          // infinities and NaN of the drafted tokens of this segment that the row sees
          for (int32_t p = max(s.ctx, static_cast<int32_t>(s.tile0 * kTcTile));
               p < min(s.len, static_cast<int32_t>((s.tile0 + s.tiles) * kTcTile)); ++p) {
            if (p < 0 || !(seen_bits(a, s, words, tok, p) & 1u)) continue;
            const uint32_t nth = static_cast<uint32_t>(p) / a.page_tokens;
            const uint32_t pg = static_cast<uint32_t>(a.table[static_cast<uint64_t>(s.b) * a.max_pages + nth]);
            if (pg >= a.n_pages) continue;
            if constexpr (FOUR) {
              const Kv4View& v4 = t.four[1];
              const int64_t slot4 = p - static_cast<int64_t>(nth) * a.page_tokens;
              if (32 * c >= a.dim) continue;
              const uint32_t* codes = reinterpret_cast<const uint32_t*>(v4.codes + static_cast<int64_t>(pg) * v4.page_stride +
                                                                        static_cast<int64_t>(s.h) * v4.head_stride + slot4 * v4.token_stride) + 4 * c;
              const uint32_t sc = quad::scale_bits<F16>(*reinterpret_cast<const uint16_t*>(
                  v4.scales + static_cast<int64_t>(pg) * v4.s_page + static_cast<int64_t>(s.h) * v4.s_head + slot4 * v4.s_token + 2 * c));
              if (!quad::odd<F16>(sc)) continue;
#pragma unroll
              for (uint32_t i = 0; i < 32; ++i) {
                const float x = quad::value<F16>(codes[i / 8], quad_element(i & 7u), sc);
                if (!(fabsf(x) < INFINITY)) o[i] += x;
              }
              continue;
            }
            const uint16_t* v = reinterpret_cast<const uint16_t*>(
                a.v.data + static_cast<int64_t>(pg) * a.v.page_stride + static_cast<int64_t>(s.h) * a.v.head_stride +
                static_cast<int64_t>(p - nth * a.page_tokens) * a.v.token_stride);
            const uint32_t ex = F16 ? 0x7C00u : 0x7F80u;
#pragma unroll
            for (uint32_t i = 0; i < 32; ++i)
              if (32 * c + i < a.dim && (v[32 * c + i] & ex) == ex)
                o[i] += F16 ? __half2float(__ushort_as_half(v[32 * c + i])) : __uint_as_float(static_cast<uint32_t>(v[32 * c + i]) << 16);
          }
        }
        if (!live)
#pragma unroll
          for (uint32_t i = 0; i < 32; ++i) o[i] = 0.f;
        if (whole) {
          if (exists)
#pragma unroll
            for (uint32_t i = 0; i < 32; i += 8)
              if (32 * c + i < a.dim) {
                uint32_t w[4];
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e)
                  w[e] = FOUR ? tc::pack2<F16>(o[i + quad_place(2 * e)] * inv, o[i + quad_place(2 * e + 1)] * inv)
                              : tc::pack2<F16>(o[i + 2 * e] * inv, o[i + 2 * e + 1] * inv);
                uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<char*>(a.out) + (orow * a.dim + 32 * c + i) * 2);
                if ((reinterpret_cast<uintptr_t>(a.out) & 15u) == 0)
                  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                else
                  dst[0] = w[0], dst[1] = w[1], dst[2] = w[2], dst[3] = w[3];
              }
        } else {
#pragma unroll
          for (uint32_t i = 0; i < 32; i += 4) {
            const uint32_t i8 = i & ~7u, e = i & 7u;
            *reinterpret_cast<float4*>(t.o_part + prow * DP + 32 * c + i) =
                FOUR ? make_float4(o[i8 + quad_place(e)], o[i8 + quad_place(e + 1)], o[i8 + quad_place(e + 2)], o[i8 + quad_place(e + 3)])
                     : make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
      }
      if (!live) top = -INFINITY, sum = 0.f;
      if (whole) {
        if (exists && a.lse) a.lse[orow] = row_lse<F16>(top, sum);
      } else {
        t.ml_part[prow] = make_float2(top, sum);
      }
      g += s.tiles;
      ++segs;
      // O is read: the next segment's first product may overwrite it
      tc::fence_before();
      if (MT == 2 && again) load_q(following, segs);
      s = following;
      more = again;
    }
  }
  __syncthreads();
  if (tid == 0 && *stop) kv_status(a.status, IBP_ETIMEOUT);
  if (warp == S::kMmaWarp) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

constexpr int kJoinThreads = 256;
constexpr uint32_t kJoinRows = kJoinThreads / 32;  // rows of a CTA, a warp each

// CTA (j, rows): joins the item that crosses the start of range j, if j is the
// first range boundary inside it.  The range before holds its first part (slot
// 1), the ranges from j on the others (slot 0), added in that order.
template <uint32_t DP, uint32_t ROWS, bool F16, uint32_t TILE = kTcTile>
__global__ void __launch_bounds__(kJoinThreads) k_kv_tree_join(const __grid_constant__ TcArgs t) {
  pdl_begin();
  const AttendArgs& a = t.a;
  const uint32_t j = blockIdx.x + 1, lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const int4 f = t.first[j], sh = t.first[t.n_ctas];
  const uint64_t share = static_cast<uint32_t>(sh.x) | (static_cast<uint64_t>(static_cast<uint32_t>(sh.y)) << 32);
  const uint64_t before = static_cast<uint32_t>(f.w);
  if (f.x < 0 || before == 0 || before > share) return;
  const uint32_t b = f.x, h = f.y;
  const uint64_t start = j * share - before, end = start + tiles_of<TILE>(a, b);
  const uint32_t last = static_cast<uint32_t>((end - 1) / share);
  constexpr uint32_t kRows = ROWS;
  const uint32_t r = blockIdx.y * kJoinRows + warp, gr = f.z * kRows + r;
  const uint32_t tok = gr / a.group, head = gr - tok * a.group;
  if (r >= kRows || tok >= a.T) return;
  auto row_of = [&](uint32_t c) { return (2ull * c + (c < j ? 1 : 0)) * kRows + r; };
  // Weights of up to 32 parts at a time, a part a lane; their rows follow with
  // four loads in flight.  The running maximum makes room for any number.  A part of
  // weight 0 is added like the others: what is not finite in it the row has seen, and
  // the result must not depend on where the ranges of the CTAs end.
  float top = -INFINITY, sum = 0.f;
  float2 acc[DP / 64];
#pragma unroll
  for (uint32_t e = 0; e < DP / 64; ++e) acc[e] = make_float2(0.f, 0.f);
  for (uint32_t c0 = j - 1; c0 <= last; c0 += 32) {
    const uint32_t n = last - c0 + 1 < 32 ? last - c0 + 1 : 32;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < n) ml = t.ml_part[row_of(c0 + lane)];
    float m = ml.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    m = fmaxf(m, top);
    const float was = top == -INFINITY ? (sum == 0.f ? 0.f : 1.f) : tc::ex2(top - m);
    top = m;
    const float w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : tc::ex2(ml.x - top);
    float s = w * ml.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    sum = was * sum + s;
#pragma unroll
    for (uint32_t e = 0; e < DP / 64; ++e) acc[e].x *= was, acc[e].y *= was;
    for (uint32_t c = 0; c < n; c += 4) {
      float2 o[4][DP / 64];
#pragma unroll
      for (uint32_t u = 0; u < 4; ++u)
#pragma unroll
        for (uint32_t e = 0; e < DP / 64; ++e)
          o[u][e] = c + u < n ? *reinterpret_cast<const float2*>(t.o_part + row_of(c0 + c + u) * DP + e * 64 + lane * 2)
                              : make_float2(0.f, 0.f);
#pragma unroll
      for (uint32_t u = 0; u < 4; ++u) {
        const float wc = __shfl_sync(0xFFFFFFFFu, w, c + u);
#pragma unroll
        for (uint32_t e = 0; e < DP / 64; ++e)
          acc[e].x += wc * o[u][e].x, acc[e].y += wc * o[u][e].y;
      }
    }
  }
  const uint64_t orow = (static_cast<uint64_t>(b) * a.T + tok) * a.kv_heads * a.group + h * a.group + head;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (uint32_t e = 0; e < DP / 64; ++e) {
    const uint32_t d = e * 64 + lane * 2;
    if (d < a.dim)
      *reinterpret_cast<uint32_t*>(static_cast<char*>(a.out) + (orow * a.dim + d) * 2) =
          tc::pack2<F16>(acc[e].x * inv, acc[e].y * inv);
  }
  if (lane == 0 && a.lse) a.lse[orow] = row_lse<F16>(top, sum);
}

}  // namespace ibp

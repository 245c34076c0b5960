// ibp_kv_weigh_tc.cu - the attention weight of cached tokens on the tensor cores
// (tcgen05), for calls of many rows (prompts, large drafts).
//
// A cluster of CTAs takes 256 tokens of a sequence and shares out the kv heads, and
// the row blocks where there are fewer heads than CTAs.  In a CTA
//   four loader warps   write two tiles of 128 keys (once a head) and blocks of 128 queries
//                       with the rows' logarithms of sums into shared memory;
//   one MMA warp        S^T = K Q^T, 128 tokens by 128 rows, two tiles and two slots
//                       each in TMEM (all 512 columns);
//   eight warps         a thread per token: exp2(S scale - lse) summed along its row of
//                       S^T in a register.
// With tokens as TMEM lanes no sum crosses threads until the cluster's CTAs are added up
// at the end, in a fixed order.  A token's key reaches its own sum alone, so what is not
// finite in it needs no care.  128 rows by 256 tokens are 32768 exponentials and 4.2 million
// multiply-adds, of 1024 cycles each on their pipes.
//
// 256 tokens a CTA share a block of queries, which is what moves most; a cluster
// shares the heads, so that the sum over heads needs no scratch and no atomics.
//
// Measured on one GB300: 511 queries a sequence, 32 heads on 8 kv heads of 128, two caches of
// up to 8192 tokens in 16 bits: 130 us with cold caches, 0.40 PFLOP/s of products; the few-row
// kernel takes 960 us.  128 rows of a CTA take 3300 to 4000 cycles, what a CTA begins and ends
// with 13 us.  Two things bound it.  In a CTA the roles wait for one another: exponentials and
// products each keep their pipe 33 % busy, issue slots are 38 % used.  And CTAs of fixed size do not
// fill the SMs evenly: 204 of them here, one a SM, so two rounds, and the SMs work for 54 % of
// the time.
//
// Every wait has a limit, as in ibp_kv_tree.cuh.
#include "ibp_kv_serve.cuh"
#include "ibp_kv_tree.cuh"

namespace ibp {

constexpr uint32_t kWtTokens = 256;   // of a CTA
constexpr uint32_t kWtStages = 4;     // blocks of queries in flight
constexpr uint32_t kWtThreads = 256 + 32 + 128;

struct WtArgs {
  WeighArgs x;
  uint32_t cluster;        // CTAs
  uint32_t heads_at_once;  // CTAs of a cluster on different heads; the others share out row blocks
  long long limit;
};

template <uint32_t DP>
struct WtShape {
  static constexpr uint32_t kHalves = DP / 64;
  static constexpr uint32_t kPanel = 128 * 128;
  static constexpr uint32_t kTile = kHalves * kPanel;  // 128 keys or queries
  static constexpr uint32_t kBytes = (2 + kWtStages) * kTile;
  static constexpr uint32_t kSmem = kBytes + 1024 + 20480;
};

struct WtShared {
  uint64_t k_full, k_empty, q_full[kWtStages], q_empty[kWtStages], s_full[2][2], s_empty[2][2], done;
  alignas(16) float back[kWtStages][128];  // -lse log2 e of a block's rows; -infinity: nothing to add
  uint32_t plain[kWtStages][4]; // every one of 32 rows has something to add
  alignas(16) uint32_t seen[kWtStages][2][4][128];  // where some row may not see a tile: bits of 32 tokens, by row
  float sums[kWtTokens];
  uint32_t tmem, stop;
};

constexpr int64_t kWtNone = INT64_MIN;

// 32 rows of a warp, lane i's at base + off, on their way into rows first_row on of a
// swizzled tile: half a warp copies a row of 128 dimensions at once.
template <uint32_t DP>
__device__ __forceinline__ void wt_rows(uint32_t tile, uint32_t first_row, const char* base, int64_t off, uint32_t dim, bool vec) {
  constexpr uint32_t kChunks = DP / 8, kPer = 32 / kChunks;
  const uint32_t lane = threadIdx.x & 31u, c = lane % kChunks;
  const uint32_t dst = tile + (c / 8) * 128 * 128;
  if (vec) {
#pragma unroll
    for (uint32_t j = 0; j < kChunks; ++j) {
      const int64_t o = __shfl_sync(0xFFFFFFFFu, off, j * kPer + lane / kChunks);
      const uint32_t r = first_row + j * kPer + lane / kChunks;
      const bool on = o != kWtNone && c * 8 < dim;
      cp16(dst + r * 128 + (((c & 7u) ^ (r & 7u)) << 4), on ? base + o + c * 16 : base, on);
    }
  } else {
#pragma unroll 1
    for (uint32_t j = 0; j < kChunks; ++j) {
      const int64_t o = __shfl_sync(0xFFFFFFFFu, off, j * kPer + lane / kChunks);
      const uint32_t r = first_row + j * kPer + lane / kChunks;
      const bool on = o != kWtNone && c * 8 < dim;
      const char* p = on ? base + o + c * 16 : base;
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + r * 128 + (((c & 7u) ^ (r & 7u)) << 4) + 4 * e), "l"(p + 4 * e), "r"(on ? 4u : 0u)
                     : "memory");
    }
  }
}

// The same with every row and dimension there, lane i's row at `row`: next to nothing to
// compute, since four warps have a block of 128 rows to keep up with.
template <uint32_t DP>
__device__ __forceinline__ void wt_sure_rows(uint32_t tile, uint32_t first_row, const char* row) {
  constexpr uint32_t kChunks = DP / 8, kPer = 32 / kChunks, kTurns = 8 / kPer;  // instructions after which the order repeats
  const uint32_t lane = threadIdx.x & 31u, c = lane % kChunks, r0 = lane / kChunks;
  uint32_t dst[kTurns];
#pragma unroll
  for (uint32_t i = 0; i < kTurns; ++i)
    dst[i] = tile + (c / 8) * 128 * 128 + (first_row + r0 + i * kPer) * 128 + (((c & 7u) ^ ((r0 + i * kPer) & 7u)) << 4);
  const uint64_t mine = reinterpret_cast<uint64_t>(row);
#pragma unroll
  for (uint32_t j = 0; j < kChunks; ++j) {
    const char* p = reinterpret_cast<const char*>(__shfl_sync(0xFFFFFFFFu, mine, j * kPer + r0)) + c * 16;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst[j % kTurns] + j / kTurns * 8 * 128), "l"(p) : "memory");
  }
}

template <uint32_t DP, bool FOUR, bool F16>
__global__ void __launch_bounds__(kWtThreads, 1) k_kv_weigh_tc(const __grid_constant__ WtArgs w) {
  using S = WtShape<DP>;
  const WeighArgs& x = w.x;
  const AttendArgs& a = x.a;
  extern __shared__ unsigned char raw_sm[];
  unsigned char* sm = raw_sm + ((1024 - (tc::s32(raw_sm) & 1023u)) & 1023u);
  const uint32_t base = tc::s32(sm);
  WtShared& sh = *reinterpret_cast<WtShared*>(sm + S::kBytes);
  static_assert(sizeof(WtShared) <= 20480, "shared");
  const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
  const uint32_t rank = blockIdx.x % w.cluster, first = blockIdx.x / w.cluster * kWtTokens, b = blockIdx.y;
  const uint32_t share = kWtTokens / w.cluster;  // tokens that a CTA adds up at the end
  pdl_begin();
  const int32_t raw = a.lens[b], all = clamp_len(raw, a.page_tokens, a.max_pages);
  const int32_t len = all < static_cast<int32_t>(x.width) ? all : static_cast<int32_t>(x.width);  // weighed positions
  const int32_t live = a.n_live ? a.n_live[b] : static_cast<int32_t>(a.T);
  const int32_t n_live = live < 0 ? 0 : (live > static_cast<int32_t>(a.T) ? static_cast<int32_t>(a.T) : live);
  if (blockIdx.x == 0 && tid == 0 && (raw != len || live != n_live || n_live > all)) kv_status(a.status, IBP_ERANGE);
  const int32_t ctx = all - n_live;
  const uint32_t rows = static_cast<uint32_t>(n_live) * a.group;
  const float* was = x.w + static_cast<uint64_t>(b) * x.width;
  float* out = x.w_out + static_cast<uint64_t>(b) * x.width;
  if (static_cast<int32_t>(first) >= len) {  // the same for the whole cluster
    const uint32_t i = first + rank * share + tid;
    if (tid < share && i < x.width) out[i] = was[i];
    return;
  }
  if (tid == 0) {
    tc::bar_init(tc::s32(&sh.k_full), 128);
    tc::bar_init(tc::s32(&sh.k_empty), 1);
    for (uint32_t i = 0; i < kWtStages; ++i) {
      tc::bar_init(tc::s32(&sh.q_full[i]), 128);
      tc::bar_init(tc::s32(&sh.q_empty[i]), 1 + 8);
    }
    for (uint32_t i = 0; i < 4; ++i) {
      tc::bar_init(tc::s32(&sh.s_full[i >> 1][i & 1]), 1);
      tc::bar_init(tc::s32(&sh.s_empty[i >> 1][i & 1]), 128);
    }
    tc::bar_init(tc::s32(&sh.done), 1);
    sh.stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::s32(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sh.tmem;
  volatile uint32_t* stop = &sh.stop;
  const uint32_t head0 = rank % w.heads_at_once, part = rank / w.heads_at_once, parts = w.cluster / w.heads_at_once;
  const uint32_t blocks = (rows + 127) / 128, mine = blocks > part ? (blocks - part + parts - 1) / parts : 0;
  const uint32_t k_sm = base, q_sm = base + 2 * S::kTile;

  if (warp >= 9) {
    // ---- loaders: thread r has keys r and r + 128, and row r of a block of queries
    const uint32_t r = tid - 288;
    bool ok = true;
    uint32_t fill = 0, heads = 0;
    const quad::Magic<F16> magic;
    const bool partly = static_cast<int32_t>(first + kWtTokens) > ctx;
    TcSeg seg = {};
    seg.len = all, seg.ctx = ctx;
    for (uint32_t h = head0; ok && mine && h < a.kv_heads; h += w.heads_at_once, ++heads) {
      ok = tc::bar_wait(tc::s32(&sh.k_empty), (heads & 1u) ^ 1u, stop, w.limit);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
#pragma unroll 1
      for (uint32_t m = 0; m < 2; ++m) {
        const uint32_t pos = first + m * 128 + r;
        uint32_t page = 0, slot = 0;
        bool there = static_cast<int32_t>(pos) < len;
        if (there) {
          const uint32_t nth = pos / a.page_tokens;
          slot = pos - nth * a.page_tokens;
          page = static_cast<uint32_t>(__ldg(a.table + static_cast<uint64_t>(b) * a.max_pages + nth));
          if (page >= a.n_pages) {
            kv_status(a.status, IBP_ERANGE);
            there = false;
            page = slot = 0;
          }
        }
        if constexpr (FOUR) {
          unsigned char* dst = sm + m * S::kTile + r * 128;
          const char* c = x.k4.codes + static_cast<int64_t>(page) * x.k4.page_stride + static_cast<int64_t>(h) * x.k4.head_stride +
                          static_cast<int64_t>(slot) * x.k4.token_stride;
          const char* sc = x.k4.scales + static_cast<int64_t>(page) * x.k4.s_page + static_cast<int64_t>(h) * x.k4.s_head +
                           static_cast<int64_t>(slot) * x.k4.s_token;
          uint4 codes[DP / 32];
          uint32_t scale[DP / 32];
#pragma unroll
          for (uint32_t g = 0; g < DP / 32; ++g) {
            const bool in = there && g * 32 < a.dim;
            codes[g] = in ? __ldg(reinterpret_cast<const uint4*>(c + g * 16)) : make_uint4(0u, 0u, 0u, 0u);
            scale[g] = in ? static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(sc + g * 2))) : 0u;
          }
#pragma unroll
          for (uint32_t g = 0; g < DP / 32; ++g) {
            const quad::Pair<F16> p(scale[g] * 0x10001u);
            const uint32_t u[4] = {codes[g].x, codes[g].y, codes[g].z, codes[g].w};
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) {
              const uint32_t i = g * 4 + e;
              const uint32_t y0 = quad::decode<F16, 0>(u[e], p, magic), y1 = quad::decode<F16, 1>(u[e], p, magic);
              const uint32_t y2 = quad::decode<F16, 2>(u[e], p, magic), y3 = quad::decode<F16, 3>(u[e], p, magic);
              *reinterpret_cast<uint4*>(dst + (i / 8) * S::kPanel + (((i & 7u) ^ (r & 7u)) << 4)) =
                  make_uint4(__byte_perm(y0, y1, 0x5410), __byte_perm(y2, y3, 0x5410), __byte_perm(y0, y1, 0x7632), __byte_perm(y2, y3, 0x7632));
            }
          }
        } else {
          const int64_t off = there ? static_cast<int64_t>(page) * a.k.page_stride + static_cast<int64_t>(slot) * a.k.token_stride : kWtNone;
          wt_rows<DP>(k_sm + m * S::kTile, r & 96u, a.k.data + static_cast<int64_t>(h) * a.k.head_stride, off, a.dim, true);
        }
      }
      cp_commit();
      cp_wait<0>();
      tc::fence_async();
      tc::bar_arrive(tc::s32(&sh.k_full));
      // Blocks of queries, up to kFly on their way; one is handed on when it has landed.
      constexpr uint32_t kFly = kWtStages - 1;
      auto hand_on = [&](uint32_t nth) {
        tc::fence_async();
        tc::bar_arrive(tc::s32(&sh.q_full[nth % kWtStages]));
      };
      auto lse_of = [&](uint32_t j, uint32_t* t, uint32_t* head, bool* on) {
        const uint32_t row = (part + j * parts) * 128 + r;
        *on = j < mine && row < rows;
        *t = *on ? row / a.group : 0, *head = *on ? h * a.group + row - *t * a.group : 0;
        return *on ? __ldg(x.lse + (static_cast<uint64_t>(b) * a.T + *t) * a.kv_heads * a.group + *head) : -INFINITY;
      };
      uint32_t t, head;
      bool on;
      float lse = lse_of(0, &t, &head, &on);
#pragma unroll 1
      for (uint32_t j = 0; j < mine; ++j, ++fill) {
        const uint32_t st = fill % kWtStages;
        ok = tc::bar_wait(tc::s32(&sh.q_empty[st]), (fill / kWtStages & 1u) ^ 1u, stop, w.limit);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        const char* q = a.q + static_cast<int64_t>(b) * a.q_seq;
        const int64_t off = static_cast<int64_t>(t) * a.q_token + static_cast<int64_t>(head) * a.q_head;
        if (x.q16 && a.dim == DP)
          wt_sure_rows<DP>(q_sm + st * S::kTile, r & 96u, q + off);  // rows past the end: the first one, which adds nothing
        else
          wt_rows<DP>(q_sm + st * S::kTile, r & 96u, q, on ? off : kWtNone, a.dim, x.q16);
        cp_commit();
        const float back = lse == -INFINITY ? -INFINITY : -lse * 1.4426950408889634f;
        sh.back[st][r] = back;
        const bool plain = __all_sync(0xFFFFFFFFu, back != -INFINITY);
        if (lane == 0) sh.plain[st][r / 32] = plain;
        if (partly) {
          const uint32_t* words = a.mask ? a.mask + (static_cast<uint64_t>(b) * a.T + t) * a.mask_words : nullptr;
#pragma unroll 1
          for (uint32_t e = 0; e < 8; ++e)
            sh.seen[st][e >> 2][e & 3u][r] = on && back != -INFINITY ? seen_bits(a, seg, words, t, static_cast<int32_t>(first + 32 * e)) : 0u;
        }
        lse = lse_of(j + 1, &t, &head, &on);
        if (j >= kFly - 1) {
          cp_wait<kFly - 1>();
          hand_on(fill - (kFly - 1));
        }
      }
      // the last ones (all of them have been asked for unless a wait gave up)
      cp_wait<0>();
      if (ok)
        for (uint32_t n = mine < kFly ? mine : kFly - 1; n > 0; --n) hand_on(fill - n);
    }
  } else if (warp == 8) {
    // ---- MMA
    const uint32_t fmt = F16 ? 0u : 1u;
    const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
    const uint64_t kd = tc::operand(k_sm, 16), qd = tc::operand(q_sm, 16);
    constexpr uint32_t kStep = S::kTile >> 4;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool r = tc::bar_wait(tc::s32(bar), parity, stop, w.limit);
      return __all_sync(0xFFFFFFFFu, r) != 0;
    };
    auto commit = [&](uint64_t* bar) {
      if (tc::elect()) tc::commit(tc::s32(bar));
      __syncwarp();
    };
    bool ok = true;
    uint32_t fill = 0, heads = 0;
    for (uint32_t h = head0; ok && mine && h < a.kv_heads; h += w.heads_at_once, ++heads) {
      if (!(ok = wait(&sh.k_full, heads & 1u))) break;
      for (uint32_t j = 0; j < mine; ++j, ++fill) {
        const uint32_t st = fill % kWtStages, slot = fill & 1u;
        if (!(ok = wait(&sh.q_full[st], fill / kWtStages & 1u))) break;
        for (uint32_t m = 0; m < 2; ++m) {
          if (!(ok = wait(&sh.s_empty[m][slot], (fill >> 1 & 1u) ^ 1u))) break;
          tc::fence_after();
          if (tc::elect()) {
            const uint64_t ka = kd + m * kStep, qa = qd + st * kStep;
            const uint32_t d = tmem + (slot * 2 + m) * 128;
#pragma unroll
            for (uint32_t kk = 0; kk < DP / 16; ++kk) {
              const uint32_t off = ((kk / 4) * S::kPanel + (kk % 4) * 32) >> 4;
              tc::mma_ss(d, ka + off, qa + off, idesc, kk > 0);
            }
            tc::commit(tc::s32(&sh.s_full[m][slot]));
          }
          __syncwarp();
        }
        if (!ok) break;
        commit(&sh.q_empty[st]);
      }
      commit(&sh.k_empty);
    }
    // the last products and the arrivals they cause end before the CTA leaves
    commit(&sh.done);
    tc::bar_drain(tc::s32(&sh.done), 0);
    __syncwarp();
  } else {
    // ---- sums: thread of tile m, token r of it
    const uint32_t m = warp / 4, r = tid & 127u;
    const uint32_t lanes = (warp & 3u) << 21;
    const bool open = static_cast<int32_t>(first + m * 128 + 128) <= ctx;  // every row sees the whole tile
    const float scale = a.scale_log2;
    float total = 0.f;
    bool ok = true;
    uint32_t fill = 0;
    for (uint32_t h = head0; ok && mine && h < a.kv_heads; h += w.heads_at_once) {
      for (uint32_t j = 0; j < mine; ++j, ++fill) {
        const uint32_t st = fill % kWtStages, slot = fill & 1u;
        ok = tc::bar_wait(tc::s32(&sh.s_full[m][slot]), fill >> 1 & 1u, stop, w.limit) &&
             tc::bar_wait(tc::s32(&sh.q_full[st]), fill / kWtStages & 1u, stop, w.limit);  // has passed: for what the loaders wrote
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc::fence_after();
        const uint32_t col = tmem + lanes + (slot * 2 + m) * 128;
        float y[2][32];
        tc::ld32(y[0], col);
        uint64_t block[2] = {0, 0};  // two sums of two lanes
        const uint64_t scale2 = tc::two(scale, scale);
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
          float(&v)[32] = y[c & 1u];
          tc::ld_wait32(v);
          if (c < 3) {
            tc::ld32(y[(c + 1) & 1u], col + 32 * (c + 1));
          } else {
            tc::fence_before();
            tc::bar_arrive(tc::s32(&sh.s_empty[m][slot]));
          }
          // two rows' exponentials; those that are not wanted are dropped, not multiplied away
          auto pair = [&](uint32_t i, uint64_t back, bool on0, bool on1) {
            float p, q;
            tc::split(tc::fma2(tc::two(v[i], v[i + 1]), scale2, back), p, q);
            p = tc::ex2(p), q = tc::ex2(q);
            block[i / 2 & 1u] = tc::add2(block[i / 2 & 1u], tc::two(on0 ? p : 0.f, on1 ? q : 0.f));
          };
          const ulonglong2* bk = reinterpret_cast<const ulonglong2*>(&sh.back[st][32 * c]);
          if (open && sh.plain[st][c]) {
#pragma unroll
            for (uint32_t i = 0; i < 32; i += 4) {
              const ulonglong2 x4 = bk[i / 4];
              pair(i, x4.x, true, true);
              pair(i + 2, x4.y, true, true);
            }
          } else if (open) {
#pragma unroll
            for (uint32_t i = 0; i < 32; i += 4) {
              const ulonglong2 x4 = bk[i / 4];
              const float* f = &sh.back[st][32 * c + i];
              pair(i, x4.x, f[0] != -INFINITY, f[1] != -INFINITY);
              pair(i + 2, x4.y, f[2] != -INFINITY, f[3] != -INFINITY);
            }
          } else {
#pragma unroll
            for (uint32_t i = 0; i < 32; i += 4) {
              const ulonglong2 x4 = bk[i / 4];
              const uint4 seen = *reinterpret_cast<const uint4*>(&sh.seen[st][m][warp & 3u][32 * c + i]);
              pair(i, x4.x, seen.x >> lane & 1u, seen.y >> lane & 1u);
              pair(i + 2, x4.y, seen.z >> lane & 1u, seen.w >> lane & 1u);
            }
          }
        }
        float s0, s1;
        tc::split(tc::add2(block[0], block[1]), s0, s1);
        total += s0 + s1;
        __syncwarp();
        if (lane == 0) tc::bar_arrive(tc::s32(&sh.q_empty[st]));
      }
    }
    sh.sums[m * 128 + r] = total;
  }
  __syncthreads();
  if (tid == 0 && *stop) kv_status(a.status, IBP_ETIMEOUT);
  if (warp == 8) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
  // The cluster's CTAs each add up their share of the tokens, in the CTAs' order.
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (tid < share) {
    const uint32_t i = rank * share + tid;
    float s = 0.f;
    for (uint32_t c = 0; c < w.cluster; ++c) {
      uint32_t addr = tc::s32(&sh.sums[i]);
      float v;
      asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(addr) : "r"(c));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
      s += v;
    }
    const int32_t p = static_cast<int32_t>(first + i);
    if (static_cast<uint32_t>(p) < x.width) out[p] = p >= len ? was[p] : (p < ctx ? fmaf(x.decay, was[p], s) : s);
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <uint32_t DP, bool FOUR, bool F16>
static int launch(const WtArgs& w, int device, cudaStream_t stream) {
  using S = WtShape<DP>;
  auto kern = k_kv_weigh_tc<DP, FOUR, F16>;
  static std::atomic<int> ready[64];
  if (device < 0 || device >= 64 || !ready[device].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) {
      set_cuda_error(e, "set-up of k_kv_weigh_tc");
      cudaGetLastError();
      return IBP_ECUDA;
    }
    if (device >= 0 && device < 64) ready[device].store(1, std::memory_order_release);
  }
  const uint32_t tiles = (w.x.width + kWtTokens - 1) / kWtTokens;
  return kv_launch("k_kv_weigh_tc", kern, dim3(tiles * w.cluster, w.x.a.n_seqs), kWtThreads, S::kSmem, w.cluster, stream, w);
}

int launch_kv_weigh_tc(const WeighArgs& x, int device, cudaStream_t stream) {
  WtArgs w;
  w.x = x;
  // Eight CTAs where all clusters of eight run at once (15 fit), else four, which leave fewer
  // SMs idle and begin fewer times; two for a single block of rows, where beginning counts most.
  // Measured (us with 2 / 4 / 8), 511 queries of 4 heads on 8 kv heads: one cache of 1024 tokens
  // 153 / 83 / 48, one of 8192 153 / 83 / 99, two 155 / 132 / 126, eight 337 / 323 / 370, three of
  // 16384 335 / 276 / 306; 16 queries: two of 8192 30 / 36 / 44, sixteen 114 / 149 / 230.
  const uint64_t rows = static_cast<uint64_t>(x.a.T) * x.a.group, clusters = (x.width + kWtTokens - 1ull) / kWtTokens * x.a.n_seqs;
  w.cluster = clusters * 10 <= static_cast<uint64_t>(sm_count(device)) ? 8 : (rows <= 128 ? 2 : 4);
  w.heads_at_once = 1;
  while (w.heads_at_once < w.cluster && 2 * w.heads_at_once <= x.a.kv_heads) w.heads_at_once *= 2;
  w.limit = kv_tree_limit();
  const bool four = x.k4.codes != nullptr, f16 = x.a.f16;
  if (x.a.dim <= 64) {
    if (four) return f16 ? launch<64, true, true>(w, device, stream) : launch<64, true, false>(w, device, stream);
    return f16 ? launch<64, false, true>(w, device, stream) : launch<64, false, false>(w, device, stream);
  }
  if (four) return f16 ? launch<128, true, true>(w, device, stream) : launch<128, true, false>(w, device, stream);
  return f16 ? launch<128, false, true>(w, device, stream) : launch<128, false, false>(w, device, stream);
}

}  // namespace ibp

// ibp_kv_weigh.cu - the attention weight that each cached token receives.
//
// The weight of a row (query and head) for a token is exp(s - lse) with the row's
// known logarithm of the sum, so a token's total needs its key once and no value.  A
// CTA takes a run of tokens; its warps share out the kv heads (and runs of 16 MT
// tokens, where there are fewer heads than warps) and add up their rows in registers;
// the warps' sums are added in a fixed order, so results do not depend on how threads
// run.  S^T = K Q^T as in the attention kernels: a lane holds neighbouring dimensions
// of a token's key, and queries are laid out to match.
//
// Measured on one GB300: 32 ragged caches of up to 16384 tokens in 4 bits, 8 kv heads of 4
// query heads of 128, one token each (202 MB): 91 us with cold caches, 2.2 TB/s.  16
// tokens of a head cost about 270 warp instructions, of which 96 decode.  Issue slots are 56 %
// used, DRAM 31 %: with 3.7 warps a scheduler, loads and the chain of products into one
// accumulator are waited for.  The same caches in 16 bits (712 MB) 183 us, 3.9 TB/s, issue slots
// 27 % used: two warps a scheduler wait for their loads.  Loads straight into registers, without the
// ring, took 325 us (4 bits).
//
// Heads of 136 to 256 come here with any number of rows, eight at a time, for each of which the
// keys are read from shared memory anew: 8 caches of up to 8192 tokens in 4 bits, 8 kv heads of
// 256, 64 rows 289 us, 256 rows 1127 us, 1024 rows 4353 us (16 bits: 332, 1237, 4711), where
// heads of 128 take 142, 105 and 201 us.
#include <type_traits>

#include "ibp_kv_serve.cuh"

namespace ibp {

constexpr uint32_t kWgWarps = 4;
constexpr uint32_t kWgTiles = 2;  // of a CTA's warps: 93 us for the batch above with 1, 91 with 2, 95 with 4
// Rows a kv head from which the tensor cores take over (ibp_kv_weigh_tc.cu).  Measured (us, few
// rows / tensor cores): two caches of up to 8192 tokens in 16 bits, 8 kv heads: 52 rows 44 / 46,
// 64 rows 48 / 44, 96 rows 65 / 42; eight of up to 16384 in 4 bits, which the few-row kernel
// reads faster: 52 rows 185 / 259, 64 rows 210 / 251, 96 rows 302 / 235.
constexpr uint64_t kWgMany = 64, kWgMany4 = 80;

// A warp's stage: the keys of 16 MT tokens of a head as the cache has them, the scales
// of codes, and which of the tokens there are.
template <uint32_t DP, uint32_t MT, bool FOUR>
struct WeighStage {
  static constexpr uint32_t kTokens = 16 * MT;
  static constexpr uint32_t kRow = FOUR ? DP / 2 : DP * 2;       // bytes of a key
  static constexpr uint32_t kScale = FOUR ? DP / 16 : 0;         // and of its scales
  static constexpr uint32_t kKeys = kTokens * kRow;
  static constexpr uint32_t kBytes = kKeys + kTokens * kScale + 16;
  static constexpr uint32_t kStages = DP == 256 && !FOUR ? 3 : 4;

  // Place of 16 bytes of a token's key, so that eight lanes on two rows meet in no bank.
  static __device__ __forceinline__ uint32_t at(uint32_t tok, uint32_t c) {
    if (FOUR) {
      const uint32_t piece = tok * (DP / 32) + c, line = piece >> 3;
      return (piece ^ (DP == 256 ? line & 7u : 0u)) * 16;
    }
    const uint32_t turn = DP == 64 ? tok & 1u : (c >> 3) ^ (tok & 1u) << (DP == 128 ? 1 : 2);
    return tok * kRow + ((c ^ (turn & 7u)) * 16);
  }
};

// Operands A of two steps (16 dimensions each) from a lane's eight of tokens g and g + 8.
template <bool FOUR, bool F16>
__device__ __forceinline__ void weigh_operands(const uint4& x, const uint4& y, uint32_t j, const quad::Pair<F16>& p0, const quad::Pair<F16>& p1,
                                               const quad::Magic<F16>& m, uint32_t (&lo)[4], uint32_t (&hi)[4]) {
  if constexpr (FOUR) {  // word j of 32 codes
    const uint32_t u = j == 0 ? x.x : (j == 1 ? x.y : (j == 2 ? x.z : x.w)), v = j == 0 ? y.x : (j == 1 ? y.y : (j == 2 ? y.z : y.w));
    lo[0] = quad::decode<F16, 0>(u, p0, m), lo[1] = quad::decode<F16, 0>(v, p1, m);
    lo[2] = quad::decode<F16, 1>(u, p0, m), lo[3] = quad::decode<F16, 1>(v, p1, m);
    hi[0] = quad::decode<F16, 2>(u, p0, m), hi[1] = quad::decode<F16, 2>(v, p1, m);
    hi[2] = quad::decode<F16, 3>(u, p0, m), hi[3] = quad::decode<F16, 3>(v, p1, m);
  } else {  // eight values
    lo[0] = x.x, lo[1] = y.x, lo[2] = x.y, lo[3] = y.y;
    hi[0] = x.z, hi[1] = y.z, hi[2] = x.w, hi[3] = y.w;
  }
}

// Eight rows of queries of a head and their logarithms of sums.
template <uint32_t DP>
struct WeighRows {
  uint32_t q[DP / 32][4];
  float lse[2];  // of rows 2t and 2t + 1; -infinity where there is none
};

// Where a lane's part of a block's queries and its rows' logarithms are in a head.
struct WeighAt {
  const char* q;
  const float* lse[2];  // nullptr: no such row
};

__device__ __forceinline__ WeighAt weigh_at(const WeighArgs& x, uint32_t b, uint32_t h, uint32_t r0, uint32_t rows, uint32_t d) {
  const AttendArgs& a = x.a;
  const uint32_t lane = threadIdx.x & 31u, g = lane >> 2, t = lane & 3u;
  const uint32_t rq = r0 + g < rows ? r0 + g : rows - 1, tq = rq / a.group;  // a row past the end is not counted
  WeighAt at;
  at.q = a.q + static_cast<int64_t>(b) * a.q_seq + static_cast<int64_t>(tq) * a.q_token +
         static_cast<int64_t>(h * a.group + rq - tq * a.group) * a.q_head + d * 2;
#pragma unroll
  for (uint32_t e = 0; e < 2; ++e) {
    const uint32_t r = r0 + 2 * t + e, tr = r / a.group;
    at.lse[e] = r < rows ? x.lse + (static_cast<uint64_t>(b) * a.T + tr) * a.kv_heads * a.group + h * a.group + r - tr * a.group : nullptr;
  }
  return at;
}

template <uint32_t DP>
__device__ __forceinline__ void weigh_rows(const WeighArgs& x, const WeighAt& at, uint32_t d, WeighRows<DP>& o) {
  const AttendArgs& a = x.a;
  if (x.q16) {
#pragma unroll
    for (uint32_t j = 0; j < DP / 32; ++j) {
      const uint4 u = d + 8 * j < a.dim ? __ldg(reinterpret_cast<const uint4*>(at.q + 16 * j)) : make_uint4(0u, 0u, 0u, 0u);
      o.q[j][0] = u.x, o.q[j][1] = u.y, o.q[j][2] = u.z, o.q[j][3] = u.w;
    }
  } else {
#pragma unroll
    for (uint32_t j = 0; j < DP / 32; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint16_t* v = reinterpret_cast<const uint16_t*>(at.q + 16 * j) + 2 * i;
        o.q[j][i] = d + 8 * j < a.dim ? __ldg(v) | static_cast<uint32_t>(__ldg(v + 1)) << 16 : 0u;
      }
  }
#pragma unroll
  for (uint32_t e = 0; e < 2; ++e) o.lse[e] = at.lse[e] ? __ldg(at.lse[e]) : -INFINITY;
}

// 16 MT tokens a warp.  head_warps of a CTA's warps share a run of tokens, each with its
// own heads; each warp has a ring of stages that asynchronous copies fill some heads
// ahead, over the ends of tiles.
// SHARED: at most 8 rows a head, whose queries the CTA lays out in shared memory as the
// products take them.
template <uint32_t DP, uint32_t MT, bool FOUR, bool F16, bool SHARED>
__global__ void __launch_bounds__(kWgWarps * 32, DP == 256 ? 3 : 4) k_kv_weigh(const __grid_constant__ WeighArgs x, uint32_t head_warps, int32_t shift, uint32_t even) {
  using S = WeighStage<DP, MT, FOUR>;
  __shared__ float sums[kWgWarps][16 * MT];
  extern __shared__ __align__(128) unsigned char dyn[];  // the rings, then (SHARED) queries and -lse log2 e
  pdl_begin();
  const AttendArgs& a = x.a;
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3u;
  const uint32_t b = blockIdx.y, runs = kWgWarps / head_warps, tokens = 16 * MT * runs;
  const int32_t raw = a.lens[b], all = clamp_len(raw, a.page_tokens, a.max_pages);
  const int32_t len = all < static_cast<int32_t>(x.width) ? all : static_cast<int32_t>(x.width);  // weighed positions
  const int32_t live = a.n_live ? a.n_live[b] : static_cast<int32_t>(a.T);
  const int32_t n_live = live < 0 ? 0 : (live > static_cast<int32_t>(a.T) ? static_cast<int32_t>(a.T) : live);
  if (blockIdx.x == 0 && threadIdx.x == 0 && (raw != len || live != n_live || n_live > all)) kv_status(a.status, IBP_ERANGE);
  const int32_t ctx = all - n_live;
  const uint32_t rows = static_cast<uint32_t>(n_live) * a.group;
  const float* was = x.w + static_cast<uint64_t>(b) * x.width;
  float* out = x.w_out + static_cast<uint64_t>(b) * x.width;
  const quad::Magic<F16> magic;
  const uint32_t tiles = len > 0 ? ceil_div(static_cast<uint32_t>(len), tokens) : 0;
  const uint32_t h0 = warp % head_warps, heads = rows && h0 < a.kv_heads ? ceil_div(a.kv_heads - h0, head_warps) : 0;  // this warp's
  uint4* sq = reinterpret_cast<uint4*>(dyn + kWgWarps * S::kStages * S::kBytes);  // [head][DP / 32][lane]
  float* sl = reinterpret_cast<float*>(sq + a.kv_heads * DP);                     // [head][8]
  if (SHARED && blockIdx.x < tiles && rows) {
#pragma unroll 4
    for (uint32_t i = threadIdx.x; i < a.kv_heads * DP; i += kWgWarps * 32) {
      const uint32_t h = i / DP, j = i / 32 % (DP / 32), l = i & 31u, r = l >> 2, d = (l & 3u) * (DP / 4) + 8 * j;
      const uint32_t tr = r / a.group;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows && d < a.dim) {
        const char* q = a.q + static_cast<int64_t>(b) * a.q_seq + static_cast<int64_t>(tr) * a.q_token +
                        static_cast<int64_t>(h * a.group + r - tr * a.group) * a.q_head + d * 2;
        if (x.q16) {
          w = __ldg(reinterpret_cast<const uint4*>(q));
        } else {
          const uint16_t* v = reinterpret_cast<const uint16_t*>(q);
          w = make_uint4(v[0] | static_cast<uint32_t>(v[1]) << 16, v[2] | static_cast<uint32_t>(v[3]) << 16, v[4] | static_cast<uint32_t>(v[5]) << 16,
                         v[6] | static_cast<uint32_t>(v[7]) << 16);
        }
      }
      if (FOUR)
        w = make_uint4(__byte_perm(w.x, w.z, 0x5410), __byte_perm(w.x, w.z, 0x7632), __byte_perm(w.y, w.w, 0x5410), __byte_perm(w.y, w.w, 0x7632));
      sq[i] = w;
    }
    for (uint32_t i = threadIdx.x; i < a.kv_heads * 8; i += kWgWarps * 32) {
      const uint32_t h = i / 8, r = i & 7u, tr = r / a.group;
      const float lse = r < rows ? __ldg(x.lse + (static_cast<uint64_t>(b) * a.T + tr) * a.kv_heads * a.group + h * a.group + r - tr * a.group) : -INFINITY;
      sl[i] = lse == -INFINITY ? -INFINITY : -lse * 1.4426950408889634f;
    }
    __syncthreads();
  }
  auto base_of = [&](uint32_t tile) { return tile * tokens + warp / head_warps * 16 * MT; };  // this warp's run
  // The page of this lane's token of a tile, on its way; none past the last.
  auto page_of = [&](uint32_t tile) -> uint32_t {
    const uint32_t pos = base_of(tile) + lane;
    if (!heads || tile >= tiles || lane >= S::kTokens || static_cast<int32_t>(pos) >= len) return 0xFFFFFFFFu;
    return static_cast<uint32_t>(__ldg(a.table + static_cast<uint64_t>(b) * a.max_pages + (shift >= 0 ? pos >> shift : pos / a.page_tokens)));
  };
  const int64_t key_step = (FOUR ? x.k4.head_stride : a.k.head_stride) * static_cast<int64_t>(head_warps);
  const int64_t scale_step = x.k4.s_head * static_cast<int64_t>(head_warps);
  unsigned char* const ring_p = dyn + warp * S::kStages * S::kBytes;
  const uint32_t ring = smem_u32(ring_p);
  uint32_t read_tile = blockIdx.x, read_left = heads, there = 0;
  uint32_t ahead = page_of(read_tile);
  const char *key = nullptr, *scale = nullptr;  // of this lane's token in the head that is read next
  auto fill = [&](uint32_t slot) {
    if (read_tile >= tiles || !heads) return;
    if (read_left == heads) {
      const uint32_t pos = base_of(read_tile) + lane;
      uint32_t pg = ahead, at = shift >= 0 ? pos & ((1u << shift) - 1u) : pos % a.page_tokens;
      const bool on = pg < a.n_pages;
      if (!on) {  // page 0 is read instead and the score made zero
        if (lane < S::kTokens && static_cast<int32_t>(pos) < len) kv_status(a.status, IBP_ERANGE);
        pg = at = 0;
      }
      there = __ballot_sync(0xFFFFFFFFu, on);
      if (FOUR) {
        key = x.k4.codes + static_cast<int64_t>(pg) * x.k4.page_stride + static_cast<int64_t>(h0) * x.k4.head_stride +
              static_cast<int64_t>(at) * x.k4.token_stride;
        scale = x.k4.scales + static_cast<int64_t>(pg) * x.k4.s_page + static_cast<int64_t>(h0) * x.k4.s_head + static_cast<int64_t>(at) * x.k4.s_token;
      } else {
        key = a.k.data + static_cast<int64_t>(pg) * a.k.page_stride + static_cast<int64_t>(h0) * a.k.head_stride + static_cast<int64_t>(at) * a.k.token_stride;
      }
      ahead = page_of(read_tile + gridDim.x);
    }
    constexpr uint32_t kChunks = S::kRow / 16, kPer = 32 / kChunks;
    const uint32_t c = lane % kChunks, r0 = lane / kChunks, stage = ring + slot * S::kBytes;
    const bool col = c * (FOUR ? 32 : 8) < a.dim;
#pragma unroll
    for (uint32_t i = 0; i < S::kTokens / kPer; ++i) {
      const char* p = reinterpret_cast<const char*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(key), r0 + i * kPer));
      cp16(stage + S::at(r0 + i * kPer, c), col ? p + c * 16 : p, col);
    }
    if constexpr (FOUR) {
      if (lane < S::kTokens) {
        const uint32_t off = S::kKeys + lane * S::kScale;
        if (even) {
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(stage + off), "l"(scale), "n"(S::kScale) : "memory");
        } else {
#pragma unroll
          for (uint32_t j = 0; j < DP / 32; ++j)
            *reinterpret_cast<uint16_t*>(ring_p + slot * S::kBytes + off + 2 * j) = j * 32 < a.dim ? __ldg(reinterpret_cast<const uint16_t*>(scale) + j) : uint16_t(0);
        }
      }
      scale += scale_step;
    }
    if (lane == 0) *reinterpret_cast<uint32_t*>(ring_p + slot * S::kBytes + S::kBytes - 16) = there;
    key += key_step;
    if (--read_left == 0) {
      read_left = heads;
      read_tile += gridDim.x;
    }
  };
  constexpr uint32_t kAhead = S::kStages - 1;
#pragma unroll
  for (uint32_t i = 0; i < kAhead; ++i) {
    fill(i);
    cp_commit();
  }
  // This lane's places in a stage.
  constexpr uint32_t kReads = FOUR ? (DP == 256 ? 2 : 1) : DP / 32;  // 16 bytes each (DP 64: 8 of codes)
  uint32_t k_at[kReads];
#pragma unroll
  for (uint32_t i = 0; i < kReads; ++i) k_at[i] = FOUR && DP == 64 ? S::at(g, t / 2) + (t & 1u) * 8 : S::at(g, t * kReads + i);
  uint32_t slot = 0;
#pragma unroll 1
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const uint32_t first = tile * tokens, base = base_of(tile);
    const bool open = static_cast<int32_t>(base + 16 * MT) <= ctx;  // every row sees the whole run
    float sum[MT][2];
#pragma unroll
    for (uint32_t m = 0; m < MT; ++m) sum[m][0] = sum[m][1] = 0.f;
    // f(j): operand B of eight dimensions; back: -lse log2 e, -infinity for a row that sees nothing
    auto work = [&](const unsigned char* st, auto f, const float (&back)[2], uint32_t r0) {
      const uint32_t there_now = *reinterpret_cast<const uint32_t*>(st + S::kBytes - 16) >> g;
      float c[MT][4];
#pragma unroll
      for (uint32_t m = 0; m < MT; ++m) {
        c[m][0] = c[m][1] = c[m][2] = c[m][3] = 0.f;
#pragma unroll
        for (uint32_t i = 0; i < kReads; ++i) {
          const unsigned char* k0 = st + k_at[i] + 16 * m * S::kRow;
          uint4 u, v;
          if constexpr (FOUR && DP == 64) {
            const uint2 u2 = *reinterpret_cast<const uint2*>(k0), v2 = *reinterpret_cast<const uint2*>(k0 + 8 * S::kRow);
            u = make_uint4(u2.x, u2.y, 0u, 0u), v = make_uint4(v2.x, v2.y, 0u, 0u);
          } else {
            u = *reinterpret_cast<const uint4*>(k0), v = *reinterpret_cast<const uint4*>(k0 + 8 * S::kRow);
          }
          uint32_t s0 = 0, s1 = 0;
          if constexpr (FOUR) {
            const unsigned char* sc = st + S::kKeys + (16 * m + g) * S::kScale + 2 * (DP == 64 ? t / 2 : t * kReads + i);
            s0 = *reinterpret_cast<const uint16_t*>(sc), s1 = *reinterpret_cast<const uint16_t*>(sc + 8 * S::kScale);
          }
          const quad::Pair<F16> p0(s0 * 0x10001u), p1(s1 * 0x10001u);
          constexpr uint32_t kWords = FOUR ? (DP == 64 ? 2 : 4) : 1;
#pragma unroll
          for (uint32_t j = 0; j < kWords; ++j) {
            const uint4 w = f(i * kWords + j);
            uint32_t lo[4], hi[4];
            weigh_operands<FOUR, F16>(u, v, j, p0, p1, magic, lo, hi);
            mma16816<F16>(c[m], lo, w.x, w.y);
            mma16816<F16>(c[m], hi, w.z, w.w);
          }
        }
      }
#pragma unroll
      for (uint32_t e = 0; e < 2; ++e) {
        const uint32_t tq = open ? 0 : (r0 + 2 * t + e) / a.group;
#pragma unroll
        for (uint32_t m = 0; m < MT; ++m)
#pragma unroll
          for (uint32_t i = 0; i < 2; ++i) {
            bool on = back[e] != -INFINITY;
            if (!open && on) {
              const int32_t pos = static_cast<int32_t>(base + 16 * m + g + 8 * i), at = pos - ctx;
              on = pos < len && (at < 0 || (a.mask ? (a.mask[(static_cast<uint64_t>(b) * a.T + tq) * a.mask_words + (at >> 5)] >> (at & 31)) & 1u
                                                  : static_cast<uint32_t>(at) <= tq));
            }
            const float p = ex2(fmaf(there_now >> (16 * m + 8 * i) & 1u ? c[m][2 * i + e] : 0.f, a.scale_log2, back[e]));
            sum[m][i] += on ? p : 0.f;
          }
      }
    };
    auto head = [&](const unsigned char* k, uint32_t h) {
      if constexpr (SHARED) {
        const float2 back = *reinterpret_cast<const float2*>(sl + h * 8 + 2 * t);
        work(k, [&](uint32_t j) { return sq[h * DP + j * 32 + lane]; }, {back.x, back.y}, 0);
      } else {
#pragma unroll 1
        for (uint32_t r0 = 0; r0 < rows; r0 += 8) {
          WeighRows<DP> q;
          weigh_rows<DP>(x, weigh_at(x, b, h, r0, rows, t * (DP / 4)), t * (DP / 4), q);
          float back[2];
#pragma unroll
          for (uint32_t e = 0; e < 2; ++e) back[e] = q.lse[e] == -INFINITY ? -INFINITY : -q.lse[e] * 1.4426950408889634f;
          work(k, [&](uint32_t j) {
            const uint32_t(&w)[4] = q.q[j];
            return FOUR ? make_uint4(__byte_perm(w[0], w[2], 0x5410), __byte_perm(w[0], w[2], 0x7632), __byte_perm(w[1], w[3], 0x5410), __byte_perm(w[1], w[3], 0x7632))
                        : make_uint4(w[0], w[1], w[2], w[3]);
          }, back, r0);
        }
      }
    };
#pragma unroll 1
    for (uint32_t n = 0, h = h0; n < heads; ++n, h += head_warps) {
      __syncwarp();  // every lane is done with the stage that is filled next
      fill(slot == 0 ? kAhead : slot - 1);
      cp_commit();
      cp_wait<kAhead>();
      __syncwarp();
      head(ring_p + slot * S::kBytes, h);
      slot = slot == kAhead ? 0 : slot + 1;
    }
    auto write = [&](uint32_t pos, float s) {
      const int32_t p = static_cast<int32_t>(pos);
      if (p < len) out[pos] = p < ctx ? fmaf(x.decay, was[pos], s) : s;
    };
#pragma unroll
    for (uint32_t m = 0; m < MT; ++m)
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        float s = sum[m][i];
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
        if (t == 0) {
          if (head_warps == 1)
            write(base + 16 * m + 8 * i + g, s);
          else
            sums[warp][16 * m + 8 * i + g] = s;
        }
      }
    if (head_warps == 1) continue;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < tokens; i += kWgWarps * 32) {
      const uint32_t run = i / (16 * MT);
      float s = 0.f;
      for (uint32_t w = 0; w < head_warps; ++w) s += sums[run * head_warps + w][i % (16 * MT)];
      write(first + i, s);
    }
    __syncthreads();
  }
  // positions without a token keep what they have
  for (uint64_t i = static_cast<uint32_t>(len > 0 ? len : 0) + static_cast<uint64_t>(blockIdx.x) * kWgWarps * 32 + threadIdx.x; i < x.width;
       i += static_cast<uint64_t>(gridDim.x) * kWgWarps * 32)
    out[i] = was[i];
}

int launch_kv_weigh(const WeighArgs& x, int device, cudaStream_t stream) {
  const AttendArgs& a = x.a;
  if (a.dim <= 128 && static_cast<uint64_t>(a.T) * a.group >= (x.k4.codes ? kWgMany4 : kWgMany)) return launch_kv_weigh_tc(x, device, stream);
  const uint32_t dp = a.dim <= 64 ? 64 : (a.dim <= 128 ? 128 : 256);
  const bool four = x.k4.codes != nullptr;
  const uint32_t mt = four && dp < 256 ? 2 : 1;
  // A warp takes all heads of its tokens where there are tokens enough to fill the GPU (4-bit
  // caches of up to 8192 tokens, 8 kv heads, 1 / 2 / 4 warps: one cache 20 / 17 / 15 us, four
  // 22 / 20 / 26 us; 32 of up to 16384 95 / 95 / 112 us).
  const uint64_t all_runs = (static_cast<uint64_t>(x.width) + 16 * mt - 1) / (16 * mt) * a.n_seqs;
  uint32_t head_warps = 1;
  while (head_warps < kWgWarps && head_warps < a.kv_heads && all_runs * head_warps < 8ull * sm_count(device)) head_warps *= 2;
  const uint32_t tokens = 16 * mt * (kWgWarps / head_warps);
  // A CTA walks a few tiles, so that what it begins with counts less; more would leave ragged
  // batches uneven.
  const uint32_t tiles = (x.width + tokens - 1) / tokens, some = kWgTiles < tiles ? kWgTiles : 1;
  const uint32_t walk = static_cast<uint64_t>(tiles) * a.n_seqs >= 4ull * some * sm_count(device) ? some : 1;
  const dim3 grid((tiles + walk - 1) / walk, a.n_seqs);
  int32_t shift = -1;
  if ((a.page_tokens & (a.page_tokens - 1)) == 0)
    for (shift = 0; (1u << shift) < a.page_tokens;) ++shift;
  const uint32_t room = a.kv_heads * (dp * 16 + 32);
  const bool shared = static_cast<uint64_t>(a.T) * a.group <= 8 && a.kv_heads <= 64 && room <= 40 * 1024;
  const uint64_t scales = reinterpret_cast<uintptr_t>(x.k4.scales) | static_cast<uint64_t>(x.k4.s_page) | static_cast<uint64_t>(x.k4.s_head) |
                          static_cast<uint64_t>(x.k4.s_token);
  const bool even = a.dim == dp && scales % (dp / 16) == 0;
  auto go = [&](auto kern, uint32_t ring, std::atomic<int>* ready) {
    if (device < 0 || device >= 64 || !ready[device].load(std::memory_order_acquire)) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
      if (e != cudaSuccess) {
        set_cuda_error(e, "set-up of k_kv_weigh");
        cudaGetLastError();
        return static_cast<int>(IBP_ECUDA);
      }
      if (device >= 0 && device < 64) ready[device].store(1, std::memory_order_release);
    }
    return kv_launch("k_kv_weigh", kern, grid, kWgWarps * 32, ring + (shared ? room : 0), 1, stream, x, head_warps, shift, even);
  };
  auto sized = [&](auto d, auto m, auto quads, auto f16, auto sh) {
    constexpr uint32_t D = decltype(d)::value, M = decltype(m)::value;
    constexpr bool Q = decltype(quads)::value, F = decltype(f16)::value, H = decltype(sh)::value;
    using S = WeighStage<D, M, Q>;
    static std::atomic<int> ready[64];
    static_assert(kWgWarps * S::kStages * S::kBytes + 40 * 1024 <= 160 * 1024, "the attribute covers it");
    return go(k_kv_weigh<D, M, Q, F, H>, kWgWarps * S::kStages * S::kBytes, ready);
  };
  auto typed = [&](auto quads, auto f16) {
    constexpr bool Q = decltype(quads)::value;
    using One = std::integral_constant<uint32_t, 1>;
    using Many = std::integral_constant<uint32_t, Q ? 2 : 1>;
    auto by_dim = [&](auto sh) {
      if (dp == 64) return sized(std::integral_constant<uint32_t, 64>{}, Many{}, quads, f16, sh);
      if (dp == 128) return sized(std::integral_constant<uint32_t, 128>{}, Many{}, quads, f16, sh);
      return sized(std::integral_constant<uint32_t, 256>{}, One{}, quads, f16, sh);
    };
    return shared ? by_dim(std::true_type{}) : by_dim(std::false_type{});
  };
  if (a.f16) return four ? typed(std::true_type{}, std::true_type{}) : typed(std::false_type{}, std::true_type{});
  return four ? typed(std::true_type{}, std::false_type{}) : typed(std::false_type{}, std::false_type{});
}

}  // namespace ibp

// ibp_kv_weigh.cu - the attention weight that each cached token receives.
//
// The weight of a row (query and head) for a token is exp(s - lse) with the row's
// known logarithm of the sum, so a token's total needs its key once and no value.  A
// CTA takes a run of tokens; its warps share out the kv heads (and runs of 16 MT
// tokens, where there are fewer heads than warps) and add up their rows in registers;
// the warps' sums are added in a fixed order, so results do not depend on how threads
// run.  S^T = K Q^T as in the attention kernels: a lane holds neighbouring dimensions
// of a token's key, and queries are laid out to match.  Bound by the keys' bytes for
// single tokens, by products and exponentials for prompts.
#include <type_traits>

#include "ibp_kv_serve.cuh"

namespace ibp {

constexpr uint32_t kWgWarps = 8;
constexpr uint64_t kWgMany = 64;  // rows a kv head from which the tensor cores take over

// Keys of 16 tokens as operands A: [step][register].
template <uint32_t DP, bool FOUR, bool F16>
struct WeighKeys {
  uint32_t f[DP / 16][4];

  // key rows g and g + 8 of this lane's DP / 4 dimensions
  __device__ __forceinline__ void load(const WeighArgs& x, const int64_t (&page)[2], const uint32_t (&slot)[2], uint32_t h, uint32_t t) {
    const AttendArgs& a = x.a;
    const uint32_t d0 = t * (DP / 4);
    if constexpr (FOUR) {
      uint32_t w[2][DP / 32], s[2][DP == 256 ? 2 : 1];
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        const bool on = page[i] >= 0;
        const int64_t pg = on ? page[i] : 0;
        const char* c = x.k4.codes + pg * x.k4.page_stride + static_cast<int64_t>(h) * x.k4.head_stride +
                        static_cast<int64_t>(slot[i]) * x.k4.token_stride + d0 / 2;
        const char* sc = x.k4.scales + pg * x.k4.s_page + static_cast<int64_t>(h) * x.k4.s_head +
                         static_cast<int64_t>(slot[i]) * x.k4.s_token + d0 / kQuadGroup * 2;
        if constexpr (DP == 256) {
#pragma unroll
          for (uint32_t j = 0; j < 2; ++j) {
            const bool in = on && d0 + 32 * j < a.dim;
            const uint4 u = in ? __ldg(reinterpret_cast<const uint4*>(c + 16 * j)) : make_uint4(0u, 0u, 0u, 0u);
            w[i][4 * j] = u.x, w[i][4 * j + 1] = u.y, w[i][4 * j + 2] = u.z, w[i][4 * j + 3] = u.w;
            s[i][j] = in ? __ldg(reinterpret_cast<const uint16_t*>(sc + 2 * j)) : 0u;
          }
        } else {
          const bool in = on && d0 < a.dim;
          if constexpr (DP == 128) {
            const uint4 u = in ? __ldg(reinterpret_cast<const uint4*>(c)) : make_uint4(0u, 0u, 0u, 0u);
            w[i][0] = u.x, w[i][1] = u.y, w[i][2] = u.z, w[i][3] = u.w;
          } else {
            const uint2 u = in ? __ldg(reinterpret_cast<const uint2*>(c)) : make_uint2(0u, 0u);
            w[i][0] = u.x, w[i][1] = u.y;
          }
          s[i][0] = in ? __ldg(reinterpret_cast<const uint16_t*>(sc)) : 0u;
        }
      }
      const quad::Magic<F16> m;
#pragma unroll
      for (uint32_t j = 0; j < DP / 32; ++j) {
        const uint32_t gi = DP == 256 ? j / 4 : 0;
        const quad::Pair<F16> p0(s[0][gi] * 0x10001u), p1(s[1][gi] * 0x10001u);
        f[2 * j][0] = quad::decode<F16, 0>(w[0][j], p0, m), f[2 * j][1] = quad::decode<F16, 0>(w[1][j], p1, m);
        f[2 * j][2] = quad::decode<F16, 1>(w[0][j], p0, m), f[2 * j][3] = quad::decode<F16, 1>(w[1][j], p1, m);
        f[2 * j + 1][0] = quad::decode<F16, 2>(w[0][j], p0, m), f[2 * j + 1][1] = quad::decode<F16, 2>(w[1][j], p1, m);
        f[2 * j + 1][2] = quad::decode<F16, 3>(w[0][j], p0, m), f[2 * j + 1][3] = quad::decode<F16, 3>(w[1][j], p1, m);
      }
    } else {
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        const bool on = page[i] >= 0;
        const char* c = a.k.data + (on ? page[i] : 0) * a.k.page_stride + static_cast<int64_t>(h) * a.k.head_stride +
                        static_cast<int64_t>(slot[i]) * a.k.token_stride + d0 * 2;
#pragma unroll
        for (uint32_t j = 0; j < DP / 32; ++j) {
          const uint4 u = on && d0 + 8 * j < a.dim ? __ldg(reinterpret_cast<const uint4*>(c + 16 * j)) : make_uint4(0u, 0u, 0u, 0u);
          f[2 * j][i] = u.x, f[2 * j][2 + i] = u.y, f[2 * j + 1][i] = u.z, f[2 * j + 1][2 + i] = u.w;
        }
      }
    }
  }
};

// Eight dimensions of a query as the keys' order has them: registers of two steps.
template <bool FOUR>
__device__ __forceinline__ void weigh_query(uint32_t (&r)[4], const char* q, bool q16) {
  uint32_t w[4];
  if (q16) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(q));
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(q) + 2 * i;
      w[i] = __ldg(h) | static_cast<uint32_t>(__ldg(h + 1)) << 16;
    }
  }
  if (FOUR) {  // elements (0, 4), (1, 5), (2, 6), (3, 7)
    r[0] = __byte_perm(w[0], w[2], 0x5410), r[1] = __byte_perm(w[0], w[2], 0x7632);
    r[2] = __byte_perm(w[1], w[3], 0x5410), r[3] = __byte_perm(w[1], w[3], 0x7632);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = w[i];
  }
}

template <uint32_t DP, uint32_t MT, bool FOUR, bool F16>
__global__ void __launch_bounds__(kWgWarps * 32) k_kv_weigh(const WeighArgs x, uint32_t head_warps) {
  __shared__ float sums[kWgWarps][16 * MT];
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
  for (uint32_t first = blockIdx.x * tokens; first < x.width; first += gridDim.x * tokens) {
    const uint32_t base = first + warp / head_warps * 16 * MT;  // this warp's run
    float sum[MT][2];
#pragma unroll
    for (uint32_t m = 0; m < MT; ++m) sum[m][0] = sum[m][1] = 0.f;
    if (static_cast<int32_t>(base) < len) {
      int64_t page[MT][2];
      uint32_t slot[MT][2];
#pragma unroll
      for (uint32_t m = 0; m < MT; ++m)
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
          const uint32_t pos = base + 16 * m + g + 8 * i, nth = pos / a.page_tokens;
          slot[m][i] = pos - nth * a.page_tokens;
          page[m][i] = -1;
          if (static_cast<int32_t>(pos) < len) {
            const uint32_t pg = static_cast<uint32_t>(__ldg(a.table + static_cast<uint64_t>(b) * a.max_pages + nth));
            if (pg < a.n_pages)
              page[m][i] = pg;
            else
              kv_status(a.status, IBP_ERANGE);
          }
        }
      const bool open = static_cast<int32_t>(base + 16 * MT) <= ctx;  // every row sees the whole run
#pragma unroll 1
      for (uint32_t h = warp % head_warps; h < a.kv_heads; h += head_warps) {
        WeighKeys<DP, FOUR, F16> k[MT];
#pragma unroll
        for (uint32_t m = 0; m < MT; ++m) k[m].load(x, page[m], slot[m], h, t);
#pragma unroll 1
        for (uint32_t r0 = 0; r0 < rows; r0 += 8) {
          const uint32_t rq = r0 + g < rows ? r0 + g : rows - 1;  // a row past the end is not counted
          const char* q = a.q + static_cast<int64_t>(b) * a.q_seq + static_cast<int64_t>(rq / a.group) * a.q_token +
                          static_cast<int64_t>(h * a.group + rq % a.group) * a.q_head + t * (DP / 4) * 2;
          float c[MT][4];
#pragma unroll
          for (uint32_t m = 0; m < MT; ++m) c[m][0] = c[m][1] = c[m][2] = c[m][3] = 0.f;
#pragma unroll
          for (uint32_t j = 0; j < DP / 32; ++j) {
            uint32_t f[4] = {0u, 0u, 0u, 0u};
            if (t * (DP / 4) + 8 * j < a.dim) weigh_query<FOUR>(f, q + 16 * j, x.q16);
#pragma unroll
            for (uint32_t m = 0; m < MT; ++m) {
              mma16816<F16>(c[m], k[m].f[2 * j], f[0], f[1]);
              mma16816<F16>(c[m], k[m].f[2 * j + 1], f[2], f[3]);
            }
          }
#pragma unroll
          for (uint32_t e = 0; e < 2; ++e) {
            const uint32_t r = r0 + 2 * t + e;
            if (r >= rows) continue;
            const uint32_t tq = r / a.group;
            const float lse = __ldg(x.lse + (static_cast<uint64_t>(b) * a.T + tq) * a.kv_heads * a.group + h * a.group + r % a.group);
            if (lse == -INFINITY) continue;  // a row that sees nothing
            const float back = -lse * 1.4426950408889634f;
#pragma unroll
            for (uint32_t m = 0; m < MT; ++m)
#pragma unroll
              for (uint32_t i = 0; i < 2; ++i) {
                bool on = true;
                if (!open) {
                  const int32_t pos = static_cast<int32_t>(base + 16 * m + g + 8 * i), at = pos - ctx;
                  on = pos < len && (at < 0 || (a.mask ? (a.mask[(static_cast<uint64_t>(b) * a.T + tq) * a.mask_words + (at >> 5)] >> (at & 31)) & 1u
                                                      : static_cast<uint32_t>(at) <= tq));
                }
                if (on) sum[m][i] += ex2(fmaf(c[m][2 * i + e], a.scale_log2, back));
              }
          }
        }
      }
    }
#pragma unroll
    for (uint32_t m = 0; m < MT; ++m)
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) {
        float s = sum[m][i];
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
        if (t == 0) sums[warp][16 * m + 8 * i + g] = s;
      }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < tokens; i += kWgWarps * 32) {
      const uint32_t pos = first + i;
      if (pos >= x.width) break;
      const uint32_t run = i / (16 * MT);
      float s = 0.f;
      for (uint32_t w = 0; w < head_warps; ++w) s += sums[run * head_warps + w][i % (16 * MT)];
      const int32_t p = static_cast<int32_t>(pos);
      out[pos] = p >= len ? was[pos] : (p < ctx ? fmaf(x.decay, was[pos], s) : s);
    }
    __syncthreads();
  }
}

int launch_kv_weigh(const WeighArgs& x, int device, cudaStream_t stream) {
  const AttendArgs& a = x.a;
  if (a.dim <= 128 && static_cast<uint64_t>(a.T) * a.group >= kWgMany) return launch_kv_weigh_tc(x, device, stream);
  uint32_t head_warps = 1;
  while (head_warps < kWgWarps && head_warps < a.kv_heads) head_warps *= 2;
  const uint32_t dp = a.dim <= 64 ? 64 : (a.dim <= 128 ? 128 : 256);
  const uint32_t mt = static_cast<uint64_t>(a.T) * a.group > 8 && dp < 256 ? 2 : 1, tokens = 16 * mt * (kWgWarps / head_warps);
  const uint64_t want = (static_cast<uint64_t>(x.width) + tokens - 1) / tokens, most = 0x7FFFFFFFull;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most), a.n_seqs);
  auto go = [&](auto kern) { return kv_launch("k_kv_weigh", kern, grid, kWgWarps * 32, 0, 1, stream, x, head_warps); };
  auto typed = [&](auto four, auto f16) {
    constexpr bool Q = decltype(four)::value, F = decltype(f16)::value;
    if (dp == 64) return mt == 2 ? go(k_kv_weigh<64, 2, Q, F>) : go(k_kv_weigh<64, 1, Q, F>);
    if (dp == 128) return mt == 2 ? go(k_kv_weigh<128, 2, Q, F>) : go(k_kv_weigh<128, 1, Q, F>);
    return go(k_kv_weigh<256, 1, Q, F>);
  };
  const bool four = x.k4.codes != nullptr;
  if (a.f16) return four ? typed(std::true_type{}, std::true_type{}) : typed(std::false_type{}, std::true_type{});
  return four ? typed(std::true_type{}, std::false_type{}) : typed(std::false_type{}, std::false_type{});
}

}  // namespace ibp

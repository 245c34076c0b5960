// ibp_kv_verify.cu - drafted tokens against the target's probabilities.
//
// A cluster takes a sequence.  Whether a token is accepted when it is the first one
// tried behind its parent depends on two probabilities alone, so all these tests are
// made at once; the walk then follows the answers.  Only a rejection needs a whole
// row of probabilities (what is left of the target's after the draft's is taken out,
// and its sum), and the last row is needed for the drawn token.  Rows are split over
// the cluster's warps in the order of the vocabulary.
//
// Sums are of whole numbers, 2^44 times the probability, in 64 bits: they do not
// depend on the order, so neither do the choices.  What is left after several
// rejections is computed anew from the rows (m subtractions and products an element)
// and not stored.
//
// Measured on one GB300: a chain of 4 over 32768 tokens 11 us, trees of 15 for 64
// sequences over 131072 tokens 63 us with cold caches (46 to 49 us where the
// probabilities have just been written), of which the rows that cannot be left out are 10.  Each
// rejection is a walk over two rows that the next step waits for, and a cluster's row comes
// out of few SMs: latency of the walks bounds it.
//
// CTAs of a sequence: 1 up to a vocabulary of 4096, 4 up to 16384, 8 beyond (64 trees of 15,
// us with 1 / 4 / 8: 4096 20 / 24 / 24, 8192 28 / 24 / 26, 16384 40 / 26 / 26, 32768
// 73 / 35 / 28, 131072 276 / 87 / 60).
#include <type_traits>

#include "ibp_kv_serve.cuh"

namespace ibp {

constexpr int kVfThreads = 256;
constexpr uint32_t kVfWarps = kVfThreads / 32;

__device__ __forceinline__ float probability(float x) { return fminf(fmaxf(x, 0.f), 1.f); }  // NaN: 0

struct VerifyShared {
  // Sums of the warps' parts of a row, and the CTA's.  Three slots: the one that is kept,
  // the one that was written last (others may still read it), and the next.
  long long warp[3][kVfWarps];
  long long cta[3];
  long long part[kVfWarps];
};

// What is left of row p behind `depth` rejections, the last one not scaled to a sum of
// one again: the weight by which a token is drawn.
struct Left {
  const float *p, *q;
  const float* scale;
  const int32_t* x;
  uint32_t depth;
  __device__ __forceinline__ float drawn(uint32_t i, float qi, uint32_t k) const {
    return q ? qi : (static_cast<int32_t>(i) == x[k] ? 1.f : 0.f);
  }
  // of element i, whose probabilities are pi and qi; DEPTH: what depth is, 2 for more
  template <uint32_t DEPTH>
  __device__ __forceinline__ float of(uint32_t i, float pi, float qi) const {
    float v = probability(pi);
    if (DEPTH == 0) return v;
    qi = probability(qi);
    v = fmaxf(__fsub_rn(v, drawn(i, qi, 0)), 0.f);
    if (DEPTH > 1)
      for (uint32_t k = 1; k < depth; ++k) v = fmaxf(__fsub_rn(__fmul_rn(v, scale[k - 1]), drawn(i, qi, k)), 0.f);
    return v;
  }
  __device__ __forceinline__ float operator()(uint32_t i) const {
    const float pi = __ldg(p + i);
    return depth ? of<2>(i, pi, q ? __ldg(q + i) : 0.f) : of<0>(i, pi, 0.f);
  }
};

// rint(w 2^44) of a weight in [0, 1] as high 2^23 + low: high = rint(w 2^21), what is left
// is exact and low its rounding, to even like the whole's since high 2^23 is.  Whole numbers
// below 2^22 are the last bits of a float of 1.5 2^23 more.  (A conversion to 64 bits
// goes through the double-precision pipe: 25 % of the kernel's time.)
__device__ __forceinline__ void whole_parts(float w, int32_t& high, int32_t& low) {
  const float h = __fmaf_rn(w, 0x1p21f, 12582912.f);
  const float rest = __fmaf_rn(__fadd_rn(h, -12582912.f), -0x1p-21f, w);
  high += __float_as_int(h) - 0x4B400000;
  low += __float_as_int(__fmaf_rn(rest, 0x1p44f, 12582912.f)) - 0x4B400000;
}
__device__ __forceinline__ long long whole(float w) {
  int32_t high = 0, low = 0;
  whole_parts(w, high, low);
  return (static_cast<long long>(high) << 23) + low;
}

__device__ __forceinline__ long long warp_total(long long s) {
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

__device__ __forceinline__ long long remote_ll(const long long* p, uint32_t rank) {
  uint32_t addr = smem_u32(p);
  long long v;
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(addr) : "r"(rank));
  asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

template <uint32_t C>
__device__ __forceinline__ void vf_sync() {
  if (C == 1)
    __syncthreads();
  else
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums of the weights, in slot `buf`: every warp's, the CTA's, and the row's (returned).
// VEC: rows of whole aligned pieces of four.
template <uint32_t C, bool VEC>
__device__ __forceinline__ long long vf_sum(VerifyShared& sh, uint32_t buf, const Left& f, uint32_t from, uint32_t to) {
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  // A lane has at most 2^18 / (8 * 256) elements of up to 2^21 and +-2^22: 32 bits hold its sums.
  static_assert(IBP_VERIFY_MAX_VOCAB / (8 * kVfThreads) <= 256, "");
  int32_t high = 0, low = 0;
  auto sum = [&](auto depth) {
    constexpr uint32_t D = decltype(depth)::value;
    const bool two = D && f.q;
    if (VEC) {
      constexpr uint32_t kFly = 4;  // 16-byte reads of each row under way
      for (uint32_t i0 = from + 4 * lane; i0 < to; i0 += 128 * kFly) {
        float4 x[kFly], y[kFly];
#pragma unroll
        for (uint32_t u = 0; u < kFly; ++u) {
          const uint32_t i = i0 + 128 * u;
          x[u] = y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < to) {
            x[u] = __ldg(reinterpret_cast<const float4*>(f.p + i));
            if (two) y[u] = __ldg(reinterpret_cast<const float4*>(f.q + i));
          }
        }
#pragma unroll
        for (uint32_t u = 0; u < kFly; ++u) {
          const uint32_t i = i0 + 128 * u;  // past the end all weights are zeros
          whole_parts(f.template of<D>(i, x[u].x, y[u].x), high, low);
          whole_parts(f.template of<D>(i + 1, x[u].y, y[u].y), high, low);
          whole_parts(f.template of<D>(i + 2, x[u].z, y[u].z), high, low);
          whole_parts(f.template of<D>(i + 3, x[u].w, y[u].w), high, low);
        }
      }
    } else {
#pragma unroll 8
      for (uint32_t i = from + lane; i < to; i += 32) whole_parts(f.template of<D>(i, __ldg(f.p + i), two ? __ldg(f.q + i) : 0.f), high, low);
    }
  };
  if (f.depth == 0)
    sum(std::integral_constant<uint32_t, 0>{});
  else if (f.depth == 1)
    sum(std::integral_constant<uint32_t, 1>{});
  else
    sum(std::integral_constant<uint32_t, 2>{});
  long long s = (static_cast<long long>(high) << 23) + low;
  s = warp_total(s);
  if (lane == 0) sh.warp[buf][warp] = s;
  __syncthreads();
  if (warp == 0) {
    const long long all = warp_total(lane < kVfWarps ? sh.warp[buf][lane] : 0);
    if (lane == 0) sh.cta[buf] = all;
  }
  vf_sync<C>();
  long long total = 0;
#pragma unroll
  for (uint32_t r = 0; r < C; ++r) total += C == 1 ? sh.cta[buf] : remote_ll(&sh.cta[buf], r);
  return total;
}

template <uint32_t C, bool VEC>
__global__ void __launch_bounds__(kVfThreads, 4) k_kv_verify(const VerifyArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ VerifyShared sh;
  pdl_begin();
  const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5, T = a.T, V = a.vocab;
  const uint32_t rank = C == 1 ? 0 : blockIdx.x % C, b = blockIdx.x / C;
  int32_t* tok = reinterpret_cast<int32_t*>(dyn);  // [T]; -1: out of range
  int32_t* par = tok + T;                          // [T]; -2: out of range
  float* ut = reinterpret_cast<float*>(par + T);   // [T]
  float* scale = ut + T;                           // [T]: of the rejections behind the present node
  int32_t* gone = reinterpret_cast<int32_t*>(scale + T);  // [T]: their tokens
  uint8_t* first = reinterpret_cast<uint8_t*>(gone + T);  // [T]: accepted if the first one tried
  const float* p = a.p + static_cast<int64_t>(b) * a.p_seq;
  const float* q = a.q ? a.q + static_cast<int64_t>(b) * a.q_seq : nullptr;
  const float* u = a.u + static_cast<uint64_t>(b) * (T + 1);
  const int32_t want = a.n_draft ? a.n_draft[b] : static_cast<int32_t>(T);
  const int32_t n = want < 0 ? 0 : (want > static_cast<int32_t>(T) ? static_cast<int32_t>(T) : want);
  bool bad = want != n;
  for (uint32_t t = tid; t < static_cast<uint32_t>(n); t += kVfThreads) {
    const uint64_t at = static_cast<uint64_t>(b) * T + t;
    int32_t x = a.tokens[at], r = a.parents ? a.parents[at] : static_cast<int32_t>(t) - 1;
    const float ux = u[t];
    if (x < 0 || static_cast<uint32_t>(x) >= V) x = -1, bad = true;
    if (r < -1 || r >= static_cast<int32_t>(t)) r = -2, bad = true;
    bool ok = false;
    if (x >= 0 && r >= -1) {
      const float px = probability(p[static_cast<int64_t>(r + 1) * a.p_row + x]);
      const float qx = q ? probability(q[static_cast<int64_t>(r + 1) * a.q_row + x]) : 1.f;
      ok = static_cast<double>(ux) * qx < px;  // the product of two floats is exact
    }
    tok[t] = x, par[t] = r, ut[t] = ux, first[t] = ok;
  }
  if (bad && rank == 0) kv_status(a.status, IBP_ERANGE);
  __syncthreads();

  // This warp's part of a row.
  constexpr uint32_t kPiece = VEC ? 128 : 32;
  const uint32_t part = (V + C * kVfWarps * kPiece - 1) / (C * kVfWarps * kPiece) * kPiece;
  auto clip = [&](uint32_t x) { return x < V ? x : V; };
  const uint32_t from = clip((rank * kVfWarps + warp) * part), to = clip(from + part);

  int32_t node = -1;
  uint32_t count = 0, keep = 0, last = 0;
  long long total = -1;  // of the weights that a token would be drawn by, in slot `keep`; -1: not known
  Left f = {p, q, scale, gone, 0u};
  for (int32_t t = 0; t < n; ++t) {
    if (par[t] != node || tok[t] < 0) continue;
    const int32_t x = tok[t];
    bool ok = first[t];
    if (f.depth) {
      const float left = __fmul_rn(f(x), scale[f.depth - 1]);
      const float qx = q ? probability(__ldg(f.q + x)) : 1.f;
      ok = static_cast<double>(ut[t]) * qx < left;
    }
    if (ok) {
      if (rank == 0 && tid == 0) a.path[static_cast<uint64_t>(b) * T + count] = t;
      ++count;
      node = t;
      f.p = p + static_cast<int64_t>(node + 1) * a.p_row;
      if (q && node + 1 < static_cast<int32_t>(T)) f.q = q + static_cast<int64_t>(node + 1) * a.q_row;
      f.depth = 0;
      total = -1;
    } else {
      // A warp behind may still read entry 0: the test of a token that was accepted behind a
      // rejection, whose node now rejects its first.
      __syncthreads();
      if (tid == 0) gone[f.depth] = x;
      __syncthreads();
      ++f.depth;
      last = keep != last ? 3 - keep - last : (keep + 1) % 3;
      const long long z = vf_sum<C, VEC>(sh, last, f, from, to);
      if (z > 0) {
        keep = last;
        total = z;
        if (tid == 0) scale[f.depth - 1] = static_cast<float>(__ddiv_rn(17592186044416.0, static_cast<double>(z)));
        __syncthreads();
      } else {
        --f.depth;  // nothing would be left: the token is out, the rest stays
      }
    }
  }
  if (total < 0) {
    keep = last = keep != last ? 3 - keep - last : (keep + 1) % 3;
    total = vf_sum<C, VEC>(sh, last, f, from, to);
  }
  if (rank == 0) {
    for (uint32_t t = count + tid; t < T; t += kVfThreads) a.path[static_cast<uint64_t>(b) * T + t] = -1;
    if (tid == 0) a.n_accept[b] = static_cast<int32_t>(count);
  }
  if (total == 0) {
    if (rank == 0 && tid == 0) {
      a.token[b] = -1;
      kv_status(a.status, IBP_ERANGE);
    }
  } else {
    // The first token whose running sum is above floor(u total): CTA, warp's part, the
    // part shared out over the warps again, token.
    const double want_sum = static_cast<double>(u[T]) * static_cast<double>(total);
    long long aim = want_sum >= static_cast<double>(total) ? total - 1 : (want_sum > 0 ? static_cast<long long>(want_sum) : 0);
    if (aim > total - 1) aim = total - 1;
    if constexpr (C > 1)
      for (uint32_t r = 0; r < rank; ++r) aim -= remote_ll(&sh.cta[keep], r);
    const bool mine = aim >= 0 && aim < sh.cta[keep];
    if (mine) {
      uint32_t w = 0;
      while (w < kVfWarps - 1 && aim >= sh.warp[keep][w]) aim -= sh.warp[keep][w++];
      const uint32_t lo = clip((rank * kVfWarps + w) * part), hi = clip(lo + part);
      const uint32_t sub = (part + kVfWarps * 32 - 1) / (kVfWarps * 32) * 32;
      const uint32_t s0 = lo + warp * sub < hi ? lo + warp * sub : hi, s1 = s0 + sub < hi ? s0 + sub : hi;
      long long s = 0;
      for (uint32_t i = s0 + lane; i < s1; i += 32) s += whole(f(i));
      s = warp_total(s);
      if (lane == 0) sh.part[warp] = s;
      __syncthreads();
      w = 0;
      while (w < kVfWarps - 1 && aim >= sh.part[w]) aim -= sh.part[w++];
      if (warp == w) {
        for (uint32_t i0 = s0; i0 < s1; i0 += 32) {
          const uint32_t i = i0 + lane;
          const long long me = i < s1 ? whole(f(i)) : 0;
          long long run = me;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, run, o);
            if (static_cast<int>(lane) >= o) run += y;
          }
          const uint32_t hit = __ballot_sync(0xFFFFFFFFu, run > aim);
          if (hit) {
            if (lane == 0) a.token[b] = static_cast<int32_t>(i0 + __ffs(hit) - 1);
            break;
          }
          aim -= __shfl_sync(0xFFFFFFFFu, run, 31);
        }
      }
    }
  }
  if (C > 1) vf_sync<C>();  // no CTA leaves while another reads its sums
}

int launch_kv_verify(const VerifyArgs& a, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(a.T) * 21;
  auto go = [&](auto kern, uint32_t c) {
    return kv_launch("k_kv_verify", kern, dim3(a.n_seqs * c), kVfThreads, smem, c, stream, a);
  };
  const uint64_t strides = static_cast<uint64_t>(a.p_seq) | static_cast<uint64_t>(a.p_row) | (a.q ? static_cast<uint64_t>(a.q_seq) | static_cast<uint64_t>(a.q_row) : 0);
  const bool vec = a.vocab % 4 == 0 && strides % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.p) | reinterpret_cast<uintptr_t>(a.q)) & 15u) == 0;
  if (a.vocab <= 4096) return vec ? go(k_kv_verify<1, true>, 1) : go(k_kv_verify<1, false>, 1);
  if (a.vocab <= 16384) return vec ? go(k_kv_verify<4, true>, 4) : go(k_kv_verify<4, false>, 4);
  return vec ? go(k_kv_verify<8, true>, 8) : go(k_kv_verify<8, false>, 8);
}

}  // namespace ibp

// ibp_kv4_tree.cu - launch of the tensor-core attention over caches held in 4 bits.
#include <type_traits>

#include "ibp_kv_tree.cuh"

namespace ibp {

static size_t align256(size_t x) { return (x + 255) / 256 * 256; }

bool kv4_tree_takes(uint32_t n_seqs, uint32_t kv_heads, uint64_t rows, uint32_t dim, uint64_t tokens, int device) {
  if (dim > 128 || tokens == 0) return false;
  const uint64_t longest = (tokens + kTcTile - 1) / kTcTile;
  return longest * n_seqs * kv_heads * ((rows + 15) / 16) >= 2ull * sm_count(device);
}

size_t kv4_tree_workspace(uint32_t dim, int device) {
  const size_t n = sm_count(device), dp = dim <= 64 ? 64 : 128;
  return align256((n + 1) * sizeof(int4)) + align256(2 * n * kTcTile * sizeof(float2)) + 2 * n * kTcTile * dp * 4;
}

template <uint32_t DP, bool F16, bool EVEN>
static int launch(TcArgs& t, int device, cudaStream_t stream) {
  using S = TcShape<DP, 1, true>;
  auto kern = k_kv_tree<DP, 1, F16, true, EVEN>;
  static std::atomic<int> ready[64];
  if (device < 0 || device >= 64 || !ready[device].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) {
      set_cuda_error(e, "set-up of k_kv_tree");
      cudaGetLastError();
      return IBP_ECUDA;
    }
    if (device >= 0 && device < 64) ready[device].store(1, std::memory_order_release);
  }
  const CUtensorMap none = {};
  int rc = kv_launch("k_kv_tree", kern, dim3(t.n_ctas), S::kThreads, S::kSmem, 1, stream, t, none, none);
  if (rc != IBP_OK || t.n_ctas == 1) return rc;
  const uint64_t rows = static_cast<uint64_t>(t.a.T) * t.a.group, most = rows < kTcTile ? rows : kTcTile;
  return kv_launch("k_kv_tree_join", k_kv_tree_join<DP, kTcTile, F16>,
                   dim3(t.n_ctas - 1, static_cast<unsigned>((most + kJoinRows - 1) / kJoinRows)), kJoinThreads, 0, 1, stream, t);
}

int launch_kv4_tree(const Attend4Args& x, int device, size_t ws_bytes, cudaStream_t stream) {
  const AttendArgs& a = x.a;
  const uint64_t rows = static_cast<uint64_t>(a.T) * a.group, tokens = static_cast<uint64_t>(a.max_pages) * a.page_tokens;
  if (!a.part || ws_bytes < kv4_tree_workspace(a.dim, device)) return IBP_EINVAL;
  TcArgs t = {};
  t.a = a;
  t.four[0] = x.k, t.four[1] = x.v;
  t.limit = kv_tree_limit();
  const uint32_t dp = a.dim <= 64 ? 64 : 128;
  t.shift = -1;
  if ((a.page_tokens & (a.page_tokens - 1)) == 0)
    for (t.shift = 0; (1u << t.shift) < a.page_tokens;) ++t.shift;
  bool even = a.dim == dp;  // all of the tile's dimensions, a token's scales aligned as one
  t.narrow = 1;
  for (int i = 0; i < 2; ++i) {
    const Kv4View& v = t.four[i];
    even = even && (reinterpret_cast<uintptr_t>(v.scales) | static_cast<uint64_t>(v.s_page) | static_cast<uint64_t>(v.s_head) |
                        static_cast<uint64_t>(v.s_token)) % (dp / 16) == 0;
    const uint64_t wide = static_cast<uint64_t>(v.page_stride) | static_cast<uint64_t>(v.token_stride) | static_cast<uint64_t>(v.s_page) |
                          static_cast<uint64_t>(v.s_token);
    t.narrow = t.narrow && wide <= 0xFFFFFFFFull;
  }
  t.row_pairs = static_cast<uint32_t>((rows + kTcTile - 1) / kTcTile);
  t.q16 = ((reinterpret_cast<uintptr_t>(a.q) | static_cast<uint64_t>(a.q_seq) | static_cast<uint64_t>(a.q_token) |
            static_cast<uint64_t>(a.q_head)) & 15u) == 0;
  const uint64_t tiles = (tokens + kTcTile - 1) / kTcTile * a.n_seqs * a.kv_heads * t.row_pairs;
  const uint64_t want = (tiles + kTcMinTiles - 1) / kTcMinTiles, n = sm_count(device);
  uint64_t ctas = want < n ? want : n;
  if (ctas > t.row_pairs) ctas -= ctas % t.row_pairs;
  t.n_ctas = static_cast<uint32_t>(ctas);
  char* w = reinterpret_cast<char*>(a.part);
  t.first = reinterpret_cast<int4*>(w);
  w += align256((n + 1) * sizeof(int4));
  t.ml_part = reinterpret_cast<float2*>(w);
  w += align256(2 * n * kTcTile * sizeof(float2));
  t.o_part = reinterpret_cast<float*>(w);
  auto go = [&](auto f16, auto e) {
    constexpr bool F = decltype(f16)::value, E = decltype(e)::value;
    return dp == 64 ? launch<64, F, E>(t, device, stream) : launch<128, F, E>(t, device, stream);
  };
  if (even) return a.f16 ? go(std::true_type{}, std::true_type{}) : go(std::false_type{}, std::true_type{});
  return a.f16 ? go(std::true_type{}, std::false_type{}) : go(std::false_type{}, std::false_type{});
}

}  // namespace ibp

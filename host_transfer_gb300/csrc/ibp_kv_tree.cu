// ibp_kv_tree.cu - launch of the tensor-core tree attention, and the join of
// items that several CTAs share.
#include "ibp_kv_tree.cuh"

namespace ibp {

constexpr int kJoinThreads = 256;
constexpr uint32_t kJoinRows = kJoinThreads / 32;  // rows of a CTA, a warp each

// CTA (j, rows): joins the item that crosses the start of range j, if j is the
// first range boundary inside it.  The range before holds its first part (slot
// 1), the ranges from j on the others (slot 0), added in that order.
template <uint32_t DP, uint32_t MT, bool F16>
__global__ void __launch_bounds__(kJoinThreads) k_kv_tree_join(const __grid_constant__ TcArgs t) {
  pdl_begin();
  const AttendArgs& a = t.a;
  const uint32_t j = blockIdx.x + 1, lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const int4 f = t.first[j], sh = t.first[t.n_ctas];
  const uint64_t share = static_cast<uint32_t>(sh.x) | (static_cast<uint64_t>(static_cast<uint32_t>(sh.y)) << 32);
  const uint64_t before = static_cast<uint32_t>(f.w);
  if (f.x < 0 || before == 0 || before > share) return;
  const uint32_t b = f.x, h = f.y;
  const uint64_t start = j * share - before, end = start + tiles_of(a, b);
  const uint32_t last = static_cast<uint32_t>((end - 1) / share);
  constexpr uint32_t kRows = MT * kTcTile;
  const uint32_t r = blockIdx.y * kJoinRows + warp, gr = f.z * kRows + r;
  const uint32_t tok = gr / a.group, head = gr - tok * a.group;
  if (tok >= a.T) return;
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

static size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Two row tiles of 128 fill TMEM beside the scores.  One row tile of 256 would fit
// too (256 columns of scores, 256 of output); it is not built, and wider heads take
// the few-row kernel.
static bool tc_shape(uint32_t dim) { return dim <= 128; }
static uint32_t tc_dim(uint32_t dim) { return dim <= 64 ? 64 : 128; }
static uint32_t tc_tiles(uint64_t rows) { return rows > kTcTile ? 2 : 1; }

// Whether the kernel takes a call.  Boxes are whole 8-row swizzle groups of a
// page.  Little work is done sooner by the few-row kernel, which has less to set
// up: counted in 16-row x 128-token pieces, below two to a SM.  Measured (us, few-row /
// this): 40 tiles of 4 rows 7.0 / 16, of 64 rows 11 / 18, of 128 rows 22 / 19; 256
// tiles of 16 rows 16 / 18, of 32 rows 23 / 18; 1024 of 16 rows 28 / 22, of 128 79 / 26.
static bool tc_takes(uint32_t n_seqs, uint32_t kv_heads, uint64_t rows, uint32_t dim, uint32_t page_tokens,
                     uint64_t tokens, int device) {
  if (!tc_shape(dim) || page_tokens % 8 || tokens == 0) return false;
  const uint64_t longest = (tokens + kTcTile - 1) / kTcTile;
  return longest * n_seqs * kv_heads * ((rows + 15) / 16) >= 2ull * sm_count(device);
}

size_t kv_tree_workspace(uint32_t n_seqs, uint32_t kv_heads, uint64_t rows, uint32_t dim, uint32_t page_tokens,
                         uint64_t tokens, int device) {
  if (!tc_takes(n_seqs, kv_heads, rows, dim, page_tokens, tokens, device)) return 0;
  const size_t n = sm_count(device), per = tc_tiles(rows) * kTcTile;
  return align256((n + 1) * sizeof(int4)) + align256(2 * n * per * sizeof(float2)) + 2 * n * per * tc_dim(dim) * 4;
}

static int encode(CUtensorMap* map, const KvView& v, const AttendArgs& a, uint32_t box, bool* ok) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<Encode> cache{nullptr};  // looked up once, any host thread
  Encode fn = cache.load(std::memory_order_acquire);
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !f) {
      set_cuda_error(e != cudaSuccess ? e : cudaErrorSymbolNotFound, "cudaGetDriverEntryPointByVersion(cuTensorMapEncodeTiled)");
      cudaGetLastError();
      return IBP_ECUDA;
    }
    fn = reinterpret_cast<Encode>(f);
    cache.store(fn, std::memory_order_release);
  }
  // (dimension, token, head, page); a stride that is never taken still has to be valid
  const cuuint64_t dims[4] = {a.dim, a.page_tokens, a.kv_heads, a.n_pages};
  const cuuint64_t token = v.token_stride;
  const cuuint64_t strides[3] = {token, a.kv_heads == 1 ? token : static_cast<cuuint64_t>(v.head_stride),
                                 a.n_pages == 1 ? token : static_cast<cuuint64_t>(v.page_stride)};
  const cuuint32_t boxes[4] = {64, box, 1, 1}, ones[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, a.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                        const_cast<char*>(v.data), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  *ok = r == CUDA_SUCCESS;
  return IBP_OK;
}

template <uint32_t DP, uint32_t MT, bool F16>
static int launch(TcArgs& t, const CUtensorMap& mk, const CUtensorMap& mv, int device, cudaStream_t stream) {
  using S = TcShape<DP, MT>;
  auto kern = k_kv_tree<DP, MT, F16>;
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
  int rc = kv_launch("k_kv_tree", kern, dim3(t.n_ctas), S::kThreads, S::kSmem, 1, stream, t, mk, mv);
  if (rc != IBP_OK || t.n_ctas == 1) return rc;
  const uint64_t rows = static_cast<uint64_t>(t.a.T) * t.a.group, most = rows < MT * kTcTile ? rows : MT * kTcTile;
  return kv_launch("k_kv_tree_join", k_kv_tree_join<DP, MT, F16>,
                   dim3(t.n_ctas - 1, static_cast<unsigned>((most + kJoinRows - 1) / kJoinRows)), kJoinThreads, 0, 1, stream, t);
}

static std::atomic<uint64_t> wait_limit{IBP_KV_WAIT_CYCLES};

uint64_t kv_tree_wait_limit(uint64_t cycles) { return wait_limit.exchange(cycles, std::memory_order_relaxed); }

int launch_kv_tree(const AttendArgs& a, int device, size_t ws_bytes, cudaStream_t stream, bool* done) {
  *done = false;
  const uint64_t rows = static_cast<uint64_t>(a.T) * a.group;
  // The softmax takes the maximum before it scales, so the scale has to be positive.
  const uint64_t tokens = static_cast<uint64_t>(a.max_pages) * a.page_tokens, sms = sm_count(device);
  if (!(a.scale_log2 > 0.f) || !tc_takes(a.n_seqs, a.kv_heads, rows, a.dim, a.page_tokens, tokens, device)) return IBP_OK;
  uint32_t box = 8;
  while (box < kTcTile && a.page_tokens % (2 * box) == 0) box *= 2;
  CUtensorMap mk, mv;
  bool ok = false;
  int rc = encode(&mk, a.k, a, box, &ok);
  if (rc == IBP_OK && ok) rc = encode(&mv, a.v, a, box, &ok);
  if (rc != IBP_OK || !ok) return rc;
  const uint32_t mt = tc_tiles(rows), dp = tc_dim(a.dim);
  TcArgs t = {};
  t.a = a;
  t.box = box;
  t.limit = static_cast<long long>(wait_limit.load(std::memory_order_relaxed));
  t.row_pairs = static_cast<uint32_t>((rows + mt * kTcTile - 1) / (mt * kTcTile));
  t.q16 = ((reinterpret_cast<uintptr_t>(a.q) | static_cast<uint64_t>(a.q_seq) | static_cast<uint64_t>(a.q_token) |
            static_cast<uint64_t>(a.q_head)) & 15u) == 0;
  const uint64_t tiles = (tokens + kTcTile - 1) / kTcTile * a.n_seqs * a.kv_heads * t.row_pairs;
  const uint64_t want = (tiles + kTcMinTiles - 1) / kTcMinTiles;
  const uint64_t n = sms;
  uint64_t ctas = want < sms ? want : sms;
  if (ctas > t.row_pairs) ctas -= ctas % t.row_pairs;
  t.n_ctas = static_cast<uint32_t>(ctas);
  char* w = reinterpret_cast<char*>(a.part);
  const size_t per = mt * kTcTile;
  t.first = reinterpret_cast<int4*>(w);
  w += align256((n + 1) * sizeof(int4));
  t.ml_part = reinterpret_cast<float2*>(w);
  w += align256(2 * n * per * sizeof(float2));
  t.o_part = reinterpret_cast<float*>(w);
  if (!a.part || ws_bytes < kv_tree_workspace(a.n_seqs, a.kv_heads, rows, a.dim, a.page_tokens, tokens, device))
    return IBP_EINVAL;
  *done = true;
  auto go = [&](auto f16) {
    constexpr bool F = decltype(f16)::value;
    if (dp == 64)
      return mt == 1 ? launch<64, 1, F>(t, mk, mv, device, stream) : launch<64, 2, F>(t, mk, mv, device, stream);
    return mt == 1 ? launch<128, 1, F>(t, mk, mv, device, stream) : launch<128, 2, F>(t, mk, mv, device, stream);
  };
  return a.f16 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace ibp

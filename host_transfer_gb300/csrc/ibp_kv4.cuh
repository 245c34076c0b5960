// ibp_kv4.cuh - paged caches held in 4 bits: views, arguments and decoding.
//
// A group of 32 elements of a token and head is 32 codes c of 4 bits and one scale
// s of the cache's type with 5 significant bits; an element stands for (c - 8) s.
// A whole number of 3 bits times 5 bits has 8, so bfloat16 and half precision hold
// every element exactly: the tensor cores' operands are the cache's values, with
// no rounding between.
#pragma once

#include "ibp_kv_mma.cuh"

namespace ibp {

constexpr uint32_t kQuadGroup = 32;  // elements that share a scale

struct Kv4View {  // K or V pages of one layer; strides in bytes
  const char* codes;
  int64_t page_stride, head_stride, token_stride;
  const char* scales;
  int64_t s_page, s_head, s_token;
};

struct Kv4Rows {  // arguments of the storing and loading kernels
  Kv4View p[2];           // K and V
  const char* x[2];       // rows: n_seqs x T x heads x dim
  int64_t x_seq[2], x_token[2], x_head[2];  // bytes
  const int32_t* table;
  const int32_t* lens;
  const int32_t* n_rows;  // rows per sequence, or nullptr: T
  uint32_t n_seqs, max_pages, n_pages, page_tokens, T, heads, dim;
  uint32_t f16;
  uint32_t vec;           // rows may be read and written 16 bytes at a time
  int32_t shift;          // set by the launch: pages of 2^shift tokens, or -1
  uint32_t loops;         // and rounds of tokens a block
  uint32_t* status;
};

int launch_kv4_store(const Kv4Rows& r, int device, cudaStream_t stream);
int launch_kv4_load(const Kv4Rows& r, int device, cudaStream_t stream);

struct Attend4Args {
  AttendArgs a;    // k and v are not used
  Kv4View k, v;
  int32_t shift;   // pages of 2^shift tokens, or -1
};

size_t kv4_attend_workspace(uint32_t n_seqs, uint32_t kv_heads, uint64_t rows, uint32_t dim, uint64_t tokens, int device);
int launch_kv4_attend(const Attend4Args& x, int device, size_t ws_bytes, cudaStream_t stream);

// The tensor-core kernel on codes (ibp_kv4_tree.cu): positive scales only.
bool kv4_tree_takes(uint32_t n_seqs, uint32_t kv_heads, uint64_t rows, uint32_t dim, uint64_t tokens, int device);
size_t kv4_tree_workspace(uint32_t dim, int device);
int launch_kv4_tree(const Attend4Args& x, int device, size_t ws_bytes, cudaStream_t stream);

// Decodes every sequence into pages of kExpand tokens (page b * ceil(tokens / kExpand) + j
// of sequence b), with a table and lengths that say so.
constexpr uint32_t kExpand = 128;
struct Kv4Expanded {
  int32_t* table;
  int32_t* lens;
  char* k;
  char* v;
};
size_t kv4_expand_workspace(uint32_t n_seqs, uint64_t tokens, uint32_t heads, uint32_t dim);
int launch_kv4_expand(const Attend4Args& x, const Kv4Expanded& e, int device, cudaStream_t stream);

namespace quad {

// A scale as `odd` and `value` take it, in the low half.  bfloat16: 5 significant bits
// (the rest are ignored), and not a number from 2^122 on, where 24 s may overflow.
template <bool F16>
__device__ __forceinline__ uint32_t scale_bits(uint32_t s) {
  if (F16) return s;
  s &= 0xFFF8u;
  return (s & 0x7FFFu) >= 0x7C80u ? 0x7FC0u : s;
}

// Whether a code times the scale may be something other than a finite number.
template <bool F16>
__device__ __forceinline__ bool odd(uint32_t s) {
  return F16 ? (s & 0x7FFFu) > 0x6FFFu : (s & 0x7FFFu) > 0x7F80u;  // half precision: above 8188, or NaN
}

template <bool F16>
__device__ __forceinline__ float to_float(uint32_t half) {
  if (!F16) return __uint_as_float(half << 16);
  float f;
  asm("{\n.reg .b16 h;\nmov.b32 {h, _}, %1;\ncvt.f32.f16 %0, h;\n}" : "=f"(f) : "r"(half));
  return f;
}

// What element i of a word of codes stands for, as a float that the type holds
// (half precision: or that it rounds to infinity).
template <bool F16>
__device__ __forceinline__ float value(uint32_t word, uint32_t i, uint32_t scale) {
  const float c = static_cast<float>(static_cast<int>((word >> (4 * i)) & 15u) - 8);
  const float v = __fmul_rn(c, to_float<F16>(scale));
  return F16 ? to_float<true>(pack2<true>(v, 0.f) & 0xFFFFu) : v;
}

// A pair of scales as read, and what the decoding adds.  bfloat16: 64 s is infinite from
// 2^122 on, and then everything decoded is NaN; the products with 1 / 64 and
// -24 / 64 are exact for 5 bits.  `keep` 0 makes the group zeros.
template <bool F16>
struct Pair {
  uint32_t s, m;
  __device__ __forceinline__ explicit Pair(uint32_t both, bool keep = true) {
    if (F16) {
      s = keep ? both : 0u;
      m = 0xCE00CE00u;  // -24
    } else {
      uint32_t w;
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(both & (keep ? 0xFFF8FFF8u : 0u)), "r"(0x42804280u));  // 64
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(s) : "r"(w), "r"(0x3C803C80u));
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(w), "r"(0xBEC0BEC0u));
    }
  }
};

// The constants of a decoding, kept in registers: with two immediates a mask with the
// exponent put in would be two instructions.
template <bool F16>
struct Magic {
  uint32_t mask, one;
  __device__ __forceinline__ Magic() {
    asm volatile("mov.u32 %0, %1;" : "=r"(mask) : "n"(F16 ? 0x03C003C0 : 0x00780078));
    asm volatile("mov.u32 %0, %1;" : "=r"(one) : "n"(F16 ? 0x4C004C00 : 0x41804180));
  }
};

// Elements I and I + 4 of a word (the codes at bits 4 I and 16 + 4 I) as a pair of
// 16-bit floats.  The code becomes the mantissa of a number between 16 and 32.
// bfloat16: (16 + c) s - 24 s in one fused operation, exact since the result is
// representable.  Half precision, where 24 s may overflow: ((16 + c) - 24) s.
template <bool F16, int I>
__device__ __forceinline__ uint32_t decode(uint32_t w, const Pair<F16>& p, const Magic<F16>& c) {
  uint32_t r;
  if (F16) {
    r = I == 0 ? w << 6 : (I == 1 ? w << 2 : (I == 2 ? w >> 2 : w >> 6));
    asm("lop3.b32 %0, %0, %1, %2, 0xEA;" : "+r"(r) : "r"(c.mask), "r"(c.one));
    asm("add.rn.f16x2 %0, %0, %1;" : "+r"(r) : "r"(p.m));
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(r) : "r"(p.s));
  } else {
    r = I == 0 ? w << 3 : (I == 1 ? w >> 1 : (I == 2 ? w >> 5 : w >> 9));
    asm("lop3.b32 %0, %0, %1, %2, 0xEA;" : "+r"(r) : "r"(c.mask), "r"(c.one));
    asm("fma.rn.bf16x2 %0, %0, %1, %2;" : "+r"(r) : "r"(p.s), "r"(p.m));
  }
  return r;
}

}  // namespace quad

}  // namespace ibp

// AdamW over a list of tensors, for sm_103a, with first and second moments in
// FP32 or in 8 bits.
//
//   g' = g * grad_scale
//   m' = b1 m + (1 - b1) g',   v' = b2 v + (1 - b2) g'^2,   r' = sqrt(v')
//   p' = p (1 - lr wd) - (lr / (1 - b1^t)) m' / (r' / sqrt(1 - b2^t) + eps)
//
// 8 bits: m and r = sqrt(v) are held as E4M3 codes with one UE8M0 scale 2^e
// for each 128 elements, e the smallest exponent that brings the block's
// largest magnitude to 448 or below.  r instead of v, because E4M3 spans 18
// powers of two and v would need twice as many as r.  Codes are rounded up
// with probability equal to the part cut off: E4M3 steps are 6 to 12 % apart
// while v moves by 0.1 % a step, so rounding to nearest would hold v where it
// is.  This rounding is right on average for each new code, and so for m, whose
// recursion is linear.  v's next step squares what is held, so steady gradients
// leave v 3 to 6 % high, and r with a spread (rms) of 12 to 17 %, whatever b2
// (normal gradients, b2 = 0.999: 4.3 % and 14.8 % measured).  The probability is
// decided by 16 bits of a hash of the element's index in its tensor, the tensor's
// place in the list and the caller's seed: the same call gives the same bits.  r
// above zero never becomes zero, which would leave m' / eps as the next update.
// The new moments enter the update before they are rounded.
//
// Every operation that a code depends on is a correctly rounded FP32
// operation in the order written above, so codes can be reproduced exactly;
// the division of the update alone is the approximate one (2 ulp of an update
// that is itself a small part of p).
//
// A code has its moment's sign, zeros included.  A non-finite moment is stored
// as NaN, code 0x7F, and takes no part in its block's scale.  A non-finite
// grad_scale leaves every tensor untouched: the usual answer to a gradient norm
// that overflowed.
//
// Bound by memory: per element 24 + g bytes with FP32 states (g = 4 or 2 bytes
// of gradient), 12 + 1/32 + g with 8-bit ones, and 2 for a BF16 copy.  201 M
// elements: 895 us with FP32 states and gradients and a copy (101 % of the copy
// rate); 517 us with 8-bit states, BF16 gradients and a copy (93 %), where 71
// instructions per element keep the schedulers two thirds busy as well.
//
// The list travels in the kernel's parameters (up to 32 KB of them), so a
// step is one launch for up to 448 tensors and nothing is copied or kept
// between calls.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "step_ops.h"

namespace dg {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 128;                 // elements of one scale
constexpr int kMinChunk = kBlock;           // elements of one warp's turn: a power of two
// chosen for the list (see launch_adamw); with 8-bit states at most a scale
// byte per lane
constexpr int kMaxChunk8 = 32 * kBlock, kMaxChunk32 = 8 * kBlock;

struct Entry {
  float *p;
  const void *g;
  void *m, *v;
  uint8_t *sm, *sv;
  __nv_bfloat16 *copy;
  int64_t n;
};

template <int kMax>
struct Params {
  AdamwHyper h;
  int n, tensor0;                           // entries, and the first one's place in the list
  int chunk;                                // elements of one warp's turn
  int64_t chunks;
  // Chunks of the entries before, apart from the entries: every CTA reads them
  // all (within the entries: 400 tensors of 1024 elements 12.8 us instead of 6.2).
  int chunk0[kMax];
  int place[kMax];                          // place in the list, less tensor0
  Entry e[kMax];
};

__device__ __forceinline__ float scale_value(uint32_t byte) {   // 2^(byte - 127)
  return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

__device__ __forceinline__ void decode4(uint32_t codes, float (&f)[4]) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(codes)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(codes >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;
// Bits of |x|, or 0 where x is not finite.
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = abs_bits(x);
  return b < kInfBits ? b : 0u;
}
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Bits of the largest |x|; at least kInfBits if one of them is not finite.
__device__ __forceinline__ uint32_t max4(const float (&x)[4]) {
  return __float_as_uint(max_nan(max_nan(fabsf(x[0]), fabsf(x[1])), max_nan(fabsf(x[2]), fabsf(x[3]))));
}
__device__ __forceinline__ uint32_t finite_max4(const float (&x)[4]) {
  return max(max(finite_bits(x[0]), finite_bits(x[1])), max(finite_bits(x[2]), finite_bits(x[3])));
}

// UE8M0 byte of the block's largest magnitude (its FP32 bits): 448 is
// 1.75 * 2^8, so a fraction above 0.75 (0x600000) carries into the exponent.
// Below 2^-126 * 2^8 the byte stays 0.
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits) {
  return static_cast<uint32_t>(max(static_cast<int>((bits + 0x1fffffu) >> 23) - 8, 0));
}

// E4M3 code of |x| 2^-e (at most 448), e = byte - 127, rounded up where r16 /
// 2^16 plus the part cut off reaches one.  Scaled down by another 2^120, E4M3's
// smallest normal number 2^-6 becomes FP32's, 2^-126, and FP32's subnormal
// numbers have E4M3's constant step below it: the code is then the FP32
// pattern from bit 20 up, in both ranges, and the 20 bits below are the part
// cut off.  `down` is 2^(7 - byte).
__device__ __forceinline__ uint32_t encode(float x, float down, uint32_t r16) {
  return (__float_as_uint(__fmul_rn(fabsf(x), down)) + (r16 << 4)) >> 20;
}

// 2^(7 - byte) for byte 0..133 (normal numbers).
constexpr uint32_t kMaxDownByte = 133;
__device__ __forceinline__ float down_of(uint32_t byte) { return __uint_as_float((134u - byte) << 23); }

// Hash of an element: two multiplications by odd constants (the fractional
// parts of the golden ratio and of sqrt 2), each followed by a shifted
// exclusive or.  `x` is (index + key) times the first constant.
constexpr uint32_t kMul1 = 0x9E3779B9u, kMul2 = 0x6A09E667u;
__device__ __forceinline__ uint32_t element_bits(uint32_t x, uint32_t turned) {
  uint32_t h = x ^ (x >> 16) ^ turned;
  h *= kMul2;
  return h ^ (h >> 15);
}

// One element's step: bm is b1 m, v in and out, m and r out.
__device__ __forceinline__ void update(const AdamwHyper &h, float g, float bm, float &p, float &m,
                                       float &v, float &r) {
  m = __fadd_rn(bm, __fmul_rn(h.a1, g));
  v = __fadd_rn(__fmul_rn(h.b2, v), __fmul_rn(h.a2, __fmul_rn(g, g)));
  r = __fsqrt_rn(v);
  // reciprocal within 1 ulp (a denominator below 2^-126, which needs eps = 0,
  // counts as zero)
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(fmaf(r, h.c2, h.eps)));
  p = fmaf(p, h.decay, -__fmul_rn(__fmul_rn(m, h.c1), inv));
}

// The arrays of a tensor from one lane's first element on.
template <bool kEight, bool kBf16Grad>
struct Lane {
  using G = std::conditional_t<kBf16Grad, uint16_t, float>;
  using S = std::conditional_t<kEight, uint8_t, float>;
  float *p;
  const G *g;
  S *m, *v;
  __nv_bfloat16 *copy;
  __device__ __forceinline__ Lane(const Entry &t, int64_t i)
      : p(t.p + i), g(static_cast<const G *>(t.g) + i), m(static_cast<S *>(t.m) + i),
        v(static_cast<S *>(t.v) + i), copy(t.copy == nullptr ? nullptr : t.copy + i) {}
  __device__ __forceinline__ void advance(int n) {
    p += n; g += n; m += n; v += n;
    if (copy != nullptr) copy += n;
  }
};

// What a lane holds of a block: four consecutive elements of each array, as
// they are loaded: load() waits for nothing, so that several blocks' loads
// are in flight at once.
template <bool kEight, bool kBf16Grad>
struct Four {
  using L = Lane<kEight, kBf16Grad>;
  float p[4], m[4], v[4];
  uint32_t gr[kBf16Grad ? 2 : 4];  // the gradient's bits
  uint32_t mc, vc;                 // 8 bits: the codes

  __device__ __forceinline__ void load(const L &t, int i) {
    const float4 a = *reinterpret_cast<const float4 *>(t.p + i);
    p[0] = a.x; p[1] = a.y; p[2] = a.z; p[3] = a.w;
    if constexpr (kBf16Grad) {
      const uint2 b = *reinterpret_cast<const uint2 *>(t.g + i);
      gr[0] = b.x; gr[1] = b.y;
    } else {
      const uint4 b = *reinterpret_cast<const uint4 *>(t.g + i);
      gr[0] = b.x; gr[1] = b.y; gr[2] = b.z; gr[3] = b.w;
    }
    if constexpr (kEight) {
      mc = *reinterpret_cast<const uint32_t *>(t.m + i);
      vc = *reinterpret_cast<const uint32_t *>(t.v + i);
    } else {
      const float4 b = *reinterpret_cast<const float4 *>(t.m + i);
      const float4 c = *reinterpret_cast<const float4 *>(t.v + i);
      m[0] = b.x; m[1] = b.y; m[2] = b.z; m[3] = b.w;
      v[0] = c.x; v[1] = c.y; v[2] = c.z; v[3] = c.w;
    }
  }
  // The first `left` of the four (none if it is not positive), zeros for the rest.
  __device__ __forceinline__ void load_part(const L &t, int i, int left) {
    mc = vc = gr[0] = gr[1] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = k < left;
      p[k] = in ? t.p[i + k] : 0.f;
      if constexpr (kBf16Grad)
        gr[k / 2] |= in ? static_cast<uint32_t>(t.g[i + k]) << (k & 1) * 16 : 0u;
      else
        gr[k] = in ? __float_as_uint(t.g[i + k]) : 0u;
      if constexpr (kEight) {
        mc |= in ? static_cast<uint32_t>(t.m[i + k]) << (8 * k) : 0u;
        vc |= in ? static_cast<uint32_t>(t.v[i + k]) << (8 * k) : 0u;
      } else {
        m[k] = in ? t.m[i + k] : 0.f;
        v[k] = in ? t.v[i + k] : 0.f;
      }
    }
  }
  __device__ __forceinline__ float grad(int k) const {
    if constexpr (kBf16Grad)
      return __uint_as_float(k & 1 ? gr[k / 2] & 0xffff0000u : gr[k / 2] << 16);
    else
      return __uint_as_float(gr[k]);
  }

  __device__ __forceinline__ void store(const L &t, int i) const {
    *reinterpret_cast<float4 *>(t.p + i) = make_float4(p[0], p[1], p[2], p[3]);
    if (t.copy != nullptr) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(p[0], p[1]), b = __floats2bfloat162_rn(p[2], p[3]);
      *reinterpret_cast<uint2 *>(t.copy + i) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                                          *reinterpret_cast<const uint32_t *>(&b));
    }
    if constexpr (kEight) {
      *reinterpret_cast<uint32_t *>(t.m + i) = mc;
      *reinterpret_cast<uint32_t *>(t.v + i) = vc;
    } else {
      *reinterpret_cast<float4 *>(t.m + i) = make_float4(m[0], m[1], m[2], m[3]);
      *reinterpret_cast<float4 *>(t.v + i) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
  __device__ __forceinline__ void store_part(const L &t, int i, int left) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= left) break;
      t.p[i + k] = p[k];
      if (t.copy != nullptr) t.copy[i + k] = __float2bfloat16_rn(p[k]);
      if constexpr (kEight) {
        t.m[i + k] = static_cast<uint8_t>(mc >> (8 * k));
        t.v[i + k] = static_cast<uint8_t>(vc >> (8 * k));
      } else {
        t.m[i + k] = m[k];
        t.v[i + k] = v[k];
      }
    }
  }

  // The step on the block whose lane this is (8 bits: the whole warp's);
  // `index` is the first element's.  Elements past the tensor's end hold zeros
  // and stay without effect on the block's scale.  sbyte: the new scale bytes,
  // m's in the low half.  bm: b1 times m's old scale, or, where that is below the
  // normal numbers and would lose bits, less that scale; vs: r's old scale.
  __device__ __forceinline__ void step(const AdamwHyper &h, float gs, uint32_t index, uint32_t key,
                                       float bm, float vs, uint32_t &sbyte) {
    float r[4];
    if constexpr (kEight) {
      decode4(mc, m);
      decode4(vc, v);
      if (bm < 0.f) {                                // warp-uniform; blocks of zeros, all but always
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = __fmul_rn(m[k], -bm);
        bm = h.b1;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (kEight) {
        v[k] = __fmul_rn(v[k], vs);
        v[k] = __fmul_rn(v[k], v[k]);
      }
      update(h, __fmul_rn(grad(k), gs), __fmul_rn(bm, m[k]), p[k], m[k], v[k], r[k]);
    }
    if constexpr (kEight) {
      uint32_t mb = __reduce_max_sync(0xffffffffu, max4(m));
      uint32_t rb = __reduce_max_sync(0xffffffffu, max4(r));
      const bool odd = max(mb, rb) >= kInfBits;      // something is not finite (warp-uniform)
      if (odd) {
        mb = __reduce_max_sync(0xffffffffu, finite_max4(m));
        rb = __reduce_max_sync(0xffffffffu, finite_max4(r));
      }
      const uint32_t mbyte = scale_byte(mb), rbyte = scale_byte(rb);
      sbyte = mbyte | rbyte << 16;
      uint32_t cm[4], cr[4];
      const uint32_t x = (index + key) * kMul1, turned = __funnelshift_l(key, key, 16);
      const float md = down_of(min(mbyte, kMaxDownByte)), rd = down_of(min(rbyte, kMaxDownByte));
      if (max(mbyte, rbyte) <= kMaxDownByte) {       // warp-uniform, and all but always
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t bits = element_bits(x + k * kMul1, turned);
          cm[k] = encode(m[k], md, bits >> 16);
          cr[k] = encode(r[k], rd, bits & 0xffffu);
        }
      } else {                                       // the rest of a larger block's scale first
        const float ms = scale_value(127u - (mbyte - min(mbyte, kMaxDownByte)));
        const float rs = scale_value(127u - (rbyte - min(rbyte, kMaxDownByte)));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t bits = element_bits(x + k * kMul1, turned);
          cm[k] = encode(__fmul_rn(m[k], ms), md, bits >> 16);
          cr[k] = encode(__fmul_rn(r[k], rs), rd, bits & 0xffffu);
        }
      }
      uint32_t sign = __byte_perm(__byte_perm(__float_as_uint(m[0]), __float_as_uint(m[1]), 0x0073),
                                  __byte_perm(__float_as_uint(m[2]), __float_as_uint(m[3]), 0x0073),
                                  0x5410);
      if (odd) {                                     // NaN is one code, without a sign
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (abs_bits(m[k]) >= kInfBits) {
            cm[k] = 0x7f;
            sign &= ~(0x80u << (8 * k));
          }
          if (abs_bits(r[k]) >= kInfBits) cr[k] = 0x7f;
        }
      }
      mc = (cm[0] + cm[1] * 0x100u + cm[2] * 0x10000u + cm[3] * 0x1000000u) | (sign & 0x80808080u);
      vc = cr[0] + cr[1] * 0x100u + cr[2] * 0x10000u + cr[3] * 0x1000000u;
      if ((vc - 0x01010101u) & ~vc & 0x80808080u) {  // a zero among the codes
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (cr[k] == 0 && r[k] > 0.f) vc |= 1u << (8 * k);
      }
    }
  }
};

// A warp takes a chunk (a.chunk consecutive elements of one tensor, at most
// one block per lane) at a time, two blocks together so that their loads are
// in flight at once, four consecutive elements per lane.
// The chunk's scale bytes come and go together, one per lane.
template <int kMax, bool kEight, bool kBf16Grad>
__global__ void __launch_bounds__(kThreads, kEight ? 4 : 1)
    adamw_kernel(const __grid_constant__ Params<kMax> a) {
  kernel_begin();
  constexpr int kU = 2;
  __shared__ int first[kMax];               // first chunk of each entry
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float gs = 1.f;
  if (a.h.grad_scale != nullptr) {
    gs = *a.h.grad_scale;
    if (!isfinite(gs)) return;
  }
  for (int i = threadIdx.x; i < a.n; i += kThreads) first[i] = a.chunk0[i];
  __syncthreads();
  for (int64_t c = static_cast<int64_t>(blockIdx.x) * kWarps + w; c < a.chunks;
       c += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int chunk = static_cast<int>(c);
    int lo = 0, hi = a.n - 1;               // the entry that owns the chunk
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    const Entry &e = a.e[lo];
    const int64_t base = static_cast<int64_t>(chunk - first[lo]) * a.chunk;
    const int len = static_cast<int>(min(static_cast<int64_t>(a.chunk), e.n - base));
    // (elements 2^32 apart share their bits)
    const uint32_t key = a.h.seed * 0x9E3779B9u +
                         static_cast<uint32_t>(a.tensor0 + a.place[lo]) * 0xBB67AE85u;
    Lane<kEight, kBf16Grad> t(e, base + lane * 4);
    uint32_t index = static_cast<uint32_t>(base) + lane * 4;
    // lane b: what block b's old scales give, and its new scale bytes
    float bm = a.h.b1, vs = 1.f;
    uint32_t s_new = 0;
    const bool has_block = lane * kBlock < len;
    if constexpr (kEight) {
      if (has_block) {
        const float s = scale_value(e.sm[base / kBlock + lane]);
        bm = __fmul_rn(a.h.b1, s);          // exact where it is a normal number
        if (bm < 0x1p-126f) bm = -s;
        vs = scale_value(e.sv[base / kBlock + lane]);
      }
    }
    int i0 = 0;
    // kN blocks from i0 on: whole ones, or (kPart) one that ends early
    auto blocks = [&](auto n_c, auto part_c) {
      constexpr int kN = decltype(n_c)::value;
      constexpr bool kPart = decltype(part_c)::value;
      Four<kEight, kBf16Grad> f[kN];
#pragma unroll
      for (int u = 0; u < kN; ++u) {
        if constexpr (kPart) f[u].load_part(t, 0, len - i0 - lane * 4);
        else f[u].load(t, u * kBlock);
      }
#pragma unroll
      for (int u = 0; u < kN; ++u) {
        const int b = i0 / kBlock + u;
        uint32_t sbyte = 0;
        f[u].step(a.h, gs, index + u * kBlock, key, kEight ? __shfl_sync(0xffffffffu, bm, b) : bm,
                  kEight ? __shfl_sync(0xffffffffu, vs, b) : vs, sbyte);
        if (lane == b) s_new = sbyte;
        if constexpr (kPart) f[u].store_part(t, 0, len - i0 - lane * 4);
        else f[u].store(t, u * kBlock);
      }
      t.advance(kN * kBlock);
      index += kN * kBlock;
      i0 += kN * kBlock;
    };
    using std::integral_constant;
    while (len - i0 >= kU * kBlock) blocks(integral_constant<int, kU>{}, std::false_type{});
    while (len - i0 >= kBlock) blocks(integral_constant<int, 1>{}, std::false_type{});
    if (len > i0) blocks(integral_constant<int, 1>{}, std::true_type{});
    if constexpr (kEight) {
      if (has_block) {
        e.sm[base / kBlock + lane] = static_cast<uint8_t>(s_new);
        e.sv[base / kBlock + lane] = static_cast<uint8_t>(s_new >> 16);
      }
    }
  }
}

// Two sizes of the parameter block: most of a short list's launch would
// otherwise be the copying of empty entries.
constexpr int kShort = 48, kLong = 448;
static_assert(sizeof(Params<kLong>) <= 32764, "kernel parameters");
static_assert(sizeof(Params<kShort>) <= 4096, "kernel parameters");

template <int kMax>
cudaError_t run_part(const Params<kMax> &a, bool eight, bool bf16, int sms, cudaStream_t stream) {
  const int blocks = static_cast<int>(std::min<int64_t>((a.chunks + kWarps - 1) / kWarps, 8ll * sms));
  const auto kernel = eight ? (bf16 ? adamw_kernel<kMax, true, true> : adamw_kernel<kMax, true, false>)
                            : (bf16 ? adamw_kernel<kMax, false, true> : adamw_kernel<kMax, false, false>);
  return launch_step(kernel, blocks, kThreads, 0, stream, 1, a);
}

// Fills the parameters from list[at...]; returns the first entry not taken.
template <int kMax>
int fill(Params<kMax> &a, const dg_adamw_tensor *list, int n, int at, int chunk) {
  a.n = 0;
  a.chunk = chunk;
  a.tensor0 = at;
  a.chunks = 0;
  for (; at < n && a.n < kMax; ++at) {
    const dg_adamw_tensor &t = list[at];
    if (t.n == 0) continue;
    Entry &e = a.e[a.n];
    e.p = t.p;
    e.g = t.g;
    e.m = t.m;
    e.v = t.v;
    e.sm = t.sm;
    e.sv = t.sv;
    e.copy = static_cast<__nv_bfloat16 *>(t.copy);
    e.n = t.n;
    const int64_t more = (t.n + chunk - 1) / chunk;
    if (a.chunks + more > 0x7FFFFFFF) break;         // chunk numbers are 32 bits: next launch
    a.chunk0[a.n] = static_cast<int>(a.chunks);
    a.place[a.n++] = at - a.tensor0;
    a.chunks += more;
  }
  return at;
}

}  // namespace

cudaError_t launch_adamw(const dg_adamw_tensor *list, int n, const AdamwHyper &h, bool eight,
                         bool bf16_grad, int sms, cudaStream_t stream) {
  int live = 0;
  int64_t elements = 0;
  for (int i = 0; i < n; ++i) {
    live += list[i].n > 0;
    elements += list[i].n;
  }
  // One block per turn while the list gives fewer turns than warps fit the
  // device, then longer ones, which share the search for the entry.
  int chunk = kMinChunk;
  while (chunk < (eight ? kMaxChunk8 : kMaxChunk32) && elements / chunk > 64ll * sms) chunk *= 2;
  for (int at = 0; at < n;) {
    cudaError_t e = cudaSuccess;
    if (live <= kShort) {
      Params<kShort> a;
      a.h = h;
      at = fill(a, list, n, at, chunk);
      live -= a.n;
      if (a.n > 0) e = run_part(a, eight, bf16_grad, sms, stream);
    } else {
      static thread_local Params<kLong> a;
      a.h = h;
      at = fill(a, list, n, at, chunk);
      live -= a.n;
      if (a.n > 0) e = run_part(a, eight, bf16_grad, sms, stream);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dg

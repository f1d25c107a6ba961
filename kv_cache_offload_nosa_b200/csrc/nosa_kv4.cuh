// The 4-bit K/V cache (kv_bits = 4): its format, and the kernels that write and read it.
//
// A row (the d values of one token and KV head) is cut in groups of 32 values. A group holds a
// bf16 scale and one 4-bit code per value:
//   a = max |x|,  s = bf16(a / 7) (nearest, ties to even),  c = 8 + sign(x) floor(|x| / s + 1/2),
// so a value reads back as (c - 8) s, with c in 1..15 and |error| <= s / 2 (plus what the
// rounding of s moves the largest value: less than s / 16). Groups with s < 2^-126 are stored as
// zeros (s = 0, c = 8); a group that holds an infinity or a NaN gets s = NaN and reads back NaN.
// 9/16 byte a value against bf16's 2.
//
// Exactness of the codes: x and s have 8-bit significands X and S, so |x| / s either is a half
// integer exactly or differs from every half integer in [1/2, 7] by at least 2^-12 of it. One
// fused multiply-add with (1/s)(1 + 2^-20), whose own rounding is below 2^-22, therefore rounds
// every value to the code above, halves away from zero included, without a division per value.
//
// A page holds one block of one group of heads: [bs][d/2] bytes of codes, then [bs][d/32] scales.
// The order of the codes in a row is the order in which the attention's matrix fragments take
// them, so that it unpacks a whole register with one mask and no shuffle:
//   K row: the 32-bit word at byte c*(d/8) + 4g holds values 32g + 8c + 0..7  (c = 0..3),
//   V row: the 16-bit word at byte r*(d/16) + 2g holds values 32g + 4r + 0..3 (r = 0..7),
// lowest bits first. Rows are independent, so a token is written without reading its page.
#pragma once

#include "nosa_common.cuh"

namespace nosa {

__host__ __device__ constexpr int kv4_page_bytes(int bs, int d) { return bs * (d / 2 + d / 16); }

// bf16 bits of the scale of a group whose largest magnitude has the bf16 bits `amax`. The product
// with 1/7 is within 2^-23 of a/7, which is at least 2^-12 away from a rounding border.
__device__ __forceinline__ uint32_t kv4_scale(uint32_t amax) {
  if (amax >= 0x7f80u) return 0x7fffu;
  const float s = __uint_as_float(amax << 16) * (1.0f / 7.0f);
  const uint32_t b = __bfloat16_as_ushort(__float2bfloat16_rn(s));
  return b < 0x0080u ? 0u : b;  // below 2^-126
}
// The multiplier that takes a value to its code minus 8.
__device__ __forceinline__ float kv4_inverse(uint32_t scale) {
  float r;  // within 2^-23 (s is normal, 2^-126 to 2^125.2, and so is its reciprocal)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__uint_as_float(scale << 16)));
  return scale == 0u ? 0.f : r * (1.0f + 0x1p-20f);
}
// 0x4b400000 + code: the sum's last place is 1, so its low bits are the rounded integer.
__device__ __forceinline__ uint32_t kv4_code(float x, float inv) {
  return __float_as_uint(fmaf(x, inv, 12582912.f + 8.f)) & 15u;
}

// Byte of a page that holds the code of value x of row r, and the value itself.
template <bool KEYS, int D>
__device__ __forceinline__ int kv4_code_byte(int row, int x) {
  const int g = x >> 5;
  return KEYS ? row * (D / 2) + ((x >> 3) & 3) * (D / 8) + 4 * g + ((x & 7) >> 1)
              : row * (D / 2) + ((x >> 2) & 7) * (D / 16) + 2 * g + ((x & 3) >> 1);
}
template <bool KEYS, int D>
__device__ __forceinline__ float kv4_value(const uint8_t* page, int bs, int row, int x) {
  const int code = (__ldcg(page + kv4_code_byte<KEYS, D>(row, x)) >> (4 * (x & 1))) & 15;
  const uint16_t s = __ldcg(reinterpret_cast<const uint16_t*>(page + bs * (D / 2) + row * (D / 16)) + (x >> 5));
  return static_cast<float>(code - 8) * bf16_bits_to_f32(s);
}

// ------------------------------------------------------------------ runs of tokens
struct KvRunArgs {
  uint16_t* k;               // rows of the run, [n_tokens][Hkv][d] with the strides below
  uint16_t* v;
  long long k_tok, k_head, v_tok, v_head;  // in values
  int n_tokens, B, Hkv;
  const int32_t* cu_tokens;  // [B + 1] first token of each sequence in the run
  const int32_t* start;      // [B] position of each sequence's first token, or NULL: 0
  uint8_t* k_pages;          // [B*Hkv][pages_per_group] pages, block j at page j of its group
  uint8_t* v_pages;
  int pages_per_group, bs, max_tokens;
  uint32_t* err;
};

// A CTA takes TOKENS tokens of one KV head (the heads of the same tokens are neighbouring CTAs, so
// that a token-major row is read by CTAs that run together); TPR threads a row for 8 values each.
template <int D>
struct KvRun {
  static constexpr int TPR = D / 8;            // threads per row
  static constexpr int THREADS = 256;
  static constexpr int RPP = THREADS / TPR;    // rows per pass
  static constexpr int U = 4;                  // passes, all in flight at once
  static constexpr int TOKENS = RPP * U;
};

// Sequences whose bounds are kept in shared memory; past them the search reads cu_tokens itself.
constexpr int kKvRunSeqs = 256;

// Page (of its pool, -1: none) and row of every token of the CTA: its sequence by binary search in
// cu_tokens. A token of no sequence, or with a position outside the cache, has none.
template <int D>
__device__ __forceinline__ void kv_run_places(const KvRunArgs& a, int t0, int h, int2* place) {
  __shared__ int cu_s[kKvRunSeqs + 1], start_s[kKvRunSeqs];
  const bool small = a.B <= kKvRunSeqs;
  if (small) {
    for (int i = threadIdx.x; i <= a.B; i += blockDim.x) {
      cu_s[i] = a.cu_tokens[i];
      if (i < a.B) start_s[i] = a.start ? a.start[i] : 0;
    }
    __syncthreads();
  }
  const int shift = 31 - __clz(a.bs);  // bs is a power of two
  for (int i = threadIdx.x; i < KvRun<D>::TOKENS; i += blockDim.x) {
    const int t = t0 + i;
    int lo = 0, hi = a.B - 1;  // the last b with cu_tokens[b] <= t, if any
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((small ? cu_s[mid] : a.cu_tokens[mid]) <= t) lo = mid;
      else hi = mid - 1;
    }
    int2 at = make_int2(-1, 0);
    const int c0 = small ? cu_s[lo] : a.cu_tokens[lo], c1 = small ? cu_s[lo + 1] : a.cu_tokens[lo + 1];
    if (t >= c0 && t < c1 && t < a.n_tokens) {
      const long long p = (long long)(small ? start_s[lo] : a.start ? a.start[lo] : 0) + t - c0;
      if (p >= 0 && p < a.max_tokens)
        at = make_int2((lo * a.Hkv + h) * a.pages_per_group + (static_cast<int>(p) >> shift),
                       static_cast<int>(p) & (a.bs - 1));
      else
        set_err(a.err, NOSA_ERR_FULL);
    }
    place[i] = at;
  }
  __syncthreads();
}

__device__ __forceinline__ uint32_t max_abs_bf162(uint32_t x, uint32_t y) {  // per half, NaN if either is
  const __nv_bfloat162 m = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&x)),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&y)));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// The code words of 16 values (pairs of consecutive ones) and the scale of their group, whose other
// half the neighbouring lane holds. A code is the low bits of 0x4b400000 + code; the words of eight
// add up in base 16, and their constant parts to a constant.
__device__ __forceinline__ uint2 kv4_pack(const uint4* x, uint32_t* scale) {
  const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  uint32_t m = max_abs_bf162(w[0], w[1]);
#pragma unroll
  for (int i = 2; i < 8; ++i) m = max_abs_bf162(m, w[i]);
  m = max_abs_bf162(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max_abs_bf162(m, __byte_perm(m, m, 0x1032));
  *scale = kv4_scale(m & 0xffffu);
  const float inv = kv4_inverse(*scale);
  uint32_t word[2] = {0u, 0u};
#pragma unroll
  for (int i = 15; i >= 0; --i) {
    const float v = __uint_as_float((i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    word[i / 8] = word[i / 8] * 16u + __float_as_uint(fmaf(v, inv, 12582912.f + 8.f));
  }
  constexpr uint32_t BASE = 0x4b400000u * 0x11111111u;
  return make_uint2(word[0] - BASE, word[1] - BASE);
}

// Writes K and V rows into their pages, 16 values of each per thread. Issue slots bound it before
// memory does: four sequences of 32768 tokens x 8 heads (d = 128) take 198 us with eight values per
// thread and index divisions per row (83 % of the slots used), 128 us without the divisions, 106 us
// with 16 values, so that the scale is found by two threads instead of four (6.5 TB/s).
template <int D>
__global__ void __launch_bounds__(256) kv4_write_kernel(KvRunArgs a) {
  using R = KvRun<D>;
  constexpr int TPR = D / 16, RPP = R::THREADS / TPR, U = R::TOKENS / RPP;
  __shared__ int2 place[R::TOKENS];
  const int h = blockIdx.x % a.Hkv, t0 = blockIdx.x / a.Hkv * R::TOKENS;
  const int i0 = threadIdx.x / TPR, sub = threadIdx.x % TPR, g = sub >> 1, half = sub & 1;
  uint4 kx[U][2], vx[U][2];
  {
    const uint16_t* kr = a.k + (size_t)(t0 + i0) * a.k_tok + (size_t)h * a.k_head + 16 * sub;
    const uint16_t* vr = a.v + (size_t)(t0 + i0) * a.v_tok + (size_t)h * a.v_head + 16 * sub;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        kx[u][j] = vx[u][j] = make_uint4(0, 0, 0, 0);
        if (t0 + i0 + u * RPP < a.n_tokens) {
          kx[u][j] = __ldcs(reinterpret_cast<const uint4*>(kr + u * (size_t)RPP * a.k_tok) + j);
          vx[u][j] = __ldcs(reinterpret_cast<const uint4*>(vr + u * (size_t)RPP * a.v_tok) + j);
        }
      }
  }
  kv_run_places<D>(a, t0, h, place);
  const size_t PB = kv4_page_bytes(a.bs, D);
  const bool odd = g & 1;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t ks, vs;
    const uint2 kw = kv4_pack(kx[u], &ks), w = kv4_pack(vx[u], &vs);
    // V: a thread's words hold r = 4 half + 0, 1 and + 2, 3 of group g. The thread of the other group
    // of a pair takes one of the words and gives its other, so that each stores two times 4 bytes.
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w.x : w.y, 2);
    const uint32_t lo = odd ? got : w.x, hi = odd ? w.y : got;  // even group, odd group
    const int2 at = place[i0 + u * RPP];
    if (at.x >= 0) {
      uint8_t* kp = a.k_pages + at.x * PB;
      uint8_t* vp = a.v_pages + at.x * PB;
      uint8_t* kc = kp + at.y * (D / 2) + 2 * half * (D / 8) + 4 * g;
      uint8_t* vc = vp + at.y * (D / 2) + (4 * half + 2 * odd) * (D / 16) + 4 * (g >> 1);
      *reinterpret_cast<uint32_t*>(kc) = kw.x;
      *reinterpret_cast<uint32_t*>(kc + D / 8) = kw.y;
      *reinterpret_cast<uint32_t*>(vc) = __byte_perm(lo, hi, 0x5410);
      *reinterpret_cast<uint32_t*>(vc + D / 16) = __byte_perm(lo, hi, 0x7632);
      *(reinterpret_cast<uint16_t*>((half ? vp : kp) + a.bs * (D / 2) + at.y * (D / 16)) + g) =
          static_cast<uint16_t>(half ? vs : ks);
    }
  }
}

// Eight codes of a word as bf16 values (c - 8) s, in pairs of consecutive values: 128 + c is a
// bf16 with the code in its low bits, the difference is exact and the product rounds once.
__device__ __forceinline__ uint4 kv4_unpack(uint32_t w, uint32_t scale) {
  const uint32_t s2 = scale | (scale << 16);
  const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&s2);
  const __nv_bfloat162 off = __floats2bfloat162_rn(136.f, 136.f);
  uint32_t p[4];  // values (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 y = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), off), s);
    p[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                    __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632));
}

// Reads rows back as bf16, 8 values of K and of V per thread. Bound by memory once enough CTAs are
// resident to cover the two round trips (places, codes) before the stores: the sequences above take
// 114 us with 48 registers (five CTAs an SM), 111 us with 40 (six), 119 us with 32 (eight).
template <int D>
__global__ void __launch_bounds__(256, 6) kv4_read_kernel(KvRunArgs a) {
  using R = KvRun<D>;
  __shared__ int2 place[R::TOKENS];
  const int h = blockIdx.x % a.Hkv, t0 = blockIdx.x / a.Hkv * R::TOKENS;
  const int i0 = threadIdx.x / R::TPR, sub = threadIdx.x % R::TPR, g = sub >> 2, c = sub & 3;
  const bool odd = g & 1;
  kv_run_places<D>(a, t0, h, place);
  const size_t PB = kv4_page_bytes(a.bs, D);
  uint32_t kw[R::U], vw[R::U], ks[R::U], vs[R::U];
  bool any[R::U];
#pragma unroll
  for (int u = 0; u < R::U; ++u) {
    kw[u] = vw[u] = ks[u] = vs[u] = 0u;
    const int2 at = place[i0 + u * R::RPP];
    any[u] = at.x >= 0;
    if (any[u]) {
      const uint8_t* kp = a.k_pages + at.x * PB;
      const uint8_t* vp = a.v_pages + at.x * PB;
      kw[u] = __ldcs(reinterpret_cast<const uint32_t*>(kp + at.y * (D / 2) + c * (D / 8) + 4 * g));
      vw[u] = __ldcs(
          reinterpret_cast<const uint32_t*>(vp + at.y * (D / 2) + (2 * c + odd) * (D / 16) + 4 * (g >> 1)));
      ks[u] = __ldcs(reinterpret_cast<const uint16_t*>(kp + a.bs * (D / 2) + at.y * (D / 16)) + g);
      vs[u] = __ldcs(reinterpret_cast<const uint16_t*>(vp + a.bs * (D / 2) + at.y * (D / 16)) + g);
    }
  }
  uint16_t* kr = a.k + (size_t)(t0 + i0) * a.k_tok + (size_t)h * a.k_head + 8 * sub;
  uint16_t* vr = a.v + (size_t)(t0 + i0) * a.v_tok + (size_t)h * a.v_head + 8 * sub;
#pragma unroll
  for (int u = 0; u < R::U; ++u) {
    // an even group's thread loaded r = 2c of groups g, g + 1; an odd one r = 2c + 1 of g - 1, g
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? vw[u] : vw[u] >> 16, 4);
    const uint32_t v = odd ? __byte_perm(got, vw[u], 0x7610) : __byte_perm(vw[u], got, 0x5410);
    if (any[u]) {
      __stcs(reinterpret_cast<uint4*>(kr + u * (size_t)R::RPP * a.k_tok), kv4_unpack(kw[u], ks[u]));
      __stcs(reinterpret_cast<uint4*>(vr + u * (size_t)R::RPP * a.v_tok), kv4_unpack(v, vs[u]));
    }
  }
}

}  // namespace nosa

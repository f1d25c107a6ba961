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

__host__ __device__ constexpr int kv4_row_bytes(int d) { return d / 2; }
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
  return (scale == 0u || scale == 0x7fffu) ? 0.f : __frcp_rn(__uint_as_float(scale << 16)) * (1.0f + 0x1p-20f);
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

// The tokens that one CTA's rows cover: their sequence and position, found by binary search in
// cu_tokens. pos < 0: the token belongs to no sequence, or its position is not in the cache.
template <int D>
struct KvRun {
  static constexpr int TPR = D / 8;            // threads per row, 8 values each
  static constexpr int THREADS = 256;
  static constexpr int RPP = THREADS / TPR;    // rows per pass
  static constexpr int U = 4;                  // passes, all in flight at once
  static constexpr int ROWS = RPP * U;
  static constexpr int TOKENS = ROWS + 1;      // tokens that ROWS rows can touch
};

template <int D>
__device__ __forceinline__ void kv_run_places(const KvRunArgs& a, int t0, int nt, int2* place) {
  for (int i = threadIdx.x; i < nt; i += blockDim.x) {
    const int t = t0 + i;
    int lo = 0, hi = a.B - 1;  // the last b with cu_tokens[b] <= t, if any
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.cu_tokens[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    int pos = -1;
    const int c0 = a.cu_tokens[lo];
    if (t >= c0 && t < a.cu_tokens[lo + 1]) {
      const long long p = (long long)(a.start ? a.start[lo] : 0) + (t - c0);
      if (p >= 0 && p < a.max_tokens) pos = static_cast<int>(p);
      else set_err(a.err, NOSA_ERR_FULL);
    }
    place[i] = make_int2(lo, pos);
  }
}

// Writes K and V rows into their pages: one thread takes 8 values of K and of V, four threads a
// group (its maximum by two shuffles). Bound by memory: 2 bytes in and 9/16 out a value.
template <int D>
__global__ void __launch_bounds__(256) kv4_write_kernel(KvRunArgs a) {
  using R = KvRun<D>;
  __shared__ int2 place[R::TOKENS];
  const int row0 = blockIdx.x * R::ROWS, rows = a.n_tokens * a.Hkv;  // below 2^31
  const int t0 = row0 / a.Hkv;
  const int sub = threadIdx.x % R::TPR, g = sub >> 2, c = sub & 3;
  uint4 kx[R::U], vx[R::U];
#pragma unroll
  for (int u = 0; u < R::U; ++u) {
    const int row = row0 + u * R::RPP + threadIdx.x / R::TPR;
    kx[u] = vx[u] = make_uint4(0, 0, 0, 0);
    if (row < rows) {
      const int t = row / a.Hkv, h = row % a.Hkv;
      kx[u] = __ldcs(reinterpret_cast<const uint4*>(a.k + t * a.k_tok + h * a.k_head) + sub);
      vx[u] = __ldcs(reinterpret_cast<const uint4*>(a.v + t * a.v_tok + h * a.v_head) + sub);
    }
  }
  const int last = min(row0 + R::ROWS, rows) - 1;
  kv_run_places<D>(a, t0, last / a.Hkv - t0 + 1, place);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < R::U; ++u) {
    const int row = row0 + u * R::RPP + threadIdx.x / R::TPR;
    uint32_t word[2], scale[2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint4 x = kv ? vx[u] : kx[u];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                            __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
      m = max(m & 0xffffu, m >> 16);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      scale[kv] = kv4_scale(m);
      const float inv = kv4_inverse(scale[kv]);
      word[kv] = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        word[kv] |= (kv4_code(__uint_as_float(w[i] << 16), inv) |
                     (kv4_code(__uint_as_float(w[i] & 0xffff0000u), inv) << 4)) << (8 * i);
    }
    // V: this thread's values are the words of r = 2c (low half) and r = 2c + 1 of group g; the
    // thread of the other group of a pair takes one of them, so that each stores 4 bytes
    const bool odd = g & 1;
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? word[1] & 0xffffu : word[1] >> 16, 4);
    const uint32_t vw = odd ? (got | (word[1] & 0xffff0000u)) : ((word[1] & 0xffffu) | (got << 16));
    if (row < rows) {
      const int2 p = place[row / a.Hkv - t0];
      if (p.y >= 0) {
        const int h = row % a.Hkv, r = p.y % a.bs;
        const size_t at = ((size_t)(p.x * a.Hkv + h) * a.pages_per_group + p.y / a.bs) * kv4_page_bytes(a.bs, D);
        uint8_t* kp = a.k_pages + at;
        uint8_t* vp = a.v_pages + at;
        *reinterpret_cast<uint32_t*>(kp + r * (D / 2) + c * (D / 8) + 4 * g) = word[0];
        *reinterpret_cast<uint32_t*>(vp + r * (D / 2) + (2 * c + odd) * (D / 16) + 4 * (g >> 1)) = vw;
        if (c < 2)
          *(reinterpret_cast<uint16_t*>((c ? vp : kp) + a.bs * (D / 2) + r * (D / 16)) + g) =
              static_cast<uint16_t>(c ? scale[1] : scale[0]);
      }
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

// Reads rows back as bf16: the write's layout of threads the other way round.
template <int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(KvRunArgs a) {
  using R = KvRun<D>;
  __shared__ int2 place[R::TOKENS];
  const int row0 = blockIdx.x * R::ROWS, rows = a.n_tokens * a.Hkv;  // below 2^31
  const int t0 = row0 / a.Hkv;
  const int sub = threadIdx.x % R::TPR, g = sub >> 2, c = sub & 3;
  const bool odd = g & 1;
  const int last = min(row0 + R::ROWS, rows) - 1;
  kv_run_places<D>(a, t0, last / a.Hkv - t0 + 1, place);
  __syncthreads();
  uint32_t kw[R::U], vw[R::U], ks[R::U], vs[R::U];
#pragma unroll
  for (int u = 0; u < R::U; ++u) {
    const int row = row0 + u * R::RPP + threadIdx.x / R::TPR;
    kw[u] = vw[u] = ks[u] = vs[u] = 0u;
    if (row < rows) {
      const int2 p = place[row / a.Hkv - t0];
      if (p.y >= 0) {
        const int h = row % a.Hkv, r = p.y % a.bs;
        const size_t at = ((size_t)(p.x * a.Hkv + h) * a.pages_per_group + p.y / a.bs) * kv4_page_bytes(a.bs, D);
        const uint8_t* kp = a.k_pages + at;
        const uint8_t* vp = a.v_pages + at;
        kw[u] = __ldcs(reinterpret_cast<const uint32_t*>(kp + r * (D / 2) + c * (D / 8) + 4 * g));
        vw[u] = __ldcs(reinterpret_cast<const uint32_t*>(vp + r * (D / 2) + (2 * c + odd) * (D / 16) + 4 * (g >> 1)));
        ks[u] = __ldcs(reinterpret_cast<const uint16_t*>(kp + a.bs * (D / 2) + r * (D / 16)) + g);
        vs[u] = __ldcs(reinterpret_cast<const uint16_t*>(vp + a.bs * (D / 2) + r * (D / 16)) + g);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < R::U; ++u) {
    const int row = row0 + u * R::RPP + threadIdx.x / R::TPR;
    // an even group's thread loaded r = 2c of groups g, g + 1; an odd one r = 2c + 1 of g - 1, g
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? vw[u] & 0xffffu : vw[u] >> 16, 4);
    const uint32_t v = odd ? (got | (vw[u] & 0xffff0000u)) : ((vw[u] & 0xffffu) | (got << 16));
    if (row < rows) {
      const int t = row / a.Hkv, h = row % a.Hkv;
      if (place[t - t0].y >= 0) {
        __stcs(reinterpret_cast<uint4*>(a.k + t * a.k_tok + h * a.k_head) + sub, kv4_unpack(kw[u], ks[u]));
        __stcs(reinterpret_cast<uint4*>(a.v + t * a.v_tok + h * a.v_head) + sub, kv4_unpack(v, vs[u]));
      }
    }
  }
}

}  // namespace nosa

// Split-K flash-decoding over the selected blocks of a 4-bit cache (kv_bits = 4).
//
// The tasks, their split over CTAs and the merge of the partials are those of the bf16 kernel:
// the B*Hkv*k (group, selected block) tasks, group after group, are cut in ranges of W, one range
// per CTA; each range writes one partial (m, l, acc) per query head and group it touches, and the
// last CTA to finish a group (atomic ticket) merges them.
#pragma once

#include "nosa_attn.cuh"
#include "nosa_kv4.cuh"

namespace nosa {

struct AttnKv4Args {
  AttnArgs a;
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  int bs;
  int pslots;  // partial slots per group
};

template <int D>
__global__ void __launch_bounds__(128) attn_kv4_kernel(AttnKv4Args x) {
  const AttnArgs& a = x.a;
  __shared__ float qs[8][D];
  __shared__ float p[8][128];
  __shared__ float red[4][8];
  __shared__ int s_L, s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = a.G, bs = x.bs;
  const int task0 = blockIdx.x * a.W, ntask = min(a.W, a.total - task0);
  const bool flags = a.sel_flag != nullptr;
  if (!flags) griddep_wait();
  const unsigned long long deadline = globaltimer() + a.wait_ns;
  const size_t PB = kv4_page_bytes(bs, D);
  const int GE = G * (D + 2);
  for (int t = 0; t < ntask;) {
    const int gi = (task0 + t) / a.k, pa = task0 + t - gi * a.k;
    const int pb = min(task0 + ntask, (gi + 1) * a.k) - gi * a.k;
    const int first = (int)(((long long)gi * a.k) / a.W);
    const int nseg = (int)(((long long)gi * a.k + a.k - 1) / a.W) - first + 1, seg = blockIdx.x - first;
    t += pb - pa;
    if (tid == 0) {
      if (flags && !wait_flag(a.sel_flag + (size_t)gi * kFlagStride, deadline)) set_err(a.err, NOSA_ERR_TIMEOUT);
      s_L = __ldcg(a.seq_len + gi);
    }
    for (int e = tid; e < G * D; e += 128)
      qs[e / D][e % D] = a.scale_log2 *
          bf16_bits_to_f32(a.q[((size_t)(gi / a.Hkv) * a.Hq + (gi % a.Hkv) * G + e / D) * D + e % D]);
    __syncthreads();
    const int L = s_L, N = (L + bs - 1) / bs;
    float acc[8], m[8], l[8];  // thread: one value of the row for every head
#pragma unroll
    for (int h = 0; h < 8; ++h) acc[h] = l[h] = 0.f, m[h] = -INFINITY;
    for (int i = pa; i < pb; ++i) {
      const int j = __ldcg(a.sel + (size_t)gi * a.k + i);
      if (j < 0) continue;
      const int page = j >= N ? -1 : a.identity ? gi * a.max_blocks + j
                                                : __ldcg(a.block_table + (size_t)gi * a.max_blocks + j);
      if (page < 0 || page >= a.total_pages) {
        if (tid == 0) set_err(a.err, j >= N ? NOSA_ERR_SEL : NOSA_ERR_BLOCK_TABLE);
        continue;
      }
      const uint8_t* kp = x.k_pages + page * PB;
      const uint8_t* vp = x.v_pages + page * PB;
      const int nval = min(bs, L - j * bs);
      float s[8];
#pragma unroll
      for (int h = 0; h < 8; ++h) s[h] = tid < nval ? 0.f : -INFINITY;
      if (tid < nval)
        for (int e = 0; e < D; ++e) {
          const float kv = kv4_value<true, D>(kp, bs, tid, e);
#pragma unroll
          for (int h = 0; h < 8; ++h)
            if (h < G) s[h] = fmaf(qs[h][e], kv, s[h]);
        }
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        float v = s[h];
        for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (lane == 0) red[warp][h] = v;
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const float mn = fmaxf(m[h], fmaxf(fmaxf(red[0][h], red[1][h]), fmaxf(red[2][h], red[3][h])));
        const float al = mn == -INFINITY ? 1.f : ex2(m[h] - mn);
        m[h] = mn;
        acc[h] *= al;
        l[h] *= al;
        p[h][tid] = tid < nval ? ex2(s[h] - mn) : 0.f;
      }
      __syncthreads();
      for (int tau = 0; tau < nval; ++tau) {
        const float kv = tid < D ? kv4_value<false, D>(vp, bs, tau, tid) : 0.f;
#pragma unroll
        for (int h = 0; h < 8; ++h)
          if (h < G) {
            l[h] += p[h][tau];
            acc[h] = fmaf(p[h][tau], kv, acc[h]);
          }
      }
      __syncthreads();
    }
    float* part = a.partials + ((size_t)gi * x.pslots + seg) * GE;
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h < G) {
        if (tid < D) part[h * (D + 2) + 2 + tid] = acc[h];
        if (tid == 0) {
          part[h * (D + 2)] = m[h];
          part[h * (D + 2) + 1] = l[h];
        }
      }
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(&a.counters[gi], 1u) == (unsigned)(nseg - 1);
    __syncthreads();
    if (s_last) {
      __threadfence();
      const float* p0 = a.partials + (size_t)gi * x.pslots * GE;
      for (int e = tid; e < G * D; e += 128) {
        const int h = e / D, col = e % D;
        float M = -INFINITY, num = 0.f, den = 0.f;
        for (int sg = 0; sg < nseg; ++sg) M = fmaxf(M, __ldcg(p0 + (size_t)sg * GE + h * (D + 2)));
        if (M != -INFINITY)
          for (int sg = 0; sg < nseg; ++sg) {
            const float* ps = p0 + (size_t)sg * GE + h * (D + 2);
            const float f = ex2(__ldcg(ps) - M);
            den += __ldcg(ps + 1) * f;
            num += __ldcg(ps + 2 + col) * f;
          }
        a.out[((size_t)(gi / a.Hkv) * a.Hq + (gi % a.Hkv) * G + h) * D + col] = den == 0.f ? 0.f : num / den;
      }
      if (tid == 0) {
        a.counters[gi] = 0u;
        if (flags) a.sel_flag[(size_t)gi * kFlagStride] = 0u;
        if (a.e_flag) {
          a.e_flag[(size_t)gi * kFlagStride] = 0u;
          a.e_flag[(size_t)gi * kFlagStride + 3] = 0u;
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace nosa

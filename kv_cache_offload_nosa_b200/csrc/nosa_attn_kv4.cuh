// Split-K flash-decoding over the selected blocks of a 4-bit cache (kv_bits = 4).
//
// The tasks, their split over CTAs and the merge of the partials are those of the bf16 kernel:
// the B*Hkv*k (group, selected block) tasks, group after group, are cut in ranges of W, one range
// per CTA; each range writes one partial (m, l, acc) per query head and group it touches, and the
// last CTA to finish a group (atomic ticket) merges them. One producer warp brings each task's K
// and V page (two bulk copies, codes and scales together) into a ring of stages; BS/16 consumer
// warps own 16 tokens of every page each.
//
// The pages are never expanded. With s the scales and c the codes,
//   score:  sum_d q_d K_td = sum_g s_tg sum_{d in g} q_d (c_td - 8),
//   output: sum_t p_t V_td = sum_t (p_t s_tg) (c_td - 8),
// so the matrix products run on the codes, and the scales enter where there are few values: the
// per-group partial scores, and the weights. Codes become fp16 operands in registers:
//   K: (w & 0x000f000f) is a pair of fp16 subnormals c 2^-24, (w & 0x00f000f0) is 16 c 2^-24; q is
//      scaled by a power of two to an fp16 row (its 16ths for the second kind), and the
//      accumulators start at -8 sum q. One mask and no arithmetic per pair.
//   V: the same masks or'ed with 1024 (0x6400) give 1024 + c and 1024 + 16 c, and one fp16 FMA
//      makes c - 8 of either: over a long axis the offset has to go before the sum, which it would
//      exceed many times.
// The weights p_t s_tg are split in two fp16 parts (22 bits). They are kept in range for every
// scale of V: the running reference m is that of x_t + e_t, where e_t is the exponent of the
// token's largest V scale, and it moves only when a weight would exceed 2^4.
#pragma once

#include <cuda_fp16.h>

#include "nosa_attn.cuh"
#include "nosa_kv4.cuh"

namespace nosa {

constexpr int kKv4MaxStages = 8;

struct AttnKv4Args {
  AttnArgs a;
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  int pslots;  // partial slots per group
};

template <int D, int BS>
struct AttnKv4Shape {
  static constexpr int NC = BS / 16;
  static constexpr int THREADS = (NC + 1) * 32;
  static constexpr int PAGE = kv4_page_bytes(BS, D);
  static constexpr int STAGE = 2 * PAGE;
  static size_t smem_bytes(int stages, int G) {
    return 128 + (size_t)stages * STAGE + 2 * kKv4MaxStages * 8 + kKv4MaxStages * sizeof(TaskInfo) + 16 +
           (size_t)NC * G * (D + 2) * 4;  // alignment, stages, barriers, tasks, flag + barrier, scratch
  }
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// D = A(16x16 f16, row) * B(16x8 f16, col) + C, fp32 accumulate.
__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, float c0, float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t hfma2_u32(uint32_t x, uint32_t m, uint32_t a) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(m), "r"(a));
  return y;
}
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <int D, int BS>
__global__ void __launch_bounds__(AttnKv4Shape<D, BS>::THREADS, BS == 128 ? 1 : 3) attn_kv4_kernel(AttnKv4Args x) {
  using SH = AttnKv4Shape<D, BS>;
  constexpr int NC = SH::NC;
  constexpr int NG = D / 32;  // groups of a row
  const AttnArgs& a = x.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  const int ST = a.stages;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + (size_t)ST * SH::STAGE);
  uint64_t* empty = full + kKv4MaxStages;
  TaskInfo* info = reinterpret_cast<TaskInfo*>(empty + kKv4MaxStages);
  uint64_t* meet = reinterpret_cast<uint64_t*>(info + kKv4MaxStages);  // the consumer warps' meeting point
  int* s_flag = reinterpret_cast<int*>(meet + 1);
  float* scr = reinterpret_cast<float*>(meet + 2);  // [NC][G][D + 2]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int task0 = blockIdx.x * a.W;
  const int ntask = min(a.W, a.total - task0);
  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], NC);
    }
    mbar_init(meet, NC);
    fence_barrier_init();
  }
  __syncthreads();
  const bool flags = a.sel_flag != nullptr;
  if (!flags) griddep_wait();
  const unsigned long long deadline = globaltimer() + a.wait_ns;

  if (warp == NC) {
    // ---------------------------------------------------------------- producer
    // As the bf16 kernel's: ranges cut at group boundaries, taken in parts that wait for the same
    // flag (a group's query-agnostic blocks may be ready before the rest of its selection); 32
    // tasks' pages are looked up at once, lane 0 issues the copies in task order.
    const bool early = a.att_list != nullptr;
    const int32_t* list = early ? a.att_list : a.sel;
    int it = 0;
    bool abort = false;
    for (int sr = 0; sr < ntask && !abort;) {
      const int gi = (task0 + sr) / a.k;
      const int pa = task0 + sr - gi * a.k;
      const int pb = min(task0 + ntask, (gi + 1) * a.k) - gi * a.k;
      const int first = (int)(((long long)gi * a.k) / a.W);
      const int lastc = (int)(((long long)gi * a.k + a.k - 1) / a.W);
      sr += pb - pa;
      for (int p = pa; p < pb && !abort;) {
        int pend = pb, L;
        const uint32_t* f = flags ? a.sel_flag + (size_t)gi * kFlagStride : nullptr;
        if (early) {
          const uint32_t* ef = a.e_flag + (size_t)gi * kFlagStride;
          if (lane == 0 && !wait_flag(ef, deadline)) set_err(a.err, NOSA_ERR_TIMEOUT);
          __syncwarp();
          L = static_cast<int>(__ldcg(ef + 1));
          const int ne = static_cast<int>(__ldcg(ef + 2));
          if (p < ne) {
            pend = min(pb, ne);
            f = nullptr;
          }
        }
        if (f) {
          if (lane == 0 && !wait_flag(f, deadline)) set_err(a.err, NOSA_ERR_TIMEOUT);
          __syncwarp();
        }
        if (!early) L = __ldcg(a.seq_len + gi);
        if (flags && lane == 0) fence_proxy_async_global();  // pages written before the flags
        const int N = (L + BS - 1) / BS;
        for (int base = p; base < pend && !abort; base += 32) {
          const int p_l = base + lane;
          int j_l = -1, page_l = -1;
          if (p_l < pend) {
            j_l = __ldcg(list + gi * a.k + p_l);
            if (j_l >= N) {
              set_err(a.err, NOSA_ERR_SEL);
              j_l = -1;
            }
            if (j_l >= 0) {
              page_l = a.identity ? gi * a.max_blocks + j_l
                                  : __ldcg(a.block_table + (size_t)gi * a.max_blocks + j_l);
              if (page_l < 0 || page_l >= a.total_pages) {
                set_err(a.err, NOSA_ERR_BLOCK_TABLE);
                j_l = -1;
              }
            }
          }
          const int nb = min(32, pend - base);
          __syncwarp();
          for (int v = 0; v < nb; ++v) {
            const int j = __shfl_sync(0xffffffffu, j_l, v);
            const int page = __shfl_sync(0xffffffffu, page_l, v);
            if (lane == 0) {
              const int s = it % ST, round = it / ST;
              if (round > 0 && !mbar_wait(&empty[s], (round - 1) & 1, deadline)) {
                set_err(a.err, NOSA_ERR_TIMEOUT);
                abort = true;
              } else {
                TaskInfo ti;
                ti.gi = gi;
                ti.j = j;
                ti.L = L;
                ti.last = (base + v == pb - 1);
                ti.seg = blockIdx.x - first;
                ti.nseg = lastc - first + 1;
                info[s] = ti;
                if (j >= 0) {
                  mbar_arrive_expect_tx(&full[s], SH::STAGE);
                  uint8_t* st = smem + (size_t)s * SH::STAGE;
                  bulk_load(st, x.k_pages + (size_t)page * SH::PAGE, SH::PAGE, &full[s]);
                  bulk_load(st + SH::PAGE, x.v_pages + (size_t)page * SH::PAGE, SH::PAGE, &full[s]);
                } else {
                  mbar_arrive(&full[s]);
                }
                ++it;
              }
            }
            abort = __shfl_sync(0xffffffffu, abort, 0);
            if (abort) break;
          }
        }
        p = pend;
      }
    }
    if (lane == 0 && !abort) {  // a task with gi < 0 stops the consumers
      const int s = it % ST, round = it / ST;
      if (round > 0 && !mbar_wait(&empty[s], (round - 1) & 1, deadline)) {
        set_err(a.err, NOSA_ERR_TIMEOUT);
      } else {
        TaskInfo ti = {-1, -1, 0, 0, 0, 0};
        info[s] = ti;
        mbar_arrive(&full[s]);
        ++it;
      }
    }
    // never leave the CTA with a copy in flight
    if (lane == 0)
      for (int i = max(0, it - ST); i < it; ++i) mbar_wait(&full[i % ST], (i / ST) & 1, deadline);
    return;
  }

  // ---------------------------------------------------------------- consumers
  // S^T = K . q^T: rows are tokens, columns heads. Row i < 8 of the tile is token (i >> 1) + 4 (i & 1)
  // and row i + 8 that plus 8: lane c4 of the second product then takes tokens c4, c4 + 4, c4 + 8
  // and c4 + 12, whose V rows lie in different banks. With G <= 4 column h + 4 repeats head h and
  // carries the low parts of its weights; with G = 8 the low parts take a second product.
  const int r = lane >> 2, c4 = lane & 3;
  const bool wide = a.G > 4;
  auto col_head = [&](int n) { return wide ? n : (n & 3); };
  const int h0 = col_head(2 * c4), h1 = col_head(2 * c4 + 1);
  const bool cv0 = h0 < a.G, cv1 = h1 < a.G;
  const float lo_sign = (!wide && c4 >= 2) ? -1.f : 0.f;  // low columns take w - fp16(w)
  const bool owner = wide || c4 < 2;
  const int tokA = 16 * warp + (r >> 1) + 4 * (r & 1), tokB = tokA + 8;
  const int tokV = 16 * warp + c4;
  uint32_t qb[NG][4];
  float qz[NG][2];
  float f0 = 0.f, f1 = 0.f;
  float acc[2 * NG][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  int cur = -1;
  // All consumer warps meet: a bounded wait like every other here, so that a warp that has given
  // up on a stage leaves the others an end too.
  uint32_t met = 0u;
  auto meeting = [&]() -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(meet);
    return mbar_wait(meet, met++ & 1u, deadline);
  };

  for (int i = 0;; ++i) {
    const int s = i % ST;
    if (!mbar_wait(&full[s], (i / ST) & 1, deadline)) {
      set_err(a.err, NOSA_ERR_TIMEOUT);
      break;
    }
    const TaskInfo ti = info[s];
    if (ti.gi < 0) break;
    const uint8_t* kst = smem + (size_t)s * SH::STAGE;
    const uint8_t* vst = kst + SH::PAGE;
    if (ti.gi != cur) {
      // q as fp16 rows: each head's largest magnitude goes to [2^13, 2^14), so that what the
      // conversion drops is 2^-38 of it
      cur = ti.gi;
      const int qhead = col_head(r);
      const bool qok = qhead < a.G;
      const uint16_t* qrow = a.q + ((size_t)(cur / a.Hkv) * a.Hq + (cur % a.Hkv) * a.G + (qok ? qhead : 0)) * D;
      uint4 qv[NG];
      uint32_t mx = 0u;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        qv[g] = qok ? *reinterpret_cast<const uint4*>(qrow + 32 * g + 8 * c4) : make_uint4(0, 0, 0, 0);
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(qv[g].x & 0x7fff7fffu, qv[g].y & 0x7fff7fffu),
                                   __vmaxu2(qv[g].z & 0x7fff7fffu, qv[g].w & 0x7fff7fffu)));
      }
      mx = max(mx & 0xffffu, mx >> 16);
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // 13 - exponent, kept where both it and what undoes it are floats
      const int e = min(max(140 - static_cast<int>(mx >> 7), -100), 100);
      const float up = __uint_as_float((127 + e) << 23), up16 = up * 0.0625f;
      float zero[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t w[4] = {qv[g].x, qv[g].y, qv[g].z, qv[g].w};  // values (0, 1) .. (6, 7)
        // even codes take q, odd ones a 16th of it; the fragments pair codes i and i + 4
        qb[g][0] = pack_f16(bf16_lo(w[0]) * up, bf16_lo(w[2]) * up);
        qb[g][1] = pack_f16(bf16_hi(w[0]) * up16, bf16_hi(w[2]) * up16);
        qb[g][2] = pack_f16(bf16_lo(w[1]) * up, bf16_lo(w[3]) * up);
        qb[g][3] = pack_f16(bf16_hi(w[1]) * up16, bf16_hi(w[3]) * up16);
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 q2 = __half22float2(*reinterpret_cast<const __half2*>(&qb[g][j]));
          z += ((j & 1) ? 16.f : 1.f) * (q2.x + q2.y);
        }
        z += __shfl_xor_sync(0xffffffffu, z, 1);
        z += __shfl_xor_sync(0xffffffffu, z, 2);
        zero[g] = -8.f * 0x1p-24f * z;
      }
      const float fq = __uint_as_float((127 - e) << 23) * a.scale_log2 * 0x1p24f;
      // from column r of B (all four c4 lanes agree) to columns 2 c4, 2 c4 + 1 of C
      f0 = __shfl_sync(0xffffffffu, fq, 8 * c4);
      f1 = __shfl_sync(0xffffffffu, fq, 8 * c4 + 4);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        qz[g][0] = __shfl_sync(0xffffffffu, zero[g], 8 * c4);
        qz[g][1] = __shfl_sync(0xffffffffu, zero[g], 8 * c4 + 4);
      }
#pragma unroll
      for (int mt = 0; mt < 2 * NG; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
    }
    const int nval = (ti.j >= 0) ? min(16, ti.L - ti.j * BS - 16 * warp) : 0;
    if (nval > 0) {
      // ---- scores
      uint32_t ka[NG], kb[NG], sk[NG], sv[NG];  // scales: [0, NG/2) row A, [NG/2, NG) row B
      lds_words<NG>(kst + tokA * (D / 2) + c4 * (D / 8), ka);
      lds_words<NG>(kst + tokB * (D / 2) + c4 * (D / 8), kb);
      lds_words<NG / 2>(kst + BS * (D / 2) + tokA * (D / 16), sk);
      lds_words<NG / 2>(kst + BS * (D / 2) + tokB * (D / 16), sk + NG / 2);
      lds_words<NG / 2>(vst + BS * (D / 2) + tokA * (D / 16), sv);
      lds_words<NG / 2>(vst + BS * (D / 2) + tokB * (D / 16), sv + NG / 2);
      float x0 = 0.f, x1 = 0.f, x2 = 0.f, x3 = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float c[4];
        mma_f16(c, ka[g] & 0x000f000fu, kb[g] & 0x000f000fu, ka[g] & 0x00f000f0u, kb[g] & 0x00f000f0u, qb[g][0],
                qb[g][1], qz[g][0], qz[g][1], qz[g][0], qz[g][1]);
        const uint32_t ah = ka[g] >> 8, bh = kb[g] >> 8;
        mma_f16(c, ah & 0x000f000fu, bh & 0x000f000fu, ah & 0x00f000f0u, bh & 0x00f000f0u, qb[g][2], qb[g][3], c[0],
                c[1], c[2], c[3]);
        const float sA = (g & 1) ? bf16_hi(sk[g / 2]) : bf16_lo(sk[g / 2]);
        const float sB = (g & 1) ? bf16_hi(sk[NG / 2 + g / 2]) : bf16_lo(sk[NG / 2 + g / 2]);
        x0 = fmaf(sA, c[0], x0);
        x1 = fmaf(sA, c[1], x1);
        x2 = fmaf(sB, c[2], x2);
        x3 = fmaf(sB, c[3], x3);
      }
      const int nA = nval - (tokA - 16 * warp);
      const bool tA = nA > 0, tB = nA > 8;
      x0 = (cv0 && tA) ? x0 * f0 : -INFINITY;
      x1 = (cv1 && tA) ? x1 * f1 : -INFINITY;
      x2 = (cv0 && tB) ? x2 * f0 : -INFINITY;
      x3 = (cv1 && tB) ? x3 * f1 : -INFINITY;
      // rows past the context may hold anything, a NaN scale among it
#pragma unroll
      for (int g = 0; g < NG / 2; ++g) {
        sv[g] = tA ? sv[g] : 0u;
        sv[NG / 2 + g] = tB ? sv[NG / 2 + g] : 0u;
      }
      // exponent of each token's largest V scale (the range keeps 2^-e and sums of it finite)
      auto top = [&](const uint32_t* w) {
        uint32_t m = w[0];
        if constexpr (NG == 4) m = __vmaxu2(m, w[1]);
        m = max(m & 0xffffu, m >> 16);
        return static_cast<float>(min(max(static_cast<int>(m >> 7) - 127, -60), 100));
      };
      const float eA = top(sv), eB = top(sv + NG / 2);
      const float y0 = fmaxf(x0 + eA, x2 + eB), y1 = fmaxf(x1 + eA, x3 + eB);
      if (__any_sync(0xffffffffu, y0 > m0 + 3.f || y1 > m1 + 3.f)) {
        float mx0 = y0, mx1 = y1;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
        }
        const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
        const float al0 = mn0 == m0 ? 1.f : ex2(m0 - mn0), al1 = mn1 == m1 ? 1.f : ex2(m1 - mn1);
        m0 = mn0;
        m1 = mn1;
        l0 *= al0;
        l1 *= al1;
#pragma unroll
        for (int mt = 0; mt < 2 * NG; ++mt) {
          acc[mt][0] *= al0;
          acc[mt][1] *= al1;
          acc[mt][2] *= al0;
          acc[mt][3] *= al1;
        }
      }
      const float mu0 = m0 == -INFINITY ? 0.f : m0, mu1 = m1 == -INFINITY ? 0.f : m1;
      const float p0 = ex2(x0 - mu0), p1 = ex2(x1 - mu1), p2 = ex2(x2 - mu0), p3 = ex2(x3 - mu1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      // ---- O^T += (c - 8)^T . (p s)^T
      uint32_t vw[4][NG / 2];
#pragma unroll
      for (int t = 0; t < 4; ++t) lds_words<NG / 2>(vst + (tokV + 4 * t) * (D / 2) + r * (D / 16), vw[t]);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float sA = (g & 1) ? bf16_hi(sv[g / 2]) : bf16_lo(sv[g / 2]);
        const float sB = (g & 1) ? bf16_hi(sv[NG / 2 + g / 2]) : bf16_lo(sv[NG / 2 + g / 2]);
        const float w0 = p0 * sA, w1 = p1 * sA, w2 = p2 * sB, w3 = p3 * sB;
        const uint32_t hA = pack_f16(w0, w1), hB = pack_f16(w2, w3);
        const float2 eA2 = __half22float2(*reinterpret_cast<const __half2*>(&hA));
        const float2 eB2 = __half22float2(*reinterpret_cast<const __half2*>(&hB));
        uint32_t b0, b1, d0 = 0u, d1 = 0u;
        if (wide) {
          b0 = movmatrix_t(hA);
          b1 = movmatrix_t(hB);
          d0 = movmatrix_t(pack_f16(w0 - eA2.x, w1 - eA2.y));
          d1 = movmatrix_t(pack_f16(w2 - eB2.x, w3 - eB2.y));
        } else {
          b0 = movmatrix_t(pack_f16(fmaf(eA2.x, lo_sign, w0), fmaf(eA2.y, lo_sign, w1)));
          b1 = movmatrix_t(pack_f16(fmaf(eB2.x, lo_sign, w2), fmaf(eB2.y, lo_sign, w3)));
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const uint32_t sel = 0x4400u + 0x1111u * (2 * (g & 1) + mt);  // byte 2 (g & 1) + mt of both tokens
          const uint32_t u = __byte_perm(vw[0][g / 2], vw[1][g / 2], sel);
          const uint32_t v = __byte_perm(vw[2][g / 2], vw[3][g / 2], sel);
          constexpr uint32_t ONE = 0x3c003c00u, M1032 = 0xe408e408u, SIXTEENTH = 0x2c002c00u, M72 = 0xd480d480u;
          const uint32_t a0 = hfma2_u32((u & 0x000f000fu) | 0x64006400u, ONE, M1032);
          const uint32_t a1 = hfma2_u32((u & 0x00f000f0u) | 0x64006400u, SIXTEENTH, M72);
          const uint32_t a2 = hfma2_u32((v & 0x000f000fu) | 0x64006400u, ONE, M1032);
          const uint32_t a3 = hfma2_u32((v & 0x00f000f0u) | 0x64006400u, SIXTEENTH, M72);
          float* o = acc[2 * g + mt];
          mma_f16(o, a0, a1, a2, a3, b0, b1, o[0], o[1], o[2], o[3]);
          if (wide) mma_f16(o, a0, a1, a2, a3, d0, d1, o[0], o[1], o[2], o[3]);
        }
      }
    }
    // the stage has been read: hand it back before the merge
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);

    if (ti.last) {
      // ------------------------------------------------ flush this group's part
      float L0 = l0, L1 = l1;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        L0 += __shfl_xor_sync(0xffffffffu, L0, o);
        L1 += __shfl_xor_sync(0xffffffffu, L1, o);
      }
      if (!wide) {
#pragma unroll
        for (int mt = 0; mt < 2 * NG; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[mt][e] += __shfl_xor_sync(0xffffffffu, acc[mt][e], 2);
      }
      bool ok = meeting();  // the previous merge has read the scratch
      if (owner) {
        float* w0 = scr + ((size_t)warp * a.G + h0) * (D + 2);
        float* w1 = scr + ((size_t)warp * a.G + h1) * (D + 2);
        if (r == 0) {
          if (cv0) w0[0] = m0, w0[1] = L0;
          if (cv1) w1[0] = m1, w1[1] = L1;
        }
        // rows r and r + 8 of tile mt of group g: values 32g + 4r + 2mt and the next
#pragma unroll
        for (int mt = 0; mt < 2 * NG; ++mt) {
          const int at = 2 + 32 * (mt / 2) + 4 * r + 2 * (mt & 1);
          if (cv0) *reinterpret_cast<float2*>(w0 + at) = make_float2(acc[mt][0], acc[mt][2]);
          if (cv1) *reinterpret_cast<float2*>(w1 + at) = make_float2(acc[mt][1], acc[mt][3]);
        }
      }
      ok = ok && meeting();
      const int gi = ti.gi, GE = a.G * (D + 2);
      float* part = a.partials + ((size_t)gi * x.pslots + ti.seg) * GE;
      for (int e = tid; e < GE; e += NC * 32) {
        const int h = e / (D + 2), col = e % (D + 2);
        float M = -INFINITY;
        for (int w = 0; w < NC; ++w) M = fmaxf(M, scr[((size_t)w * a.G + h) * (D + 2)]);
        float v = M;
        if (col != 0) {
          v = 0.f;
          for (int w = 0; w < NC; ++w) {
            const float* ww = scr + ((size_t)w * a.G + h) * (D + 2);
            v += ww[col] * (ww[0] == M ? 1.f : ex2(ww[0] - M));
          }
        }
        part[e] = v;
      }
      __threadfence();
      ok = ok && meeting();
      if (ok && tid == 0) *s_flag = (atomicAdd(&a.counters[gi], 1u) == (unsigned)(ti.nseg - 1));
      ok = ok && meeting();
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        set_err(a.err, NOSA_ERR_TIMEOUT);
        break;
      }
      if (*s_flag) {
        __threadfence();
        const float* p0 = a.partials + (size_t)gi * x.pslots * GE;
        const int b = gi / a.Hkv, g = gi % a.Hkv;
        for (int e = tid; e < a.G * D; e += NC * 32) {
          const int h = e / D, col = e % D;
          float M = -INFINITY;
          for (int sg = 0; sg < ti.nseg; ++sg) M = fmaxf(M, __ldcg(p0 + (size_t)sg * GE + h * (D + 2)));
          float num = 0.f, den = 0.f;
          for (int sg = 0; sg < ti.nseg; ++sg) {
            const float* ps = p0 + (size_t)sg * GE + h * (D + 2);
            const float m = __ldcg(ps), f = m == M ? 1.f : ex2(m - M);
            den += __ldcg(ps + 1) * f;
            num += __ldcg(ps + 2 + col) * f;
          }
          a.out[((size_t)b * a.Hq + g * a.G + h) * D + col] = den == 0.f ? 0.f : num / den;
        }
        if (tid == 0) {
          a.counters[gi] = 0u;
          if (flags) a.sel_flag[(size_t)gi * kFlagStride] = 0u;  // every CTA of the group passed its wait
          if (a.e_flag) {
            a.e_flag[(size_t)gi * kFlagStride] = 0u;
            a.e_flag[(size_t)gi * kFlagStride + 3] = 0u;
          }
        }
      }
      cur = -1;
    }
  }
}

}  // namespace nosa

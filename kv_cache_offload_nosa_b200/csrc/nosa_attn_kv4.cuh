// Split-K flash-decoding over the selected blocks of a 4-bit cache (kv_bits = 4).
//
// The tasks and the merge of the partials are those of the bf16 kernel: the B*Hkv*k (group, selected
// block) tasks, group after group, are cut in ranges of W, one range per CTA (or each group in ranges
// of its own); each range writes one partial per query head and group it touches (the mean of V under
// its weights, and their sum as l 2^m), and the last CTA to finish a group (atomic ticket) merges them.
// One producer warp brings each task's K and V page (two bulk copies, codes and scales together) into a
// ring of stages; the consumer warps take 32 tokens each, a page's units going to neighbouring warps and
// page after page to the next.
//
// Time: the pages are 3.6 times smaller than bf16 ones, so it is unpacking them that costs, not memory.
// Over four sequences of 131072 tokens, 8 KV heads of 4 query heads each, it takes 147 us replayed from a
// graph and up to 156 us in other company (4.1 to 3.9 TB/s; the same pages copied and not unpacked: 97
// us), over one of them 48 us. There a warp issues 390 instructions per 16 tokens, start, end and merge
// included, and no unit is full: issue slots 55 %, integer pipe 43 %, shared memory 33 % (58 wavefronts
// per 16 tokens and warp, 17 of them bank conflicts), FMA pipe 33 %, tensor pipe 18 %. Fewer
// instructions made it faster, more warps did not (8 or 12 consumer warps an SM take the same time);
// what leaves the other issue slots empty has not been found. mma.sync and not tcgen05: a group has
// G <= 8 query rows, and codes have to pass through registers on their way to an operand.
//
// The pages are never expanded. With s the scales and c the codes,
//   score:  sum_d q_d K_td = sum_g s_tg sum_{d in g} q_d (c_td - 8),
//   output: sum_t p_t V_td = sum_t (p_t s_tg) (c_td - 8),
// so the matrix products run on the codes, and the scales enter where there are few values: the
// per-group partial scores, and the weights. Codes become fp16 operands in registers: a word's pairs
// of codes 16 bits apart, masked and or'ed with 1024, are the fp16 pair 1024 + c, or 1024 + 16 c of the
// next code, and one fp16 FMA makes c - 8 of either. (The offset has to go before the products: as a
// start value -8 sum q of the accumulators it cost the scores a bit and a half, 8e-7 against 3e-7 of
// the output, for 2 % of the time.) q is scaled by a power of two to an fp16 row.
// The weights p_t s_tg, p_t = 2^(x_t - m), are split in two fp16 parts. They are kept in fp16's
// range for every scale of V: the reference m is 10 below the largest x_t + e_t seen, where e_t is
// about the base-2 logarithm of the token's largest V scale, and it moves only when an x_t + e_t
// exceeds it by more than 13. Weights are thus below 2^15, and one of 2^-14 of the largest still
// has all 22 bits of its two parts. (e_t is at least -90, which keeps p and its sum finite: V below
// 2^-100 loses digits, and below 2^-120 vanishes. With scales of 2^e weights under 2^(e - 136) of the
// largest do, 2^-11 at most. In a group 2^n smaller than the row's largest, n > 13, the parts' last place,
// 2^-35 of the largest weight, is about 2^(n-35) of the result.)
// Beyond 2^20 a score plus e_t is not e_t precise enough, and a warp that meets one there carries its
// references as pairs a + b: a near the scores and taken from them first, b for the scales of V.
#pragma once

#include <cuda_fp16.h>

#include "nosa_attn.cuh"
#include "nosa_kv4.cuh"

namespace nosa {

constexpr int kKv4MaxStages = 16;
constexpr int kKv4MaxSlots = 128;  // partial slots per group, at most
constexpr float kKv4None = -0x1.fffffep127f;  // the reference where no token has been seen

// Floats of one partial slot: means [G][D], then (m, l) [G], in 16-byte steps.
__host__ __device__ constexpr int kv4_part_floats(int G, int D) { return G * D + ((2 * G + 3) & ~3); }

struct AttnKv4Args {
  AttnArgs a;
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  int pslots;  // partial slots per group
  int parts;   // > 0: every group in this many ranges of W (the last one shorter), none across groups
};

template <int D, int BS>
struct AttnKv4Shape {
  static constexpr int NC = 4;             // consumer warps
  static constexpr int U = BS / 32;        // units of 32 tokens in a page, a warp each
  static constexpr int STEP = NC / U;      // pages in work at once; the stages are a multiple of it,
                                           // so that a warp comes to its stages in every round of the
                                           // ring (a barrier's parity tells one round from the next only)
  static constexpr int THREADS = (NC + 1) * 32;
  static constexpr int CTAS = D == 128 ? 3 : 4;  // per SM (128 and 96 registers a thread)
  static constexpr int PAGE = kv4_page_bytes(BS, D);
  static constexpr int STAGE = 2 * PAGE;
  static constexpr int most(int a, int b) { return a > b ? a : b; }
  // Shared memory for up to GM query heads a group: alignment, barriers, tasks, meeting point, q, the
  // warps' pairs; what the sums, the warps' partials and the merge share; the stages.
  template <int GM>
  static constexpr int FIXED =
      128 + kKv4MaxStages * (8 + 8 + 8) + 16 + (D / 32) * 512 + NC * 128 +
      most(NC * D * 8 * 4, most(NC * kv4_part_floats(GM, D), GM * kKv4MaxSlots + NC * GM * D) * 4);
  // As many stages as the CTAs of an SM leave room for, a multiple of STEP, at least two pages.
  template <int GM>
  static constexpr int stages() {
    const int room = (227 * 1024 / CTAS - 1024 - FIXED<GM>) / STAGE;
    const int n = (room > kKv4MaxStages ? kKv4MaxStages : room) / STEP * STEP;
    return n < 2 ? 2 : n;
  }
  template <int GM>
  static constexpr int SMEM = FIXED<GM> + stages<GM>() * STAGE;
  template <int GM>
  static constexpr int ctas_per_sm() {
    return 227 * 1024 / (SMEM<GM> + 1024) < CTAS ? 227 * 1024 / (SMEM<GM> + 1024) : CTAS;
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
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
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
__device__ __forceinline__ uint32_t mul_bf162(uint32_t x, uint32_t y) {
  const __nv_bfloat162 z =
      __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&z);
}
// (x & m) | o in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t o) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(m), "r"(o));
  return y;
}
// c - 8 of the codes in bits 0..3, or 4..7, of both halves of w as fp16 pairs; kilo: (1024, 1024), in
// a register so that masking and or'ing are one instruction.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t kilo) {
  return hfma2_u32(and_or(w, 0x000f000fu, kilo), 0x3c003c00u, 0xe408e408u);  // 1, -1032
}
__device__ __forceinline__ uint32_t next_code_pair(uint32_t w, uint32_t kilo) {
  return hfma2_u32(and_or(w, 0x00f000f0u, kilo), 0x2c002c00u, 0xd480d480u);  // 1/16, -72
}
__device__ __forceinline__ int warp_id() { return threadIdx.x >> 5; }
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

// All warps of a CTA meet: a bounded wait like every other here, so that a warp that has given up on
// a stage leaves the others an end too. met: the number of meetings before.
__device__ __forceinline__ bool kv4_meeting(uint64_t* meet, uint32_t met, unsigned long long deadline) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(meet);
  return __all_sync(0xffffffffu, mbar_wait(meet, met & 1u, deadline));
}

// The square root of the factor that takes sums from the reference `from` to `to`, the larger one.
// References hold the scales of V, so that they may lie 220 apart while the scores do not: the factor
// itself would be zero below 2^-126, where an l of up to 2^103 and more still counts; it is applied to l
// in two halves. (The sums of V are at most 2^15 a weight at any reference, so that theirs may vanish.)
__device__ __forceinline__ float half_factor(float from, float to) { return from == to ? 1.f : ex2(0.5f * (from - to)); }

// The last CTA of a group merges its partials p0 [nseg] into outg [G][D]: the segments' shares of the
// weights (a head per warp, a segment per lane) with the first values under way, then every NC-th
// segment per warp, the warps' sums last. (A share below 2^-126 is zero, as in any fp32 softmax.) scr:
// shared memory for [G] x 128 shares and [NC][G][D] values. Two meetings. Out of line: its registers
// would cost the main loop.
template <int D, int NC, bool WIDE>
__device__ __noinline__ bool kv4_merge(const float* p0, float* outg, float* scr, int nseg, int G, uint64_t* meet,
                                       uint32_t met, unsigned long long deadline) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, GE = kv4_part_floats(G, D);
  float* share = scr;
  float4* add = reinterpret_cast<float4*>(scr + G * kKv4MaxSlots);
  constexpr int E = (WIDE ? 8 : 4) * D / 128;  // four values of a head each, 32 apart
  constexpr int AT = 8 / E;                    // segments in flight
  const int ne = G * (D / 4);
  float4 y[AT][E];
  auto load = [&](int sg) {
#pragma unroll
    for (int t = 0; t < AT; ++t)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        y[t][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (sg + t * NC < nseg && lane + 32 * i < ne)
          y[t][i] = __ldcg(reinterpret_cast<const float4*>(p0 + (size_t)(sg + t * NC) * GE) + lane + 32 * i);
      }
  };
  load(warp);
  for (int h = warp; h < G; h += NC) {
    float2 ml[kKv4MaxSlots / 32];
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int i = 0; i < kKv4MaxSlots / 32; ++i) {
      const int sg = 32 * i + lane;
      ml[i] = make_float2(-INFINITY, 0.f);
      if (sg < nseg) ml[i] = __ldcg(reinterpret_cast<const float2*>(p0 + (size_t)sg * GE + G * D) + h);
      M = fmaxf(M, ml[i].x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int i = 0; i < kKv4MaxSlots / 32; ++i) {
      const float f = half_factor(ml[i].x, M);
      ml[i].y = ml[i].y * f * f;
      L += ml[i].y;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const float inv = L == 0.f ? 0.f : 1.f / L;  // (no token at all)
#pragma unroll
    for (int i = 0; i < kKv4MaxSlots / 32; ++i)
      if (32 * i + lane < nseg) share[h * kKv4MaxSlots + 32 * i + lane] = ml[i].y * inv;
  }
  if (!kv4_meeting(meet, met, deadline)) return false;
  float4 v[E];
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int sg = warp; sg < nseg; sg += AT * NC) {
    if (sg != warp) load(sg);
#pragma unroll
    for (int t = 0; t < AT; ++t)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int h = min((lane + 32 * i) / (D / 4), G - 1);
        const float f = share[h * kKv4MaxSlots + min(sg + t * NC, nseg - 1)];
        v[i].x = fmaf(y[t][i].x, f, v[i].x);
        v[i].y = fmaf(y[t][i].y, f, v[i].y);
        v[i].z = fmaf(y[t][i].z, f, v[i].z);
        v[i].w = fmaf(y[t][i].w, f, v[i].w);
      }
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (lane + 32 * i < ne) add[warp * ne + lane + 32 * i] = v[i];
  if (!kv4_meeting(meet, met + 1u, deadline)) return false;
  for (int e = tid; e < ne; e += NC * 32) {
    float4 y = add[e];
#pragma unroll
    for (int w = 1; w < NC; ++w) {
      const float4 z = add[w * ne + e];
      y.x += z.x;
      y.y += z.y;
      y.z += z.z;
      y.w += z.w;
    }
    reinterpret_cast<float4*>(outg)[e] = y;
  }
  return true;
}

// WIDE: more than four query heads a group.
template <int D, int BS, bool WIDE>
__global__ void __launch_bounds__(AttnKv4Shape<D, BS>::THREADS, AttnKv4Shape<D, BS>::CTAS)
    attn_kv4_kernel(AttnKv4Args x) {
  using SH = AttnKv4Shape<D, BS>;
  constexpr int NC = SH::NC, U = SH::U;
  constexpr int NG = D / 32;  // groups of a row
  const AttnArgs& a = x.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  const int ST = a.stages;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + kKv4MaxStages;
  int2* info = reinterpret_cast<int2*>(empty + kKv4MaxStages);  // a stage's block (-1: none) and length
  uint64_t* meet = reinterpret_cast<uint64_t*>(info + kKv4MaxStages);  // the consumer warps' meeting point
  int* s_flag = reinterpret_cast<int*>(meet + 1);
  uint4* sq = reinterpret_cast<uint4*>(meet + 2);       // [NG][32] a lane's q operands of a group
  // [NC][4] of a lane column's two heads: (a, a, b, b) of the pairs, and the factors of the scores
  float4* pairs = reinterpret_cast<float4*>(sq + NG * 32);
  float* scr = reinterpret_cast<float*>(pairs + NC * 8);  // [NC] partials at a merge
  float4* sums = reinterpret_cast<float4*>(scr) + warp_id() * NG * 2 * 32;  // this warp's sums, between merges
  uint8_t* stages = smem + SH::template FIXED<WIDE ? 8 : 4> - 128;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int task0 = x.parts ? blockIdx.x / x.parts * a.k + blockIdx.x % x.parts * a.W : blockIdx.x * a.W;
  const int ntask = min(a.W, x.parts ? a.k - blockIdx.x % x.parts * a.W : a.total - task0);
  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], U);
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
    // tasks' pages are looked up at once, and their copies issued by a lane each.
    const bool early = a.att_list != nullptr;
    const int32_t* list = early ? a.att_list : a.sel;
    int it = 0, s = 0, round = 0;  // next task, its stage, and how often the ring has gone round
    bool abort = false;
    for (int sr = 0; sr < ntask && !abort;) {
      const int gi = (task0 + sr) / a.k;
      const int pa = task0 + sr - gi * a.k;
      const int pb = min(task0 + ntask, (gi + 1) * a.k) - gi * a.k;
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
        if (flags) fence_proxy_async_global();  // pages written before the flags; every lane copies
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
          // as many of them at once as there are free stages, a lane each (the first STEP wait); STEP at
          // a time in the first round, so that the first pages of an SM's CTAs are not behind the later
          // ones of their neighbours (2 to 4 % of the kernel's time)
          for (int v = 0; v < nb;) {
            int sl = s + lane, rl = round;  // the stage of task it + lane, for lanes below ST
            if (sl >= ST) {
              sl -= ST;
              ++rl;
            }
            bool free = lane < min(round == 0 ? SH::STEP : ST, nb - v);
            if (free && rl > 0)
              free = lane < SH::STEP ? mbar_wait(&empty[sl], (rl - 1) & 1, deadline)
                                     : mbar_test(&empty[sl], (rl - 1) & 1);
            const int n = __ffs(~__ballot_sync(0xffffffffu, free)) - 1;  // (32 of them: ~0 has no bit)
            const int cnt = n < 0 ? 32 : n;
            if (cnt == 0) {
              if (lane == 0) set_err(a.err, NOSA_ERR_TIMEOUT);
              abort = true;
              break;
            }
            const int j = __shfl_sync(0xffffffffu, j_l, (v + lane) & 31);
            const int page = __shfl_sync(0xffffffffu, page_l, (v + lane) & 31);
            if (lane < cnt) {
              info[sl] = make_int2(j, L);
              if (j >= 0) {
                mbar_arrive_expect_tx(&full[sl], SH::STAGE);
                uint8_t* st = stages + (size_t)sl * SH::STAGE;
                bulk_load(st, x.k_pages + (size_t)page * SH::PAGE, SH::PAGE, &full[sl]);
                bulk_load(st + SH::PAGE, x.v_pages + (size_t)page * SH::PAGE, SH::PAGE, &full[sl]);
              } else {
                mbar_arrive(&full[sl]);
              }
            }
            __syncwarp();
            v += cnt;
            it += cnt;
            s += cnt;
            if (s >= ST) {
              s -= ST;
              ++round;
            }
          }
        }
        p = pend;
      }
    }
    // never leave the CTA with a copy in flight
    if (lane < min(ST, it)) {
      const int i = it - 1 - lane;
      mbar_wait(&full[i % ST], (i / ST) & 1, globaltimer() + a.wait_ns);
    }
    return;
  }

  // ---------------------------------------------------------------- consumers
  // S^T = K . q^T: rows are tokens, columns heads. Row i < 8 of a tile of 16 is token
  // (i >> 1) + 4 (i & 1) and row i + 8 that plus 8: lane c4 of the second product then takes tokens
  // c4, c4 + 4, c4 + 8 and c4 + 12, neighbouring rows in one load (two bank conflicts, not four). With
  // G <= 4 column h + 4 repeats head h and carries the low parts of its weights; with G = 8 the low
  // parts take a second product. Columns without a head have q = 0 and are not written.
  const int r = lane >> 2, c4 = lane & 3;
  auto col_head = [&](int n) { return WIDE ? n : (n & 3); };
  const float lo_sign = (!WIDE && c4 >= 2) ? -1.f : 0.f;  // low columns take w - fp16(w)
  const int tok0 = 32 * (warp % U);                       // the unit's first token in its page
  const int rowA = (r >> 1) + 4 * (r & 1);
  // K and V row, and scale, of this lane in tile 0 of the unit
  const uint32_t offK = (tok0 + rowA) * (D / 2) + c4 * (D / 8);
  const uint32_t offV = SH::PAGE + (tok0 + c4) * (D / 2) + r * (D / 16);
  const uint32_t offS = BS * (D / 2) + (tok0 + rowA) * (D / 16);
  constexpr float Y0 = 65536.f + 127.f;  // what x + e is offset by below
  uint32_t met = 0u;
  auto meeting = [&]() -> bool { return kv4_meeting(meet, met++, deadline); };
  auto clear_flags = [&](int gi) {  // every CTA of the group has passed its waits
    if (flags) a.sel_flag[(size_t)gi * kFlagStride] = 0u;
    if (a.e_flag) {
      a.e_flag[(size_t)gi * kFlagStride] = 0u;
      a.e_flag[(size_t)gi * kFlagStride + 3] = 0u;
    }
  };
  uint32_t kilo = 0x64006400u;  // fp16 (1024, 1024), kept in a register
  asm volatile("" : "+r"(kilo));
  int page = warp / U;  // next page of this warp, counted over the CTA's tasks
  int s = page % ST;
  uint32_t phase = (page / ST) & 1;

  for (int sr = 0; sr < ntask;) {
    const int gi = (task0 + sr) / a.k;
    const int pend = min(task0 + ntask, (gi + 1) * a.k) - task0;
    sr = pend;
    // q as fp16 rows: each head's largest magnitude goes to [2^13, 2^14), so that what the
    // conversion drops is 2^-38 of it
    float f0, f1;
    uint32_t down;  // 2^-e1, twice
    {
      const int qhead = col_head(r);
      const bool qok = qhead < a.G;
      const uint16_t* qrow = a.q + ((size_t)(gi / a.Hkv) * a.Hq + (gi % a.Hkv) * a.G + (qok ? qhead : 0)) * D;
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
      // 2^e takes the largest there, or within fp16's range where that is more than 2^126 (q is below
      // 2^-112, and still whole)
      const int e = min(max(140 - static_cast<int>(mx >> 7), -114), 126);
      const float up = __uint_as_float((127 + e) << 23);
      // The sums with q 2^e are up to 2^22 times K's scale: beyond fp32 for large keys of small queries,
      // although the scores are ordinary. So K's scales are taken times 2^-e1 (exact in bf16; it costs
      // nothing that could be measured on long axes), e1 being the least e of the group's finite heads
      // and at least 0: the sums are then no larger than that head's scores, the group's largest, and
      // what a scale loses below 2^-126 changes no score by 2^-100.
      const uint32_t top = __reduce_max_sync(0xffffffffu, mx < 0x7f80u ? mx : 0u);
      const int e1 = min(max(140 - static_cast<int>(top >> 7), 0), 126);
      down = static_cast<uint32_t>(127 - e1) << 7;
      down |= down << 16;
      if (WIDE && lane == 0) s_flag[1] = static_cast<int>(down);  // the same from every warp
      // (above zero, so that a masked score's -inf stays one)
      const float fq = fmaxf(
          __uint_as_float((127 + e1) << 23) * __uint_as_float((127 - e) << 23) * a.scale_log2, 0x1p-126f);
      // from column r of B (all four c4 lanes agree) to columns 2 c4, 2 c4 + 1 of C
      f0 = __shfl_sync(0xffffffffu, fq, 8 * c4);
      f1 = __shfl_sync(0xffffffffu, fq, 8 * c4 + 4);
      // warp g leaves group g's operands in shared memory (all of them would take 16 registers)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (g != warp) continue;
        const uint32_t w[4] = {qv[g].x, qv[g].y, qv[g].z, qv[g].w};  // values (0, 1) .. (6, 7)
        // the fragments pair codes i and i + 4
        sq[g * 32 + lane] = make_uint4(pack_f16(bf16_lo(w[0]) * up, bf16_lo(w[2]) * up),
                                       pack_f16(bf16_hi(w[0]) * up, bf16_hi(w[2]) * up),
                                       pack_f16(bf16_lo(w[1]) * up, bf16_lo(w[3]) * up),
                                       pack_f16(bf16_hi(w[1]) * up, bf16_hi(w[3]) * up));
      }
    }
    bool ok = meeting();
    float acc[2 * NG][4];
#pragma unroll
    for (int mt = 0; mt < 2 * NG; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
    // m: reference of the weights; y: what x + e may reach before m moves (offset by Y0). With pairs
    // m = 0 and f = 1, the pair goes off the scores as they come, and y stays at -inf, so that it does.
    float m0 = kKv4None, m1 = kKv4None, y0 = -INFINITY, y1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    auto paired = [&]() -> bool {
      return __any_sync(0xffffffffu, (y0 == -INFINITY && m0 != kKv4None) || (y1 == -INFINITY && m1 != kKv4None));
    };
    // The tensor cores truncate as they add: an error of about 2^-24 a step, all one way. Every
    // 16 units the accumulators go to sums in shared memory, held relative to (r0, r1).
    float r0 = -INFINITY, r1 = -INFINITY;
    int units = 0;
    auto to_sums = [&](bool first) {
      const float al0 = r0 == m0 ? 1.f : ex2(r0 - m0), al1 = r1 == m1 ? 1.f : ex2(r1 - m1);
#pragma unroll
      for (int mt = 0; mt < 2 * NG; ++mt) {
        float4 v = first ? make_float4(0.f, 0.f, 0.f, 0.f) : sums[mt * 32 + lane];
        v.x = fmaf(v.x, al0, acc[mt][0]);
        v.y = fmaf(v.y, al1, acc[mt][1]);
        v.z = fmaf(v.z, al0, acc[mt][2]);
        v.w = fmaf(v.w, al1, acc[mt][3]);
        sums[mt * 32 + lane] = v;
        acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
      }
      r0 = m0;
      r1 = m1;
    };

    for (; page < pend; page += SH::STEP) {
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], phase, deadline))) {
        set_err(a.err, NOSA_ERR_TIMEOUT);
        return;
      }
      const int2 ti = info[s];
      const uint8_t* st = stages + (size_t)s * SH::STAGE;
      const int nval = ti.x >= 0 ? ti.y - ti.x * BS - tok0 : 0;
      if (nval > 0) {
        // ---- scores of two tiles of 16 tokens: [tile][row A, row B][column]
        float xs[2][2][2];
        uint32_t sv[2][2][NG / 2];
        const uint32_t dn = WIDE ? static_cast<uint32_t>(s_flag[1]) : down;  // (no register left for it)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint32_t ka[NG], kb[NG], sk[2][NG / 2];
          lds_words<NG>(st + offK + (16 * t) * (D / 2), ka);
          lds_words<NG>(st + offK + (16 * t + 8) * (D / 2), kb);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            lds_words<NG / 2>(st + offS + (16 * t + 8 * b) * (D / 16), sk[b]);
#pragma unroll
            for (int g = 0; g < NG / 2; ++g) sk[b][g] = mul_bf162(sk[b][g], dn);
            lds_words<NG / 2>(st + SH::PAGE + offS + (16 * t + 8 * b) * (D / 16), sv[t][b]);
            xs[t][b][0] = xs[t][b][1] = 0.f;
          }
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const uint4 qb = sq[g * 32 + lane];
            const uint32_t kh = ka[g] >> 8, lh = kb[g] >> 8;
            float c[4];
            mma_f16(c, code_pair(ka[g], kilo), code_pair(kb[g], kilo), next_code_pair(ka[g], kilo),
                    next_code_pair(kb[g], kilo), qb.x, qb.y, 0.f, 0.f, 0.f, 0.f);
            mma_f16(c, code_pair(kh, kilo), code_pair(lh, kilo), next_code_pair(kh, kilo), next_code_pair(lh, kilo),
                    qb.z, qb.w, c[0], c[1], c[2], c[3]);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float sc = (g & 1) ? bf16_hi(sk[b][g / 2]) : bf16_lo(sk[b][g / 2]);
              xs[t][b][0] = fmaf(sc, c[2 * b], xs[t][b][0]);
              xs[t][b][1] = fmaf(sc, c[2 * b + 1], xs[t][b][1]);
            }
          }
        }
        if (nval < 32) {
          // rows past the context may hold anything, a NaN scale among it
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int b = 0; b < 2; ++b)
              if (16 * t + 8 * b + rowA >= nval) {
                xs[t][b][0] = xs[t][b][1] = -INFINITY;
#pragma unroll
                for (int g = 0; g < NG / 2; ++g) sv[t][b][g] = 0u;
              }
        }
        // Y0 + e of a token. The bf16 bits of a scale, as an integer over 128, are its base-2 logarithm
        // plus 127 within 0.09. 0x4b000000 + bits is 2^23 + bits as a float: over 128 that is Y0 + e. (e is
        // at least -90, so that 2^-e and sums of it stay finite.)
        auto top_exponent = [&](const uint32_t* scales) {
          float top = 0x1p-90f;
#pragma unroll
          for (int g = 0; g < NG / 2; ++g) top = fmaxf(top, fmaxf(bf16_lo(scales[g]), bf16_hi(scales[g])));
          return 0x1p-7f * __uint_as_float(__byte_perm(__float_as_uint(top), 0x4b000000u, 0x7632));
        };
        float yn0 = -INFINITY, yn1 = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float e = top_exponent(sv[t][b]);
            yn0 = fmaxf(yn0, fmaf(xs[t][b][0], f0, e));
            yn1 = fmaxf(yn1, fmaf(xs[t][b][1], f1, e));
          }
        if (__any_sync(0xffffffffu, yn0 > y0 || yn1 > y1)) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            yn0 = fmaxf(yn0, __shfl_xor_sync(0xffffffffu, yn0, o));
            yn1 = fmaxf(yn1, __shfl_xor_sync(0xffffffffu, yn1, o));
          }
          float hf0, hf1;
          const bool were = paired();
          if (!__any_sync(0xffffffffu, were || fabsf(yn0 == -INFINITY ? 0.f : yn0) > 0x1p20f ||
                                           fabsf(yn1 == -INFINITY ? 0.f : yn1) > 0x1p20f)) {
            const float mn0 = fmaxf(m0, yn0 - (Y0 + 10.f)), mn1 = fmaxf(m1, yn1 - (Y0 + 10.f));
            y0 = fmaxf(y0, yn0 + 3.f);
            y1 = fmaxf(y1, yn1 + 3.f);
            hf0 = half_factor(m0, mn0);
            hf1 = half_factor(m1, mn1);
            m0 = mn0;
            m1 = mn1;
          } else {
            // a becomes the largest score, rounded as the scores are, so that x - a is exact where the
            // weight counts; b what x - a + e reaches, less 10
            float4* pr = pairs + (warp * 4 + c4) * 2;
            const float4 ab = were ? pr[0] : make_float4(m0, m1, 0.f, 0.f);
            const float4 ff = were ? pr[1] : make_float4(f0, f1, 0.f, 0.f);
            float a0 = ab.x, a1 = ab.y, b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                xs[t][b][0] = __fmul_rn(xs[t][b][0], ff.x);
                xs[t][b][1] = __fmul_rn(xs[t][b][1], ff.y);
                a0 = fmaxf(a0, xs[t][b][0]);
                a1 = fmaxf(a1, xs[t][b][1]);
              }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, o));
              a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, o));
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const float e = top_exponent(sv[t][b]) - Y0;
                xs[t][b][0] -= a0;
                xs[t][b][1] -= a1;
                b0 = fmaxf(b0, xs[t][b][0] + e);
                b1 = fmaxf(b1, xs[t][b][1] + e);
              }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, o));
              b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, o));
            }
            const float da0 = ab.x - a0, da1 = ab.y - a1;  // the old pair is a0 + (b + da0)
            b0 = fmaxf(ab.z + da0, b0 - 10.f);
            b1 = fmaxf(ab.w + da1, b1 - 10.f);
            hf0 = ex2(0.5f * (da0 + (ab.z - b0)));
            hf1 = ex2(0.5f * (da1 + (ab.w - b1)));
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                xs[t][b][0] -= b0;
                xs[t][b][1] -= b1;
              }
            if (units >= 16) {  // the sums follow at once, so that their reference stays m
              const float g0 = hf0 * hf0 * (r0 == m0 ? 1.f : ex2(r0 - m0)), g1 = hf1 * hf1 * (r1 == m1 ? 1.f : ex2(r1 - m1));
#pragma unroll 1
              for (int mt = 0; mt < 2 * NG; ++mt) {
                const float4 v = sums[mt * 32 + lane];
                sums[mt * 32 + lane] = make_float4(v.x * g0, v.y * g1, v.z * g0, v.w * g1);
              }
            }
            r0 = r1 = m0 = m1 = 0.f;
            y0 = y1 = -INFINITY;
            f0 = f1 = 1.f;
            __syncwarp();
            if (r == 0) {
              pr[0] = make_float4(a0, a1, b0, b1);
              pr[1] = ff;
            }
            __syncwarp();
          }
          const float al0 = hf0 * hf0, al1 = hf1 * hf1;
          l0 = l0 * hf0 * hf0;
          l1 = l1 * hf1 * hf1;
#pragma unroll
          for (int mt = 0; mt < 2 * NG; ++mt) {
            acc[mt][0] *= al0;
            acc[mt][1] *= al1;
            acc[mt][2] *= al0;
            acc[mt][3] *= al1;
          }
        }
        // ---- O^T += (c - 8)^T . (p s)^T
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float p0 = ex2(fmaf(xs[t][0][0], f0, -m0)), p1 = ex2(fmaf(xs[t][0][1], f1, -m1));
          const float p2 = ex2(fmaf(xs[t][1][0], f0, -m0)), p3 = ex2(fmaf(xs[t][1][1], f1, -m1));
          l0 += p0 + p2;
          l1 += p1 + p3;
          uint32_t vw[4][NG / 2];
#pragma unroll
          for (int i = 0; i < 4; ++i) lds_words<NG / 2>(st + offV + (16 * t + 4 * i) * (D / 2), vw[i]);
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float sA = (g & 1) ? bf16_hi(sv[t][0][g / 2]) : bf16_lo(sv[t][0][g / 2]);
            const float sB = (g & 1) ? bf16_hi(sv[t][1][g / 2]) : bf16_lo(sv[t][1][g / 2]);
            const float w0 = p0 * sA, w1 = p1 * sA, w2 = p2 * sB, w3 = p3 * sB;
            const uint32_t hA = pack_f16(w0, w1), hB = pack_f16(w2, w3);
            const float2 eA2 = __half22float2(*reinterpret_cast<const __half2*>(&hA));
            const float2 eB2 = __half22float2(*reinterpret_cast<const __half2*>(&hB));
            uint32_t b0, b1, d0 = 0u, d1 = 0u;
            if constexpr (WIDE) {
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
              const uint32_t a0 = code_pair(u, kilo), a1 = next_code_pair(u, kilo);
              const uint32_t a2 = code_pair(v, kilo), a3 = next_code_pair(v, kilo);
              float* o = acc[2 * g + mt];
              mma_f16(o, a0, a1, a2, a3, b0, b1, o[0], o[1], o[2], o[3]);
              if constexpr (WIDE) mma_f16(o, a0, a1, a2, a3, d0, d1, o[0], o[1], o[2], o[3]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      if ((++units & 15) == 0) to_sums(units == 16);
      s += SH::STEP;
      if (s >= ST) {
        s -= ST;
        phase ^= 1u;
      }
    }

    // -------------------------------------------------- this CTA's part of the group
    if (units >= 16) {
      const float al0 = r0 == m0 ? 1.f : ex2(r0 - m0), al1 = r1 == m1 ? 1.f : ex2(r1 - m1);
#pragma unroll
      for (int mt = 0; mt < 2 * NG; ++mt) {
        const float4 v = sums[mt * 32 + lane];
        acc[mt][0] = fmaf(v.x, al0, acc[mt][0]);
        acc[mt][1] = fmaf(v.y, al1, acc[mt][1]);
        acc[mt][2] = fmaf(v.z, al0, acc[mt][2]);
        acc[mt][3] = fmaf(v.w, al1, acc[mt][3]);
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    if (paired()) {
      // relative to a alone: with a the largest score, l is at least 1 and the sums are those of
      // 2^(x - a) V, floats for V up to 2^107 (of less than 2^20 tokens)
      const float4 ab = pairs[(warp * 4 + c4) * 2];
      const float h0 = ex2(0.5f * ab.z), h1 = ex2(0.5f * ab.w);
      l0 = l0 * h0 * h0;
      l1 = l1 * h1 * h1;
#pragma unroll
      for (int mt = 0; mt < 2 * NG; ++mt) {
        acc[mt][0] = acc[mt][0] * h0 * h0;
        acc[mt][1] = acc[mt][1] * h1 * h1;
        acc[mt][2] = acc[mt][2] * h0 * h0;
        acc[mt][3] = acc[mt][3] * h1 * h1;
      }
      m0 = ab.x;
      m1 = ab.y;
    }
    if constexpr (!WIDE) {
#pragma unroll
      for (int mt = 0; mt < 2 * NG; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[mt][e] += __shfl_xor_sync(0xffffffffu, acc[mt][e], 2);
    }
    ok = meeting() && ok;  // everyone has read q and its sums
    const int GE = kv4_part_floats(a.G, D);
    if (WIDE || c4 < 2) {
      const int h0 = col_head(2 * c4), h1 = col_head(2 * c4 + 1);
      const bool cv0 = h0 < a.G, cv1 = h1 < a.G;
      float* w = scr + warp * GE;
      if (r == 0) {
        float2* ml = reinterpret_cast<float2*>(w + a.G * D);
        if (cv0) ml[h0] = make_float2(m0, l0);
        if (cv1) ml[h1] = make_float2(m1, l1);
      }
      // rows r and r + 8 of tile mt of group g: values 32g + 4r + 2mt and the next
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int at = 32 * g + 4 * r;
        if (cv0)
          *reinterpret_cast<float4*>(w + h0 * D + at) =
              make_float4(acc[2 * g][0], acc[2 * g][2], acc[2 * g + 1][0], acc[2 * g + 1][2]);
        if (cv1)
          *reinterpret_cast<float4*>(w + h1 * D + at) =
              make_float4(acc[2 * g][1], acc[2 * g][3], acc[2 * g + 1][1], acc[2 * g + 1][3]);
      }
    }
    if (!ok || !meeting()) {
      set_err(a.err, NOSA_ERR_TIMEOUT);
      return;
    }
    // the group's first CTA and how many it has
    const int first = x.parts ? gi * x.parts : gi * a.k / a.W;
    const int nseg = x.parts ? x.parts : (gi * a.k + a.k - 1) / a.W - first + 1;
    // the warps' parts, four values per thread: to the output where this CTA has the whole group,
    // else to its slot of the group's partials
    float* part = a.partials + ((size_t)gi * x.pslots + blockIdx.x - first) * GE;
    float* outg = a.out + ((size_t)(gi / a.Hkv) * a.Hq + (gi % a.Hkv) * a.G) * D;
#pragma unroll 1
    for (int e = tid; e < a.G * (D / 4); e += NC * 32) {
      const int head = e / (D / 4);
      float2 ml[NC];
      float M = -INFINITY, L = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < NC; ++w) {
        ml[w] = reinterpret_cast<const float2*>(scr + w * GE + a.G * D)[head];
        M = fmaxf(M, ml[w].x);
      }
#pragma unroll
      for (int w = 0; w < NC; ++w) {
        const float h = half_factor(ml[w].x, M), f = h * h;
        const float4 y = reinterpret_cast<const float4*>(scr + w * GE)[e];
        L = fmaf(ml[w].y * h, h, L);
        v.x = fmaf(y.x, f, v.x);
        v.y = fmaf(y.y, f, v.y);
        v.z = fmaf(y.z, f, v.z);
        v.w = fmaf(y.w, f, v.w);
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;  // (no token at all: zeros)
      v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
      if (nseg == 1) {
        reinterpret_cast<float4*>(outg)[e] = v;
      } else {
        reinterpret_cast<float4*>(part)[e] = v;
        if (e % (D / 4) == 0) reinterpret_cast<float2*>(part + a.G * D)[head] = make_float2(M, L);
      }
    }
    if (nseg == 1) {
      if (tid == 0) clear_flags(gi);
    } else {
      // The last CTA to publish its part (atomic ticket, no spinning) merges the group. One thread's
      // release and acquire stand for the CTA's: the meetings order the others before and after it.
      if (!meeting()) {
        set_err(a.err, NOSA_ERR_TIMEOUT);
        return;
      }
      if (tid == 0) {
        uint32_t before;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                     : "=r"(before)
                     : "l"(&a.counters[gi])
                     : "memory");
        *s_flag = before == (unsigned)(nseg - 1);
      }
      if (!meeting()) {
        set_err(a.err, NOSA_ERR_TIMEOUT);
        return;
      }
      if (*s_flag) {
        if (!kv4_merge<D, NC, WIDE>(a.partials + (size_t)gi * x.pslots * GE, outg, scr, nseg, a.G, meet, met,
                                    deadline)) {
          set_err(a.err, NOSA_ERR_TIMEOUT);
          return;
        }
        met += 2u;
        if (tid == 0) {
          a.counters[gi] = 0u;
          clear_flags(gi);
        }
      }
    }
    // the scratch turns into sums again once everyone is done with it
    if (sr < ntask && !meeting()) {
      set_err(a.err, NOSA_ERR_TIMEOUT);
      return;
    }
  }
}

}  // namespace nosa

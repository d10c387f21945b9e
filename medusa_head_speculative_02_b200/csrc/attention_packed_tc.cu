// Tree attention over the 4-bit cache on the 5th-generation tensor cores
// (tcgen05), bf16 queries, dh = 128.
//
// out_i = sum_j p_ij s_j c_j / sum_j p_ij over the slots j that query row i
// sees (visible.cuh), p_ij = 2^(x_ij - m_i), x_ij = log2(e) scale sk_j (q_i . c_j),
// where a cached row is scale * c with c = code - zero an integer of at most
// 4 bits and a sign.  The row scales factor out of both products: sk_j
// multiplies a score, sv_j a weight, so the tensor cores only ever see
// integers, exact in fp16.
//
// Keys are the M dimension.  With 64-node trees and no head grouping a
// kv-head has 64 query rows, with single tokens a handful, and an MMA is 128
// rows high; taking the 128 keys of a tile as its rows and the query rows as
// its N (16 to 128) columns wastes none of it:
//   S^T [128 keys x NC rows]  = K   (A, from TMEM)  x Q   (B, shared memory)
//   O^T [128 dims x NC rows] += V^T (A, shared memory, MN-major)
//                             x P^T (B, shared memory, MN-major)
// Unpacking: a code word holds 8 elements; (w & 0x000f000f) read as two fp16
// numbers is code * 2^-24 (subnormal, exact), (w & 0x00f000f0) code * 2^-20,
// and w >> 8 the other four.  One packed subtraction takes off zero.  The
// factor 16 between even and odd nibbles goes into Q (K side) and into the
// output dims (V side), the element order 0 4 1 5 2 6 3 7 into the order of
// Q's dims and of the output rows.  Unpacked K goes straight from registers to
// TMEM, unpacked V to shared memory.
//
// A softmax thread owns one key and NC/2 query rows, so scores need no
// cross-thread work in the common case: the running row maxima are kept in
// shared memory and move only when a score exceeds its row's maximum by more
// than 2^8 (one barrier vote of 128 threads per tile); the row sums stay in
// each thread's registers, one per row, until the end.  Weights times value
// scales, relative to a power of two >= the largest value scale seen times
// 2^-7, are rounded once to fp16.  Statistics, sums and products are fp32.
//
// Warps: 0 TMA (codes and scales, a ring of tiles), 1 MMA issue, then the
// unpack warps (4 for K and 4 for V, or 4 for both with 128 rows) and 8
// softmax warps (2 per TMEM lane quadrant, NC/2 rows each).  TMEM: O^T, two
// S^T buffers, two K buffers.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "visible.cuh"

namespace medusa {
namespace {

constexpr int BK = 128;   // keys per tile
constexpr int DH = 128;
constexpr uint32_t kCodeTile = BK * DH / 2;   // 8 KB
constexpr uint32_t kVTile = BK * DH * 2;      // 32 KB of fp16
constexpr uint32_t kAtom = BK * 128;          // 128 rows of 128 bytes: 16 KB
constexpr float kGrow = 8.0f;                 // log2 of the growth that moves a row maximum
constexpr int kParStages = 8;

template <int NC>
struct Cfg {
  static constexpr int UW = NC <= 64 ? 8 : 4;  // unpack warps
  static constexpr int SW = 8;                 // softmax warps
  static constexpr int kThreads = 32 * (2 + UW + SW);
  static constexpr int CP = NC / 2;            // query rows per softmax thread
  static constexpr int SB = CP < 32 ? CP : 32; // of them at a time
  static constexpr int NSB = CP / SB;
  static constexpr int kStages = NC <= 64 ? 6 : 3;
  static constexpr uint32_t kQ = NC * DH * 2;
  static constexpr uint32_t kP = kAtom * ((NC + 63) / 64);
  static constexpr uint32_t oV = kQ;
  static constexpr uint32_t oP = oV + 2 * kVTile;
  static constexpr uint32_t oCode = oP + 2 * kP;
  static constexpr uint32_t oPar = oCode + kStages * 2 * kCodeTile;
  static constexpr uint32_t oMisc = oPar + kParStages * 2 * BK * 4;
  static constexpr uint32_t kMisc = 512 + 4 * NC * 4 + NC * 8 + 4 * NC * 4 + 2 * 4 * 32 * 4 + 256;
  static constexpr size_t kSmem = 1024 + oMisc + kMisc;
  static constexpr uint32_t kTmemCols = NC <= 32 ? 256 : 512;  // O | S S | K K
  static constexpr uint32_t tS = NC;
  static constexpr uint32_t tK = 3 * NC;
  static_assert(3 * NC + 2 * 64 <= (int)kTmemCols, "TMEM columns");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kQ % 1024 == 0 && oCode % 1024 == 0 && oPar % 128 == 0, "operand alignment");
};

struct PackedParams {
  const __nv_bfloat16* q;
  const int32_t* L;
  const uint32_t* anc;
  const int32_t* depth;
  int B, N, W, K, Hq, Hkv, G, Lcap, R, groups, P, window, sinks;
  float scale2;  // softmax scale * log2(e)
  __nv_bfloat16* out;
  float* po;
  float2* pml;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The 8 codes of a word as four fp16 pairs of (code - zero), pair j holding
// elements j and j + 4; z24 and z20 are -zero * 2^-24 and -zero * 2^-20.
__device__ __forceinline__ void unpack_word(uint32_t w, __half2 z24, __half2 z20, uint32_t* r) {
  const uint32_t v = w >> 8;
  const uint32_t e[4] = {w & 0x000f000fu, w & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 h = __hadd2(*reinterpret_cast<const __half2*>(&e[j]), (j & 1) ? z20 : z24);
    r[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
}
__device__ __forceinline__ void zero_pairs(uint32_t par, __half2& z24, __half2& z20) {
  // unused slots may hold anything: the operands stay finite (their scale,
  // finite or not, only meets scores and weights of rows that see the key)
  const float z = fminf(fmaxf(bf16_hi(par), 0.f), 15.f);
  z24 = __float2half2_rn(-z * 0x1p-24f);
  z20 = __float2half2_rn(-z * 0x1p-20f);
}

template <int SB>
__device__ __forceinline__ void tmem_ld_cols(uint32_t t, float (&v)[SB]) {
  if constexpr (SB == 8) tmem_ld8(t, v);
  else if constexpr (SB == 16) tmem_ld16(t, v);
  else tmem_ld32(t, v);
}

// Tiles of a sequence: the sinks' first, then from the root's window start.
struct Tiles {
  int nh, t_lo, n;  // list index j is tile j (j < nh) or j - nh + t_lo
  __device__ __forceinline__ int tile(int j) const { return j < nh ? j : j - nh + t_lo; }
};
__device__ __forceinline__ Tiles tile_list(int Lb, int N, int window, int sinks) {
  const VisibleRuns vr = visible_runs(Lb, N, window, sinks);
  Tiles t;
  t.t_lo = vr.tail / BK;
  t.nh = min((vr.head + BK - 1) / BK, t.t_lo);
  t.n = t.nh + (Lb + N + BK - 1) / BK - t.t_lo;
  return t;
}

template <int NC>
__global__ void __launch_bounds__(Cfg<NC>::kThreads, 1)
    tree_attn_packed_kernel(const __grid_constant__ CUtensorMap tmKc,
                            const __grid_constant__ CUtensorMap tmVc,
                            const __grid_constant__ CUtensorMap tmKp,
                            const __grid_constant__ CUtensorMap tmVp, const PackedParams p) {
  using C = Cfg<NC>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = sm;
  uint8_t* sV = sm + C::oV;
  uint8_t* sP = sm + C::oP;
  uint8_t* sCode = sm + C::oCode;                // [stage][K 8 KB | V 8 KB]
  uint32_t* sPar = (uint32_t*)(sm + C::oPar);    // [stage][K 128 | V 128]
  uint64_t* bars = (uint64_t*)(sm + C::oMisc);
  uint64_t* code_full = bars;                    // [kStages]
  uint64_t* code_empty = code_full + C::kStages; // [kStages]
  uint64_t* par_full = code_empty + C::kStages;  // [kParStages]
  uint64_t* par_empty = par_full + kParStages;   // [kParStages]
  uint64_t* k_ready = par_empty + kParStages;    // [2] K unpacked in TMEM
  uint64_t* v_ready = k_ready + 2;               // [2] V unpacked in smem
  uint64_t* s_full = v_ready + 2;                // [2] S^T done (K buffer free)
  uint64_t* s_free = s_full + 2;                 // [2] S^T read
  uint64_t* p_full = s_free + 2;                 // [2] P^T written
  uint64_t* pv_done = p_full + 2;                // [2] O^T updated (P and V buffers free)
  uint64_t* mma_done = pv_done + 2;
  uint32_t* tmem_slot = (uint32_t*)(mma_done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  unsigned* qmax = (unsigned*)(tmem_slot + 2);
  static_assert((2 * 6 + 2 * kParStages + 13) * 8 + 16 <= 512, "barrier block");
  float* nm = (float*)(sm + C::oMisc + 512);  // [NC] minus the row maximum (base 2)
  float* fl = nm + NC;                        // [NC] rescale of the sums
  float* fo = fl + NC;                        // [NC] rescale of O
  float* lsum = fo + NC;                      // [NC]
  int* cnode = (int*)(lsum + NC);             // [NC] node of the query row
  int* cdepth = cnode + NC;                   // [NC]
  float* lred = (float*)(cdepth + NC);        // [4][NC]
  unsigned* red = (unsigned*)(lred + 4 * NC); // [2][4][32]
  float* redv = (float*)(red + 2 * 4 * 32);   // [2][4]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kWarps = C::kThreads / 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&code_full[i], 1);
      mbar_init(&code_empty[i], C::UW);
    }
    for (int i = 0; i < kParStages; ++i) {
      mbar_init(&par_full[i], 1);
      mbar_init(&par_empty[i], C::UW + C::SW);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_ready[i], 4);
      mbar_init(&v_ready[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], C::SW);
      mbar_init(&p_full[i], C::SW);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    *qmax = 0u;
    fence_mbar_init();
  }
  griddep_wait();  // prefix lengths, queries and the cache may come from the kernel ahead

  const int id = blockIdx.x;
  const int grp = id % p.groups;
  const int chunk = (id / p.groups) % p.P;
  const int bk = id / p.groups / p.P;
  const int b = bk / p.Hkv, kvh = bk - b * p.Hkv;
  const int row0 = grp * NC;
  const int Lb = p.L[b];
  const bool seq_ok = Lb >= 0 && (long long)Lb + p.N <= p.Lcap;
  Tiles tl{0, 0, 0};
  if (seq_ok) tl = tile_list(Lb, p.N, p.window, p.sinks);
  const int j0 = (int)((long long)tl.n * chunk / p.P);
  const int T = (int)((long long)tl.n * (chunk + 1) / p.P) - j0;

  if (T == 0) {  // no key in this chunk
    griddep_launch_dependents();
    for (int e = threadIdx.x; e < NC; e += C::kThreads) {
      const int r = row0 + e;
      if (r >= p.R) continue;
      if (p.P > 1) {
        p.pml[((size_t)bk * p.P + chunk) * p.R + r] = make_float2(-INFINITY, 0.f);
      } else {
        const int node = r / p.G, g = r - node * p.G;
        uint4* dst = (uint4*)(p.out + (((size_t)b * p.N + node) * p.Hq + (size_t)kvh * p.G + g) * DH);
        for (int i = 0; i < DH / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    return;
  }

  __syncthreads();  // qmax
  // Q: a warp per query row, a lane 4 dims; the largest |q| of the CTA's rows
  // sets one power-of-two factor (fp16 then holds every bf16 value down to
  // 2^-28 of it exactly)
  constexpr int RPW = (NC + kWarps - 1) / kWarps;
  uint2 qv[RPW];
  float qm = 0.f;
#pragma unroll
  for (int i = 0; i < RPW; ++i) {
    const int c = warp + i * kWarps, r = row0 + c;
    qv[i] = make_uint2(0u, 0u);
    if (c < NC && r < p.R) {
      const int node = r / p.G, g = r - node * p.G;
      qv[i] = __ldg(reinterpret_cast<const uint2*>(
                        p.q + (((size_t)b * p.N + node) * p.Hq + (size_t)kvh * p.G + g) * DH) +
                    lane);
    }
    const float f[4] = {bf16_lo(qv[i].x), bf16_hi(qv[i].x), bf16_lo(qv[i].y), bf16_hi(qv[i].y)};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = fabsf(f[e]);
      if (a <= 3.3895314e38f) qm = fmaxf(qm, a);  // finite
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) qm = fmaxf(qm, __shfl_xor_sync(0xffffffffu, qm, o));
  if (lane == 0) atomicMax(qmax, __float_as_uint(qm));
  if (warp == 0) {
    __syncwarp();
    tmem_alloc(tmem_slot, C::kTmemCols);
  }
  for (int c = threadIdx.x; c < NC; c += C::kThreads) {
    const int node = min((row0 + c) / p.G, p.N - 1);
    cnode[c] = node;
    cdepth[c] = p.depth[node];
    nm[c] = 1e30f;  // no maximum yet
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();  // TMEM taken: the next kernel may be scheduled
  // 2^k brings the largest |q| into [2^13, 2^14)
  int kexp = 0;
  if (*qmax != 0u) kexp = min(120, 13 - ((int)(*qmax >> 23) - 127));
  const float qs = __uint_as_float((uint32_t)(127 + kexp) << 23);
#pragma unroll
  for (int i = 0; i < RPW; ++i) {
    const int c = warp + i * kWarps;
    if (c < NC) {
      // dim 8 w + jj + 4 h at position 8 w + 2 jj + h
      const int w = lane >> 1, h = lane & 1;
      __half* dst = (__half*)(sQ + (w >> 3) * (NC * 128) + c * 128 + (((w & 7) ^ (c & 7)) << 4));
      const float f[4] = {bf16_lo(qv[i].x), bf16_hi(qv[i].x), bf16_lo(qv[i].y), bf16_hi(qv[i].y)};
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
        dst[2 * jj + h] = __float2half_rn(f[jj] * ((jj & 1) ? qs * 0.0625f : qs));
    }
  }
  fence_proxy_async_smem();
  __syncthreads();

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      const uint64_t pol = policy_evict_normal();
      int issued = 0;
      for (int j = 0; j < T; ++j) {
        const int st = j % C::kStages, ps = j % kParStages;
        const int key0 = tl.tile(j0 + j) * BK;
        dbg_ok(key0 >= 0 && key0 < Lb + p.N && key0 < p.Lcap, DBG_ATTN_KEY_TILE);
        if (!mbar_wait(&code_empty[st], ((uint32_t)(j / C::kStages) & 1u) ^ 1u, abort_flag)) break;
        if (!mbar_wait(&par_empty[ps], ((uint32_t)(j / kParStages) & 1u) ^ 1u, abort_flag)) break;
        mbar_arrive_expect_tx(&par_full[ps], 2 * BK * 4);
        tma_load_2d(sPar + ps * 2 * BK, &tmKp, &par_full[ps], key0, bk, pol);
        tma_load_2d(sPar + ps * 2 * BK + BK, &tmVp, &par_full[ps], key0, bk, pol);
        mbar_arrive_expect_tx(&code_full[st], 2 * kCodeTile);
        uint8_t* dst = sCode + st * 2 * kCodeTile;
        tma_load_3d(dst, &tmKc, &code_full[st], 0, key0, bk, pol);
        tma_load_3d(dst + kCodeTile, &tmVc, &code_full[st], 0, key0, bk, pol);
        issued = j + 1;
      }
      if (issued < T) {
        // aborted: let the loads already issued land before the CTA exits
        for (int j = (issued > C::kStages ? issued - C::kStages : 0); j < issued; ++j)
          mbar_wait(&code_full[j % C::kStages], (uint32_t)(j / C::kStages) & 1u, nullptr);
        for (int j = (issued > kParStages ? issued - kParStages : 0); j < issued; ++j)
          mbar_wait(&par_full[j % kParStages], (uint32_t)(j / kParStages) & 1u, nullptr);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    // S(0), S(1), then PV(t), S(t + 2): S runs two tiles ahead
    if (lane == 0) {
      constexpr uint32_t idesc_s = umma_idesc_f16_f32(BK, NC, false, false);
      constexpr uint32_t idesc_o = umma_idesc_f16_f32(DH, NC, true, true);
      const uint64_t dq = umma_desc_sw128_kmajor(smem_u32(sQ));
      auto issue_s = [&](int t) -> bool {
        const int bf = t & 1;
        const uint32_t ph = (uint32_t)(t >> 1) & 1u;
        if (!mbar_wait(&k_ready[bf], ph, abort_flag)) return false;
        if (t >= 2 && !mbar_wait(&s_free[bf], ph ^ 1u, abort_flag)) return false;
        tc_fence_after();
        const uint32_t a = tmem + C::tK + (uint32_t)bf * 64u;
        const uint32_t d = tmem + C::tS + (uint32_t)bf * NC;
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk)
          umma_bf16_ts(d, a + (uint32_t)kk * 8u,
                       dq + (uint64_t)(((kk >> 2) * (NC * 128) + (kk & 3) * 32) >> 4), idesc_s,
                       kk > 0 ? 1u : 0u);
        umma_commit(&s_full[bf]);
        return true;
      };
      auto issue_pv = [&](int t) -> bool {
        const int bf = t & 1;
        const uint32_t ph = (uint32_t)(t >> 1) & 1u;
        if (!mbar_wait(&v_ready[bf], ph, abort_flag)) return false;
        if (!mbar_wait(&p_full[bf], ph, abort_flag)) return false;
        tc_fence_after();
        const uint64_t dv = umma_desc_sw128(smem_u32(sV + bf * kVTile), kAtom, 1024u);
        const uint64_t dp = umma_desc_sw128(smem_u32(sP + bf * C::kP), kAtom, 1024u);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          umma_bf16(tmem, dv + (uint64_t)((kk * 16 * 128) >> 4), dp + (uint64_t)((kk * 16 * 128) >> 4),
                    idesc_o, (t > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&pv_done[bf]);
        return true;
      };
      bool ok = true;
      for (int t = 0; t < 2 && t < T && ok; ++t) ok = issue_s(t);
      for (int t = 0; t < T && ok; ++t) {
        ok = issue_pv(t);
        if (ok && t + 2 < T) ok = issue_s(t + 2);
      }
      umma_commit(mma_done);
      mbar_wait(mma_done, 0u, nullptr);
    }
  } else if (warp < 2 + C::UW) {
    // ---------------------------------------------------------------- unpack
    const bool doK = C::UW == 4 || warp < 6, doV = C::UW == 4 || warp >= 6;
    const int qd = warp & 3;
    const int key = qd * 32 + lane;
    const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
    const int sw = (key >> 1) & 3;  // 64-byte swizzle of the code rows
    bool ok = true;
    for (int t = 0; t < T && ok; ++t) {
      const int st = t % C::kStages, ps = t % kParStages, bf = t & 1;
      const uint32_t prev = ((uint32_t)(t >> 1) & 1u) ^ 1u;
      bool good = mbar_wait(&par_full[ps], (uint32_t)(t / kParStages) & 1u, abort_flag) &&
                  mbar_wait(&code_full[st], (uint32_t)(t / C::kStages) & 1u, abort_flag);
      if (!__all_sync(0xffffffffu, good)) break;
      uint32_t kw[16], vw[16], kp = 0u, vp = 0u;
      const uint8_t* row = sCode + st * 2 * kCodeTile + key * 64;
      if (doK) {
        kp = sPar[ps * 2 * BK + key];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(&kw[4 * i]) = *reinterpret_cast<const uint4*>(row + ((i ^ sw) << 4));
      }
      if (doV) {
        vp = sPar[ps * 2 * BK + BK + key];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(&vw[4 * i]) =
              *reinterpret_cast<const uint4*>(row + kCodeTile + ((i ^ sw) << 4));
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&par_empty[ps]);
        mbar_arrive(&code_empty[st]);
      }
      if (doK) {
        if (t >= 2) {  // S(t - 2) has read this K buffer
          good = mbar_wait(&s_full[bf], prev, abort_flag);
          if (!__all_sync(0xffffffffu, good)) break;
        }
        tc_fence_after();
        __half2 z24, z20;
        zero_pairs(kp, z24, z20);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t r[32];
#pragma unroll
          for (int w = 0; w < 8; ++w) unpack_word(kw[hh * 8 + w], z24, z20, r + 4 * w);
          tmem_st32(tmem + lane_base + C::tK + (uint32_t)(bf * 64 + hh * 32), r);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_ready[bf]);
      }
      if (doV) {
        if (t >= 2) {  // PV(t - 2) has read this V buffer
          good = mbar_wait(&pv_done[bf], prev, abort_flag);
          if (!__all_sync(0xffffffffu, good)) break;
        }
        __half2 z24, z20;
        zero_pairs(vp, z24, z20);
        uint8_t* dst = sV + bf * kVTile + key * 128;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
          uint32_t r[4];
          unpack_word(vw[w], z24, z20, r);
          *reinterpret_cast<uint4*>(dst + (w >> 3) * kAtom + (((w & 7) ^ (key & 7)) << 4)) =
              make_uint4(r[0], r[1], r[2], r[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_ready[bf]);
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int hf = (warp - (2 + C::UW)) >> 2;  // query rows [hf CP, hf CP + CP)
    const int qd = warp & 3;
    const int key = qd * 32 + lane;
    const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
    const int gt = (int)threadIdx.x - 32 * (2 + C::UW + 4 * hf);  // thread of the group
    // scores: acc * 2^24 / 2^k * scale * log2(e) * sk
    const float cscale = p.scale2 * ldexpf(1.f, 24 - kexp);
    unsigned long long lacc[C::CP / 2];
#pragma unroll
    for (int c = 0; c < C::CP / 2; ++c) lacc[c] = 0ull;
    float vref[C::NSB];
#pragma unroll
    for (int s = 0; s < C::NSB; ++s) vref[s] = 0x1p-120f;
    bool ok = true, err = false;
    for (int t = 0; t < T && ok; ++t) {
      const int bf = t & 1, ps = t % kParStages;
      const uint32_t ph = (uint32_t)(t >> 1) & 1u;
      const int tile = tl.tile(j0 + t);
      bool good = mbar_wait(&par_full[ps], (uint32_t)(t / kParStages) & 1u, abort_flag);
      const uint32_t kp = sPar[ps * 2 * BK + key], vp = sPar[ps * 2 * BK + BK + key];
      __syncwarp();
      if (lane == 0) mbar_arrive(&par_empty[ps]);
      good = good && mbar_wait(&s_full[bf], ph, abort_flag);
      // the P buffer: PV(t - 2) has read it
      if (t >= 2) good = good && mbar_wait(&pv_done[bf], ph ^ 1u, abort_flag);
      err = err || !__all_sync(0xffffffffu, good);
      tc_fence_after();
      const float ks = bf16_lo(kp) * cscale;
      const unsigned long long ks2 = f2_pack(ks, ks);
      const int slot = tile * BK + key;
      // tiles with a tree or unused slot, or one that is not in every row's window
      const bool masked = (long long)(tile + 1) * BK > Lb ||
                          (p.window > 0 && (long long)tile * BK <= (long long)Lb + p.K - p.window);
#pragma unroll
      for (int s = 0; s < C::NSB; ++s) {
        const int col0 = hf * C::CP + s * C::SB;
        uint32_t vm = 0xffffffffu;  // rows that see this key
        if (masked) {
          vm = 0u;
          if (slot < Lb + p.N) {
            const int a = slot - Lb;
            const int pos = a < 0 ? slot : Lb + __ldg(p.depth + a);
            for (int c = 0; c < C::SB; ++c) {
              bool vis = in_window(pos, Lb + cdepth[col0 + c], p.window, p.sinks);
              if (a >= 0)
                vis = vis && ((__ldg(p.anc + (size_t)cnode[col0 + c] * p.W + (a >> 5)) >> (a & 31)) & 1u);
              vm |= (uint32_t)vis << c;
            }
          }
        }
        const uint32_t ts = tmem + lane_base + C::tS + (uint32_t)(bf * NC + col0);
        const float sv = vm != 0u ? bf16_lo(vp) : 0.f;
        unsigned long long y[C::SB / 2];
        const ulonglong2* nm2 = reinterpret_cast<const ulonglong2*>(nm + col0);
        float ymax = -INFINITY;
        auto scores = [&]() {  // relative to the row maxima, base 2
          constexpr int LD = C::SB < 16 ? C::SB : 16;
#pragma unroll
          for (int c0 = 0; c0 < C::SB; c0 += LD) {
            float v[LD];
            tmem_ld_cols<LD>(ts + (uint32_t)c0, v);
#pragma unroll
            for (int c = 0; c < LD / 4; ++c) {
              const ulonglong2 n2 = nm2[c0 / 4 + c];
              y[c0 / 2 + 2 * c] = f2_fma(f2_pack(v[4 * c], v[4 * c + 1]), ks2, n2.x);
              y[c0 / 2 + 2 * c + 1] = f2_fma(f2_pack(v[4 * c + 2], v[4 * c + 3]), ks2, n2.y);
            }
          }
          if (masked) {
#pragma unroll
            for (int c = 0; c < C::SB / 2; ++c) {
              float a, d;
              f2_unpack(y[c], a, d);
              a = (vm >> (2 * c)) & 1u ? a : -INFINITY;
              d = (vm >> (2 * c + 1)) & 1u ? d : -INFINITY;
              y[c] = f2_pack(a, d);
            }
          }
        };
        scores();
#pragma unroll
        for (int c = 0; c < C::SB / 2; ++c) {
          float a, d;
          f2_unpack(y[c], a, d);
          ymax = fmaxf(ymax, fmaxf(a, d));
        }
        if (bar_red_or(1 + hf, 128, err || ymax > kGrow || fabsf(sv) > vref[s])) {
          // a row maximum or the value scale grew: move both for the whole
          // group, rescale the sums and O
#pragma unroll 1
          for (int c = 0; c < C::SB; ++c) {
            float x = tmem_ld1(ts + (uint32_t)c);
            x = (vm >> c) & 1u ? x * ks : -INFINITY;
            const unsigned o = __reduce_max_sync(0xffffffffu, f32_order(x));
            if (lane == 0) red[(hf * 4 + qd) * 32 + c] = o;
          }
          const unsigned sb = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(sv)) < 0x7f800000u
                                                                  ? __float_as_uint(fabsf(sv))
                                                                  : 0u);
          if (lane == 0) redv[hf * 4 + qd] = __uint_as_float(sb);
          if (bar_red_or(1 + hf, 128, err)) {
            ok = false;
            break;
          }
          // power of two >= the largest scale, kept in [2^-120, 2^119]
          const float big = fmaxf(fmaxf(redv[hf * 4], redv[hf * 4 + 1]),
                                  fmaxf(redv[hf * 4 + 2], redv[hf * 4 + 3]));
          const uint32_t bb = __float_as_uint(big);
          const int ex = min(246, max(7, (int)((bb >> 23) + ((bb & 0x7fffffu) ? 1 : 0))));
          const float nref = fmaxf(vref[s], __uint_as_float((uint32_t)ex << 23));
          const float fv = vref[s] / nref;
          vref[s] = nref;
          if (gt < C::SB) {
            const unsigned* rr = red + hf * 128 + gt;
            const float x = order_f32(max(max(rr[0], rr[32]), max(rr[64], rr[96])));
            const float old = nm[col0 + gt];
            float f = 1.f;
            if (x != -INFINITY && (old == 1e30f || !(x + old <= kGrow))) {
              f = old == 1e30f ? 0.f : exp2f(-old - x);
              nm[col0 + gt] = -x;
            }
            fl[col0 + gt] = f;
            fo[col0 + gt] = f * fv;
          }
          named_bar_sync(1 + hf, 128);
#pragma unroll
          for (int c = 0; c < C::SB / 2; ++c)
            lacc[s * (C::SB / 2) + c] =
                f2_mul(lacc[s * (C::SB / 2) + c],
                       *reinterpret_cast<const unsigned long long*>(fl + col0 + 2 * c));
          if (t > 0) {  // O holds PV(0 .. t - 1)
            const bool w_ok = mbar_wait(&pv_done[(t - 1) & 1], (uint32_t)((t - 1) >> 1) & 1u, abort_flag);
            if (__all_sync(0xffffffffu, w_ok)) {
              tc_fence_after();
#pragma unroll 1
              for (int c0 = 0; c0 < C::SB; c0 += 8) {
                float o8[8];
                const uint32_t ta = tmem + lane_base + (uint32_t)(col0 + c0);
                tmem_ld8(ta, o8);
#pragma unroll
                for (int e = 0; e < 8; ++e) o8[e] *= fo[col0 + c0 + e];
                tmem_st8(ta, o8);
              }
            } else {
              err = true;  // reported at the next vote
            }
          }
          scores();
        }
        if (s == C::NSB - 1) {  // S^T read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[bf]);
        }
        // weights, and weights x value scales as fp16 in this key's row of P^T
        const float vn = sv * __uint_as_float((261u << 23) - __float_as_uint(vref[s]));
        const unsigned long long vn2 = f2_pack(vn, vn);
        uint8_t* prow = sP + bf * C::kP + (col0 >> 6) * kAtom + key * 128;
#pragma unroll
        for (int c8 = 0; c8 < C::SB / 8; ++c8) {
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = c8 * 4 + e;
            float a, d;
            f2_unpack(y[c], a, d);
            const unsigned long long w2 = f2_pack(ex2_approx(a), ex2_approx(d));
            lacc[s * (C::SB / 2) + c] = f2_add(lacc[s * (C::SB / 2) + c], w2);
            f2_unpack(f2_mul(w2, vn2), a, d);
            if (masked) {  // 0, not 0 * NaN, for rows that do not see the key
              a = (vm >> (2 * c)) & 1u ? a : 0.f;
              d = (vm >> (2 * c + 1)) & 1u ? d : 0.f;
            }
            const __half2 hh = __floats2half2_rn(a, d);
            h[e] = *reinterpret_cast<const uint32_t*>(&hh);
          }
          *reinterpret_cast<uint4*>(prow + (((((col0 & 63) >> 3) + c8) ^ (key & 7)) << 4)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      if (!ok) break;
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[bf]);
    }
    ok = ok && !err;
    if (ok) {
      const bool good = mbar_wait(&pv_done[(T - 1) & 1], (uint32_t)((T - 1) >> 1) & 1u, abort_flag);
      ok = __all_sync(0xffffffffu, good);
    }
    // row sums over the 128 keys
#pragma unroll
    for (int c = 0; c < C::CP / 2; ++c) {
      float a, d;
      f2_unpack(lacc[c], a, d);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        d += __shfl_xor_sync(0xffffffffu, d, o);
      }
      if (lane == 0) {
        lred[qd * NC + hf * C::CP + 2 * c] = a;
        lred[qd * NC + hf * C::CP + 2 * c + 1] = d;
      }
    }
    const bool bad = bar_red_or(1 + hf, 128, !ok);
    if (gt < C::CP) {
      const int c = hf * C::CP + gt;
      lsum[c] = (lred[c] + lred[NC + c]) + (lred[2 * NC + c] + lred[3 * NC + c]);
    }
    named_bar_sync(1 + hf, 128);
    if (!bad) {
      tc_fence_after();
      // TMEM lane = position 8 w + 2 jj + h of dim 8 w + jj + 4 h
      const int jj = (key >> 1) & 3;
      const int dim = (key & ~7) + jj + 4 * (key & 1);
      const float unit = (jj & 1) ? 0x1p13f : 0x1p17f;  // 2^20 or 2^24, times 2^-7
#pragma unroll
      for (int s = 0; s < C::NSB; ++s) {
#pragma unroll 1
        for (int c0 = 0; c0 < C::SB; c0 += 8) {
          const int col = hf * C::CP + s * C::SB + c0;
          if (row0 + col >= p.R) break;  // warp-uniform
          float o8[8];
          tmem_ld8(tmem + lane_base + (uint32_t)col, o8);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = row0 + col + e;
            if (r >= p.R) continue;
            const float o = o8[e] * unit * vref[s];
            const float l = lsum[col + e];
            if (p.P == 1) {
              const int node = r / p.G, g = r - node * p.G;
              p.out[(((size_t)b * p.N + node) * p.Hq + (size_t)kvh * p.G + g) * DH + dim] =
                  __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
            } else {
              const size_t prow = ((size_t)bk * p.P + chunk) * p.R + r;
              p.po[prow * DH + dim] = o;
              if (key == 0) {
                const float m = nm[col + e];
                // a sum of NaN must reach the merge, which skips m = -inf
                p.pml[prow] = make_float2(m == 1e30f ? (l != l ? 0.f : -INFINITY) : (m != m ? 0.f : -m), l);
              }
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

struct PackedPlan {
  int NC, R, groups, P;
  long long ctas;
  size_t off_o, off_ml, total;
};

PackedPlan packed_plan(const medusa_tree* t, int B, int Hq, int Hkv, int Lcap, int window,
                       int sinks) {
  PackedPlan p;
  p.R = t->N * (Hq / Hkv);
  p.NC = p.R <= 16 ? 16 : p.R <= 32 ? 32 : p.R <= 64 ? 64 : 128;
  p.groups = (p.R + p.NC - 1) / p.NC;
  const long long units = (long long)B * Hkv * p.groups;
  const long long T = (ext_max_keys(Lcap, t->N, window, sinks) + BK - 1) / BK + (window > 0 ? 1 : 0);
  // key chunks: least (waves of CTAs) x (tiles of a CTA + its start and end,
  // about 4 tiles' time)
  const long long sms = num_sms();
  long long best = 0;
  p.P = 1;
  for (long long P = 1; units > 0 && P <= 64 && P <= T; ++P) {
    const long long cost = ((units * P + sms - 1) / sms) * ((T + P - 1) / P + 4 + (P > 1 ? 2 : 0));
    if (best == 0 || cost < best) {
      best = cost;
      p.P = (int)P;
    }
  }
  p.ctas = units * p.P;
  WsCarver w;
  const size_t rows = p.P > 1 ? (size_t)B * Hkv * p.P * p.R : 0;
  p.off_o = w.take<float>(rows * DH);
  p.off_ml = w.take<float2>(rows);
  p.total = w.total();
  return p;
}

template <int NC>
int packed_run(const CUtensorMap& kc, const CUtensorMap& vc, const CUtensorMap& kp,
               const CUtensorMap& vp, const PackedParams& p, long long ctas, cudaStream_t st) {
  using C = Cfg<NC>;
  static std::atomic<bool> done[64];
  int rc = ensure_max_smem(tree_attn_packed_kernel<NC>, (int)C::kSmem, done,
                           "cudaFuncSetAttribute(tree_attn_packed_kernel)");
  if (rc) return rc;
  cudaError_t e = launch_pdl(tree_attn_packed_kernel<NC>, dim3((unsigned)ctas), dim3(C::kThreads),
                             C::kSmem, st, kc, vc, kp, vp, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail(e, "tree_attn_packed_kernel launch");
}

}  // namespace

bool attention_packed_tc_eligible(int dtype, int dh) { return dtype == MEDUSA_BF16 && dh == DH; }

size_t attention_packed_tc_workspace(const medusa_tree* t, int B, int Hq, int Hkv, int Lcap,
                                     int window, int sinks) {
  return packed_plan(t, B, Hq, Hkv, Lcap, window, sinks).total;
}

int attention_packed_tc_launch(const AttnArgs& a, const PackedCache& c, cudaStream_t st) {
  const medusa_tree* t = a.tree;
  const PackedPlan pl = packed_plan(t, a.B, a.Hq, a.Hkv, a.Lcap, a.window, a.sinks);
  if (pl.ctas > 0x7fffffffLL || (long long)a.B * a.Hkv > 0x7fffffffLL)
    return fail(MEDUSA_ERR_UNSUPPORTED, "too many query rows for one launch");
  alignas(64) CUtensorMap mKc, mVc, mKp, mVp;
  const uint64_t heads = (uint64_t)a.B * a.Hkv;
  {
    const uint64_t dims[3] = {DH / 2, (uint64_t)a.Lcap, heads};
    const uint64_t strides[2] = {DH / 2, (uint64_t)a.Lcap * (DH / 2)};
    const uint32_t box[3] = {DH / 2, BK, 1};
    int rc = make_tmap_u8_sw64(&mKc, c.k_codes, 3, dims, strides, box);
    if (rc) return rc;
    rc = make_tmap_u8_sw64(&mVc, c.v_codes, 3, dims, strides, box);
    if (rc) return rc;
  }
  {
    const uint64_t dims[2] = {(uint64_t)a.Lcap, heads};
    const uint64_t strides[1] = {(uint64_t)a.Lcap * 4};
    const uint32_t box[2] = {BK, 1};
    int rc = make_tmap_u32(&mKp, c.k_par, 2, dims, strides, box);
    if (rc) return rc;
    rc = make_tmap_u32(&mVp, c.v_par, 2, dims, strides, box);
    if (rc) return rc;
  }
  PackedParams p;
  p.q = (const __nv_bfloat16*)a.q;
  p.L = a.L;
  p.anc = t->d_anc;
  p.depth = t->d_depth;
  p.B = a.B;
  p.N = t->N;
  p.W = t->W;
  p.K = t->K;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.Lcap = a.Lcap;
  p.R = pl.R;
  p.groups = pl.groups;
  p.P = pl.P;
  p.window = a.window;
  p.sinks = a.sinks;
  p.scale2 = a.scale * 1.4426950408889634f;
  p.out = (__nv_bfloat16*)a.out;
  p.po = (float*)((uint8_t*)a.ws + pl.off_o);
  p.pml = (float2*)((uint8_t*)a.ws + pl.off_ml);
  int rc;
  switch (pl.NC) {
    case 16: rc = packed_run<16>(mKc, mVc, mKp, mVp, p, pl.ctas, st); break;
    case 32: rc = packed_run<32>(mKc, mVc, mKp, mVp, p, pl.ctas, st); break;
    case 64: rc = packed_run<64>(mKc, mVc, mKp, mVp, p, pl.ctas, st); break;
    default: rc = packed_run<128>(mKc, mVc, mKp, mVp, p, pl.ctas, st); break;
  }
  if (rc || pl.P == 1) return rc;
  return attention_combine_launch(a, p.po, p.pml, pl.P, st);
}

}  // namespace medusa

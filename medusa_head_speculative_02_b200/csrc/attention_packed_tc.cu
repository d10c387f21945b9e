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
// its N (32, 64 or 128) columns wastes none of it:
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
// A softmax thread owns one key and up to 64 query rows, so scores need no
// cross-thread work in the common case: the running row maxima are kept in
// shared memory and move only when a score exceeds its row's maximum by more
// than 2^8 (one barrier vote of 128 threads per tile); the row sums stay in
// each thread's registers, one per row, until the end.  Weights times value
// scales, relative to a power of two >= the largest value scale seen times
// 2^-7, are rounded once to fp16.  Statistics, sums and products are fp32.
//
// What bounds it (64-node trees): the chain products -> softmax -> products of
// a tile, and per tile and softmax thread the 16 to 64 rows' multiply-add,
// exponential and rounding.  64 rows, 37 heads x 4 sequences of 8K: 104 us of 26
// at the HBM rate, one wave of 148 CTAs with 65 tiles each; 40 heads x 8
// sequences of 1K to 4K: 125 us of 19; 64 rows, 32 heads, 2K prefix (the 7B
// verify step): 20.9 us launch to launch, against a cache of 1.6 us of HBM time.
//
// Key chunks fill the GPU when there are few (sequence, kv-head) pairs; up to 8
// of them form a cluster and merge through distributed shared memory when all
// clusters run at once (7B: 23.6 us with partial rows in the workspace and a
// second kernel).
//
// TMEM: O^T, two S^T buffers, two K buffers.
// This source is compiled without relocatable device code: register splits
// between warpgroups (setmaxnreg) are only honoured then, and without them the
// softmax threads' 64 rows would spill.  (With 128 columns 20 bytes a thread
// still do; 32 and 64 columns spill nothing.)
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <type_traits>

#define MEDUSA_OWN_STATUS
#include "common.cuh"
#include "internal.h"
#include "visible.cuh"

namespace medusa {
namespace cg = cooperative_groups;
namespace {

constexpr int kMaxClusterChunks = 8;  // portable cluster size
constexpr int BK = 128;   // keys per tile
constexpr int DH = 128;
constexpr uint32_t kCodeTile = BK * DH / 2;   // 8 KB
constexpr uint32_t kVTile = BK * DH * 2;      // 32 KB of fp16
constexpr uint32_t kAtom = BK * 128;          // 128 rows of 128 bytes: 16 KB
constexpr float kGrow = 8.0f;                 // log2 of the growth that moves a row maximum
constexpr uint32_t kStage = 2 * kCodeTile + 2 * BK * 4;  // K | V codes, K | V (scale, zero)
constexpr int kScaleBufs = 4;

// Warpgroups: 0 TMA and MMA issue, then unpack, then two of softmax.  Up to
// 32 query rows the two softmax warpgroups take alternate key tiles, all rows
// each, with their own maxima, sums and O^T (merged at the end): a tile's
// chain of waits may then last two tiles.  64 and 128 rows are split in halves
// (at 64 rows, 37 heads x 4 sequences of 8K: halves 104 us, alternate tiles 121).
template <int NC>
struct Cfg {
  static constexpr int kSets = NC <= 32 ? 2 : 1;
  static constexpr int CP = kSets == 2 ? NC : NC / 2;  // query rows per softmax thread
  static constexpr int BS = 32;                        // of them in one mask word
  static constexpr int NB = CP / BS;
  static constexpr int kState = 2 * CP;                // (softmax warpgroup, row) states
  static constexpr int kUnpackWgs = NC <= 32 ? 2 : 1;  // K and V apart, or one for both
  static constexpr int kThreads = 128 * (3 + kUnpackWgs);
  // registers per thread after the split; their sum stays within the launch's
  static constexpr int kRegs0 = NC <= 32 ? 64 : 56;
  static constexpr int kRegsUnpack = NC <= 32 ? 72 : 80;
  static constexpr int kRegsSoftmax = NC <= 32 ? 136 : 184;
  static constexpr int kRegsLaunch = NC <= 32 ? 96 : 128;  // what 640 or 512 threads get
  static_assert(kRegs0 + kUnpackWgs * kRegsUnpack + 2 * kRegsSoftmax <=
                    (3 + kUnpackWgs) * kRegsLaunch, "register split");
  static constexpr int kStages = NC <= 64 ? 6 : 3;
  static constexpr uint32_t kQ = NC * DH * 2;
  static constexpr uint32_t kP = kAtom * ((NC + 63) / 64);
  static constexpr uint32_t oV = kQ;
  static constexpr uint32_t oP = oV + 2 * kVTile;
  static constexpr uint32_t oCode = oP + 2 * kP;
  static constexpr uint32_t oScale = oCode + kStages * kStage;
  static constexpr uint32_t oMisc = oScale + kScaleBufs * 2 * BK * 4;
  static constexpr uint32_t kMisc = 256 + 4 * kState * 4 + 3 * NC * 4 + 2 * 4 * CP * 4 +
                                    2 * (4 * 4 + NB * 4 + 4) + (NC / BS) * (MEDUSA_MAX_K + 2) * 4;
  static constexpr size_t kSmem = 1024 + oMisc + kMisc;
  static constexpr uint32_t kTmemCols = NC <= 32 ? 256 : 512;  // O (per set) | S S | K K
  // fused merge: partial rows [NC][kOS] fp32 and their (maximum, sum), over V and P^T
  static constexpr int kOS = DH + 4;
  static constexpr uint32_t oMl = oV + NC * kOS * 4;
  static_assert(oMl + NC * 8 <= oCode, "partial rows");
  static constexpr uint32_t tS = kSets * NC;
  static constexpr uint32_t tK = tS + 2 * NC;
  static_assert(tK + 2 * 64 <= kTmemCols, "TMEM columns");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kQ % 1024 == 0 && oCode % 1024 == 0 && oScale % 128 == 0, "operand alignment");
};

struct PackedParams {
  const __nv_bfloat16* q;
  const int32_t* L;
  const uint32_t* anc;
  const int32_t* depth;
  const int32_t* parent;
  int B, N, W, K, Hq, Hkv, G, Lcap, R, groups, P, window, sinks;
  int fuse;      // key-major: the P chunks are a cluster and merge in it
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

// Reduction over the lanes of a warp of 32 per-lane values each, transposed
// on the way: lane i returns value i over all lanes.
template <typename Op>
__device__ __forceinline__ float col_reduce(float (&a)[32], int lane, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float keep = up ? a[i + o] : a[i], send = up ? a[i] : a[i + o];
      a[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  return a[0];
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// Merge of the P chunks of a (sequence, kv-head) by the cluster they form,
// between two cluster_sync of every thread: rank c takes rows [c per, (c + 1)
// per), one of `warps` warps a row, from every rank's shared memory.
template <int NC>
__device__ __forceinline__ void merge_chunks(uint8_t* sm, int rank, int b, int kvh, int warp, int warps,
                                             const PackedParams& p) {
  using C = Cfg<NC>;
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  const int per = (p.R + p.P - 1) / p.P;
  const int r1 = min(p.R, (rank + 1) * per);
  for (int r = rank * per + warp; r < r1; r += warps) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < p.P) ml = cl.map_shared_rank(reinterpret_cast<float2*>(sm + C::oMl), lane)[r];
    float M = ml.x;
#pragma unroll
    for (int o = kMaxClusterChunks / 2; o > 0; o >>= 1)
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    M = __shfl_sync(0xffffffffu, M, 0);
    // a chunk without a visible key has no row; one whose weight is 0 counts, as
    // its sum or row may be NaN
    const bool has = ml.x != -INFINITY;
    const unsigned seen = __ballot_sync(0xffffffffu, has);
    const float w = has ? exp2f(ml.x - M) : 0.f;
    float Ls = has ? w * ml.y : 0.f;
#pragma unroll
    for (int o = kMaxClusterChunks / 2; o > 0; o >>= 1) Ls += __shfl_xor_sync(0xffffffffu, Ls, o);
    Ls = __shfl_sync(0xffffffffu, Ls, 0);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < p.P; ++c) {
      const float wc = __shfl_sync(0xffffffffu, w, c);
      if (!((seen >> c) & 1u)) continue;
      const float4 o = reinterpret_cast<const float4*>(
          cl.map_shared_rank(reinterpret_cast<float*>(sm + C::oV), c) + (size_t)r * C::kOS)[lane];
      acc.x = fmaf(wc, o.x, acc.x);
      acc.y = fmaf(wc, o.y, acc.y);
      acc.z = fmaf(wc, o.z, acc.z);
      acc.w = fmaf(wc, o.w, acc.w);
    }
    const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
    const int node = r / p.G, g = r - node * p.G;
    __nv_bfloat16* dst =
        p.out + (((size_t)b * p.N + node) * p.Hq + (size_t)kvh * p.G + g) * DH + 4 * lane;
    __align__(8) __nv_bfloat162 h[2] = {__floats2bfloat162_rn(acc.x * inv, acc.y * inv),
                                        __floats2bfloat162_rn(acc.z * inv, acc.w * inv)};
    *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(h);
  }
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
  uint8_t* sCode = sm + C::oCode;                // [stage]
  float* sScale = (float*)(sm + C::oScale);      // [4][K 128 | V 128]
  uint64_t* bars = (uint64_t*)(sm + C::oMisc);
  uint64_t* code_full = bars;                    // [kStages]
  uint64_t* code_empty = code_full + C::kStages; // [kStages]
  uint64_t* k_ready = code_empty + C::kStages;   // [2] K unpacked in TMEM, scales in smem
  uint64_t* pv_ready = k_ready + 2;              // [2] V unpacked and P^T written
  uint64_t* s_full = pv_ready + 2;               // [2] S^T done (K buffer free)
  uint64_t* s_free = s_full + 2;                 // [2] S^T and scales read
  uint64_t* pv_done = s_free + 2;                // [2] O^T updated (P and V buffers free)
  uint64_t* mma_done = pv_done + 2;
  uint32_t* tmem_slot = (uint32_t*)(mma_done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  unsigned* qmax = (unsigned*)(tmem_slot + 2);
  static_assert((2 * 6 + 11) * 8 + 16 <= 256, "barrier block");
  // per (softmax warpgroup, row)
  float* nm = (float*)(sm + C::oMisc + 256);  // minus the row maximum (base 2)
  float* fl = nm + C::kState;                 // rescale of the sums; at the end the row sum
  float* fo = fl + C::kState;                 // rescale of O; at the end its factor (< 0: no O)
  float* fd = fo + C::kState;                 // shift of the scores
  int* cnode = (int*)(fd + C::kState);        // [NC] node of the query row
  int* cdepth = cnode + NC;                   // [NC]
  int* crow = cdepth + NC;                    // [NC] node * Hq + query head, -1 past the last row
  float* red = (float*)(crow + NC);           // [warpgroup][4][CP]
  float* redv = red + 2 * 4 * C::CP;          // [warpgroup][4]
  uint32_t* unset_s = (uint32_t*)(redv + 8);  // [warpgroup][NB] rows without a maximum yet
  float* vref_s = (float*)(unset_s + 2 * C::NB);      // [warpgroup]
  uint32_t* shallow = (uint32_t*)(vref_s + 2);        // [NC / BS][x]: rows of depth < x

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr int kWarps = C::kThreads / 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&code_full[i], 1);
      mbar_init(&code_empty[i], 4 * C::kUnpackWgs);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_ready[i], 4);
      mbar_init(&pv_ready[i], 4 + 8 / C::kSets);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 8 / C::kSets);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    *qmax = 0u;
    fence_mbar_init();
  }
  griddep_wait();  // prefix lengths, queries and the cache may come from the kernel ahead

  const int chunk = blockIdx.x % p.P;  // (fused: the rank in the cluster)
  const int bk = blockIdx.x / p.P;
  const int b = bk / p.Hkv, kvh = bk - b * p.Hkv;
  const int Lb = p.L[b];
  const bool seq_ok = Lb >= 0 && (long long)Lb + p.N <= p.Lcap;
  Tiles tl{0, 0, 0};
  if (seq_ok) tl = tile_list(Lb, p.N, p.window, p.sinks);
  const int j0 = (int)((long long)tl.n * chunk / p.P);
  const int T = (int)((long long)tl.n * (chunk + 1) / p.P) - j0;

  if (T == 0) {  // no key in this chunk
    griddep_launch_dependents();
    if (p.fuse) {
      if (threadIdx.x < NC)
        reinterpret_cast<float2*>(sm + C::oMl)[threadIdx.x] = make_float2(-INFINITY, 0.f);
      cluster_sync();
      merge_chunks<NC>(sm, chunk, b, kvh, warp, kWarps, p);
      cluster_sync();
      return;
    }
    for (int r = threadIdx.x; r < p.R; r += C::kThreads) {
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

  // the first code tiles are under way while Q is prepared
  const uint64_t pol = policy_evict_normal();
  auto load_tile = [&](int j) {
    const int st = j % C::kStages;
    const int key0 = tl.tile(j0 + j) * BK;
    dbg_ok(key0 >= 0 && key0 < Lb + p.N && key0 < p.Lcap, DBG_ATTN_KEY_TILE);
    mbar_arrive_expect_tx(&code_full[st], kStage);
    uint8_t* dst = sCode + st * kStage;
    tma_load_3d(dst, &tmKc, &code_full[st], 0, key0, bk, pol);
    tma_load_2d(dst + 2 * kCodeTile, &tmKp, &code_full[st], key0, bk, pol);
    tma_load_2d(dst + 2 * kCodeTile + BK * 4, &tmVp, &code_full[st], key0, bk, pol);
    tma_load_3d(dst + kCodeTile, &tmVc, &code_full[st], 0, key0, bk, pol);
  };
  const int early = min(T, C::kStages);
  if (threadIdx.x == 0)
    for (int j = 0; j < early; ++j) load_tile(j);
  __syncthreads();  // qmax
  // Q: a warp per query row, a lane 4 dims; the largest |q| of the CTA's rows
  // sets one power-of-two factor (fp16 then holds every bf16 value down to
  // 2^-26 of it exactly, the odd pairs' 1/16 included)
  constexpr int RPW = (NC + kWarps - 1) / kWarps;
  uint2 qv[RPW];
  float qm = 0.f;
#pragma unroll
  for (int i = 0; i < RPW; ++i) {
    const int r = warp + i * kWarps;
    qv[i] = make_uint2(0u, 0u);
    if (r < p.R) {
      const int node = r / p.G, g = r - node * p.G;
      qv[i] = reinterpret_cast<const uint2*>(
          p.q + (((size_t)b * p.N + node) * p.Hq + (size_t)kvh * p.G + g) * DH)[lane];
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
    const int node = min(c / p.G, p.N - 1);
    cnode[c] = node;
    cdepth[c] = p.depth[node];
    crow[c] = c < p.R ? node * p.Hq + kvh * p.G + (c - node * p.G) : -1;
  }
  for (int c = threadIdx.x; c < C::kState; c += C::kThreads) nm[c] = 0.f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);  // warp-uniform
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
  for (int e = threadIdx.x; e < (NC / C::BS) * (MEDUSA_MAX_K + 2); e += C::kThreads) {
    const int g = e / (MEDUSA_MAX_K + 2), x = e - g * (MEDUSA_MAX_K + 2);
    uint32_t m = 0u;
    for (int c = 0; c < C::BS; ++c) m |= (uint32_t)(cdepth[g * C::BS + c] < x) << c;
    shallow[e] = m;
  }
  fence_proxy_async_smem();
  __syncthreads();

  const int wg = warp >> 2, qd = warp & 3;
  const int key = qd * 32 + lane;                          // this thread's key of a tile
  const uint32_t lane_base = (uint32_t)(qd * 32) << 16;   // its TMEM lane quadrant
  if (wg == 0) {
    reg_dec<C::kRegs0>();
    if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- TMA producer
      int issued = early;
      for (int j = early; j < T; ++j) {
        const int st = j % C::kStages;
        if (!mbar_wait(&code_empty[st], ((uint32_t)(j / C::kStages) & 1u) ^ 1u, abort_flag)) break;
        load_tile(j);
        issued = j + 1;
      }
      if (issued < T) {
        // aborted: let the loads already issued land before the CTA exits
        for (int j = (issued > C::kStages ? issued - C::kStages : 0); j < issued; ++j)
          mbar_wait(&code_full[j % C::kStages], (uint32_t)(j / C::kStages) & 1u, nullptr);
      }
    }
    if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    // S(0), S(1), then S(t + 2) once S(t) has been read, and PV(t)
    constexpr uint32_t idesc_s = umma_idesc_f16_f32(BK, NC, false, false);
    constexpr uint32_t idesc_o = umma_idesc_f16_f32(DH, NC, true, true);
    const uint64_t dq = umma_desc_sw128_kmajor(smem_u32(sQ));
    const uint64_t dv0 = umma_desc_sw128(smem_u32(sV), kAtom, 1024u);
    const uint64_t dp0 = umma_desc_sw128(smem_u32(sP), kAtom, 1024u);
    auto issue_s = [&](int t) -> bool {
      const int bf = t & 1;
      const uint32_t ph = (uint32_t)(t >> 1) & 1u;
      if (!mbar_wait_warp(&k_ready[bf], ph, abort_flag)) return false;
      tc_fence_after();
      const uint32_t a = tmem + C::tK + (uint32_t)bf * 64u;
      const uint32_t d = tmem + C::tS + (uint32_t)bf * NC;
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk)
        umma_f16_ts_warp(d, a + (uint32_t)kk * 8u,
                         dq + (uint64_t)(((kk >> 2) * (NC * 128) + (kk & 3) * 32) >> 4), idesc_s,
                         kk > 0 ? 1u : 0u);
      umma_commit_warp(&s_full[bf]);
      return true;
    };
    auto issue_pv = [&](int t) -> bool {
      const int bf = t & 1;
      const uint32_t ph = (uint32_t)(t >> 1) & 1u;
      if (!mbar_wait_warp(&pv_ready[bf], ph, abort_flag)) return false;
      tc_fence_after();
      const uint64_t dv = dv0 + (uint64_t)(bf * (kVTile >> 4));
      const uint64_t dp = dp0 + (uint64_t)(bf * (C::kP >> 4));
#pragma unroll
      for (int kk = 0; kk < BK / 16; ++kk)
        umma_f16_warp(tmem + (uint32_t)((t & (C::kSets - 1)) * NC), dv + (uint64_t)((kk * 16 * 128) >> 4),
                      dp + (uint64_t)((kk * 16 * 128) >> 4), idesc_o,
                      (t >= C::kSets || kk > 0) ? 1u : 0u);
      umma_commit_warp(&pv_done[bf]);
      return true;
    };
    bool ok = true;
    for (int t = 0; t < 2 && t < T && ok; ++t) ok = issue_s(t);
    for (int t = 0; t < T && ok; ++t) {
      if (t + 2 < T)
        ok = mbar_wait_warp(&s_free[t & 1], (uint32_t)(t >> 1) & 1u, abort_flag) && issue_s(t + 2);
      ok = ok && issue_pv(t);
    }
    umma_commit_warp(mma_done);
    mbar_wait(mma_done, 0u, nullptr);
    }
  } else if (wg <= C::kUnpackWgs) {
    // ---------------------------------------------------------------- unpack
    reg_dec<C::kRegsUnpack>();
    const bool doK = wg == 1, doV = wg == C::kUnpackWgs;
    const int sw = (key >> 1) & 3;  // 64-byte swizzle of the code rows
    // cscale: scores are acc * 2^24 / 2^k * scale * log2(e) * sk
    const float cscale = p.scale2 * ldexpf(1.f, 24 - kexp);
    // One warpgroup for both unpacks K two tiles ahead of V: K(t) only waits
    // for S(t - 2), V(t - 2) for PV(t - 4), so the products of one tile never
    // wait for the softmax of the tile before it.
    constexpr int kLag = C::kUnpackWgs == 1 ? 2 : 0;
    bool ok = true;
    for (int s = 0; s < T + kLag && ok; ++s) {
      uint32_t w[16];
      __half2 z24, z20;
      if (doK && s < T) {
        const int st = s % C::kStages, bf = s & 1;
        ok = mbar_wait_warp(&code_full[st], (uint32_t)(s / C::kStages) & 1u, abort_flag);
        if (!ok) break;
        const uint8_t* row = sCode + st * kStage + key * 64;
        const uint32_t* par = (const uint32_t*)(sCode + st * kStage + 2 * kCodeTile);
        const uint32_t kp = par[key], vp = par[BK + key];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(&w[4 * i]) = *reinterpret_cast<const uint4*>(row + ((i ^ sw) << 4));
        if (!doV) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&code_empty[st]);
        }
        if (s >= 2) {  // S(s - 2) has read this K buffer
          ok = mbar_wait_warp(&s_full[bf], ((uint32_t)(s >> 1) & 1u) ^ 1u, abort_flag);
          if (!ok) break;
        }
        // softmax(s - 4) has read this scale buffer: S(s - 2) was issued after s_free(s - 4)
        sScale[(s & (kScaleBufs - 1)) * 2 * BK + key] = bf16_lo(kp) * cscale;
        sScale[(s & (kScaleBufs - 1)) * 2 * BK + BK + key] = bf16_lo(vp);
        tc_fence_after();
        zero_pairs(kp, z24, z20);
#pragma unroll
        for (int hh = 0; hh < 4; ++hh) {
          uint32_t r[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) unpack_word(w[hh * 4 + i], z24, z20, r + 4 * i);
          tmem_st16_nowait(tmem + lane_base + C::tK + (uint32_t)(bf * 64 + hh * 16), r);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_ready[bf]);
      }
      if (doV && s >= kLag) {
        const int t = s - kLag, st = t % C::kStages, bf = t & 1;
        ok = mbar_wait_warp(&code_full[st], (uint32_t)(t / C::kStages) & 1u, abort_flag);
        if (!ok) break;
        const uint8_t* row = sCode + st * kStage + kCodeTile + key * 64;
        const uint32_t vp = ((const uint32_t*)(sCode + st * kStage + 2 * kCodeTile))[BK + key];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(&w[4 * i]) = *reinterpret_cast<const uint4*>(row + ((i ^ sw) << 4));
        __syncwarp();
        if (lane == 0) mbar_arrive(&code_empty[st]);
        if (t >= 2) {  // PV(t - 2) has read this V buffer
          ok = mbar_wait_warp(&pv_done[bf], ((uint32_t)(t >> 1) & 1u) ^ 1u, abort_flag);
          if (!ok) break;
        }
        zero_pairs(vp, z24, z20);
        uint8_t* dst = sV + bf * kVTile + key * 128;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint32_t r[4];
          unpack_word(w[i], z24, z20, r);
          *reinterpret_cast<uint4*>(dst + (i >> 3) * kAtom + (((i & 7) ^ (key & 7)) << 4)) =
              make_uint4(r[0], r[1], r[2], r[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pv_ready[bf]);
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    reg_inc<C::kRegsSoftmax>();
    const int g = wg - 1 - C::kUnpackWgs;       // softmax warpgroup
    const int bar_id = 1 + g;
    const int st0 = g * C::CP;                   // its row states
    const int col0 = C::kSets == 2 ? 0 : st0;    // its query rows
    const uint32_t tO = tmem + lane_base + (uint32_t)st0;  // (sets: its own O^T)
    float lacc[C::CP];
#pragma unroll
    for (int c = 0; c < C::CP; ++c) lacc[c] = 0.f;
    float vref = 0x1p-120f;
    constexpr uint32_t kAll = 0xffffffffu;
    uint32_t unset[C::NB];  // rows that have seen no key: their maximum is still open
#pragma unroll
    for (int n = 0; n < C::NB; ++n) unset[n] = kAll;
    // tiles with tree or unused slots (from m_hi), or slots outside some row's window (to m_lo)
    const int m_hi = Lb / BK;
    const long long wl = (long long)Lb + p.K - p.window;
    const int m_lo = p.window > 0 && wl >= 0 ? (int)(wl / BK) : -1;
    bool ok = true, err = false;
    for (int t = C::kSets == 2 ? g : 0; t < T; t += C::kSets) {
      const int bf = t & 1;
      const uint32_t ph = (uint32_t)(t >> 1) & 1u;
      const int tile = tl.tile(j0 + t);
      err = err || !mbar_wait_warp(&s_full[bf], ph, abort_flag);
      tc_fence_after();
      const float ks = sScale[(t & (kScaleBufs - 1)) * 2 * BK + key];
      float sv = sScale[(t & (kScaleBufs - 1)) * 2 * BK + BK + key];
      // scores relative to the row maxima, base 2
      float y[C::CP];
      if constexpr (C::CP == 64) tmem_ld64(tmem + lane_base + C::tS + (uint32_t)(bf * NC + col0), y);
      else tmem_ld32(tmem + lane_base + C::tS + (uint32_t)(bf * NC + col0), y);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_free[bf]);
      const bool masked = tile >= m_hi || tile <= m_lo;
      uint32_t vm[C::NB];  // rows that see this key
#pragma unroll
      for (int n = 0; n < C::NB; ++n) vm[n] = kAll;
      if (masked) {
        const int a0 = tile * BK + qd * 32 - Lb;  // tree node of lane 0 (negative: a prefix slot)
        const int a = a0 + lane;
        uint32_t any = 0u;
#pragma unroll
        for (int n = 0; n < C::NB; ++n) {
          if (a0 > -32) {
            // lane c: row c's ancestor bits of this warp's 32 keys, then transposed
            const uint32_t* ar = p.anc + (size_t)cnode[col0 + n * C::BS + lane] * p.W;
            const int wi = a0 >> 5;  // -1: prefix slots first
            const uint32_t w0 = wi >= 0 && wi < p.W ? __ldg(ar + wi) : 0u;
            const uint32_t w1 = wi + 1 < p.W ? __ldg(ar + wi + 1) : 0u;
            const uint32_t w = __funnelshift_r(w0, w1, a0 & 31);
            uint32_t tm = 0u;
#pragma unroll
            for (int c = 0; c < C::BS; ++c)
              tm |= ((__shfl_sync(0xffffffffu, w, c) >> lane) & 1u) << c;
            if (a >= 0) vm[n] = a < p.N ? tm : 0u;
          }
          if (p.window > 0 && a < p.N) {
            const int dp = a < 0 ? a : __ldg(p.depth + a);  // position - L_b
            if (Lb + dp >= p.sinks)
              vm[n] &= shallow[(col0 / C::BS + n) * (MEDUSA_MAX_K + 2) +
                               (int)min((long long)MEDUSA_MAX_K + 1, max(0ll, (long long)dp + p.window))];
          }
          any |= vm[n];
        }
        if (any == 0u) sv = 0.f;
      }
      const float4* nm4 = reinterpret_cast<const float4*>(nm + st0);
#pragma unroll
      for (int c = 0; c < C::CP / 4; ++c) {
        const float4 n = nm4[c];
        y[4 * c] = fmaf(y[4 * c], ks, n.x);
        y[4 * c + 1] = fmaf(y[4 * c + 1], ks, n.y);
        y[4 * c + 2] = fmaf(y[4 * c + 2], ks, n.z);
        y[4 * c + 3] = fmaf(y[4 * c + 3], ks, n.w);
      }
      if (masked) {
#pragma unroll
        for (int c = 0; c < C::CP; ++c) y[c] = (vm[c / C::BS] >> (c % C::BS)) & 1u ? y[c] : -INFINITY;
      }
      float ym[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < C::CP / 2; ++c) ym[c & 3] = max3(ym[c & 3], y[2 * c], y[2 * c + 1]);
      uint32_t fresh = 0u;
#pragma unroll
      for (int n = 0; n < C::NB; ++n) fresh |= vm[n] & unset[n];
      if (bar_red_or(bar_id, 128,
                     err || max3(ym[0], ym[1], fmaxf(ym[2], ym[3])) > kGrow || fabsf(sv) > vref ||
                         fresh != 0u)) {
        // a row maximum or the value scale grew (or a row met its first key):
        // move them for the whole warpgroup, rescale the sums and O
#pragma unroll
        for (int n = 0; n < C::NB; ++n) {
          float a[C::BS];
#pragma unroll
          for (int c = 0; c < C::BS; ++c) a[c] = y[n * C::BS + c];
          const float m = col_reduce(a, lane, [](float x, float z) { return fmaxf(x, z); });
          red[(g * 4 + qd) * C::CP + n * C::BS + lane] = m;
        }
        const uint32_t av = __float_as_uint(fabsf(sv));
        const unsigned sb = __reduce_max_sync(0xffffffffu, av < 0x7f800000u ? av : 0u);
        if (lane == 0) redv[g * 4 + qd] = __uint_as_float(sb);
        if (bar_red_or(bar_id, 128, err)) {
          ok = false;
          break;
        }
        // power of two >= the largest scale, kept in [2^-120, 2^119]
        const float* rv = redv + g * 4;
        const uint32_t bb = __float_as_uint(fmaxf(fmaxf(rv[0], rv[1]), fmaxf(rv[2], rv[3])));
        const int ex = min(246, max(7, (int)((bb >> 23) + ((bb & 0x7fffffu) ? 1 : 0))));
        const float nref = fmaxf(vref, __uint_as_float((uint32_t)ex << 23));
        const float fv = vref / nref;
        vref = nref;
        if (qd == 0) {  // the warpgroup's first warp: lane c is row c of each block
#pragma unroll
          for (int n = 0; n < C::NB; ++n) {
            const int c = n * C::BS + lane;
            const float* rr = red + g * 4 * C::CP + c;
            const float x = fmaxf(fmaxf(rr[0], rr[C::CP]), fmaxf(rr[2 * C::CP], rr[3 * C::CP]));
            const bool open = (unset[n] >> lane) & 1u;
            const bool seen = x != -INFINITY;
            float d = 0.f, f = 1.f;  // shift of the maximum, factor of the sums
            if (seen && (open || x > kGrow)) {
              d = -x;
              f = open ? 0.f : exp2f(-x);
            }
            nm[st0 + c] += d;
            fd[st0 + c] = d;
            fl[st0 + c] = f;
            fo[st0 + c] = f * fv;
            const unsigned sn = __ballot_sync(0xffffffffu, seen);
            if (lane == 0) unset_s[g * C::NB + n] = unset[n] & ~sn;
          }
        }
        named_bar_sync(bar_id, 128);
#pragma unroll
        for (int n = 0; n < C::NB; ++n) unset[n] = unset_s[g * C::NB + n];
#pragma unroll
        for (int c = 0; c < C::CP; ++c) {
          lacc[c] *= fl[st0 + c];
          y[c] += fd[st0 + c];
        }
        if (t >= C::kSets) {  // O holds the PV of this warpgroup's earlier tiles
          const int tp = t - C::kSets;
          if (mbar_wait_warp(&pv_done[tp & 1], (uint32_t)(tp >> 1) & 1u, abort_flag)) {
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < C::CP; c0 += 8) {
              float o8[8];
              tmem_ld8(tO + (uint32_t)c0, o8);
#pragma unroll
              for (int e = 0; e < 8; ++e) o8[e] *= fo[st0 + c0 + e];
              tmem_st8(tO + (uint32_t)c0, o8);
            }
          } else {
            err = true;  // reported at the next vote
          }
        }
      }
      // PV(t - 2) has read this P buffer
      if (t >= 2) err = err || !mbar_wait_warp(&pv_done[bf], ph ^ 1u, abort_flag);
      // weights, and weights x value scales as fp16 in this key's row of P^T
      const float vn = sv * __uint_as_float((261u << 23) - __float_as_uint(vref));
      uint8_t* prow = sP + bf * C::kP + (col0 >> 6) * kAtom + key * 128;
      auto weights = [&](auto is_masked) {
#pragma unroll
        for (int c8 = 0; c8 < C::CP / 8; ++c8) {
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = c8 * 8 + 2 * e;
            float a = ex2_approx(y[c]), d = ex2_approx(y[c + 1]);
            lacc[c] += a;
            lacc[c + 1] += d;
            a *= vn;
            d *= vn;
            if constexpr (decltype(is_masked)::value) {
              // 0, not 0 * NaN, for rows that do not see the key
              a = (vm[c / C::BS] >> (c % C::BS)) & 1u ? a : 0.f;
              d = (vm[c / C::BS] >> (c % C::BS + 1)) & 1u ? d : 0.f;
            }
            const __half2 hh = __floats2half2_rn(a, d);
            h[e] = *reinterpret_cast<const uint32_t*>(&hh);
          }
          *reinterpret_cast<uint4*>(prow + (((((col0 & 63) >> 3) + c8) ^ (key & 7)) << 4)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
      };
      if (masked) weights(std::true_type{});
      else weights(std::false_type{});
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pv_ready[bf]);
    }
    ok = ok && !err;
    if (ok) {  // the last PV: every earlier one is done too
      const bool good = mbar_wait(&pv_done[(T - 1) & 1], (uint32_t)((T - 1) >> 1) & 1u, abort_flag);
      ok = __all_sync(0xffffffffu, good);
    }
    // row sums over the keys of this warpgroup
#pragma unroll
    for (int n = 0; n < C::NB; ++n) {
      float a[C::BS];
#pragma unroll
      for (int c = 0; c < C::BS; ++c) a[c] = lacc[n * C::BS + c];
      const float ls = col_reduce(a, lane, [](float x, float z) { return x + z; });
      red[(g * 4 + qd) * C::CP + n * C::BS + lane] = ls;
    }
    if (qd == 0 && lane == 0) {
      vref_s[g] = vref;
#pragma unroll
      for (int n = 0; n < C::NB; ++n) unset_s[g * C::NB + n] = unset[n];
    }
    const bool bad = bar_red_or(3, 256, !ok);  // both warpgroups
    // each warpgroup writes half of the rows; its first 64 threads find their
    // factors (and with sets the weights of the two O^T)
    constexpr int EC = NC / 2;
    const int e0 = g * EC;
    const int gt = (int)threadIdx.x & 127;
    if (!bad && gt < EC) {
      const int c = e0 + gt;
      float m[2], l[2], w[2];
      float M = -INFINITY;
#pragma unroll
      for (int s = 0; s < C::kSets; ++s) {
        const int gs = C::kSets == 2 ? s : g, cc = C::kSets == 2 ? c : gt;
        const float* rr = red + gs * 4 * C::CP + cc;
        l[s] = (rr[0] + rr[C::CP]) + (rr[2 * C::CP] + rr[3 * C::CP]);
        const bool open = (unset_s[gs * C::NB + cc / C::BS] >> (cc % C::BS)) & 1u;
        // an open row with a sum of NaN (a NaN score) must still count
        m[s] = open ? (l[s] != l[s] ? 0.f : -INFINITY) : -nm[gs * C::CP + cc];
        M = fmaxf(M, m[s]);
      }
      float Ls = 0.f;
#pragma unroll
      for (int s = 0; s < C::kSets; ++s) {
        w[s] = m[s] == -INFINITY ? 0.f : exp2f(m[s] - M);
        if (m[s] != -INFINITY) Ls += w[s] * l[s];  // (a weight of 0 too: the sum may be NaN)
      }
      const float inv = p.P == 1 ? (Ls == 0.f ? 0.f : 1.f / Ls) : 1.f;
#pragma unroll
      for (int s = 0; s < C::kSets; ++s) {
        const int gs = C::kSets == 2 ? s : g;
        fo[s * NC + c] = m[s] == -INFINITY ? -1.f : w[s] * inv * vref_s[gs];
      }
      if (p.fuse)
        reinterpret_cast<float2*>(sm + C::oMl)[c] = make_float2(M, Ls);
      else if (p.P > 1 && crow[c] >= 0)
        p.pml[((size_t)bk * p.P + chunk) * p.R + c] = make_float2(M, Ls);
    }
    named_bar_sync(bar_id, 128);
    if (!bad) {
      tc_fence_after();
      // TMEM lane = position 8 w + 2 jj + h of dim 8 w + jj + 4 h
      const int jj = (key >> 1) & 3;
      const int dim = (key & ~7) + jj + 4 * (key & 1);
      const float unit = (jj & 1) ? 0x1p13f : 0x1p17f;  // 2^20 or 2^24, times 2^-7
      __nv_bfloat16* ob = p.out + (size_t)b * p.N * p.Hq * DH + dim;
      float* pb = p.po + ((size_t)bk * p.P + chunk) * p.R * DH + dim;
      float* sb = reinterpret_cast<float*>(sm + C::oV) + dim;
#pragma unroll 1
      for (int c0 = e0; c0 < e0 + EC; c0 += 8) {
        if (c0 >= p.R) break;  // warp-uniform
        float o8[8], x8[8];
        tmem_ld8(tmem + lane_base + (uint32_t)c0, o8);
        if constexpr (C::kSets == 2) tmem_ld8(tmem + lane_base + (uint32_t)(NC + c0), x8);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = crow[c0 + e];
          if (r < 0) continue;
          // below 0: that warpgroup saw no key of the row (its O^T may be unwritten)
          float o = fo[c0 + e] < 0.f ? 0.f : o8[e] * unit * fo[c0 + e];
          if constexpr (C::kSets == 2)
            o += fo[NC + c0 + e] < 0.f ? 0.f : x8[e] * unit * fo[NC + c0 + e];
          if (p.P == 1) ob[(size_t)r * DH] = __float2bfloat16_rn(o);
          else if (p.fuse) sb[(c0 + e) * C::kOS] = o;
          else pb[(size_t)(c0 + e) * DH] = o;
        }
      }
    }
    if (p.fuse) {
      cluster_sync();
      // (the softmax warps: the others have too few registers left)
      merge_chunks<NC>(sm, chunk, b, kvh, warp - 4 * (1 + C::kUnpackWgs), 8, p);
      cluster_sync();
    }
  }
  if (wg <= C::kUnpackWgs && p.fuse) {
    cluster_sync();
    cluster_sync();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

#include "attention_packed_pair.cuh"

struct PackedPlan {
  int NC, R, groups, P;  // NC = 256: two query tiles a CTA (attention_packed_pair.cuh)
  bool fuse;             // chunks merge in a cluster
  long long ctas;
  size_t off_o, off_ml, total;
};

template <int NC>
int max_active_clusters(int P) {
  static std::atomic<bool> done[64];
  static std::atomic<int> cache[64][kMaxClusterChunks + 1];
  using C = Cfg<NC>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  const int v = cache[dev][P].load(std::memory_order_relaxed);
  if (v) return v - 1;
  if (ensure_max_smem(tree_attn_packed_kernel<NC>, (int)C::kSmem, done,
                      "cudaFuncSetAttribute(tree_attn_packed_kernel)"))
    return 0;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = P;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, tree_attn_packed_kernel<NC>, &cfg) != cudaSuccess) {
    cudaGetLastError();  // not an error of the caller's stream: no in-cluster merge
    return 0;
  }
  cache[dev][P].store(n + 1, std::memory_order_relaxed);
  return n;
}

PackedPlan packed_plan(const medusa_tree* t, int B, int Hq, int Hkv, int Lcap, int window,
                       int sinks) {
  PackedPlan p;
  p.R = t->N * (Hq / Hkv);
  p.NC = p.R <= 32 ? 32 : p.R <= 64 ? 64 : p.R <= 128 ? 128 : 256;
  p.groups = (p.R + p.NC - 1) / p.NC;
  const long long units = (long long)B * Hkv * p.groups;
  const long long T = (ext_max_keys(Lcap, t->N, window, sinks) + BK - 1) / BK + (window > 0 ? 1 : 0);
  // key chunks: least (waves of CTAs) x (tiles of a CTA + its start and end,
  // about 4 tiles' time, and the merge: 1 in a cluster, which takes every
  // cluster running at once, 2 with a second kernel)
  const long long sms = num_sms();
  long long best = 0;
  p.P = 1;
  p.fuse = false;
  for (long long P = 1; units > 0 && P <= 64 && P <= T; ++P) {
    bool fuse = false;
    if (p.NC <= 128 && P > 1 && P <= kMaxClusterChunks && units * P <= sms) {
      const int n = p.NC == 32   ? max_active_clusters<32>((int)P)
                    : p.NC == 64 ? max_active_clusters<64>((int)P)
                                 : max_active_clusters<128>((int)P);
      fuse = units <= n;
    }
    const long long cost =
        ((units * P + sms - 1) / sms) * ((T + P - 1) / P + 4 + (P == 1 ? 0 : fuse ? 1 : 2));
    if (best == 0 || cost < best) {
      best = cost;
      p.P = (int)P;
      p.fuse = fuse;
    }
  }
  p.ctas = units * p.P;
  WsCarver w;
  const size_t rows = p.P > 1 && !p.fuse ? (size_t)B * Hkv * p.P * p.R : 0;
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
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.P;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = p.fuse ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, tree_attn_packed_kernel<NC>, kc, vc, kp, vp, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail(e, "tree_attn_packed_kernel launch");
}

}  // namespace

int attention_packed_tc_status(unsigned* status, unsigned* site, bool clear) {
  const unsigned zero = 0u;
  *status = *site = 0u;
  cudaError_t e = cudaMemcpyFromSymbol(status, g_dev_status, sizeof(unsigned));
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(site, g_dev_debug_site, sizeof(unsigned));
  if (e == cudaSuccess && clear) {
    e = cudaMemcpyToSymbol(g_dev_status, &zero, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_dev_debug_site, &zero, sizeof(unsigned));
  }
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail(e, "device status");
}

namespace {
// One thread waits for phase 0 of a barrier that no thread arrives at.
__global__ void packed_selftest_wait_kernel(unsigned long long limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) mbar_wait_limit(&bar, 0u, &abort_flag, limit_ns);
}
}  // namespace

int attention_packed_tc_selftest(unsigned long long limit_ns, cudaStream_t st) {
  packed_selftest_wait_kernel<<<1, 32, 0, st>>>(limit_ns);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail(e, "packed_selftest_wait_kernel launch");
}

namespace {
int pair_run(const CUtensorMap& kc, const CUtensorMap& vc, const CUtensorMap& kp,
             const CUtensorMap& vp, const PackedParams& p, long long ctas, cudaStream_t st) {
  static std::atomic<bool> done[64];
  int rc = ensure_max_smem(tree_attn_packed_pair_kernel, (int)PairCfg::kSmem, done,
                           "cudaFuncSetAttribute(tree_attn_packed_pair_kernel)");
  if (rc) return rc;
  cudaError_t e = launch_pdl(tree_attn_packed_pair_kernel, dim3((unsigned)ctas),
                             dim3(PairCfg::kThreads), PairCfg::kSmem, st, kc, vc, kp, vp, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail(e, "tree_attn_packed_pair_kernel launch");
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
  p.parent = t->d_parent;
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
  p.fuse = pl.fuse ? 1 : 0;
  p.window = a.window;
  p.sinks = a.sinks;
  p.scale2 = a.scale * 1.4426950408889634f;
  p.out = (__nv_bfloat16*)a.out;
  p.po = (float*)((uint8_t*)a.ws + pl.off_o);
  p.pml = (float2*)((uint8_t*)a.ws + pl.off_ml);
  int rc;
  switch (pl.NC) {
    case 32: rc = packed_run<32>(mKc, mVc, mKp, mVp, p, pl.ctas, st); break;
    case 64: rc = packed_run<64>(mKc, mVc, mKp, mVp, p, pl.ctas, st); break;
    case 128: rc = packed_run<128>(mKc, mVc, mKp, mVp, p, pl.ctas, st); break;
    default: rc = pair_run(mKc, mVc, mKp, mVp, p, pl.ctas, st); break;
  }
  if (rc || pl.P == 1 || pl.fuse) return rc;
  return attention_combine_launch(a, p.po, p.pml, pl.P, st);
}

}  // namespace medusa

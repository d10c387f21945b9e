// Tree attention over the 4-bit cache for few query rows (at most 16 per
// kv-head: single tokens, small trees), bf16 queries, dh = 128.
//
// Same arithmetic as tree_attn_packed_kernel: the codes as integers, exact in
// fp16, through the tensor cores, the row scales applied to the fp32 scores
// and to the weights.  K's zero comes off the fp32 sums, q . code - zero
// sum(q), which costs two multiply-adds a key and row instead of a packed
// subtraction per two elements.  V's does not: a row whose weight rests on
// keys with code = zero in some dim would be left with the rounding of the
// two large sums there.  With so few rows a tile's products are small and what
// counts is that nothing waits: here a warp works alone.  It streams its own
// 16-key groups (cp.async into a private ring, no barrier but its own),
// unpacks them in registers straight into mma.sync (m16n8k16) fragments, and
// keeps its own maxima, sums and O, merged once at the end.
//   S^T [16 keys x 8 rows]   A = K: a lane's 16 bytes of a key's row are its own
//                            32 of the 128 dims (any assignment of dims to k
//                            positions will do as long as Q follows it),
//                            B = Q (registers, fixed)
//   O^T [16 dims x 8 rows]  += A = V^T: pairs of keys per register, byte-permuted
//                            from the two keys' words before unpacking,
//                            B = P^T: the score fragment as fp16, transposed
//                            by two movmatrix
// Keys 4 t .. 4 t + 3 of a group belong to the lanes of thread-in-group t (k
// positions 2 t, 2 t + 1, 2 t + 8, 2 t + 9), so V's scales are one 16-byte load.
//
// The tcgen05 kernel reads and waits per 128-key tile in about 2000 cycles
// whatever the number of rows; 8 KB + 8 KB of codes arrive in 750.  Measured:
// single tokens of 16 sequences of 32K, 8 kv-heads, 4 rows each: 147 us of 87
// at the HBM rate; 9K to 32K: 95 of 55.  Bound: instruction issue (61 %) and the
// integer pipe (57 %: 88 logic operations per 16 keys and lane).  Four blocks
// per SM with up to 128 registers: five with 102 take 154 us, six (spilling)
// 224, three 155; the scores in two chains of MMAs instead of one 150.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "visible.cuh"

namespace medusa {
namespace {

constexpr int DH = 128;
constexpr int kWarps = 4;
constexpr int KB = 16 * kWarps;  // keys of a block: one 16-key group per warp
constexpr int kStages = 4;
constexpr int kGroupBytes = 2 * 16 * (DH / 2) + 2 * 16 * 4;  // K, V codes, K, V (scale, zero)
constexpr float kGrow = 8.0f;
constexpr int OS = DH + 4;  // merged rows: float4 stores of different rows fall in different banks

struct RowsParams {
  const __nv_bfloat16* q;
  const uint8_t* kc;
  const uint8_t* vc;
  const uint32_t* kp;
  const uint32_t* vp;
  const int32_t* L;
  const uint32_t* anc;
  const int32_t* depth;
  int B, N, W, K, Hq, Hkv, G, Lcap, R, P, window, sinks;
  float scale2;
  __nv_bfloat16* out;
  float* po;
  float2* pml;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 8 x 8 fp16 fragment, transposed
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// zero of a (scale, zero) word; unused slots may hold anything: kept finite
__device__ __forceinline__ float zero_point(uint32_t par) {
  return fminf(fmaxf(hi16(par), 0.f), 15.f);
}
// The same as an integer (the low bits of 2^23 + zero; four bits of anything).
__device__ __forceinline__ uint32_t zero_bits(uint32_t par) {
  return __float_as_uint(hi16(par) + 8388608.f) & 0xfu;
}
// -za * 2^-24 and -zb * 2^-24 as an fp16 pair (subnormals: the bits are the
// integers), and the same * 2^-20
__device__ __forceinline__ void zero_pairs(uint32_t za, uint32_t zb, __half2& z24, __half2& z20) {
  const uint32_t z = za + (zb << 16);
  const uint32_t lo = z | 0x80008000u, hi = (z << 4) | 0x80008000u;
  z24 = *reinterpret_cast<const __half2*>(&lo);
  z20 = *reinterpret_cast<const __half2*>(&hi);
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint32_t add_h2(uint32_t a, __half2 b) {
  return h2_bits(__hadd2(*reinterpret_cast<const __half2*>(&a), b));
}

// grid x: (sequence, kv-head) x chunk, chunks fastest
template <int NQ>  // blocks of 8 query rows
__global__ void __launch_bounds__(32 * kWarps, NQ == 1 ? 4 : 3)
    tree_attn_packed_rows_kernel(const RowsParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int chunk = blockIdx.x % p.P, place = blockIdx.x / p.P;
  // the longest sequences start first (up to 32 sequences; ties by index)
  int b = place / p.Hkv;
  const int kvh = place - b * p.Hkv;
  if (p.B > 1 && p.B <= 32) {
    const int mine = lane < p.B ? p.L[lane] : -1;
    int rank = 0;
    for (int i = 0; i < p.B; ++i) {
      const int x = __shfl_sync(0xffffffffu, mine, i);
      rank += (x > mine || (x == mine && i < lane)) ? 1 : 0;
    }
    const unsigned who = __ballot_sync(0xffffffffu, lane < p.B && rank == b);
    b = __ffs(who) - 1;
  }
  const int bk = b * p.Hkv + kvh;
  const int Lb = p.L[b];
  const bool seq_ok = Lb >= 0 && (long long)Lb + p.N <= p.Lcap;

  // visible 64-key blocks: the sinks', then from the root's window start
  int nh = 0, b_lo = 0, nb = 0;
  if (seq_ok) {
    const VisibleRuns vr = visible_runs(Lb, p.N, p.window, p.sinks);
    b_lo = vr.tail / KB;
    nh = min((vr.head + KB - 1) / KB, b_lo);
    nb = nh + (Lb + p.N + KB - 1) / KB - b_lo;
  }
  const int j0 = (int)((long long)nb * chunk / p.P);
  const int T = (int)((long long)nb * (chunk + 1) / p.P) - j0;

  // this lane's pieces of a group: 16 bytes of keys lane / 4 and + 8 of K and
  // of V; V's rows and pieces are placed so that the 8-byte reads of keys
  // 4 t + i fall in different banks
  const size_t row0 = (size_t)bk * p.Lcap;
  const uint32_t ring_a = smem_u32(smem) + warp * (kStages * kGroupBytes);
  const uint8_t* ring = smem + warp * (kStages * kGroupBytes);
  const int ck = lane >> 2, cc = lane & 3;
  const uint8_t* ksrc = p.kc + row0 * (DH / 2) + lane * 16;
  const uint8_t* vsrc = p.vc + row0 * (DH / 2) + lane * 16;
  const uint8_t* psrc = (const uint8_t*)((lane < 4 ? p.kp : p.vp) + row0) + (lane & 3) * 16;
  const uint32_t kdst = lane * 16;
  const uint32_t vdst = 1024 + (ck ^ ((ck >> 2) & 1)) * 64 + cc * 16;
  const uint32_t vdst8 = 1024 + ((ck + 8) ^ ((ck >> 2) & 1)) * 64 + (cc ^ 2) * 16;
  auto slot0 = [&](int j) {  // first slot of this warp's group in block j0 + j
    const int jj = j0 + j;
    return (jj < nh ? jj : jj - nh + b_lo) * KB + warp * 16;
  };
  auto issue = [&](int j) {
    if (j < T) {
      const int s0 = slot0(j);
      const uint32_t dst = ring_a + (j % kStages) * kGroupBytes;
      const size_t off = (size_t)s0 * (DH / 2);
      if (s0 + 16 <= p.Lcap) {
        cp16(dst + kdst, ksrc + off);
        cp16(dst + kdst + 512, ksrc + off + 512);
        cp16(dst + vdst, vsrc + off);
        cp16(dst + vdst8, vsrc + off + 512);
        if (lane < 8) cp16(dst + 2048 + lane * 16, psrc + (size_t)s0 * 4);
      } else {
      const bool l0 = s0 + ck < p.Lcap, l8 = s0 + ck + 8 < p.Lcap;  // past the cache: zeros
      cp16(dst + kdst, l0 ? ksrc + off : p.kc, l0);
      cp16(dst + kdst + 512, l8 ? ksrc + off + 512 : p.kc, l8);
      cp16(dst + vdst, l0 ? vsrc + off : p.vc, l0);
      cp16(dst + vdst8, l8 ? vsrc + off + 512 : p.vc, l8);
      if (lane < 8) {  // 16 K words, 16 V words (Lcap is a multiple of 4)
        const bool lp = s0 + (lane & 3) * 4 < p.Lcap;
        cp16(dst + 2048 + lane * 16, lp ? psrc + (size_t)s0 * 4 : (const uint8_t*)p.kp, lp);
      }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  for (int j = 0; j < kStages - 1; ++j) issue(j);  // in flight while Q is prepared

  // Q fragments (row 8 n + g): pair j of this lane's word wi is dims
  // 8 (4 t4 + wi) + j, + 4
  uint32_t qf[NQ][8][2];  // [row block][k step][register half]
  float qm = 0.f;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int r = 8 * n + g, nd = r / p.G;
    const __nv_bfloat16* qrow =
        p.q + (((size_t)b * p.N + nd) * p.Hq + (size_t)kvh * p.G + (r - nd * p.G)) * DH;
#pragma unroll
    for (int wi = 0; wi < 4; ++wi) {
      uint4 u = make_uint4(0u, 0u, 0u, 0u);
      if (r < p.R) u = *reinterpret_cast<const uint4*>(qrow + 8 * (4 * t4 + wi));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};  // dims (0,1) (2,3) (4,5) (6,7)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x0 = fabsf(lo16(w[e])), x1 = fabsf(hi16(w[e]));
        if (x0 <= 3.3895314e38f) qm = fmaxf(qm, x0);
        if (x1 <= 3.3895314e38f) qm = fmaxf(qm, x1);
      }
      // bf16 pairs (d_j, d_{j+4}), turned into fp16 below
      qf[n][2 * wi][0] = (w[0] & 0xffffu) | (w[2] << 16);
      qf[n][2 * wi][1] = (w[0] >> 16) | (w[2] & 0xffff0000u);
      qf[n][2 * wi + 1][0] = (w[1] & 0xffffu) | (w[3] << 16);
      qf[n][2 * wi + 1][1] = (w[1] >> 16) | (w[3] & 0xffff0000u);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) qm = fmaxf(qm, __shfl_xor_sync(0xffffffffu, qm, o));
  // 2^kexp brings the largest |q| into [2^13, 2^14)
  int kexp = 0;
  if (qm != 0.f) kexp = min(120, 13 - ((int)(__float_as_uint(qm) >> 23) - 127));
  const float qs = __uint_as_float((uint32_t)(127 + kexp) << 23);
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float f = e == 0 ? qs : qs * 0.0625f;  // odd pairs: codes carry 2^-20, not 2^-24
        qf[n][ks][e] = h2_bits(__floats2half2_rn(lo16(qf[n][ks][e]) * f, hi16(qf[n][ks][e]) * f));
      }
  const float cscale = p.scale2 * ldexpf(1.f, 24 - kexp);
  // The products take the codes as they are; zero comes off after the sums:
  // q . (code - zero) = q . code - zero sum(q), with sum(q) of the rounded q
  // (in the codes' unit 2^-24) for this lane's score columns 8 n + 2 t4 + e
  float qsum[NQ][2];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float x = 0.f;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&qf[n][ks][0]));
      const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&qf[n][ks][1]));
      x += (f0.x + f0.y) * 0x1p-24f + (f1.x + f1.y) * 0x1p-20f;
    }
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);  // row 8 n + g
    qsum[n][0] = __shfl_sync(0xffffffffu, x, 8 * t4);
    qsum[n][1] = __shfl_sync(0xffffffffu, x, 8 * t4 + 4);
  }

  // O^T: [dim block][row block]; fragment register 2 i + e is dim row g + 8 i,
  // query row 8 n + 2 t4 + e
  float o[8][NQ][4];
#pragma unroll
  for (int d = 0; d < 8; ++d)
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][n][e] = 0.f;
  float nm[NQ][2], l[NQ][2];  // minus the row maximum (base 2), row sum
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) nm[n][e] = l[n][e] = 0.f;
  uint32_t open = NQ == 1 ? 0x3u : 0x33u;  // bit 4 n + e: the row has seen no key, its maximum is open
  float vref = 0x1p-120f;
  // groups with tree or unused slots (from m_hi), or slots outside some row's window (to m_lo)
  const int m_hi = Lb - 15;
  const long long wl = (long long)Lb + p.K - p.window;
  const int m_lo = p.window > 0 && wl >= 0 ? (int)wl : -1;
  const int kg = 4 * (g >> 1) + (g & 1);  // key of row g of the K fragment; row g + 8 is kg + 2

  for (int j = 0; j < T; ++j) {
    issue(j + kStages - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const int s0 = slot0(j);
    const uint8_t* st = ring + (j % kStages) * kGroupBytes;
    if (s0 < Lb + p.N) {  // (warp-uniform) the group has a slot in use
      const uint32_t* kpar = reinterpret_cast<const uint32_t*>(st + 2048);
      const uint32_t kp[2] = {kpar[kg], kpar[kg + 2]};
      const uint32_t vp[2] = {kpar[16 + kg], kpar[16 + kg + 2]};
      float sv[2] = {lo16(vp[0]), lo16(vp[1])};
      // ---------------- scores
      float s[NQ][4];
#pragma unroll
      for (int n = 0; n < NQ; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
      {
        uint32_t w[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<uint4*>(w[i]) =
              *reinterpret_cast<const uint4*>(st + (kg + 2 * i) * 64 + t4 * 16);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          uint32_t a[2], c[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t v = (ks & 1) ? w[i][ks >> 1] >> 8 : w[i][ks >> 1];
            a[i] = v & 0x000f000fu;
            c[i] = v & 0x00f000f0u;
          }
#pragma unroll
          for (int n = 0; n < NQ; ++n) mma16816(s[n], a[0], a[1], c[0], c[1], qf[n][ks][0], qf[n][ks][1]);
        }
      }
      // ---------------- relative to the row maxima, base 2
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float ks = lo16(kp[i]) * cscale, z = zero_point(kp[i]);
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            s[n][2 * i + e] = fmaf(fmaf(-z, qsum[n][e], s[n][2 * i + e]), ks, nm[n][e]);
      }
      const bool masked = s0 >= m_hi || s0 <= m_lo;
      uint32_t vis = NQ == 1 ? 0xfu : 0xffu;  // bit 4 n + 2 i + e: key row g + 8 i, query row 8 n + 2 t4 + e
      if (masked) {
        vis = 0u;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int slot = s0 + kg + 2 * i, a = slot - Lb;
          if (a < p.N) {
            const int pos = a < 0 ? slot : Lb + __ldg(p.depth + a);
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int nd = min((8 * n + 2 * t4 + e) / p.G, p.N - 1);
                bool ok = in_window(pos, Lb + __ldg(p.depth + nd), p.window, p.sinks);
                if (a >= 0) ok = ok && ((__ldg(p.anc + (size_t)nd * p.W + (a >> 5)) >> (a & 31)) & 1u);
                vis |= (uint32_t)ok << (4 * n + 2 * i + e);
              }
          }
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!((vis >> (4 * n + 2 * i + e)) & 1u)) s[n][2 * i + e] = -INFINITY;
        }
        // a key no row of the warp sees must not move the value scale
        uint32_t any = vis;
        any |= __shfl_xor_sync(0xffffffffu, any, 1);
        any |= __shfl_xor_sync(0xffffffffu, any, 2);
        if (!(any & 0x33u)) sv[0] = 0.f;
        if (!(any & 0xccu)) sv[1] = 0.f;
      }
      const float svm = fmaxf(fabsf(sv[0]), fabsf(sv[1]));
      float smax = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3]));
      if (NQ == 2)
        smax = fmaxf(smax, fmaxf(fmaxf(s[NQ - 1][0], s[NQ - 1][1]), fmaxf(s[NQ - 1][2], s[NQ - 1][3])));
      if (__any_sync(0xffffffffu, smax > kGrow || svm > vref || ((vis | (vis >> 2)) & open) != 0u)) {
        // a row maximum or the value scale grew (or a row met its first key):
        // move them, rescale sums and O
        const uint32_t sb = __reduce_max_sync(
            0xffffffffu, __float_as_uint(svm) < 0x7f800000u ? __float_as_uint(svm) : 0u);
        const int ex = min(246, max(7, (int)((sb >> 23) + ((sb & 0x7fffffu) ? 1 : 0))));
        const float nref = fmaxf(vref, __uint_as_float((uint32_t)ex << 23));
        const float fv = vref / nref;
        vref = nref;
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(s[n][e], s[n][2 + e]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const uint32_t bit = 1u << (4 * n + e);
            float f = 1.f, d = 0.f;
            if (mx != -INFINITY && ((open & bit) || mx > kGrow)) {
              f = (open & bit) ? 0.f : exp2f(-mx);
              d = -mx;
            }
            if (mx != -INFINITY) open &= ~bit;
            nm[n][e] += d;
            s[n][e] += d;
            s[n][2 + e] += d;
            l[n][e] *= f;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              o[q][n][e] *= f * fv;
              o[q][n][2 + e] *= f * fv;
            }
          }
      }
      // ---------------- weights: fp16, transposed into the B fragment
      const float inv = __uint_as_float((261u << 23) - __float_as_uint(vref));  // 2^7 / vref
      uint32_t pb[NQ][2];
      float x[NQ][4];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float w = ex2_approx(s[n][2 * i + e]);
            l[n][e] += w;
            x[n][2 * i + e] = w * (sv[i] * inv);
          }
      if (masked) {  // 0, not 0 * NaN, for a key a row does not see
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] = (vis >> (4 * n + e)) & 1u ? x[n][e] : 0.f;
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          pb[n][i] = movmatrix_t(h2_bits(__floats2half2_rn(x[n][2 * i], x[n][2 * i + 1])));
      // ---------------- O^T += V^T P^T: words 2 g, 2 g + 1 of keys 4 t4 + i
      const uint4 vq = *reinterpret_cast<const uint4*>(kpar + 16 + 4 * t4);
      __half2 z24[2], z20[2];
      zero_pairs(zero_bits(vq.x), zero_bits(vq.y), z24[0], z20[0]);
      zero_pairs(zero_bits(vq.z), zero_bits(vq.w), z24[1], z20[1]);
      uint2 vv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 4 * t4 + i;
        vv[i] = *reinterpret_cast<const uint2*>(st + 1024 + (key ^ (t4 & 1)) * 64 +
                                                (((g >> 1) ^ ((t4 >> 1) << 1)) * 16) + (g & 1) * 8);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {  // elements 0-3, then 4-7 of the words
          const uint32_t sel = hf ? 0x7632u : 0x5410u;
          uint32_t a = __byte_perm(x ? vv[0].y : vv[0].x, x ? vv[1].y : vv[1].x, sel);
          uint32_t c = __byte_perm(x ? vv[2].y : vv[2].x, x ? vv[3].y : vv[3].x, sel);
#pragma unroll
          for (int q = 0; q < 2; ++q) {  // element 2 q in dim row g, 2 q + 1 in row g + 8
            const uint32_t a0 = add_h2(a & 0x000f000fu, z24[0]), a1 = add_h2(a & 0x00f000f0u, z20[0]);
            const uint32_t a2 = add_h2(c & 0x000f000fu, z24[1]), a3 = add_h2(c & 0x00f000f0u, z20[1]);
#pragma unroll
            for (int n = 0; n < NQ; ++n)
              mma16816(o[4 * x + 2 * hf + q][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            a >>= 8;
            c >>= 8;
          }
        }
      }
    }
    __syncwarp();  // every lane has read the stage before it is filled again
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");

  // ---------------- merge of the warps
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
    }
  __syncthreads();  // the rings are free
  float* so = reinterpret_cast<float*>(smem);        // [warp][8 NQ][OS]
  float2* sml = reinterpret_cast<float2*>(so + kWarps * 8 * NQ * OS);
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = warp * 8 * NQ + 8 * n + 2 * t4 + e;
      float* row = so + (size_t)r * OS + 16 * g;
      // block d, register halves i: element 2 d + i of dims 16 g .. 16 g + 15
#pragma unroll
      for (int d = 0; d < 8; d += 2) {
        float4 v;
        // codes carry 2^-24 (even elements) or 2^-20, weights 2^7 / vref
        v.x = o[d][n][e] * 0x1p17f * vref;
        v.y = o[d][n][2 + e] * 0x1p13f * vref;
        v.z = o[d + 1][n][e] * 0x1p17f * vref;
        v.w = o[d + 1][n][2 + e] * 0x1p13f * vref;
        *reinterpret_cast<float4*>(row + 2 * d) = v;
      }
      // an open row with a sum of NaN (only NaN scores) must still count
      const bool none = ((open >> (4 * n + e)) & 1u) && l[n][e] == l[n][e];
      if (g == 0) sml[r] = make_float2(none ? -INFINITY : -nm[n][e], l[n][e]);
    }
  __syncthreads();
  for (int e = threadIdx.x; e < p.R * (DH / 4); e += 32 * kWarps) {
    const int r = e / (DH / 4), c = e - r * (DH / 4);
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[w * 8 * NQ + r].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float Ls = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = sml[w * 8 * NQ + r];
      if (ml.x == -INFINITY) continue;
      const float f = exp2f(ml.x - M);
      const float4 v = *reinterpret_cast<const float4*>(so + ((size_t)w * 8 * NQ + r) * OS + 4 * c);
      Ls += f * ml.y;
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    if (p.P == 1) {
      const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
      const int nd = r / p.G;
      __nv_bfloat16* dst = p.out + (((size_t)b * p.N + nd) * p.Hq + (size_t)kvh * p.G +
                                    (r - nd * p.G)) * DH + 4 * c;
      __align__(8) __nv_bfloat162 h2[2] = {__floats2bfloat162_rn(acc.x * inv, acc.y * inv),
                                           __floats2bfloat162_rn(acc.z * inv, acc.w * inv)};
      *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(h2);
    } else {
      const size_t prow = ((size_t)bk * p.P + chunk) * p.R + r;
      *reinterpret_cast<float4*>(p.po + prow * DH + 4 * c) = acc;
      if (c == 0) p.pml[prow] = make_float2(M, Ls);
    }
  }
}

template <int NQ>
constexpr size_t rows_smem() {
  const size_t ring = (size_t)kWarps * kStages * kGroupBytes;
  const size_t merge = (size_t)kWarps * 8 * NQ * (OS * 4 + 8);
  return ring > merge ? ring : merge;
}

struct RowsPlan {
  int R, P;
  long long ctas;
  size_t off_o, off_ml, total;
};
RowsPlan rows_plan(const medusa_tree* t, int B, int Hq, int Hkv, int Lcap, int window, int sinks) {
  RowsPlan p;
  p.R = t->N * (Hq / Hkv);
  const long long units = (long long)B * Hkv;
  const long long nb = (ext_max_keys(Lcap, t->N, window, sinks) + KB - 1) / KB + (window > 0 ? 1 : 0);
  // key chunks: least time of the resident CTAs, each with its start and end of
  // about 4 blocks' time (6 with the merge), and half a chunk for the uneven
  // end: the CTAs of an SM share it, so a part wave costs little, and the
  // sequences' lengths are not known here.  (Whole waves and no end: 8
  // sequences of 4K to 16K, 16 rows, 62 us instead of 54; 64 of 500 to 4096, 4
  // rows, 71 instead of 64.)
  const double slots = (p.R <= 8 ? 4.0 : 3.0) * num_sms();
  double best = 0.0;
  long long P = 1;
  for (long long x = 1; units > 0 && x <= 64 && x <= nb; ++x) {
    const double waves = (double)(units * x) / slots, T = (double)((nb + x - 1) / x);
    const double cost = (waves > 1.0 ? waves : 1.0) * (T + (x > 1 ? 6.0 : 4.0)) + 0.5 * T;
    if (x == 1 || cost < best) {
      best = cost;
      P = x;
    }
  }
  p.P = (int)P;
  p.ctas = units * p.P;
  WsCarver w;
  const size_t rows = p.P > 1 ? (size_t)B * Hkv * p.P * p.R : 0;
  p.off_o = w.take<float>(rows * DH);
  p.off_ml = w.take<float2>(rows);
  p.total = w.total();
  return p;
}

template <int NQ>
int rows_run(const RowsParams& p, long long ctas, cudaStream_t st) {
  static std::atomic<bool> done[64];
  int rc = ensure_max_smem(tree_attn_packed_rows_kernel<NQ>, (int)rows_smem<NQ>(), done,
                           "cudaFuncSetAttribute(tree_attn_packed_rows_kernel)");
  if (rc) return rc;
  cudaError_t e = launch_pdl(tree_attn_packed_rows_kernel<NQ>, dim3((unsigned)ctas), dim3(32 * kWarps),
                             rows_smem<NQ>(), st, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail(e, "tree_attn_packed_rows_kernel launch");
}

}  // namespace

bool attention_packed_rows_eligible(int dtype, int dh, int rows) {
  return dtype == MEDUSA_BF16 && dh == DH && rows <= 16;
}

size_t attention_packed_rows_workspace(const medusa_tree* t, int B, int Hq, int Hkv, int Lcap,
                                       int window, int sinks) {
  return rows_plan(t, B, Hq, Hkv, Lcap, window, sinks).total;
}

int attention_packed_rows_launch(const AttnArgs& a, const PackedCache& c, cudaStream_t st) {
  const medusa_tree* t = a.tree;
  const RowsPlan pl = rows_plan(t, a.B, a.Hq, a.Hkv, a.Lcap, a.window, a.sinks);
  if (pl.ctas > 0x7fffffffLL) return fail(MEDUSA_ERR_UNSUPPORTED, "too many query rows for one launch");
  RowsParams p;
  p.q = (const __nv_bfloat16*)a.q;
  p.kc = (const uint8_t*)c.k_codes;
  p.vc = (const uint8_t*)c.v_codes;
  p.kp = (const uint32_t*)c.k_par;
  p.vp = (const uint32_t*)c.v_par;
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
  p.P = pl.P;
  p.window = a.window;
  p.sinks = a.sinks;
  p.scale2 = a.scale * 1.4426950408889634f;
  p.out = (__nv_bfloat16*)a.out;
  p.po = (float*)((uint8_t*)a.ws + pl.off_o);
  p.pml = (float2*)((uint8_t*)a.ws + pl.off_ml);
  const int rc = pl.R <= 8 ? rows_run<1>(p, pl.ctas, st) : rows_run<2>(p, pl.ctas, st);
  if (rc || pl.P == 1) return rc;
  return attention_combine_launch(a, p.po, p.pml, pl.P, st);
}

}  // namespace medusa

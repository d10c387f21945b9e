// Tree attention over the 4-bit cache and with a sliding window: dispatch,
// and the SIMT kernel for fp32 and dh = 64.
//
// For node i of sequence b and query head h:
//   out = softmax_j(scale q . k_j) v_j over the slots j that node i sees
// (visible.cuh), k_j and v_j read from a bf16/fp32 cache or decoded from
// 4-bit rows, scale_j * (code - zero).
//
// SIMT kernel: a CTA takes RB query rows (tree nodes x the GQA group) of one
// (sequence, kv-head) and one chunk of its visible keys, 64 keys at a time.
// 128 threads as 8 row groups x 16 key (or dim) groups, each with an
// RB/8 x 4 block of scores and an RB/8 x dh/16 block of the output in
// registers, so a 16-byte shared-memory load feeds about 10 (Q K^T) and 16
// (P V) multiply-adds and the FMA pipe, not shared memory, bounds it.
// Running row maximum and sum in fp32 (base 2).  Chunks leave unnormalised
// partial rows that tree_attn_combine_kernel merges.  At the small sizes it
// serves it is bound by its two launches (smallest configuration, fp32, 4-bit
// cache: 15 us); large fp32 shapes run at the FMA rate.
#include "internal.h"
#include "visible.cuh"

namespace medusa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int TK = 64;
constexpr int kThreads = 128;

struct SimtParams {
  const void* q;
  const void* k;      // cache values, or packed code words
  const void* v;
  const uint32_t* kp;  // packed: (scale, zero) words
  const uint32_t* vp;
  const int32_t* L;
  const uint32_t* anc;
  const int32_t* depth;
  int N, W, Hq, Hkv, G, Lcap, R, rblocks, P, window, sinks;
  float qscale;
  float* po;
  float2* pml;
};

template <int DH, int RB>
struct SimtSmem {
  float q[RB][DH + 4];
  float k[TK][DH + 4];
  float v[TK][DH];
  float p[RB][TK + 4];
  uint32_t am[RB][MEDUSA_MAX_N / 32];
  int depth[MEDUSA_MAX_N];
};

// 8 values (dims 8 c .. 8 c + 7) of slot `slot` of one kv-head.
template <typename T, int DH, bool kPacked>
__device__ __forceinline__ void load_row8(const void* base, const uint32_t* par, int b, int kvh,
                                          int Hkv, int Lcap, int slot, int c, float (&x)[8]) {
  if constexpr (kPacked) {
    const size_t row = ((size_t)b * Hkv + kvh) * Lcap + slot;
    const uint32_t w = reinterpret_cast<const uint32_t*>(base)[row * (DH / 8) + c];
    const uint32_t p = par[row];
    const float s = __uint_as_float(p << 16), z = __uint_as_float(p & 0xffff0000u);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = s * ((float)((w >> (4 * e)) & 15u) - z);
  } else {
    const T* p = reinterpret_cast<const T*>(base) + (((size_t)b * Lcap + slot) * Hkv + kvh) * DH + c * 8;
    if constexpr (sizeof(T) == 4) {
      const float4 a0 = reinterpret_cast<const float4*>(p)[0];
      const float4 a1 = reinterpret_cast<const float4*>(p)[1];
      x[0] = a0.x, x[1] = a0.y, x[2] = a0.z, x[3] = a0.w;
      x[4] = a1.x, x[5] = a1.y, x[6] = a1.z, x[7] = a1.w;
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    }
  }
}

// grid x: ((sequence, kv-head), chunk, row block), row blocks fastest
template <typename T, int DH, int RB, bool kPacked>
__global__ void __launch_bounds__(kThreads) tree_attn_ext_simt_kernel(const SimtParams a) {
  griddep_launch_dependents();
  griddep_wait();
  extern __shared__ __align__(16) uint8_t smem_raw[];
  auto& s = *reinterpret_cast<SimtSmem<DH, RB>*>(smem_raw);
  constexpr int RT = RB / 8;    // rows per thread
  constexpr int DT = DH / 16;   // output dims per thread
  const long long id = blockIdx.x;
  const int rb = (int)(id % a.rblocks);
  const int chunk = (int)((id / a.rblocks) % a.P);
  const int bk = (int)(id / a.rblocks / a.P);
  const int b = bk / a.Hkv, kvh = bk - b * a.Hkv;
  const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15;
  const int Lb = a.L[b];
  const bool seq_ok = Lb >= 0 && (long long)Lb + a.N <= a.Lcap;

  for (int e = tid; e < RB * DH; e += kThreads) {
    const int i = e / DH, d = e - i * DH, r = rb * RB + i;
    float val = 0.f;
    if (r < a.R) {
      const int n = r / a.G, g = r - n * a.G;
      val = to_f32(reinterpret_cast<const T*>(
                a.q)[(((size_t)b * a.N + n) * a.Hq + (size_t)kvh * a.G + g) * DH + d]) *
            a.qscale;
    }
    s.q[i][d] = val;
  }
  for (int e = tid; e < RB * a.W; e += kThreads) {
    const int i = e / a.W, w = e - i * a.W, r = rb * RB + i;
    s.am[i][w] = r < a.R ? a.anc[(size_t)(r / a.G) * a.W + w] : 0u;
  }
  for (int e = tid; e < a.N; e += kThreads) s.depth[e] = a.depth[e];

  VisibleRuns vr{0, 0, 0};
  if (seq_ok) vr = visible_runs(Lb, a.N, a.window, a.sinks);
  int per = (vr.total + a.P - 1) / a.P;
  per = (per + TK - 1) / TK * TK;
  const int u_lo = (int)min((long long)vr.total, (long long)chunk * per);
  const int u_hi = (int)min((long long)vr.total, (long long)u_lo + per);

  float m[RT], l[RT], o[RT][DT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[i][d] = 0.f;
  }

  for (int u0 = u_lo; u0 < u_hi; u0 += TK) {
    __syncthreads();
    for (int e = tid; e < TK * (DH / 8); e += kThreads) {
      const int j = e / (DH / 8), c = e - j * (DH / 8);
      float x[8] = {}, y[8] = {};
      if (u0 + j < u_hi) {
        const int u = u0 + j;
        const int slot = u < vr.head ? u : u - vr.head + vr.tail;
        if (dbg_ok(slot < a.Lcap, DBG_ATTN_SLOT)) {
          load_row8<T, DH, kPacked>(a.k, a.kp, b, kvh, a.Hkv, a.Lcap, slot, c, x);
          load_row8<T, DH, kPacked>(a.v, a.vp, b, kvh, a.Hkv, a.Lcap, slot, c, y);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        reinterpret_cast<float4*>(&s.k[j][c * 8])[h] =
            make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
        reinterpret_cast<float4*>(&s.v[j][c * 8])[h] =
            make_float4(y[4 * h], y[4 * h + 1], y[4 * h + 2], y[4 * h + 3]);
      }
    }
    __syncthreads();
    // scores: rows rg + 8 i, keys cg + 16 j
    float acc[RT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 2
    for (int d = 0; d < DH; d += 4) {
      float4 kv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(&s.k[cg + 16 * j][d]);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const float4 qv = *reinterpret_cast<const float4*>(&s.q[rg + 8 * i][d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = fmaf(qv.x, kv[j].x, acc[i][j]);
          acc[i][j] = fmaf(qv.y, kv[j].y, acc[i][j]);
          acc[i][j] = fmaf(qv.z, kv[j].z, acc[i][j]);
          acc[i][j] = fmaf(qv.w, kv[j].w, acc[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int ri = rg + 8 * i, r = rb * RB + ri;
      const int dq = s.depth[min(r / a.G, a.N - 1)];
      float tmax = -INFINITY;
      bool see[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int u = u0 + cg + 16 * j;
        const int slot = u < vr.head ? u : u - vr.head + vr.tail;
        bool vis = r < a.R && u < u_hi;
        if (vis && slot >= Lb) {
          const int n = slot - Lb;
          vis = ((s.am[ri][n >> 5] >> (n & 31)) & 1u) &&
                in_window(Lb + s.depth[n], Lb + dq, a.window, a.sinks);
        } else if (vis) {
          vis = in_window(slot, Lb + dq, a.window, a.sinks);
        }
        see[j] = vis;
        acc[i][j] = vis ? acc[i][j] : -INFINITY;
        tmax = fmaxf(tmax, acc[i][j]);
      }
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, off));
      const float m_new = fmaxf(m[i], tmax);
      const float corr = (m_new == -INFINITY) ? 1.f : exp2f(m[i] - m_new);
      float psum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = (acc[i][j] == -INFINITY) ? 0.f : exp2f(acc[i][j] - m_new);
        s.p[ri][cg + 16 * j] = see[j] ? p : -1.f;  // a negative weight: masked
        psum += p;
      }
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) psum += __shfl_xor_sync(0xffffffffu, psum, off);
      l[i] = l[i] * corr + psum;
      m[i] = m_new;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[i][d] *= corr;
    }
    __syncwarp();
    // O: rows rg + 8 i, dims 4 cg + 64 c .. + 3; a masked key's V row may hold
    // anything, so it is skipped, not multiplied (a visible one with p = 0 is
    // not: 0 x NaN is NaN)
#pragma unroll 1
    for (int j = 0; j < TK; j += 4) {
      float4 pv[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) pv[i] = *reinterpret_cast<const float4*>(&s.p[rg + 8 * i][j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float vv[DT];
#pragma unroll
        for (int c = 0; c < DT / 4; ++c) {
          const float4 t = *reinterpret_cast<const float4*>(&s.v[j + e][4 * cg + 64 * c]);
          vv[4 * c] = t.x, vv[4 * c + 1] = t.y, vv[4 * c + 2] = t.z, vv[4 * c + 3] = t.w;
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float p = e == 0 ? pv[i].x : e == 1 ? pv[i].y : e == 2 ? pv[i].z : pv[i].w;
          if (!(p < 0.f)) {
#pragma unroll
            for (int d = 0; d < DT; ++d) o[i][d] = fmaf(p, vv[d], o[i][d]);
          }
        }
      }
    }
  }

#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = rb * RB + rg + 8 * i;
    if (r >= a.R) continue;
    const size_t prow = ((size_t)bk * a.P + chunk) * a.R + r;
#pragma unroll
    for (int c = 0; c < DT / 4; ++c)
      *reinterpret_cast<float4*>(&a.po[prow * DH + 4 * cg + 64 * c]) =
          make_float4(o[i][4 * c], o[i][4 * c + 1], o[i][4 * c + 2], o[i][4 * c + 3]);
    // a sum of NaN (a NaN score) must reach the merge, which skips m = -inf
    if (cg == 0) a.pml[prow] = make_float2(l[i] != l[i] ? 0.f : m[i], l[i]);
  }
}

struct SimtPlan {
  int RB, R, rblocks, P;
  long long ctas;
  size_t off_o, off_ml, total;
};

SimtPlan simt_plan(const medusa_tree* t, int B, int Hq, int Hkv, int dh, int Lcap, int window,
                   int sinks) {
  SimtPlan p;
  p.R = t->N * (Hq / Hkv);
  p.RB = p.R <= 32 ? 16 : 64;  // few rows: smaller blocks, less idle work
  p.rblocks = (p.R + p.RB - 1) / p.RB;
  const long long base = (long long)p.rblocks * B * Hkv;
  const long long keys = ext_max_keys(Lcap, t->N, window, sinks);
  long long want = base > 0 ? (4LL * num_sms() + base - 1) / base : 1;
  const long long max_p = (keys + 2 * TK - 1) / (2 * TK);  // >= 2 tiles each
  if (want > max_p) want = max_p;
  if (want < 1) want = 1;
  p.P = (int)want;
  p.ctas = base * p.P;
  WsCarver w;
  const size_t rows = (size_t)B * Hkv * p.P * p.R;
  p.off_o = w.take<float>(rows * dh);
  p.off_ml = w.take<float2>(rows);
  p.total = w.total();
  return p;
}

template <typename T, int DH, int RB, bool kPacked>
int simt_run_t(const SimtParams& p, long long ctas, cudaStream_t st) {
  static std::atomic<bool> done[64];
  auto* fn = tree_attn_ext_simt_kernel<T, DH, RB, kPacked>;
  constexpr int smem = (int)sizeof(SimtSmem<DH, RB>);
  int rc = ensure_max_smem(fn, smem, done, "cudaFuncSetAttribute(tree_attn_ext_simt_kernel)");
  if (rc) return rc;
  cudaError_t e = launch_pdl(fn, dim3((unsigned)ctas), dim3(kThreads), smem, st, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail(e, "tree_attn_ext_simt_kernel launch");
}
template <typename T, int DH, bool kPacked>
int simt_run(const SimtParams& p, int RB, long long ctas, cudaStream_t st) {
  return RB == 16 ? simt_run_t<T, DH, 16, kPacked>(p, ctas, st)
                  : simt_run_t<T, DH, 64, kPacked>(p, ctas, st);
}

int simt_launch(const AttnExtArgs& x, cudaStream_t st) {
  const AttnArgs& a = x.a;
  const medusa_tree* t = a.tree;
  const SimtPlan pl = simt_plan(t, a.B, a.Hq, a.Hkv, a.dh, a.Lcap, a.window, a.sinks);
  if (pl.ctas > 0x7fffffffLL) return fail(MEDUSA_ERR_UNSUPPORTED, "too many query rows for one launch");
  SimtParams p;
  p.q = a.q;
  p.k = x.packed ? x.packed->k_codes : a.k;
  p.v = x.packed ? x.packed->v_codes : a.v;
  p.kp = x.packed ? (const uint32_t*)x.packed->k_par : nullptr;
  p.vp = x.packed ? (const uint32_t*)x.packed->v_par : nullptr;
  p.L = a.L;
  p.anc = t->d_anc;
  p.depth = t->d_depth;
  p.N = t->N;
  p.W = t->W;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.Lcap = a.Lcap;
  p.R = pl.R;
  p.rblocks = pl.rblocks;
  p.P = pl.P;
  p.window = a.window;
  p.sinks = a.sinks;
  p.qscale = a.scale * kLog2e;
  p.po = (float*)((uint8_t*)a.ws + pl.off_o);
  p.pml = (float2*)((uint8_t*)a.ws + pl.off_ml);
  int rc;
  const bool f32 = a.dtype == MEDUSA_F32, d64 = a.dh == 64;
  if (x.packed)
    rc = f32 ? (d64 ? simt_run<float, 64, true>(p, pl.RB, pl.ctas, st)
                    : simt_run<float, 128, true>(p, pl.RB, pl.ctas, st))
             : (d64 ? simt_run<__nv_bfloat16, 64, true>(p, pl.RB, pl.ctas, st)
                    : simt_run<__nv_bfloat16, 128, true>(p, pl.RB, pl.ctas, st));
  else
    rc = f32 ? (d64 ? simt_run<float, 64, false>(p, pl.RB, pl.ctas, st)
                    : simt_run<float, 128, false>(p, pl.RB, pl.ctas, st))
             : (d64 ? simt_run<__nv_bfloat16, 64, false>(p, pl.RB, pl.ctas, st)
                    : simt_run<__nv_bfloat16, 128, false>(p, pl.RB, pl.ctas, st));
  if (rc) return rc;
  return attention_combine_launch(a, p.po, p.pml, pl.P, st);
}

}  // namespace

long long ext_max_keys(int Lcap, int N, int window, int sinks) {
  if (window <= 0) return Lcap;
  const long long k = (long long)window + sinks + N;
  return k < Lcap ? k : Lcap;
}

namespace {

// Windowed bf16 path: the launch shape is the plain kernels' for a cache that
// holds what a sequence's nodes can see, whole tiles for the sinks.
int window_tc_lcap(int Lcap, int N, int window, int sinks) {
  const long long s = ((long long)sinks + 127) / 128 * 128;
  const long long k = ext_max_keys(Lcap, N, window, (int)(s < 0x7fffffff ? s : 0x7fffffff));
  return (int)k;
}
struct WindowTcPlan {
  TcShape sh;
  size_t off_o, off_ml, total;
};
WindowTcPlan window_tc_plan(const medusa_tree* t, int B, int Hq, int Hkv, int dh, int Lcap,
                            int window, int sinks) {
  WindowTcPlan p;
  p.sh = attention_tc_shape(B, Hq, Hkv, t->N, window_tc_lcap(Lcap, t->N, window, sinks), true);
  WsCarver w;
  const size_t rows = p.sh.P > 1 && !p.sh.fuse ? (size_t)B * Hkv * p.sh.P * t->N * (Hq / Hkv) : 0;
  p.off_o = w.take<float>(rows * dh);
  p.off_ml = w.take<float2>(rows);
  p.total = w.total();
  return p;
}

}  // namespace

size_t attention_ext_workspace(const medusa_tree* t, int B, int Hq, int Hkv, int dh, int Lcap,
                               int dtype, int window, int sinks, bool packed) {
  if (!packed && window <= 0) return attention_workspace(t, B, Hq, Hkv, dh, Lcap, dtype);
  if (!packed && attention_tc_eligible(dtype, dh, Hq, Hkv))
    return window_tc_plan(t, B, Hq, Hkv, dh, Lcap, window, sinks).total;
  if (packed && attention_packed_rows_eligible(dtype, dh, t->N * (Hq / Hkv)))
    return attention_packed_rows_workspace(t, B, Hq, Hkv, Lcap, window, sinks);
  if (packed && attention_packed_tc_eligible(dtype, dh))
    return attention_packed_tc_workspace(t, B, Hq, Hkv, Lcap, window, sinks);
  return simt_plan(t, B, Hq, Hkv, dh, Lcap, window, sinks).total;
}

int attention_ext_launch(const AttnExtArgs& x, cudaStream_t st) {
  const AttnArgs& a = x.a;
  if (!x.packed && a.window <= 0) return attention_launch(a, st);  // no window: the plain call
  if (!x.packed && attention_tc_eligible(a.dtype, a.dh, a.Hq, a.Hkv)) {
    const WindowTcPlan p =
        window_tc_plan(a.tree, a.B, a.Hq, a.Hkv, a.dh, a.Lcap, a.window, a.sinks);
    float* po = (float*)((uint8_t*)a.ws + p.off_o);
    float2* pml = (float2*)((uint8_t*)a.ws + p.off_ml);
    int rc = attention_tc_run(a, p.sh, po, pml, st);
    if (rc || p.sh.P == 1 || p.sh.fuse) return rc;
    return attention_combine_launch(a, po, pml, p.sh.P, st);
  }
  if (x.packed && attention_packed_rows_eligible(a.dtype, a.dh, a.tree->N * (a.Hq / a.Hkv)))
    return attention_packed_rows_launch(a, *x.packed, st);
  if (x.packed && attention_packed_tc_eligible(a.dtype, a.dh))
    return attention_packed_tc_launch(a, *x.packed, st);
  return simt_launch(x, st);
}

}  // namespace medusa

// The 4-bit KV cache: storing K/V rows, reading them back, and the compaction
// of the accepted path.
//
// A cached row (one token's K or V of one kv-head, dh values x) is held as
// dh 4-bit codes, a bf16 scale and an integer zero point:
//   lo = min(0, min x), hi = max(0, max x)
//   scale = bf16((hi - lo) / 15)
//   zero  = clamp(rint(-lo / scale), 0, 15)
//   code  = clamp(rint(x / scale) + zero, 0, 15)
// and stands for scale * (code - zero).  Every step is an fp32 operation
// rounded to nearest, rint rounds ties to even, so the codes are defined to
// the last bit.  The range always holds 0, hence 0 is stored exactly, and
// code - zero is a small integer, exact in every type the readers use.  A
// row of zeros has scale 0; a row with a NaN, an infinity or a range beyond
// fp32 gets a NaN scale (it reads back as NaN).
//
// Layout: codes [B][Hkv][Lcap][dh/2] bytes (element 2i in the low half of byte
// i), (scale, zero) [B][Hkv][Lcap] bf16 pairs: the keys of one kv-head are
// contiguous, so a 128-key tile is one 8 KB block (dh = 128) and its scales
// 512 bytes.  68 bytes per row of 128 values, 3.8 x less than bf16.
//
// A row is taken by dh/8 lanes of a warp, 8 values (one 32-bit code word) each,
// so loads of values are 16 or 32 bytes per lane and coalesced along the
// heads.  The read back is bound by HBM (16 ragged prompts of up to 8192
// tokens, 8 heads of 128 in bf16: 108 us, 5.7 TB/s), the store by instruction issue (118
// us, see row_grid), both and the compaction by launch latency at a tree's
// few rows.  In fp32 the same store takes 148 us of 101 at the HBM rate (its
// four rows in flight spill 28 bytes a thread), the read back 258 of 176.
#include "common.cuh"
#include "internal.h"

namespace medusa {
namespace {

constexpr int kThreads = 256;

// 8 consecutive values of a row as loaded, and as four fp32 pairs.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float x[8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
  }
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ float get(int i) const { return x[i]; }
  // min(0, min x) and max(0, max x) over the row's LPR lanes; hi is infinite
  // or NaN if a value is
  template <int LPR>
  __device__ __forceinline__ void range(float& lo, float& hi) const {
    float nan = 0.f;
    lo = hi = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
      nan = fmaf(x[i], 0.f, nan);  // NaN from a NaN or an infinity
    }
    if (nan != 0.f) hi = INFINITY;  // reaches every lane through the row maximum
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
  }
};
__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <>
struct Raw8<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
  // in pairs, exact in bf16: (lo, -hi) in one register, so a step over the
  // lanes is one shuffle and one minimum
  template <int LPR>
  __device__ __forceinline__ void range(float& lo, float& hi) const {
    const uint32_t mn = min_nan2(min_nan2(w[0], w[1]), min_nan2(w[2], w[3]));
    const uint32_t mx = max_nan2(max_nan2(w[0], w[1]), max_nan2(w[2], w[3]));
    uint32_t m = min_nan2(__byte_perm(mn, mx, 0x5410) ^ 0x80000000u,
                          __byte_perm(mn, mx, 0x7632) ^ 0x80000000u);
    m = min_nan2(m, 0u);
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) m = min_nan2(m, __shfl_xor_sync(0xffffffffu, m, o));
    lo = __uint_as_float(m << 16);
    hi = -__uint_as_float(m & 0xffff0000u);
  }
};
// Decodes a code word and stores its 8 values scale * (code - zero).  Small
// integers by their bits: 2^23 + code in fp32, 128 + code in bf16; code - zero
// is exact either way, and the product is rounded once.  (bf16 through fp32:
// 132 us instead of 108 for the read back of row_grid's example.)
__device__ __forceinline__ void decode8(float* p, uint32_t w, uint32_t par) {
  const float s = __uint_as_float(par << 16), z = 8388608.f + __uint_as_float(par & 0xffff0000u);
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = s * (__uint_as_float(0x4b000000u | ((w >> (4 * e)) & 15u)) - z);
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void decode8(__nv_bfloat16* p, uint32_t w, uint32_t par) {
  const uint32_t s2 = __byte_perm(par, 0u, 0x1010);
  const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&s2);
  const __nv_bfloat162 z = __float2bfloat162_rn(128.f + __uint_as_float(par & 0xffff0000u));
  uint32_t h[4];  // elements j and j + 4
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t c = ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 v = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&c), z), s);
    h[j] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(p) =
      make_uint4(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410),
                 __byte_perm(h[0], h[1], 0x7632), __byte_perm(h[2], h[3], 0x7632));
}

// The codes of 8 values, divided: rint of the correctly rounded quotients.
template <typename T>
__device__ __forceinline__ uint32_t codes_by_division(const Raw8<T>& x, float s, float zero) {
  uint32_t w = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = fminf(fmaxf(rintf(__fdiv_rn(x.get(i), s)) + zero, 0.f), 15.f);
    w |= (uint32_t)(int)c << (4 * i);
  }
  return w;
}

// Encodes one row held 8 values to a lane by LPR neighbouring lanes: this
// lane's code word, and the row's (scale, zero) word.
//
// rint(x / s) without a division: x times the hardware's 1 / s (1 ulp) is
// within 4e-6 of the quotient (|x / s| < 16).
//   bf16: x and s have 8 significant bits, so a quotient that is no tie is at
//   least 1/512 away from one.  Adding 1.5 * 2^13 rounds to the nearest
//   multiple of 2^-10: ties come out exact, the others stay on their side.
//   (One value in 400 is a tie: testing for them and dividing there cost 4
//   warps in 10 eight divisions.)
//   fp32: the nearest integer of the product is the quotient's unless it lies
//   that close to a tie; a lane with such a value (one in 6000) divides.
// Adding 1.5 * 2^23 rounds to nearest even and leaves the integer in the low
// bits, so no conversion instruction is used (rint and float-to-int run at an
// eighth of the rate of an addition); the eight integers go into the word by
// shifts and additions, the offsets of all by one multiply-add.  A code is
// never negative: rint is odd and monotone, so rint(x / s) >= rint(lo / s) =
// -zero.  It is 16 at most, and clamped, in a row whose lo and hi both round
// away from 0 (one in 90).
template <typename T, int LPR>
__device__ __forceinline__ uint32_t encode(const Raw8<T>& x, uint32_t& par) {
  float lo, hi;
  x.template range<LPR>(lo, hi);
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
  const float s = __bfloat162float(sb);
  if (!(s <= 3.4028234e38f)) {
    par = 0x7fc0u;  // scale NaN, zero 0
    return 0u;
  }
  if (s == 0.f) {
    par = 0u;
    return 0u;
  }
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  constexpr bool kFine = sizeof(T) == 2;  // ties made exact
  constexpr float kMagic = 12582912.f;    // 1.5 * 2^23
  constexpr float kFirst = kFine ? 12288.f : kMagic;  // 1.5 * 2^13
  constexpr uint32_t kBits = 0x4b400000u;  // kMagic's bits: those of kMagic + n are kBits + n
  float tz = fmaf(-lo, r, kFirst), th = fmaf(hi, r, kFirst);
  if (kFine) {
    tz = __fadd_rn(tz, kMagic - kFirst);
    th = __fadd_rn(th, kMagic - kFirst);
  }
  float zero = __fsub_rn(tz, kMagic);
  float far = fabsf(fmaf(-lo, r, -zero));  // fp32: largest distance from an integer
  const uint32_t bias = __float_as_uint(tz) - 2u * kBits;  // (modulo 2^32: t[i] + bias is the code)
  const bool over = __float_as_uint(th) + bias > 15u;
  const unsigned long long r2 = f2_pack(r, r), first2 = f2_pack(kFirst, kFirst);
  uint32_t t[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned long long x2 = f2_pack(x.get(2 * i), x.get(2 * i + 1));
    unsigned long long t2 = f2_fma(x2, r2, first2);
    if (kFine) {
      t2 = f2_add(t2, f2_pack(kMagic - kFirst, kMagic - kFirst));
    } else {
      float d0, d1;
      f2_unpack(f2_fma(x2, r2, f2_fma(t2, f2_pack(-1.f, -1.f), first2)), d0, d1);
      far = fmaxf(far, fmaxf(fabsf(d0), fabsf(d1)));
    }
    float t0, t1;
    f2_unpack(t2, t0, t1);
    t[2 * i] = __float_as_uint(t0);
    t[2 * i + 1] = __float_as_uint(t1);
  }
  uint32_t w = 0u;
  if (!over) {
#pragma unroll
    for (int i = 7; i >= 0; --i) w = w * 16u + t[i];
    w += bias * 0x11111111u;
  } else {
#pragma unroll
    for (int i = 7; i >= 0; --i) w = w * 16u + __viaddmin_u32(t[i], bias, 15u);
  }
  // (1 / s may overflow for the smallest scales; far is the lane's own: every
  // lane of a row finds the same zero either way)
  if ((!kFine && !(far <= 0.49999f)) || s < 1e-30f) {
    zero = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f);
    w = codes_by_division(x, s, zero);
  }
  par = (uint32_t)__bfloat16_as_ushort(sb) | (__float_as_uint(zero) & 0xffff0000u);
  return w;
}

// idx / d for idx < 2^31 with m = floor(2^32 / d) (d = 1: 2^32 - 1): the high
// product is at most 2 short.
__device__ __forceinline__ uint32_t fast_div(uint32_t idx, uint32_t d, uint32_t m) {
  uint32_t q = __umulhi(idx, m);
  uint32_t r = idx - q * d;
  if (r >= d) {
    ++q;
    r -= d;
  }
  return r >= d ? q + 1 : q;
}

// Grid: x over the (token, head) rows of a sequence, y the sequences, z K and
// V; RPT rows per lane group in flight at once.  The rows' slots are those of
// tokens start_b + t, t < count_b.
struct RowGrid {
  const int32_t* start;
  const int32_t* count;
  int B, T, H, Lcap;
  uint32_t rows, hmul;  // T * H, floor(2^32 / H)
  uint32_t dt, dh;      // a step of one block's rows in (token, head)
};

// Cache rows of rows `row`, `row` + one block's rows, ... of sequence b; -1: not
// one of its tokens, or outside the cache.
template <int RPT>
__device__ __forceinline__ void cache_rows(const RowGrid& g, int b, int start, int count, uint32_t row,
                                           long long (&out)[RPT]) {
  uint32_t t = fast_div(row, g.H, g.hmul), h = row - t * g.H;
  const uint32_t n = (uint32_t)min(count, g.T);
  const long long base = (long long)b * g.H * g.Lcap;
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const long long slot = (long long)start + t;
    const bool in = t < n && slot >= 0 && slot < g.Lcap;
    out[i] = in ? base + (long long)h * g.Lcap + slot : -1;
    t += g.dt;
    h += g.dh;
    if (h >= (uint32_t)g.H) {
      h -= g.H;
      ++t;
    }
  }
}

template <typename T, int DH, int RPT>
__global__ void __launch_bounds__(kThreads, 4)
    kv_pack_kernel(const T* k, const T* v, const RowGrid g, uint32_t* kc, uint32_t* kp,
                   uint32_t* vc, uint32_t* vp) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int LPR = DH / 8;
  constexpr int GROUPS = kThreads / LPR;
  const T* src = blockIdx.z ? v : k;
  uint32_t* codes = blockIdx.z ? vc : kc;
  uint32_t* par = blockIdx.z ? vp : kp;
  const int sub = threadIdx.x % LPR;
  const uint32_t first = blockIdx.x * (GROUPS * RPT);
  for (int b = blockIdx.y; b < g.B; b += gridDim.y) {
    const int count = g.count ? g.count[b] : g.T, start = g.start[b];
    if (count <= 0 || (long long)first >= (long long)count * g.H) continue;  // (uniform) past its tokens
    Raw8<T> x[RPT];
    long long dst[RPT];
    const uint32_t row = first + threadIdx.x / LPR;
    cache_rows<RPT>(g, b, start, count, row, dst);
    const T* from = src + ((size_t)b * g.rows + row) * DH + sub * 8;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      x[i].clear();
      if (dst[i] >= 0) x[i].load(from + i * (GROUPS * DH));
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      uint32_t p;
      const uint32_t w = encode<T, LPR>(x[i], p);  // every lane: the row maxima are shuffles
      if (dst[i] >= 0) {
        codes[dst[i] * LPR + sub] = w;
        if (sub == 0) par[dst[i]] = p;
      }
    }
  }
}

// The values of slots start_b .. start_b + T - 1; zeros past a sequence's
// count and outside the cache.
template <typename T, int DH, int RPT>
__global__ void __launch_bounds__(kThreads)
    kv_unpack_kernel(const uint32_t* kc, const uint32_t* kp, const uint32_t* vc,
                     const uint32_t* vp, const RowGrid g, T* k, T* v) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int LPR = DH / 8;
  constexpr int GROUPS = kThreads / LPR;
  const uint32_t* codes = blockIdx.z ? vc : kc;
  const uint32_t* par = blockIdx.z ? vp : kp;
  T* out = blockIdx.z ? v : k;
  const int sub = threadIdx.x % LPR;
  for (int b = blockIdx.y; b < g.B; b += gridDim.y) {
    const int count = g.count ? g.count[b] : g.T, start = g.start[b];
    const uint32_t row0 = blockIdx.x * (GROUPS * RPT) + threadIdx.x / LPR;
    uint32_t w[RPT], p[RPT];
    long long src[RPT];
    cache_rows<RPT>(g, b, start, max(count, 0), row0, src);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      w[i] = src[i] >= 0 ? codes[src[i] * LPR + sub] : 0u;
      p[i] = src[i] >= 0 ? par[src[i]] : 0u;
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const uint32_t row = row0 + i * GROUPS;
      if (row >= g.rows) continue;
      decode8(out + ((size_t)b * g.rows + row) * DH + sub * 8, w[i], p[i]);
    }
  }
}

// Accepted path of every (layer, sequence, kv-head): slot L_b + j <- slot
// L_b + n_j, j = 1..a.  A thread owns one 32-bit word of a slot (code words
// of K and V, then the two (scale, zero) words) and reads all its sources
// before it writes: n_j >= j, so no source is overwritten by an earlier move
// and the moves are those of the in-order copy.
__global__ void __launch_bounds__(kThreads)
    kv_compact_packed_kernel(uint32_t* __restrict__ kc, uint32_t* __restrict__ kp,
                             uint32_t* __restrict__ vc, uint32_t* __restrict__ vp,
                             const int32_t* L, const int32_t* alen,
                             const int32_t* anodes, long long total, int B, int H,
                             int words, int Lcap, int K, int32_t* __restrict__ new_len) {
  griddep_launch_dependents();
  griddep_wait();
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i < B && new_len != nullptr) {
    const int a = alen[i], Lb = L[i];
    new_len[i] = (a >= 0 && a <= K && Lb >= 0) ? Lb + 1 + a : -1;
  }
  if (i >= total) return;
  const int per = 2 * words + 2;
  const long long lbh = i / per;  // (layer, sequence, kv-head)
  const int w = (int)(i - lbh * per);
  const int b = (int)((lbh / H) % B);
  const int a = alen[b], Lb = L[b];
  if (a < 0 || a > K || Lb < 0) return;
  // word w of a slot: K codes, V codes, K (scale, zero), V (scale, zero)
  uint32_t* base;
  int stride;
  if (w < 2 * words) {
    base = (w < words ? kc : vc) + lbh * Lcap * words + (w < words ? w : w - words);
    stride = words;
  } else {
    base = (w == 2 * words ? kp : vp) + lbh * Lcap;
    stride = 1;
  }
  uint32_t val[MEDUSA_MAX_K];
  bool ok[MEDUSA_MAX_K];
#pragma unroll
  for (int j = 1; j <= MEDUSA_MAX_K; ++j) {
    ok[j - 1] = false;
    if (j <= a) {
      const int n = anodes[(size_t)b * (K + 1) + j];
      const long long src = (long long)Lb + n;
      ok[j - 1] = n >= j && src < Lcap && (long long)Lb + j < Lcap;
      if (w == 0) dbg_ok(ok[j - 1], DBG_COMPACT_NODE);
      if (ok[j - 1]) val[j - 1] = base[src * stride];
    }
  }
#pragma unroll
  for (int j = 1; j <= MEDUSA_MAX_K; ++j)
    if (ok[j - 1]) base[((long long)Lb + j) * stride] = val[j - 1];
}

// Few rows: one per lane group (latency); many: four in flight, in 64 registers
// (16 ragged prompts of up to 8192 tokens, 8 heads: the store takes 118 us; when
// it took 181, two rows in flight took 198, one 241).  It is bound by
// instruction issue (the row's range and the 8 codes of a lane), the read back
// by HBM writes.
int row_grid(const PackedRows& a, int groups, bool* many, RowGrid* g, dim3* grid) {
  const long long rows = (long long)a.T * a.c.Hkv;
  if (rows > 0x7fffffffLL - 4 * kThreads)
    return fail(MEDUSA_ERR_UNSUPPORTED, "T * Hkv does not fit 31 bits");
  *many = rows * a.B >= 4LL * groups * num_sms();
  g->start = a.start;
  g->count = a.count;
  g->B = a.B;
  g->T = a.T;
  g->H = a.c.Hkv;
  g->Lcap = a.c.Lcap;
  g->rows = (uint32_t)rows;
  g->dt = (uint32_t)(groups / a.c.Hkv);
  g->dh = (uint32_t)(groups % a.c.Hkv);
  g->hmul = a.c.Hkv == 1 ? 0xffffffffu : (uint32_t)((1ull << 32) / (uint32_t)a.c.Hkv);
  const int per = groups * (*many ? 4 : 1);
  *grid = dim3((unsigned)((rows + per - 1) / per), (unsigned)(a.B < 65535 ? a.B : 65535), 2);
  return MEDUSA_OK;
}

template <typename T, int DH>
int pack_launch_t(const PackedRows& a, cudaStream_t st) {
  bool many = false;
  RowGrid g = {};
  dim3 grid;
  int rc = row_grid(a, kThreads / (DH / 8), &many, &g, &grid);
  if (rc) return rc;
  auto* fn = many ? kv_pack_kernel<T, DH, 4> : kv_pack_kernel<T, DH, 1>;
  cudaError_t e = launch_pdl(fn, grid, dim3(kThreads), 0, st, (const T*)a.k, (const T*)a.v, g,
                             (uint32_t*)a.c.k_codes, (uint32_t*)a.c.k_par, (uint32_t*)a.c.v_codes,
                             (uint32_t*)a.c.v_par);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail(e, "kv_pack_kernel launch");
}
template <typename T, int DH>
int unpack_launch_t(const PackedRows& a, cudaStream_t st) {
  bool many = false;
  RowGrid g = {};
  dim3 grid;
  int rc = row_grid(a, kThreads / (DH / 8), &many, &g, &grid);
  if (rc) return rc;
  auto* fn = many ? kv_unpack_kernel<T, DH, 4> : kv_unpack_kernel<T, DH, 1>;
  cudaError_t e = launch_pdl(fn, grid, dim3(kThreads), 0, st, (const uint32_t*)a.c.k_codes,
                             (const uint32_t*)a.c.k_par, (const uint32_t*)a.c.v_codes,
                             (const uint32_t*)a.c.v_par, g, (T*)a.k_out, (T*)a.v_out);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail(e, "kv_unpack_kernel launch");
}

}  // namespace

int kv_pack_launch(const PackedRows& a, cudaStream_t st) {
  if (a.dtype == MEDUSA_F32)
    return a.c.dh == 64 ? pack_launch_t<float, 64>(a, st) : pack_launch_t<float, 128>(a, st);
  return a.c.dh == 64 ? pack_launch_t<__nv_bfloat16, 64>(a, st)
                      : pack_launch_t<__nv_bfloat16, 128>(a, st);
}

int kv_unpack_launch(const PackedRows& a, cudaStream_t st) {
  if (a.dtype == MEDUSA_F32)
    return a.c.dh == 64 ? unpack_launch_t<float, 64>(a, st) : unpack_launch_t<float, 128>(a, st);
  return a.c.dh == 64 ? unpack_launch_t<__nv_bfloat16, 64>(a, st)
                      : unpack_launch_t<__nv_bfloat16, 128>(a, st);
}

int kv_compact_packed_launch(const PackedCache& c, int layers, int B, const int32_t* L,
                             const int32_t* alen, const int32_t* anodes, int K, int32_t* new_len,
                             cudaStream_t st) {
  const int words = c.dh / 8;
  const long long total = (long long)layers * B * c.Hkv * (2 * words + 2);
  const long long blocks = ((total > B ? total : B) + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return fail(MEDUSA_ERR_UNSUPPORTED, "too many rows for one launch");
  cudaError_t e = launch_pdl(kv_compact_packed_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, st,
                             (uint32_t*)c.k_codes, (uint32_t*)c.k_par, (uint32_t*)c.v_codes,
                             (uint32_t*)c.v_par, L, alen, anodes, total, B, c.Hkv, words, c.Lcap,
                             K, new_len);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? MEDUSA_OK : cuda_fail(e, "kv_compact_packed_kernel launch");
}

}  // namespace medusa

// Tree attention over the 4-bit cache with many query rows per kv-head (more
// than 128): two 128-row query tiles per CTA, query rows as the MMAs' rows.
// Included by attention_packed_tc.cu.
//
// With this many rows the products bound the call, not the cache, and a tile's
// work per softmax thread decides: a thread here owns one query row and all 128 keys of a
// tile, keeps the row's maximum and sum to itself (no votes, no weights
// through shared memory: P goes back to TMEM over the S columns just read),
// where the key-major kernel needs a vote of 128 threads per tile and 64 row
// sums per thread.  8B-GQA batch of 16 (512 rows per kv-head, 8K prefixes): 360
// us, key-major 604; 52 heads, 256-node trees, 4 x 32K: 1.11 ms.  The products
// and the exponentials take 2048 cycles each per pair of tiles and 128 keys;
// 4400 to 5000 pass: the waits between them.
//   S = Q K^T   M 128 rows x N 128 keys, Q and K K-major in shared memory
//   O += P V    A = P from TMEM (fp16), B = V MN-major
// Both tiles read every unpacked K/V tile.  MMA order S_a(0), S_b(0), then
// PV_a(t), S_a(t+1), PV_b(t), S_b(t+1): one tile's products run during the
// other's softmax.  K and V are unpacked with their scales, relative to a power
// of two >= the tile's largest for K (one factor on the tile's scores) and >=
// the largest so far for V (its growth rescales O), 2^-117 at least, and rounded
// once to fp16 (scales read from shared memory by every softmax thread, 128 a
// tile, made the call 1.25 x as long).  The weights of a tile's first 64 keys are
// rounded to fp16 a second time when the other 64 raise the row's maximum by
// more than 2^8.  A row whose K or V has no finite scale is stored as 0
// and put back as NaN scores, so that it reaches the rows that see it only.
// Warpgroups: 0 TMA (ring of K and V code tiles) and MMA issue, 1 unpack, 2
// and 3 the softmax of query tiles a and b.

struct PairCfg {
  static constexpr int kThreads = 512;
  static constexpr int kRegs0 = 56, kRegsUnpack = 80, kRegsSoftmax = 184, kRegsLaunch = 128;
  static_assert(kRegs0 + kRegsUnpack + 2 * kRegsSoftmax <= 4 * kRegsLaunch, "register split");
  static constexpr uint32_t kTile = 2 * kAtom;  // 128 rows of 128 fp16: 32 KB
  static constexpr int kItems = 3;              // ring of K and V code tiles, K, V, K, V, ...
  static constexpr uint32_t kItem = kCodeTile + 2 * BK * 4;  // K's carries both (scale, zero) rows
  static constexpr uint32_t oK = 2 * kTile;
  static constexpr uint32_t oV = oK + 2 * kTile;
  static constexpr uint32_t oRing = oV + 2 * kTile;
  static constexpr uint32_t oMisc = oRing + kItems * kItem;
  static constexpr size_t kSmem = 1024 + oMisc + 512;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// The 8 codes of a word as four fp16 pairs of scale * (code - zero), rounded
// once: 1024 + code and 1024 + 16 code are fp16 numbers by their bits, z1 =
// -(1024 + zero) and z16 = -(1024 + 16 zero) bring them to code - zero and 16
// times it, a1 and a16 = a1 / 16 are the scale.
__device__ __forceinline__ void unpack_word_scaled(uint32_t w, __half2 z1, __half2 z16, __half2 a1,
                                                   __half2 a16, uint32_t* r) {
  const uint32_t v = w >> 8;
  const uint32_t e[4] = {(w & 0x000f000fu) | 0x64006400u, (w & 0x00f000f0u) | 0x64006400u,
                         (v & 0x000f000fu) | 0x64006400u, (v & 0x00f000f0u) | 0x64006400u};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 h = __hmul2(__hadd2(*reinterpret_cast<const __half2*>(&e[j]), (j & 1) ? z16 : z1),
                              (j & 1) ? a16 : a1);
    r[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

// 2^(q2 x s + m2) for the 64 scores of one key half as fp16 pairs (pk[c]: keys
// 2c, 2c + 1); returns their fp32 sum.  Every exponential on MUFU (one pair in
// two, four or eight by polynomial on the FMA pipe: 132, 124 and 120 us against
// 119 at the 8B-GQA shape, 4 sequences).
__device__ __forceinline__ float exp_pack64_f16(const float (&v)[64], unsigned long long q2,
                                                unsigned long long m2, uint32_t (&pk)[32]) {
  unsigned long long sum2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int c2 = 0; c2 < 32; ++c2) {
    float x0, x1, e0, e1;
    f2_unpack(f2_fma(f2_pack(v[2 * c2], v[2 * c2 + 1]), q2, m2), x0, x1);
    e0 = ex2_approx(x0);
    e1 = ex2_approx(x1);
    sum2[c2 & 3] = f2_add(sum2[c2 & 3], f2_pack(e0, e1));
    const __half2 h2 = __floats2half2_rn(e0, e1);
    pk[c2] = *reinterpret_cast<const uint32_t*>(&h2);
  }
  float a0, a1, b0, b1, c0f, c1f, d0, d1;
  f2_unpack(sum2[0], a0, a1);
  f2_unpack(sum2[1], b0, b1);
  f2_unpack(sum2[2], c0f, c1f);
  f2_unpack(sum2[3], d0, d1);
  return ((a0 + a1) + (b0 + b1)) + ((c0f + c1f) + (d0 + d1));
}

// Visible keys of the 32 slots from s0 for a query row (node, depth): prefix
// slots, ancestors, both within the row's window.
__device__ __forceinline__ uint32_t row_mask(int s0, int Lb, int node, int depth,
                                             const PackedParams& p) {
  const int a0 = s0 - Lb;
  uint32_t m = 0u;
  if (a0 > -32) {
    const uint32_t* ar = p.anc + (size_t)node * p.W;
    const int wi = a0 >> 5;  // -1: prefix slots first
    const uint32_t w0 = wi >= 0 && wi < p.W ? __ldg(ar + wi) : 0u;
    const uint32_t w1 = wi + 1 < p.W ? __ldg(ar + wi + 1) : 0u;
    m = __funnelshift_r(w0, w1, a0 & 31);
    if (p.window > 0 && p.window <= depth) {  // ancestors that have left the window
      int a = node;
      for (int d = depth; a >= 0; --d) {
        if (d <= depth - p.window && Lb + d >= p.sinks && a >= a0 && a < a0 + 32)
          m &= ~(1u << (a - a0));
        a = __ldg(p.parent + a);
      }
    }
  }
  if (a0 < 0) {
    const int n = min(32, -a0);  // prefix slots s0 .. s0 + n - 1
    uint32_t pre = 0xffffffffu >> (32 - n);
    if (p.window > 0) {
      const long long low = (long long)Lb + depth - p.window + 1 - s0;  // first in the window
      const uint32_t in = low <= 0 ? 0xffffffffu : low >= 32 ? 0u : 0xffffffffu << (int)low;
      const long long sk = (long long)p.sinks - s0;
      const uint32_t sink = sk <= 0 ? 0u : sk >= 32 ? 0xffffffffu : 0xffffffffu >> (32 - (int)sk);
      pre &= in | sink;
    }
    m |= pre;
  }
  return m;
}

// The power of two >= a scale (its bits), kept in [2^-117, 2^119], where 2^10
// over it is an fp32 number too.
constexpr float kMinRef = 0x1p-117f;
__device__ __forceinline__ float scale_ref(uint32_t bits) {
  const int ex = min(246, max(10, (int)((bits >> 23) + ((bits & 0x7fffffu) ? 1 : 0))));
  return __uint_as_float((uint32_t)ex << 23);
}

__global__ void __launch_bounds__(PairCfg::kThreads, 1)
    tree_attn_packed_pair_kernel(const __grid_constant__ CUtensorMap tmKc,
                                 const __grid_constant__ CUtensorMap tmVc,
                                 const __grid_constant__ CUtensorMap tmKp,
                                 const __grid_constant__ CUtensorMap tmVp, const PackedParams p) {
  using C = PairCfg;
  constexpr int BM = 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = sm;
  uint8_t* sK = sm + C::oK;
  uint8_t* sV = sm + C::oV;
  uint8_t* sRing = sm + C::oRing;
  uint64_t* it_full = (uint64_t*)(sm + C::oMisc);  // [kItems]
  uint64_t* it_empty = it_full + C::kItems;  // [kItems]
  uint64_t* k_ready = it_empty + C::kItems;  // [2]
  uint64_t* k_empty = k_ready + 2;           // [2]
  uint64_t* v_ready = k_empty + 2;           // [2]
  uint64_t* v_empty = v_ready + 2;           // [2]
  uint64_t* s_full = v_empty + 2;            // [query tile]
  uint64_t* p_full = s_full + 2;             // [query tile]
  uint64_t* pv_done = p_full + 2;            // [query tile]
  uint64_t* mma_done = pv_done + 2;
  uint32_t* tmem_slot = (uint32_t*)(mma_done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  unsigned* qmax = (unsigned*)(tmem_slot + 2);
  float* sGrow = (float*)(tmem_slot + 4);  // [4] factor on O before the tile
  float* sRef = sGrow + 4;                 // [4] power of two of the value scales
  float* sScore = sRef + 4;                // [4] scale of the scores
  unsigned* sNan = (unsigned*)(sScore + 4);  // [4][4] keys in use without a finite scale
  unsigned* sMax = sNan + 16;                // [2][K 4 | V 4] largest scales of the unpack warps
  static_assert((2 * C::kItems + 15) * 8 + 16 + 48 + 64 + 64 <= 512, "barrier block");

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kItems; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_ready[i], 4);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_ready[i], 4);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    *qmax = 0u;
    fence_mbar_init();
  }
  griddep_wait();  // prefix lengths, queries and the cache may come from the kernel ahead

  const int id = blockIdx.x;
  const int grp = id % p.groups;  // pair of query tiles
  const int chunk = (id / p.groups) % p.P;
  const int bk = id / p.groups / p.P;
  const int b = bk / p.Hkv, kvh = bk - b * p.Hkv;
  const int row0 = grp * 2 * BM;
  const int Lb = p.L[b];
  const bool seq_ok = Lb >= 0 && (long long)Lb + p.N <= p.Lcap;
  Tiles tl{0, 0, 0};
  if (seq_ok) tl = tile_list(Lb, p.N, p.window, p.sinks);
  const int j0 = (int)((long long)tl.n * chunk / p.P);
  const int T = (int)((long long)tl.n * (chunk + 1) / p.P) - j0;
  if (T == 0) {  // no key in this chunk
    griddep_launch_dependents();
    const int r = row0 + (int)threadIdx.x;
    if ((int)threadIdx.x < 2 * BM && r < p.R) {
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
  auto load_item = [&](int i) {
    const int st = i % C::kItems;
    const int key0 = tl.tile(j0 + (i >> 1)) * BK;
    dbg_ok(key0 >= 0 && key0 < Lb + p.N && key0 < p.Lcap, DBG_ATTN_KEY_TILE);
    uint8_t* dst = sRing + st * C::kItem;
    if (i & 1) {
      mbar_arrive_expect_tx(&it_full[st], kCodeTile);
      tma_load_3d(dst, &tmVc, &it_full[st], 0, key0, bk, pol);
    } else {
      mbar_arrive_expect_tx(&it_full[st], C::kItem);
      tma_load_3d(dst, &tmKc, &it_full[st], 0, key0, bk, pol);
      tma_load_2d(dst + kCodeTile, &tmKp, &it_full[st], key0, bk, pol);
      tma_load_2d(dst + kCodeTile + BK * 4, &tmVp, &it_full[st], key0, bk, pol);
    }
  };
  const int early = min(2 * T, C::kItems);
  if (threadIdx.x == 0)
    for (int i = 0; i < early; ++i) load_item(i);
  __syncthreads();  // qmax
  // Q as fp16 under one power of two, dims in the unpacked codes' order (as in
  // tree_attn_packed_kernel): 16 rows per warp
  uint2 qv[16];
  float qm = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = row0 + warp + 16 * i;
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
    tmem_alloc(tmem_slot, 512);  // S/P a | S/P b | O a | O b
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  griddep_launch_dependents();  // TMEM taken: the next kernel may be scheduled
  int kexp = 0;
  if (*qmax != 0u) kexp = min(120, 13 - ((int)(*qmax >> 23) - 127));
  const float qs = __uint_as_float((uint32_t)(127 + kexp) << 23);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int rr = warp + 16 * i, c = rr & 127;
    const int w = lane >> 1, h = lane & 1;  // dim 8 w + jj + 4 h at position 8 w + 2 jj + h
    __half* dst = (__half*)(sQ + (rr >> 7) * C::kTile + (w >> 3) * kAtom + c * 128 +
                            (((w & 7) ^ (c & 7)) << 4));
    const float f[4] = {bf16_lo(qv[i].x), bf16_hi(qv[i].x), bf16_lo(qv[i].y), bf16_hi(qv[i].y)};
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
      dst[2 * jj + h] = __float2half_rn(f[jj] * qs);
  }
  fence_proxy_async_smem();
  __syncthreads();

  const int wg = warp >> 2, qd = warp & 3;
  const int key = qd * 32 + lane;  // (softmax: the row of the query tile)
  const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
  if (wg == 0) {
    reg_dec<C::kRegs0>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- TMA producer
      int issued = early;
      for (int i = early; i < 2 * T; ++i) {
        const int st = i % C::kItems;
        if (!mbar_wait(&it_empty[st], ((uint32_t)(i / C::kItems) & 1u) ^ 1u, abort_flag)) break;
        load_item(i);
        issued = i + 1;
      }
      if (issued < 2 * T) {
        // aborted: let the loads already issued land before the CTA exits
        for (int i = (issued > C::kItems ? issued - C::kItems : 0); i < issued; ++i)
          mbar_wait(&it_full[i % C::kItems], (uint32_t)(i / C::kItems) & 1u, nullptr);
      }
    }
    if (warp == 1) {
      // -------------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_s = umma_idesc_f16_f32(BM, BK, false, false);
      constexpr uint32_t idesc_o = umma_idesc_f16_f32(BM, DH, false, true);
      const uint64_t dq0 = umma_desc_sw128_kmajor(smem_u32(sQ));
      const uint64_t dk0 = umma_desc_sw128_kmajor(smem_u32(sK));
      const uint64_t dv0 = umma_desc_sw128(smem_u32(sV), kAtom, 1024u);
      auto issue_s = [&](int t, int q) -> bool {
        const int st = t & 1;
        if (q == 0 && !mbar_wait_warp(&k_ready[st], (uint32_t)(t >> 1) & 1u, abort_flag)) return false;
        // the S/P columns of tile q hold P_q(t - 1) until its PV has run
        if (t > 0 && !mbar_wait_warp(&pv_done[q], (uint32_t)(t - 1) & 1u, abort_flag)) return false;
        tc_fence_after();
        const uint64_t dq = dq0 + (uint64_t)(q * (C::kTile >> 4));
        const uint64_t dk = dk0 + (uint64_t)(st * (C::kTile >> 4));
        const uint32_t dS = tmem + (uint32_t)q * 128u;
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * kAtom + (kk & 3) * 32) >> 4);
          umma_f16_warp(dS, dq + off, dk + off, idesc_s, kk > 0 ? 1u : 0u);
        }
        if (q == 1) umma_commit_warp(&k_empty[st]);  // both tiles have read K(t)
        umma_commit_warp(&s_full[q]);
        return true;
      };
      auto issue_pv = [&](int u, int q) -> bool {
        const int st = u & 1;
        if (q == 0 && !mbar_wait_warp(&v_ready[st], (uint32_t)(u >> 1) & 1u, abort_flag)) return false;
        if (!mbar_wait_warp(&p_full[q], (uint32_t)u & 1u, abort_flag)) return false;
        tc_fence_after();
        const uint64_t dv = dv0 + (uint64_t)(st * (C::kTile >> 4));
        const uint32_t aP = tmem + (uint32_t)q * 128u;
        const uint32_t tOq = tmem + 256u + (uint32_t)q * 128u;
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          umma_f16_ts_warp(tOq, aP + (uint32_t)((kk >> 2) * 64 + (kk & 3) * 8),
                           dv + (uint64_t)((kk * 16 * 128) >> 4), idesc_o,
                           (u > 0 || kk > 0) ? 1u : 0u);
        if (q == 1) umma_commit_warp(&v_empty[st]);  // both tiles have read V(u)
        umma_commit_warp(&pv_done[q]);
        return true;
      };
      bool ok = issue_s(0, 0) && issue_s(0, 1);
      for (int t = 0; t < T && ok; ++t) {
        ok = issue_pv(t, 0);
        if (ok && t + 1 < T) ok = issue_s(t + 1, 0);
        if (ok) ok = issue_pv(t, 1);
        if (ok && t + 1 < T) ok = issue_s(t + 1, 1);
      }
      umma_commit_warp(mma_done);
      mbar_wait(mma_done, 0u, nullptr);
    }
  } else if (wg == 1) {
    // ---------------------------------------------------------------- unpack
    reg_dec<C::kRegsUnpack>();
    const int sw = (key >> 1) & 3;  // 64-byte swizzle of the code rows
    float vref = kMinRef;
    bool ok = true;
    uint32_t kp = 0u, vp = 0u;
    float kref = 0.f;
    for (int i = 0; i < 2 * T && ok; ++i) {
      const int t = i >> 1, st = i % C::kItems, bf = t & 1;
      const bool isV = i & 1;
      const uint32_t prev = ((uint32_t)(t >> 1) & 1u) ^ 1u;
      ok = mbar_wait_warp(&it_full[st], (uint32_t)(i / C::kItems) & 1u, abort_flag);
      if (isV) {
        if (!ok) {  // the other warps meet this at the next vote
          if (i + 1 < 2 * T) bar_red_or(1, 128, true);
          break;
        }
      } else {
        const uint32_t* par = (const uint32_t*)(sRing + st * C::kItem + kCodeTile);
        kp = par[key];
        vp = par[BK + key];
        // the largest scales of the keys in use; every warp of the group takes
        // part (an error ends them together)
        const int slot = tl.tile(j0 + t) * BK + key;
        const bool live = slot < Lb + p.N && in_window(slot, Lb, p.window, p.sinks);
        const uint32_t ak = __float_as_uint(fabsf(bf16_lo(kp)));
        const uint32_t av = __float_as_uint(fabsf(bf16_lo(vp)));
        const bool fin = ak < 0x7f800000u && av < 0x7f800000u;
        const unsigned mk = __reduce_max_sync(0xffffffffu, live && fin ? ak : 0u);
        const unsigned mv = __reduce_max_sync(0xffffffffu, live && fin ? av : 0u);
        const unsigned nan = __ballot_sync(0xffffffffu, live && !fin);
        if (lane == 0) {
          sMax[bf * 8 + qd] = mk;
          sMax[bf * 8 + 4 + qd] = mv;
        }
        if (bar_red_or(1, 128, !ok)) break;
        const unsigned* sx = sMax + bf * 8;
        const float nk = scale_ref(max(max(sx[0], sx[1]), max(sx[2], sx[3])));
        const float nref = fmaxf(vref, scale_ref(max(max(sx[4], sx[5]), max(sx[6], sx[7]))));
        const float grow = vref / nref;
        kref = nk;
        vref = nref;
        if (t >= 2) ok = mbar_wait_warp(&k_empty[bf], prev, abort_flag);
        // softmax(t - 4) has read these slots: S(t - 2) followed its P(t - 3)
        if (lane == 0) sNan[(t & 3) * 4 + qd] = nan;
        if (key == 0) {
          // Q carries 2^kexp, K 2^10 / kref.  Never 0, which would turn the -inf
          // of a masked score into NaN: below 2^-126 (K rows of zeros, small
          // queries) the scores, |S| < 2^35, are 0 to fp32 with either factor
          sScore[t & 3] = fmaxf(p.scale2 * ldexpf(1.f, -kexp) * (kref * 0x1p-10f), 0x1p-126f);
          sGrow[t & 3] = grow;
          sRef[t & 3] = vref;
        }
      }
      uint32_t w[16];
      const uint8_t* row = sRing + st * C::kItem + key * 64;
      // scale 2^10 / ref; none for a scale that is not finite or larger than
      // those in use (a slot that no row sees)
      const uint32_t par = isV ? vp : kp;
      const float ref = isV ? vref : kref;
      const float z = fminf(fmaxf(bf16_hi(par), 0.f), 15.f);
      float sc = bf16_lo(par);
      sc = fabsf(sc) <= ref ? sc * __uint_as_float((264u << 23) - __float_as_uint(ref)) : 0.f;
      const __half2 z1 = __float2half2_rn(-1024.f - z), z16 = __float2half2_rn(-1024.f - 16.f * z);
      const __half2 a1 = __float2half2_rn(sc), a16 = __float2half2_rn(sc * 0.0625f);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<uint4*>(&w[4 * e]) = *reinterpret_cast<const uint4*>(row + ((e ^ sw) << 4));
      __syncwarp();
      if (lane == 0) mbar_arrive(&it_empty[st]);
      if (isV && t >= 2) ok = mbar_wait_warp(&v_empty[bf], prev, abort_flag);
      if (ok) {
        uint8_t* dst = (isV ? sV : sK) + bf * C::kTile + key * 128;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          uint32_t r[4];
          unpack_word_scaled(w[e], z1, z16, a1, a16, r);
          *reinterpret_cast<uint4*>(dst + (e >> 3) * kAtom + (((e & 7) ^ (key & 7)) << 4)) =
              make_uint4(r[0], r[1], r[2], r[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(isV ? &v_ready[bf] : &k_ready[bf]);
      }
      if (isV) {  // an error after the vote: the other warps meet it at the next one
        if (!ok && i + 1 < 2 * T) {
          bar_red_or(1, 128, true);
          break;
        }
      } else if (!ok) {
        // K's wait failed: skip V, end together at the next vote
        if (i + 2 < 2 * T) bar_red_or(1, 128, true);
        break;
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    reg_inc<C::kRegsSoftmax>();
    const int q = wg - 2;
    const uint32_t tS = tmem + lane_base + (uint32_t)q * 128u;
    const uint32_t tO = tmem + lane_base + 256u + (uint32_t)q * 128u;
    const int grow_ = row0 + q * BM + key;  // this thread's query row
    const bool row_ok = grow_ < p.R;
    const bool live = row0 + q * BM + qd * 32 < p.R;  // warp-uniform
    const int node = min(grow_ / p.G, p.N - 1);
    const int depth = __ldg(p.depth + node);
    const int m_hi = Lb / BK;
    const long long wl = (long long)Lb + p.K - p.window;
    const int m_lo = p.window > 0 && wl >= 0 ? (int)(wl / BK) : -1;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    for (int t = 0; t < T; ++t) {
      if (!mbar_wait_warp(&s_full[q], (uint32_t)t & 1u, abort_flag)) {
        ok = false;
        break;
      }
      if (live) {
        const int tile = tl.tile(j0 + t);
        const bool masked = tile >= m_hi || tile <= m_lo;
        const uint32_t* nk = sNan + (t & 3) * 4;
        const bool bad_key = (nk[0] | nk[1] | nk[2] | nk[3]) != 0u;  // (rare) rows without a scale
        const float sf = sScore[t & 3];  // scores of this tile: S x sf, base 2
        float fv = sGrow[t & 3];         // growth of the value scale, once per tile
        const unsigned long long q2 = f2_pack(sf, sf);
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          float v[64];
          tc_fence_after();
          tmem_ld64(tS + (uint32_t)(hf * 64), v);
          if (masked || bad_key) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t m = row_mask(tile * BK + hf * 64 + h * 32, Lb, node, depth, p);
              const uint32_t nan = sNan[(t & 3) * 4 + hf * 2 + h];
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const float x = (nan >> c) & 1u ? NAN : v[h * 32 + c];
                v[h * 32 + c] = (m >> c) & 1u ? x : -INFINITY;
              }
            }
          }
          float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int c = 4; c < 64; c += 2) mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], v[c], v[c + 1]);
          const float tmax = max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * sf;
          // Moves the row maximum when it grew by more than 2^kGrow (and, with
          // the tile's first half, follows the value scale): rescales l, the O
          // row and, for the second half, the first half's P
          const bool grow_m = tmax > m_used + kGrow;
          if (__any_sync(0xffffffffu, grow_m) || fv != 1.f) {
            float corr = 1.f;
            if (grow_m) {
              corr = ex2_approx(m_used - tmax);  // 0 when m_used is -inf
              m_used = tmax;
              l *= corr;
            }
            const float fo = corr * fv;
            fv = 1.f;
            if (t > 0) {
              ok = mbar_wait_warp(&pv_done[q], (uint32_t)(t - 1) & 1u, abort_flag);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c0 = 0; c0 < DH; c0 += 16) {
                float o16[16];
                tmem_ld16(tO + (uint32_t)c0, o16);
#pragma unroll
                for (int e = 0; e < 16; ++e) o16[e] *= fo;
                tmem_st16(tO + (uint32_t)c0, o16);
              }
            }
            if (hf == 1) {
#pragma unroll 1
              for (int c0 = 0; c0 < 32; c0 += 16) {
                float w16[16];
                tmem_ld16(tS + (uint32_t)c0, w16);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w16[e]));
                  const __half2 h2 = __floats2half2_rn(f.x * corr, f.y * corr);
                  w16[e] = *reinterpret_cast<const float*>(&h2);
                }
                tmem_st16(tS + (uint32_t)c0, w16);
              }
            }
          }
          // weights x 2^7 as fp16 pairs over the S columns just read
          const float moff = (m_used == -INFINITY ? 0.f : m_used) - 7.f;
          const unsigned long long m2 = f2_pack(-moff, -moff);
          uint32_t pk[32];
          l += exp_pack64_f16(v, q2, m2, pk);
          tmem_st32(tS + (uint32_t)(hf * 64), pk);
        }
        if (!ok) break;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[q]);
    }
    if (ok && live) {
      ok = mbar_wait_warp(&pv_done[q], (uint32_t)(T - 1) & 1u, abort_flag);
      if (ok) {
        tc_fence_after();
        // weights and l carry 2^7, V 2^10 / vref; the power of two comes last, as
        // its product with 1 / l may lose bits below 2^-126
        const float vref = sRef[(T - 1) & 3];
        const float f = p.P == 1 ? (l == 0.f ? 0.f : 0x1p-10f / l) : 0x1p-17f;
        const int g = grow_ - node * p.G;
        __nv_bfloat16* ob =
            p.out + (((size_t)b * p.N + node) * p.Hq + (size_t)kvh * p.G + g) * DH;
        const size_t prow = ((size_t)bk * p.P + chunk) * p.R + grow_;
#pragma unroll 1
        for (int c0 = 0; c0 < DH; c0 += 16) {
          float o16[16];
          tmem_ld16(tO + (uint32_t)c0, o16);
          if (!row_ok) continue;
          float d[16];  // position 8 w + 2 jj + h is dim 8 w + jj + 4 h
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int jj = (e >> 1) & 3;
            d[(e & 8) + jj + 4 * (e & 1)] = o16[e] * f * vref;
          }
          if (p.P == 1) {
            __align__(16) __nv_bfloat162 h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = __floats2bfloat162_rn(d[2 * e], d[2 * e + 1]);
            reinterpret_cast<uint4*>(ob + c0)[0] = reinterpret_cast<const uint4*>(h)[0];
            reinterpret_cast<uint4*>(ob + c0)[1] = reinterpret_cast<const uint4*>(h)[1];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              reinterpret_cast<float4*>(p.po + prow * DH + c0)[e] =
                  make_float4(d[4 * e], d[4 * e + 1], d[4 * e + 2], d[4 * e + 3]);
          }
        }
        // (a sum of NaN must reach the merge, which skips m = -inf)
        if (p.P > 1 && row_ok) p.pml[prow] = make_float2(l != l && m_used == -INFINITY ? 0.f : m_used, l * 0x1p-7f);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

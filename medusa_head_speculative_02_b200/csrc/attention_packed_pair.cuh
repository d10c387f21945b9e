// Tree attention over the 4-bit cache with many query rows per kv-head (more
// than 128): two 128-row query tiles per CTA, query rows as the MMAs' rows.
// Included by attention_packed_tc.cu.
//
// Same arithmetic as tree_attn_packed_kernel.  With this many rows the
// products bound the call, not the cache, and a tile's work per softmax
// thread decides: a thread here owns one query row and all 128 keys of a
// tile, keeps the row's maximum and sum to itself (no votes, no weights
// through shared memory: P goes back to TMEM over the S columns just read),
// where the key-major kernel needs a vote of 128 threads per tile and 64 row
// sums per thread.  8B-GQA batch of 16 (512 rows per kv-head): key-major 604
// us.
//   S = Q K^T   M 128 rows x N 128 keys, Q and K K-major in shared memory
//   O += P V    A = P from TMEM (fp16), B = V MN-major
// Both tiles read every unpacked K/V tile.  MMA order S_a(0), S_b(0), then
// PV_a(t), S_a(t+1), PV_b(t), S_b(t+1): one tile's products run during the
// other's softmax.  The unpack warps write the scales of a tile beside it:
// sk * softmax scale, and sv relative to a power of two >= the largest sv so
// far times 2^-7, whose growth (a factor they pass on) rescales O.
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
  static constexpr uint32_t oScale = oRing + kItems * kItem;
  static constexpr uint32_t oMisc = oScale + 4 * BK * 4;
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
  float* sScale = (float*)(sm + C::oScale);  // [4][128]: K scale x softmax scale
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
  unsigned* sMax = (unsigned*)(sRef + 4);  // [2][4] largest value scale of the unpack warps
  static_assert((2 * C::kItems + 15) * 8 + 16 + 32 + 32 <= 512, "barrier block");

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
      dst[2 * jj + h] = __float2half_rn(f[jj] * ((jj & 1) ? qs * 0.0625f : qs));
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
      const uint64_t pol = policy_evict_normal();
      int issued = 0;
      for (int i = 0; i < 2 * T; ++i) {
        const int st = i % C::kItems;
        const int key0 = tl.tile(j0 + (i >> 1)) * BK;
        dbg_ok(key0 >= 0 && key0 < Lb + p.N && key0 < p.Lcap, DBG_ATTN_KEY_TILE);
        if (!mbar_wait(&it_empty[st], ((uint32_t)(i / C::kItems) & 1u) ^ 1u, abort_flag)) break;
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
          umma_f16_ts_warp(tOq, aP + (uint32_t)(kk * 8),
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
    const float cscale = p.scale2 * ldexpf(1.f, 24 - kexp);
    float vref = 0x1p-120f;
    bool ok = true;
    uint32_t vp = 0u;
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
        vp = par[BK + key];
        // the largest value scale of the keys in use; every warp of the group
        // takes part (an error ends them together)
        const int slot = tl.tile(j0 + t) * BK + key;
        const bool live = slot < Lb + p.N && in_window(slot, Lb, p.window, p.sinks);
        const uint32_t av = __float_as_uint(fabsf(bf16_lo(vp)));
        const unsigned sb = __reduce_max_sync(0xffffffffu, live && av < 0x7f800000u ? av : 0u);
        if (lane == 0) sMax[bf * 4 + qd] = sb;
        if (bar_red_or(1, 128, !ok)) break;
        const unsigned bb = max(max(sMax[bf * 4], sMax[bf * 4 + 1]), max(sMax[bf * 4 + 2], sMax[bf * 4 + 3]));
        // power of two >= the largest scale, kept in [2^-120, 2^119]
        const int ex = min(246, max(7, (int)((bb >> 23) + ((bb & 0x7fffffu) ? 1 : 0))));
        const float nref = fmaxf(vref, __uint_as_float((uint32_t)ex << 23));
        const float grow = vref / nref;
        vref = nref;
        if (t >= 2) ok = mbar_wait_warp(&k_empty[bf], prev, abort_flag);
        // softmax(t - 4) has read this scale buffer: S(t - 2) followed its P(t - 3)
        // (a V row with no finite scale is stored as 0 and shows in the scores instead,
        // so that it reaches the rows that see it and no other)
        sScale[(t & 3) * BK + key] =
            fabsf(bf16_lo(vp)) <= 3.3895314e38f ? bf16_lo(par[key]) * cscale : NAN;
        if (key == 0) {
          sGrow[t & 3] = grow;
          sRef[t & 3] = vref;
        }
      }
      uint32_t w[16];
      const uint8_t* row = sRing + st * C::kItem + key * 64;
      __half2 z24, z20;
      __half2 a1, a16;
      if (isV) {
        const float z = fminf(fmaxf(bf16_hi(vp), 0.f), 15.f);
        z24 = __float2half2_rn(-1024.f - z);
        z20 = __float2half2_rn(-1024.f - 16.f * z);
        // sv 2^10 / vref; none for a scale that is not finite or larger than
        // those in use (a slot that no row sees)
        float sv = bf16_lo(vp);
        sv = fabsf(sv) <= vref ? sv * __uint_as_float((264u << 23) - __float_as_uint(vref)) : 0.f;
        a1 = __float2half2_rn(sv);
        a16 = __float2half2_rn(sv * 0.0625f);
      } else {
        zero_pairs(((const uint32_t*)(sRing + st * C::kItem + kCodeTile))[key], z24, z20);
      }
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
          if (isV) unpack_word_scaled(w[e], z24, z20, a1, a16, r);
          else unpack_word(w[e], z24, z20, r);
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
        const float* sc = sScale + (t & 3) * BK;
        const float fv = sGrow[t & 3];  // growth of the value scale
        // scores relative to the row maximum, base 2
        float x[128];
        tc_fence_after();
        tmem_ld128(tS, x);
        const float moff = m_used == -INFINITY ? 0.f : m_used;
        {
          const unsigned long long m2 = f2_pack(-moff, -moff);
          const ulonglong2* k2 = reinterpret_cast<const ulonglong2*>(sc);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const ulonglong2 k = k2[c];
            f2_unpack(f2_fma(f2_pack(x[4 * c], x[4 * c + 1]), k.x, m2), x[4 * c], x[4 * c + 1]);
            f2_unpack(f2_fma(f2_pack(x[4 * c + 2], x[4 * c + 3]), k.y, m2), x[4 * c + 2], x[4 * c + 3]);
          }
        }
        if (masked) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const uint32_t m = row_mask(tile * BK + h * 32, Lb, node, depth, p);
#pragma unroll
            for (int c = 0; c < 32; ++c) x[h * 32 + c] = (m >> c) & 1u ? x[h * 32 + c] : -INFINITY;
          }
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < 128; c += 2) mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], x[c], x[c + 1]);
        const float tmax = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
        // Moves the row maximum when it grew by more than 2^kGrow (or the row
        // met its first key), and follows the value scale: rescales l and O
        const bool grow_m = tmax > kGrow || (m_used == -INFINITY && tmax != -INFINITY);
        if (__any_sync(0xffffffffu, grow_m) || fv != 1.f) {
          float corr = 1.f, d = 0.f;
          if (grow_m) {
            d = -tmax;
            corr = m_used == -INFINITY ? 0.f : ex2_approx(d);
            m_used = moff + tmax;
            l *= corr;
          }
          const float fo = corr * fv;
#pragma unroll
          for (int c = 0; c < 128; ++c) x[c] += d;
          if (t > 0) {
            ok = mbar_wait_warp(&pv_done[q], (uint32_t)(t - 1) & 1u, abort_flag);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < DH; c0 += 8) {
              float o8[8];
              tmem_ld8(tO + (uint32_t)c0, o8);
#pragma unroll
              for (int e = 0; e < 8; ++e) o8[e] *= fo;
              tmem_st8(tO + (uint32_t)c0, o8);
            }
          }
        }
        // weights x 2^7, as fp16 pairs over the S columns just read; a masked
        // tile takes every exponential on MUFU, which gives exactly 0 there
        unsigned long long sum2[4] = {0ull, 0ull, 0ull, 0ull};
        auto weights = [&](auto is_masked) {
          const unsigned long long seven = f2_pack(7.f, 7.f);
#pragma unroll
          for (int c0 = 0; c0 < 64; c0 += 16) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const int c2 = c0 + c;
              float x0, x1, e0, e1;
              f2_unpack(f2_add(f2_pack(x[2 * c2], x[2 * c2 + 1]), seven), x0, x1);
              if (!decltype(is_masked)::value && (c2 & 3) == 3) {
                exp2_fma2(x0, x1, e0, e1);  // one pair in four on the FMA pipe
              } else {
                e0 = ex2_approx(x0);
                e1 = ex2_approx(x1);
              }
              sum2[c2 & 3] = f2_add(sum2[c2 & 3], f2_pack(e0, e1));
              const __half2 hh = __floats2half2_rn(e0, e1);
              pk[c] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            tmem_st16_nowait(tS + (uint32_t)c0, pk);
          }
          tmem_wait_st();
        };
        if (masked) weights(std::true_type{});
        else weights(std::false_type{});
        float a0, a1, b0, b1, c0, c1, d0, d1;
        f2_unpack(sum2[0], a0, a1);
        f2_unpack(sum2[1], b0, b1);
        f2_unpack(sum2[2], c0, c1);
        f2_unpack(sum2[3], d0, d1);
        l += ((a0 + a1) + (b0 + b1)) + ((c0 + c1) + (d0 + d1));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[q]);
    }
    if (ok && live) {
      ok = mbar_wait_warp(&pv_done[q], (uint32_t)(T - 1) & 1u, abort_flag);
      if (ok) {
        tc_fence_after();
        // weights and l carry 2^7, V 2^10 / vref
        const float vref = sRef[(T - 1) & 3] * 0x1p-10f;
        const float f = p.P == 1 ? (l == 0.f ? 0.f : vref / l) : vref * 0x1p-7f;
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
            d[(e & 8) + jj + 4 * (e & 1)] = o16[e] * f;
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

// paged_tiles.cu -- attention of chunks of query rows over cached keys on the tensor cores.
//
// The sums of paged_rows.cu, for calls whose rows fill tensor-core tiles: row r of (sequence, key head) is token
// r / G, head r % G, and 256 such rows share one pass over their keys. One CTA an SM = (256 rows, split of the
// key tiles, key head, sequence); S = Q . K^T and O += P . V are tcgen05.mma (M = 128, two row halves) with S,
// P and O in TMEM; 128-key tiles of K and V lie in shared memory in two stages each.
//   warps 0-3, 4-7  load Q; softmax of row half 0, 1: thread r owns row r. Reads S from TMEM 32 columns at a
//                   time, writes the weights back over it, raises the running maximum only when a row's
//                   weights sum past a bound (O in TMEM is rescaled then), writes the output.
//   warp 8          issues the products: PV of a half, then that half's QK of the next key tile, so that one
//                   half's softmax runs under the other's products.
//   warp 9 (bf16)   brings the key tiles by TMA, a box a page (or 128 rows of a contiguous tensor);
//   warps 12-15     (INT8) bring the codes through registers, widened to bf16 (K) and f16 (V), exact.
//                   Value rows behind the sequence or before the window become zeros: P is zero there, but
//                   what unwritten memory holds need not be finite. (Key rows: their logits are masked.)
// The scales of INT8 keys and values enter in the softmax, x = S * (s_k scale log2 e), w = p * (s_v c): one
// vector of 128 of each a tile, with the power of two c (paged.cuh).
// Widened words hold four codes as pairs (0, 2), (1, 3): K keeps that order within every group of four d
// values and Q is stored to match; V's columns, and so O's, have it too and the output undoes it.
// Every wait is bounded as in attn_sm100.cu.
#include <climits>

#include "paged.cuh"

namespace bsva {
namespace {

template <bool I8>
constexpr int kTileThreads = I8 ? 512 : 384;
constexpr int KT = 128;                 // keys of a tile
constexpr int MS = 4;                   // stages of the scale vectors
constexpr uint32_t kTileTmem = 512;

template <int D>
struct __align__(1024) TileSmem {
  __nv_bfloat16 q[2][128 * D];          // K-major, D/64 panels of [128 rows x 64], 128-byte swizzle
  uint16_t k[2][KT * D];                // the same
  uint16_t v[2][KT * D];                // MN-major: D/64 panels of [128 keys x 64], 128-byte swizzle
  float fk[MS][KT];                     // INT8: s_k * scale * log2 e
  float sv[MS][KT];                     // INT8: s_v * c
  float rs[MS];                         // INT8: c of this tile / c of the last one
  float cn[MS];                         // INT8: c
  uint32_t red[2][4];
  long long rows[2][KT];                // INT8: cache row of each key of the tile whose loads come next, -1: none
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], v_raw, q_full, m_full[MS], r_full, s_full[2],
      p_full[2], pv_done[2];
  uint32_t tmem_base;
  int abort;
};

// D[tmem] (+)= A[smem] * B[smem]^T, bf16 in, fp32 accumulate.
__device__ __forceinline__ void mma_bf16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16-byte chunk c (8 values) of row `row` in a tile of [rows x D] 16-bit values, 64-value panels, swizzled.
template <int D>
__device__ __forceinline__ void* chunk_at(void* tile, int row, int c) {
  return static_cast<char*>(tile) + (c / 8) * (128 * 128) + row * 128 + (((c % 8) ^ (row & 7)) * 16);
}

template <int D, bool I8>
__global__ void __launch_bounds__(kTileThreads<I8>, 1)
    paged_tiles_kernel(const PagedArgs a, const __grid_constant__ PagedMaps maps) {
  extern __shared__ unsigned char smem_raw[];
  TileSmem<D>& sm = *reinterpret_cast<TileSmem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s = blockIdx.z, h = blockIdx.y;
  const int sp = blockIdx.x % a.nsplit;
  // the last rows of a causal chunk have the most keys: they start first
  const int rt = int(gridDim.x) / a.nsplit - 1 - int(blockIdx.x) / a.nsplit;

  const SeqView sv = seq_view(a, s);
  const int R = sv.n * a.G;
  const int rb = rt * 256;
  if (rb >= R) return;
  const int rows = min(256, R - rb);
  const int past = sv.kv - sv.n;
  const int i0 = rb / a.G, i1 = (rb + rows - 1) / a.G;
  const int hi_all = a.causal ? min(sv.kv, past + i1 + 1) : sv.kv;
  const int lo_all = a.window ? max(0, past + i0 - a.window + 1) : 0;
  int t0 = lo_all / KT, N = 0;
  if (hi_all > lo_all) {
    const int all = (hi_all + KT - 1) / KT - t0, per = (all + a.nsplit - 1) / a.nsplit;
    t0 += sp * per;
    N = max(0, min(per, all - sp * per));
  }
  const int nh = rows > 128 ? 2 : 1;

  // output element offset of this thread's row (softmax threads), -1 where there is none
  auto out_offset = [&](int rr) -> long long {
    if (rr >= R) return -1;
    return (long long)s * a.o_seq + (long long)(sv.q0 + rr / a.G) * a.o_tok + (long long)(h * a.G + rr % a.G) * a.o_head;
  };

  if (N == 0) {   // no key tile: out = 0, lse = -inf, or a split's empty part
    if (tid < 256) {
      const long long off = out_offset(rb + tid);
      if (off >= 0) {
        if (a.nsplit > 1) {
          a.part_ml[size_t(sp) * a.out_rows + off / D] = make_float2(-INFINITY, 0.f);
        } else {
          for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4*>(a.out + off)[c] = make_uint4(0, 0, 0, 0);
          if (a.lse) a.lse[off / D] = -INFINITY;
        }
      }
    }
    return;
  }

  constexpr uint32_t O_COL = 0, S_COL = 256;      // O halves at 0 and D, S (and P over it) at 256 and 384
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_full[i], I8 ? 4 : 1);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], I8 ? 4 : 1);
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 128);
      mbar_init(&sm.pv_done[i], 1);
    }
    for (int i = 0; i < MS; ++i) mbar_init(&sm.m_full[i], 4);
    mbar_init(&sm.r_full, 4);
    mbar_init(&sm.v_raw, 1);
    mbar_init(&sm.q_full, 8);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(&sm.tmem_base, kTileTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;
  const uint64_t lim = a.wait_limit_ns;
  auto wait = [&](uint64_t* bar, uint32_t par) {
    return __all_sync(0xffffffffu, mbar_wait(bar, par & 1, abort, a.status, lim)) != 0;
  };

  if (I8 && warp >= 12) {
    // ---------------------------------------------------------------------------- key tiles, INT8 codes
    const int lt = tid - 384;
    constexpr int CPR = D / 16, RP = 128 / CPR, NP = KT / RP;   // 16-byte chunks a row, rows a pass, passes
    const int c = lt % CPR, r0 = lt / CPR;
    auto arrive = [&](uint64_t* bar) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // the page table is read once a key (lt of the tile), a tile ahead of the loads that need it
    auto row_of = [&](int j) -> long long {
      const int key = (t0 + j) * KT + lt;
      return j < N && key >= lo_all && key < sv.kv ? (long long)kv_row(a, page_of(a, s, key), h, key) : -1;
    };
    uint4 kr[NP], vr[NP];
    auto load = [&](const void* base, uint4 (&x)[NP], int j) {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const long long row = sm.rows[j & 1][p * RP + r0];
        x[p] = row >= 0 ? __ldg(reinterpret_cast<const uint4*>(base) + row * CPR + c) : make_uint4(0, 0, 0, 0);
      }
    };
    float sk = 0.f, svv = 0.f;
    auto load_scales = [&](long long row) {
      sk = row >= 0 ? __ldg(a.k_scale + row) : 0.f;
      svv = row >= 0 ? __ldg(a.v_scale + row) : 0.f;
    };
    long long next = row_of(0);
    sm.rows[0][lt] = next;
    load_scales(next);
    next = row_of(1);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.r_full);
    bool ok = wait(&sm.r_full, 0);
    if (ok) {
      load(a.k, kr, 0);
      load(a.v, vr, 0);
    }
    float cn = 0.f;
    for (int j = 0; ok && j < N; ++j) {
      const int st = j & 1, ms = j % MS;
      // k_empty(j) = QK of tile j - 2 done, so the softmax of tile j - 3 is through: stage ms is free
      if (j >= 2 && !(ok = wait(&sm.k_empty[st], (j >> 1) - 1))) break;
      const uint32_t top_w = __reduce_max_sync(0xffffffffu, __float_as_uint(svv));
      sm.rows[st ^ 1][lt] = next;
      if (lane == 0) sm.red[st][warp - 12] = top_w;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.r_full);
      if (!(ok = wait(&sm.r_full, j + 1))) break;
      const float top = __uint_as_float(max(max(sm.red[st][0], sm.red[st][1]), max(sm.red[st][2], sm.red[st][3])));
      float rs = 1.f;
      if (top * cn >= kScaleGrow || (cn == 0.f && top > 0.f)) {
        const float n = scale_norm(top);
        if (cn != 0.f) rs = n / cn;
        cn = n;
      }
      sm.fk[ms][lt] = sk * a.scale_log2;
      sm.sv[ms][lt] = svv * cn;
      if (lt == 0) {
        sm.rs[ms] = rs;
        sm.cn[ms] = cn;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.m_full[ms]);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        uint32_t o[8];
        widen_bf16(kr[p].x, o[0], o[1]);
        widen_bf16(kr[p].y, o[2], o[3]);
        widen_bf16(kr[p].z, o[4], o[5]);
        widen_bf16(kr[p].w, o[6], o[7]);
        *static_cast<uint4*>(chunk_at<D>(sm.k[st], p * RP + r0, 2 * c)) = make_uint4(o[0], o[1], o[2], o[3]);
        *static_cast<uint4*>(chunk_at<D>(sm.k[st], p * RP + r0, 2 * c + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      arrive(&sm.k_full[st]);
      load(a.k, kr, j + 1);
      load_scales(next);
      next = row_of(j + 2);
      if (j >= 2 && !(ok = wait(&sm.v_empty[st], (j >> 1) - 1))) break;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        uint32_t o[8];
        widen_f16(vr[p].x, o[0], o[1]);
        widen_f16(vr[p].y, o[2], o[3]);
        widen_f16(vr[p].z, o[4], o[5]);
        widen_f16(vr[p].w, o[6], o[7]);
        *static_cast<uint4*>(chunk_at<D>(sm.v[st], p * RP + r0, 2 * c)) = make_uint4(o[0], o[1], o[2], o[3]);
        *static_cast<uint4*>(chunk_at<D>(sm.v[st], p * RP + r0, 2 * c + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      arrive(&sm.v_full[st]);
      load(a.v, vr, j + 1);
    }
  } else if (!I8 && warp == 9) {
    // --------------------------------------------------------------------------- key tiles, bf16 by TMA
    const int box = min(a.box_rows, KT), nb = KT / box;      // rows of a box, boxes of a panel of the tile
    const int sub = lane % nb, panel = lane / nb;
    auto issue = [&](const CUtensorMap* map, void* tile, int j, uint64_t* bar) {
      const int key = (t0 + j) * KT + sub * box;
      const bool in = panel < D / 64 && key + box > lo_all && key < sv.kv;
      const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, in));
      if (lane == 0) mbar_arrive_expect_tx(bar, boxes * box * 128);
      __syncwarp();
      if (in) {
        const int off = a.page_table ? key & ((1 << a.page_shift) - 1) : key;
        tma_load_3d(static_cast<char*>(tile) + panel * (128 * 128) + sub * box * 128, map, panel * 64, off,
                    page_of(a, s, key) * a.Hkv + h, bar);
      }
      __syncwarp();
    };
    if (lane == 0) {
      tma_prefetch_desc(&maps.k);
      tma_prefetch_desc(&maps.v);
    }
    int raw = 0;
    for (int j = 0; j < N; ++j) {
      const int st = j & 1, key0 = (t0 + j) * KT;
      const int v0 = max(lo_all - key0, 0), v1 = min(sv.kv - key0, KT);   // rows that some query row may see
      if (j >= 2 && !wait(&sm.k_empty[st], (j >> 1) - 1)) break;
      issue(&maps.k, sm.k[st], j, &sm.k_full[st]);
      if (j >= 2 && !wait(&sm.v_empty[st], (j >> 1) - 1)) break;
      if (v0 == 0 && v1 == KT) {
        issue(&maps.v, sm.v[st], j, &sm.v_full[st]);
      } else {                                   // the first tile of a window, the last one of the sequence
        issue(&maps.v, sm.v[st], j, &sm.v_raw);
        if (!wait(&sm.v_raw, raw++)) break;
        for (int x = lane; x < (v0 + KT - v1) * (D / 8); x += 32) {
          const int r = x / (D / 8);
          *static_cast<uint4*>(chunk_at<D>(sm.v[st], r < v0 ? r : v1 + r - v0, x % (D / 8))) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.v_full[st]);
      }
    }
  } else if (warp == 8) {
    // -------------------------------------------------------------------------------------- products
    constexpr uint32_t IDESC_QK = make_idesc(1, 1, 1, false, false, 128, KT);
    constexpr uint32_t kFmt = I8 ? 0u : 1u;
    constexpr uint32_t IDESC_PV = make_idesc(1, kFmt, kFmt, false, true, 128, D);
    constexpr uint32_t kPanel = (128 * 128) >> 4, kTile = (KT * D * 2) >> 4;
    const uint64_t dq0 = make_sdesc(smem_u32(sm.q[0]), 16, 1024, 2u);
    const uint64_t dk0 = make_sdesc(smem_u32(sm.k[0]), 16, 1024, 2u);
    const uint64_t dv0 = make_sdesc(smem_u32(sm.v[0]), 128 * 128, 1024, 2u);
    auto qk = [&](int hf, int j) {
      const uint64_t dq = dq0 + uint64_t(hf * kTile), dk = dk0 + uint64_t((j & 1) * kTile);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t at = (kk / 4) * kPanel + (kk % 4) * 2;
          mma_bf16_ss(tmem + S_COL + hf * KT, dq + at, dk + at, IDESC_QK, kk > 0 ? 1u : 0u);
        }
        tc_commit(&sm.s_full[hf]);
        if (hf == nh - 1) tc_commit(&sm.k_empty[j & 1]);
      }
      __syncwarp();
    };
    auto pv = [&](int hf, int j) {
      const uint64_t dv = dv0 + uint64_t((j & 1) * kTile);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk)
          mma_bf16_ts(tmem + O_COL + hf * D, tmem + S_COL + hf * KT + 8 * kk, dv + kk * ((16 * 128) >> 4), IDESC_PV,
                      (j > 0 || kk > 0) ? 1u : 0u);
        tc_commit(&sm.pv_done[hf]);
        if (hf == nh - 1) tc_commit(&sm.v_empty[j & 1]);
      }
      __syncwarp();
    };
    bool ok = wait(&sm.q_full, 0) && wait(&sm.k_full[0], 0);
    tc_fence_after();
    for (int hf = 0; ok && hf < nh; ++hf) qk(hf, 0);
    for (int j = 0; ok && j < N; ++j) {
      for (int hf = 0; ok && hf < nh; ++hf) {
        ok = wait(&sm.p_full[hf], j) && (hf > 0 || wait(&sm.v_full[j & 1], j >> 1));
        if (!ok) break;
        tc_fence_after();
        pv(hf, j);
        if (j + 1 < N) {
          if (hf == 0) {
            ok = wait(&sm.k_full[(j + 1) & 1], (j + 1) >> 1);
            tc_fence_after();
          }
          if (ok) qk(hf, j + 1);
        }
      }
    }
  } else if (warp < 8) {
    // Q rows, zeros behind the last one: 16-byte chunks, eight loads in flight
    {
      constexpr int CPR = D / 8, RP = 256 / CPR;
      const int c = tid % CPR, q0 = tid / CPR;
      for (int p0 = 0; p0 < nh * 128; p0 += 8 * RP) {
        uint4 w[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const int rr = rb + p0 + p * RP + q0;
          w[p] = make_uint4(0, 0, 0, 0);
          if (rr < R)
            w[p] = __ldg(reinterpret_cast<const uint4*>(a.q + (long long)s * a.q_seq +
                                                        (long long)(sv.q0 + rr / a.G) * a.q_tok +
                                                        (long long)(h * a.G + rr % a.G) * a.q_head) + c);
        }
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const int r = p0 + p * RP + q0;
          if constexpr (I8)
            w[p] = make_uint4(__byte_perm(w[p].x, w[p].y, 0x5410), __byte_perm(w[p].x, w[p].y, 0x7632),
                              __byte_perm(w[p].z, w[p].w, 0x5410), __byte_perm(w[p].z, w[p].w, 0x7632));
          *static_cast<uint4*>(chunk_at<D>(sm.q[r / 128], r % 128, c)) = w[p];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full);
    }
    if (warp / 4 < nh) {
    // --------------------------------------------------------------------------------------- softmax
    const int hf = warp / 4, r = tid & 127;
    const int rr = rb + hf * 128 + r;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + S_COL + hf * KT, tO = tmem + lanes + O_COL + hf * D;
    int lo = 0, hi = sv.kv - 1;                  // first and last key of the row (rows past the end: all)
    if (rr < R) {
      const int pos = past + rr / a.G;
      if (a.causal) hi = min(hi, pos);
      if (a.window) lo = max(0, pos - a.window + 1);
    }
    float m = -INFINITY, l = 0.f, cn = 1.f;
    bool alive = true;
    for (int j = 0; j < N; ++j) {
      const int key0 = (t0 + j) * KT, ms = j % MS;
      alive = wait(&sm.s_full[hf], j);
      if (I8 && alive) alive = wait(&sm.m_full[ms], j / MS);
      if (!alive) break;
      tc_fence_after();
      const int clo = max(lo - key0, 0), chi = min(hi - key0, KT - 1);   // columns the row sees
      const bool full = __all_sync(0xffffffffu, clo == 0 && chi == KT - 1);
      uint32_t pk[64];
      float ls = 0.f, f = 1.f;                   // f: factor of O so far
      if constexpr (I8) {
        f = sm.rs[ms];
        cn = sm.cn[ms];
      }
      // weights 2^(x - mu) of the tile, 32 columns at a time
      auto weights = [&](float mu) {
        float2 acc = make_float2(0.f, 0.f);
        const float2 nm = make_float2(-mu, -mu), sc = make_float2(a.scale_log2, a.scale_log2);
        // x f - m in one rounding is off the product that tile_max rounded by half a step of m: nothing below 2^20,
        // but past 2^24 whole octaves, so rows with such logits round the product first
        const bool far = __any_sync(0xffffffffu, fabsf(mu) >= 0x1p20f);
#pragma unroll
        for (int c0 = 0; c0 < KT; c0 += 32) {
          uint32_t x[32];
          tmem_ld32(tS + c0, x);
          tmem_wait_ld(x);
          float2 y[16];
          if (!far) {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              float2 fk = sc;
              if constexpr (I8) fk = *reinterpret_cast<const float2*>(&sm.fk[ms][c0 + 2 * c]);
              y[c] = __ffma2_rn(make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), fk, nm);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              float2 fk = sc;
              if constexpr (I8) fk = *reinterpret_cast<const float2*>(&sm.fk[ms][c0 + 2 * c]);
              y[c].x = __fadd_rn(__fmul_rn(__uint_as_float(x[2 * c]), fk.x), nm.x);
              y[c].y = __fadd_rn(__fmul_rn(__uint_as_float(x[2 * c + 1]), fk.y), nm.y);
            }
          }
          if (!full) {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              if (c0 + 2 * c < clo || c0 + 2 * c > chi) y[c].x = -INFINITY;
              if (c0 + 2 * c + 1 < clo || c0 + 2 * c + 1 > chi) y[c].y = -INFINITY;
            }
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float2 p = make_float2(ex2_approx(y[c].x), ex2_approx(y[c].y));
            acc = __fadd2_rn(acc, p);
            if constexpr (I8) {
              const float2 w = __fmul2_rn(p, *reinterpret_cast<const float2*>(&sm.sv[ms][c0 + 2 * c]));
              pk[c0 / 2 + c] = pack_f16x2(w.x, w.y);
            } else {
              pk[c0 / 2 + c] = pack_bf16x2(p.x, p.y);
            }
          }
        }
        ls = acc.x + acc.y;
      };
      auto tile_max = [&]() {
        float mx = -INFINITY;
#pragma unroll 1
        for (int c0 = 0; c0 < KT; c0 += 32) {
          uint32_t x[32];
          tmem_ld32(tS + c0, x);
          tmem_wait_ld(x);
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            float4 fk = make_float4(a.scale_log2, a.scale_log2, a.scale_log2, a.scale_log2);
            if constexpr (I8) fk = *reinterpret_cast<const float4*>(&sm.fk[ms][c0 + c]);
            float y[4] = {__fmul_rn(__uint_as_float(x[c]), fk.x), __fmul_rn(__uint_as_float(x[c + 1]), fk.y),
                          __fmul_rn(__uint_as_float(x[c + 2]), fk.z), __fmul_rn(__uint_as_float(x[c + 3]), fk.w)};
            if (!full) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (c0 + c + e < clo || c0 + c + e > chi) y[e] = -INFINITY;
            }
            mx = fmaxf(mx, fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])));
          }
        }
        return mx;
      };
      // The running maximum holds nearly always (a row whose weights sum to at most kFar has none above that): it is
      // looked at only where it does not, and the weights taken again. f16 weights bound kFar: 2^12 with the factor
      // kScaleGrow of s_v c stays below 2^15; bf16 weights have the range of fp32.
      constexpr float kFar = I8 ? 0x1p12f : 0x1p40f;
      bool redo = __any_sync(0xffffffffu, m == -INFINITY);
#pragma unroll 1
      while (true) {
        if (redo) {
          const float mx = tile_max();
          if (mx > m + 8.f) {
            const float al = m == -INFINITY ? 0.f : ex2_approx(m - mx);
            f *= al;
            l *= al;
            m = mx;
          }
        }
        weights(m == -INFINITY ? 0.f : m);
        if (redo || !__any_sync(0xffffffffu, !(ls <= kFar))) break;
        redo = true;
      }
      if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {
        if (!(alive = wait(&sm.pv_done[hf], j - 1))) break;
        tc_fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c0, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
          tmem_st32(tO + c0, o);
        }
      }
      l += ls;
      tmem_st32(tS, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
      tmem_st32(tS + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm.p_full[hf]);
    }
    // ----------------------------------------------------------------------------------------- output
    if (alive && wait(&sm.pv_done[hf], N - 1)) {
      tc_fence_after();
      const long long off = out_offset(rr);
      const float up = I8 && cn != 0.f ? 1.f / cn : 1.f;
      const float inv = a.nsplit > 1 ? up : l > 0.f ? up / l : 0.f;
      const size_t pr = size_t(sp) * a.out_rows + (off < 0 ? 0 : off / D);
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        tmem_ld32(tO + c0, o);
        tmem_wait_ld(o);
        if (off < 0) continue;
        float y[32];
#pragma unroll
        for (int c = 0; c < 32; ++c)             // INT8: columns 4g + 1 and 4g + 2 stand for each other's d value
          y[c] = __uint_as_float(o[I8 ? (c & ~3) | ((c & 1) << 1) | ((c >> 1) & 1) : c]) * inv;
        if (a.nsplit > 1) {
          float4* dst = reinterpret_cast<float4*>(a.part_o + pr * D + c0);
#pragma unroll
          for (int c = 0; c < 8; ++c) dst[c] = make_float4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(a.out + off + c0);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            dst[c] = make_uint4(pack_bf16x2(y[8 * c], y[8 * c + 1]), pack_bf16x2(y[8 * c + 2], y[8 * c + 3]),
                                pack_bf16x2(y[8 * c + 4], y[8 * c + 5]), pack_bf16x2(y[8 * c + 6], y[8 * c + 7]));
        }
      }
      if (off >= 0) {
        if (a.nsplit > 1) a.part_ml[pr] = make_float2(m, l);
        else if (a.lse) a.lse[off / D] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
      }
    }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTileTmem);
  }
}

template <int D, bool I8>
cudaError_t launch_tiles(const PagedArgs& a, const PagedMaps& maps, cudaStream_t st) {
  // one CTA an SM: its TMEM allocation is the whole of it
  const size_t need = sizeof(TileSmem<D>) + 1024, smem = need > 120 * 1024 ? need : 120 * 1024;
  cudaError_t e = cudaFuncSetAttribute(paged_tiles_kernel<D, I8>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.max_q * a.G;
  const dim3 grid(unsigned((rows + 255) / 256 * a.nsplit), a.Hkv, a.S);
  paged_tiles_kernel<D, I8><<<grid, kTileThreads<I8>, smem, st>>>(a, maps);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tiles(const PagedArgs& a, const PagedMaps& maps, bool int8, cudaStream_t st) {
  if (a.d == 128) return int8 ? launch_tiles<128, true>(a, maps, st) : launch_tiles<128, false>(a, maps, st);
  return int8 ? launch_tiles<64, true>(a, maps, st) : launch_tiles<64, false>(a, maps, st);
}

}  // namespace bsva

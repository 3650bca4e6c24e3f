// paged_tiles.cu -- attention of chunks of query rows over cached keys on the tensor cores.
//
// The sums of paged_rows.cu, for calls whose rows fill tensor-core tiles: row r of (sequence, key head) is token
// r / G, head r % G, and 256 such rows share one pass over their keys: an item = (256 rows, split of the key
// tiles, key head, sequence). S = Q . K^T and O += P . V are tcgen05.mma (M = 128, two row halves) with S, P and
// O in TMEM, all 512 columns of it, so one CTA an SM; 128-key tiles of K and V lie in shared memory in two stages
// each. A CTA takes items until none is left: the grid has a CTA an item, and a running CTA cancels the launch of
// a waiting one and does its work, so that keys, queries and S of the next item are on their way while this one's
// output is written.
//   warps 0-3, 4-7  softmax of row half 0, 1: thread r owns row r. Reads S from TMEM, 64 keys at a time, writes
//                   the weights back over it, raises the running maximum only when a row's weights sum past a
//                   bound (O in TMEM is rescaled then), writes the output.
//   warp 8          issues the products: PV of a half, 64 keys as soon as their weights are there, then that
//                   half's QK of the next key tile, so that one half's softmax runs under the other's products.
//   warp 9 (bf16)   brings the key tiles by TMA, a box a page (or 128 rows of a contiguous tensor);
//   warps 12-15     (INT8) bring the codes through registers, widened to bf16 (K) and f16 (V), exact.
//                   Value rows behind the sequence or before the window become zeros: P is zero there, but
//                   what unwritten memory holds need not be finite. (Key rows: their logits are masked.)
//   warps 9, 10 (INT8), 10 (bf16)  bring Q: by TMA where G divides 128 (a tile's rows are then whole tokens), by
//                   cp.async otherwise.
//   warp 11         finds the next item.
// The scales of INT8 keys enter in the softmax, x = S * (s_k scale log2 e), a vector of 128 a tile; those of the
// values in their f16 widening, v8 * (s_v c) with the power of two c (paged.cuh), which costs a value two roundings of
// 2^-11 at most, as the f16 weight has one. (Both scales as vectors of the softmax took 4000 cycles a half and tile
// where one takes 2600.)
// Widened words hold four codes as pairs (0, 2), (1, 3): K's bytes are put in order first; V's columns, and so
// O's, keep that order and the output undoes it.
// bf16 values take bf16 weights; O is divided by the sum of the rounded ones, so that the rounding of a key that
// outweighs the others cancels, and the log-sum-exp takes the sum of the unrounded ones (LSE). f16 weights round eight
// times finer and need neither.
// Measured, heads of 128 (floor: 4 flops a row, key and d value at 1634 TFLOP/s): 1536 new of 12288 tokens, 12 heads,
// bf16 pages 129 us, 140 with the log-sum-exp (floor 66); tensor and exponential pipes 48 % busy, issue slots 35 %: a
// half waits for its own chain, weights - product - next logits, which P over S leaves in a row. 32760 x 512 tokens,
// 40 heads, contiguous: 390 us after a pause, 434 back to back (floor 210), a quarter of it each item's output and start.
// 2048 of 32760 tokens, 40 query and 8 key heads, INT8 pages: 2100 us (floor 815); the loaders widen every key once an
// item, which takes shared memory (44 %) and issue slots (38 %) from the softmax. No pipe is full in any of the three:
// these are costs of this arrangement, not bounds of the operators.
// Every wait is bounded as in attn_sm100.cu.
#include "paged.cuh"

namespace bsva {
namespace {

template <bool I8>
constexpr int kTileThreads = I8 ? 512 : 384;
constexpr int KT = 128;                 // keys of a tile
constexpr int MS = 4;                   // stages of the scale vectors
constexpr uint32_t kTileTmem = 512;

// One item, as warp 11 leaves it for the others.
struct Item {
  int s, h, sp, rb;                     // sequence, key head, split, first row
  int R, kv, past, q0;                  // rows of (sequence, key head), keys, keys before the chunk, first token row
  int lo_all, hi_all;                   // first key that some row sees, one past the last
  int t0, N;                            // first key tile, key tiles
  int nh;                               // row halves in use; 0 = no more items
};

template <int D, bool I8>
struct __align__(1024) TileSmem {
  __nv_bfloat16 q[2][128 * D];          // K-major, D/64 panels of [128 rows x 64], 128-byte swizzle
  uint16_t k[2][KT * D];                // the same
  uint16_t v[2][KT * D];                // MN-major: D/64 panels of [128 keys x 64], 128-byte swizzle
  float fk[MS][KT];                     // INT8: s_k * scale * log2 e
  uint32_t sv[2][KT];                   // INT8: s_v * c as a pair of f16
  float rs[MS];                         // INT8: c of this tile / c of the last one
  float cn[MS];                         // INT8: c
  uint32_t red[2][4];
  int rows[2][KT];                      // INT8: cache row of each key of the tile whose loads come next, -1: none
  uint4 stage[8][32 * 4];               // a softmax warp's rows on their way out: 64 bytes of each of 32
  uint4 next_cta;                       // answer to the request for a waiting CTA
  Item item[2];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], v_raw, q_full[2], q_empty[2], m_full[MS], r_full, s_full[2],
      p_full[2][2], pv_done[2][2], item_full[2], item_empty[2], next_full, next_go;
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}

// Cluster launch control: ask for a CTA of this grid that has not started (16 bytes, with the barrier's
// transaction count), and read the answer: false, or the CTA's index, whose work is now the caller's.
__device__ __forceinline__ void ask_next_cta(uint4* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ bool next_cta(const uint4* answer, int& x, int& y, int& z) {
  uint32_t got;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 r, [%4];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, %3, _}, r;\n\t}"
      : "=r"(got), "=&r"(x), "=&r"(y), "=&r"(z)
      : "r"(smem_u32(answer))
      : "memory");
  return got != 0;
}

// Words hold four codes b0 .. b3, the results the pairs (b0, b2) and (b1, b3).
// bf16, with one multiply-add a pair: a code b xor 0x80 = b + 128 in the low byte of a bf16 is the subnormal
// (b + 128) 2^-133, which both the multiply-add and its exact product take as it is: times 2^127, - 2 = b / 64, exact.
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t& even, uint32_t& odd) {
  auto pair = [](uint32_t x) {
    uint32_t u = lop_and_xor(x, 0x00ff00ffu, 0x00800080u), r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(u), "r"(0x7f007f00u), "r"(0xc000c000u));
    return r;
  };
  even = pair(w);
  odd = pair(w >> 8);
}
// f16 times f (a pair of equal f16): the codes exactly (paged.cuh), then one rounding. (The subnormals above would do it
// in one multiply-add, but only up to 2^-1, where values 2^10 below the largest are subnormal themselves.)
__device__ __forceinline__ void values_f16(uint32_t w, uint32_t f, uint32_t& even, uint32_t& odd) {
  widen_f16(w, even, odd);
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(even) : "r"(f));
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(odd) : "r"(f));
}

// sum += both halves of a pair of bf16
__device__ __forceinline__ void add_bf16x2(float& sum, uint32_t w) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\t"
      "add.rn.f32.bf16 %0, a, %0;\n\tadd.rn.f32.bf16 %0, b, %0;\n\t}"
      : "+f"(sum)
      : "r"(w));
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// 16-byte chunk c (8 values) of row `row` in a tile of [rows x D] 16-bit values, 64-value panels, swizzled.
template <int D>
__device__ __forceinline__ void* chunk_at(void* tile, int row, int c) {
  return static_cast<char*>(tile) + (c / 8) * (128 * 128) + row * 128 + (((c % 8) ^ (row & 7)) * 16);
}

template <int D, bool I8, bool LSE>
__global__ void __launch_bounds__(kTileThreads<I8>, 1)
    paged_tiles_kernel(const PagedArgs a, const __grid_constant__ PagedMaps maps) {
  extern __shared__ unsigned char smem_raw[];
  using Smem = TileSmem<D, I8>;
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kQWarps = I8 ? 2 : 1, kLoadWarps = I8 ? 4 : 1;

  constexpr uint32_t O_COL = 0, S_COL = 256;      // O halves at 0 and D, S (and P over it) at 256 and 384
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_full[i], kLoadWarps);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], kLoadWarps);
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.q_full[i], kQWarps);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], 128);
      mbar_init(&sm.p_full[i][1], 128);
      mbar_init(&sm.pv_done[i][0], 1);
      mbar_init(&sm.pv_done[i][1], 1);
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], 9 + kQWarps + kLoadWarps);
    }
    for (int i = 0; i < MS; ++i) mbar_init(&sm.m_full[i], 4);
    mbar_init(&sm.r_full, kLoadWarps);
    mbar_init(&sm.v_raw, 1);
    mbar_init(&sm.next_full, 1);
    mbar_init(&sm.next_go, 1);
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
  // the same for warps that wait for most of the time: their polls would take issue slots from the others
  auto wait_idle = [&](uint64_t* bar, uint32_t par) {
    const uint64_t t0 = globaltimer_ns();
    while (!__all_sync(0xffffffffu, mbar_test_wait(bar, par & 1))) {
      __nanosleep(200);
      if (__any_sync(0xffffffffu, *abort != 0 || globaltimer_ns() - t0 > lim))
        return wait(bar, par);                   // which gives up the usual way
    }
    return true;
  };
  // item `no` for this warp: false when there are no more (or a wait ran out)
  auto take = [&](Item& it, uint32_t no, bool idle = false) -> bool {
    if (!(idle ? wait_idle(&sm.item_full[no & 1], no >> 1) : wait(&sm.item_full[no & 1], no >> 1))) return false;
    it = sm.item[no & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.item_empty[no & 1]);
    return it.nh > 0;
  };

  // Registers go to the softmax. INT8, 512 threads with 128 each: 2 x 168 + 64 + 112 = 4 x 128 for the four warpgroups
  // (2048 x 32760 tokens, us: 2100; 56 and 120 for the last two 2096; 2 x 176 + 56 + 104 2102; 2 x 160 + 72 + 120 2170).
  // bf16, 384 threads with 168 each: 2 x 184 + 136 = 2 x 192 + 120 = 3 x 168, with which nothing is spilled. (A fourth
  // warpgroup for the output leaves the others too few: 32760 x 512 tokens, 40 heads, 446 us for 393.)
  if (warp < 8) {
    regs_up<I8 ? 168 : LSE ? 192 : 184>();
    // --------------------------------------------------------------------------------------- softmax
    const int hf = warp / 4, r = tid & 127;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + S_COL + hf * KT, tO = tmem + lanes + O_COL + hf * D;
    // how far a row's weights may sum before its maximum is raised: f16 holds 2^15 (and a maximum that was looked
    // for leaves 64 weights of 2^8 at most), bf16 the range of fp32
    // (times kDown there; it bounds all that a row has summed, and one that is past it goes on 2^32 lower, so that no sum
    // comes near one. A bound of 2^24 makes more rows look: 12 heads, 1536 of 12288 tokens 143 us for 140.)
    constexpr float kFar = I8 ? 0x1p15f : 0x1p40f * kDown;
    Item it;
    uint32_t gt = 0, cnt = 0;                    // key tiles, key tiles of this half
    bool alive = true;
    for (uint32_t no = 0; alive && take(it, no); gt += it.N, ++no) {
      if (hf >= it.nh) continue;
      const int rr = it.rb + hf * 128 + r;
      long long off = -1;                        // output element of the row, -1 behind the last one
      int lo = 0, hi = it.kv - 1;                // first and last key of the row (rows past the end: all)
      if (rr < it.R) {
        const int i = rr / a.G, pos = it.past + i;
        off = (long long)it.s * a.o_seq + (long long)(it.q0 + i) * a.o_tok + (long long)(it.h * a.G + rr % a.G) * a.o_head;
        if (a.causal) hi = min(hi, pos);
        if (a.window) lo = max(0, pos - a.window + 1);
      }
      // Rows behind the sequence's last one hold what the next sequence's queries or the caller's padding give. They compute
      // along with a NaN as their maximum, which no comparison raises, and the votes on how a warp's rows are computed are
      // put so that a NaN never stops the others. (Columns they see: all, as a live row does that sees a sub-tile whole.)
      auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
      float m = off < 0 ? NAN : -INFINITY, l = 0.f, le = 0.f, cn = 1.f;   // l divides O, le is of the unrounded weights
      for (int j = 0; j < it.N; ++j) {
        const int ms = (gt + j) % MS;
        alive = wait(&sm.s_full[hf], cnt);
        if (I8 && alive) alive = wait(&sm.m_full[ms], (gt + j) / MS);
        if (!alive) break;
        tc_fence_after();
        float f = 1.f;                           // factor of O so far
        if constexpr (I8) {
          f = sm.rs[ms];
          cn = sm.cn[ms];
        }
        // O so far times f, once the products before sub-tile `sub` have landed
        auto rescale = [&](int sub) {
          if (j > 0 || sub > 0) {
            if (!wait(&sm.pv_done[hf][sub ^ 1], sub ? cnt : cnt - 1)) return false;
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
          f = 1.f;
          return true;
        };
        auto publish = [&](int sub) {
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&sm.p_full[hf][sub]);
        };
        // 64 columns of S at a time become weights over their own place. The quick way takes the running maximum as it
        // is, which holds nearly always: a row whose weights sum to at most kFar has no logit far above it. Where one
        // does not, the maximum is looked for and the weights are taken again. Columns that some row does not see whole,
        // and logits past 2^20, go the slow way.
        const float* fkp = sm.fk[ms];
        const int key0 = (it.t0 + j) * KT;
        const int clo = max(lo - key0, 0), chi = min(hi - key0, KT - 1);   // columns the row sees
        const bool whole = all(clo == 0 && chi == KT - 1);
        uint32_t xa[32], xb[32], pk[32];
        bool ahead = false;                      // xa holds the sub-tile's first 32 columns
#pragma unroll 1
        for (int sub = 0; sub < 2; ++sub) {
          const int col = 64 * sub;
          float ls = 0.f, es = 0.f;
          bool quick = whole || all(clo <= col && chi >= col + 63), done = false, late = sub > 0;   // late: the first half's weights are still to be published
          auto far = [&](float ls) { return (I8 ? ls : l + ls) > kFar; };
          auto raise = [&](float mx) {
            if (!I8 && l > kFar) mx = fmaxf(mx, m + 32.f);
            if (mx > m + 8.f) {
              const float al = m == -INFINITY ? 0.f : ex2_approx(m - mx);
              f *= al;
              l *= al;
              if constexpr (LSE) le *= al;
              m = mx;
            }
          };
          auto scaled_max = [&](const uint32_t (&x)[32], int c0, float mx) {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              float4 f4 = make_float4(a.scale_log2, a.scale_log2, a.scale_log2, a.scale_log2);
              if constexpr (I8) f4 = *reinterpret_cast<const float4*>(fkp + col + c0 + c);
              mx = fmaxf(mx, fmaxf(__fmul_rn(__uint_as_float(x[c]), f4.x), __fmul_rn(__uint_as_float(x[c + 1]), f4.y)));
              mx = fmaxf(mx, fmaxf(__fmul_rn(__uint_as_float(x[c + 2]), f4.z), __fmul_rn(__uint_as_float(x[c + 3]), f4.w)));
            }
            return mx;
          };
          if (quick) {
            if (!ahead) {
              tmem_ld32(tS + col, xa);
              tmem_wait_ld(xa);
            }
            // no key seen so far, l and O are zero: a first guess from 32 of the logits, the check covers the others
            if (__any_sync(0xffffffffu, m == -INFINITY)) {
              const float mx = scaled_max(xa, 0, -INFINITY);
              if (m == -INFINITY) m = mx;
            }
            quick = all(!(fabsf(m) >= 0x1p20f));
          }
          bool looked = false;
#pragma unroll 1
          while (quick) {
            const float mu = I8 ? m : m + kDownLog2;
            const float2 nm = make_float2(-mu, -mu), sc = make_float2(a.scale_log2, a.scale_log2);
            float2 acc = make_float2(0.f, 0.f);
            float ls1 = 0.f;
            ls = 0.f;
            auto quick32 = [&](const uint32_t (&x)[32], int c0) {   // c0 = 0 or 32
#pragma unroll
              for (int c = 0; c < 16; c += 2) {
                float2 f0 = sc, f1 = sc;
                if constexpr (I8) {
                  const float4 f4 = *reinterpret_cast<const float4*>(fkp + col + c0 + 2 * c);
                  f0 = make_float2(f4.x, f4.y);
                  f1 = make_float2(f4.z, f4.w);
                }
                const float2 y = __ffma2_rn(make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), f0, nm);
                const float2 z = __ffma2_rn(make_float2(__uint_as_float(x[2 * c + 2]), __uint_as_float(x[2 * c + 3])), f1, nm);
                const float2 p = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                const float2 q = make_float2(ex2_approx(z.x), ex2_approx(z.y));
                pk[c0 / 2 + c] = I8 ? pack_f16x2(p.x, p.y) : pack_bf16x2(p.x, p.y);
                pk[c0 / 2 + c + 1] = I8 ? pack_f16x2(q.x, q.y) : pack_bf16x2(q.x, q.y);
                if constexpr (!I8) {
                  add_bf16x2(ls, pk[c0 / 2 + c]);
                  add_bf16x2(ls1, pk[c0 / 2 + c + 1]);
                }
                if constexpr (I8 || LSE) acc = __fadd2_rn(acc, __fadd2_rn(p, q));
              }
            };
            tmem_ld32(tS + col + 32, xb);
            // INT8 has no registers to spare, and one that a load still fills must not be spilled: it waits at once
            if constexpr (I8) tmem_wait_ld(xb);
            quick32(xa, 0);
            if (late) publish(0);                // its stores landed under this work
            late = false;
            tmem_wait_ld(xb);
            tmem_ld32(tS + 64, xa);              // the second sub-tile's (in the second, of no use)
            if constexpr (I8) tmem_wait_ld(xa);
            quick32(xb, 32);
            es = acc.x + acc.y;
            ls = I8 ? es : ls + ls1;
            tmem_wait_ld(xa);
            done = looked || all(!far(ls));
            if (done) break;
            tmem_ld32(tS + col, xa);
            tmem_wait_ld(xa);
            raise(scaled_max(xa, 0, scaled_max(xb, 32, -INFINITY)));
            looked = true;
            quick = all(!(fabsf(m) >= 0x1p20f));
          }
          ahead = done;
          if (late) publish(0);
          if ((I8 || looked) && __any_sync(0xffffffffu, f != 1.f) && !(alive = rescale(sub))) break;
          if (!done && all(clo > col + 63 || chi < col)) {
#pragma unroll
            for (int c = 0; c < 32; ++c) pk[c] = 0;   // no row of the warp sees any of the 64 keys
          } else if (!done) {
            // scaled logits of 32 columns in xa, -inf where the row does not see. They are rounded before the maximum is
            // taken off (fused, those past 2^24 would come out above it by half their own step), so the largest is
            // exactly 0.
            auto masked = [&](int c0) {
              tmem_ld32(tS + col + c0, xa);
              tmem_wait_ld(xa);
              const int l0 = clo - col - c0, h0 = chi - col - c0;
              const uint32_t seen = (h0 > 30 ? ~0u : h0 < 0 ? 0u : (2u << h0) - 1u) & (l0 < 1 ? ~0u : l0 > 31 ? 0u : ~0u << l0);
#pragma unroll
              for (int c = 0; c < 32; c += 4) {
                float4 f4 = make_float4(a.scale_log2, a.scale_log2, a.scale_log2, a.scale_log2);
                if constexpr (I8) f4 = *reinterpret_cast<const float4*>(fkp + col + c0 + c);
                const float fs[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float y = __fmul_rn(__uint_as_float(xa[c + e]), fs[e]);
                  xa[c + e] = __float_as_uint(seen >> (c + e) & 1u ? y : -INFINITY);
                }
              }
            };
            looked = __any_sync(0xffffffffu, m == -INFINITY);
#pragma unroll 1
            while (true) {
              if (looked) {
                float mx = -INFINITY;
#pragma unroll 1
                for (int c0 = 0; c0 < 64; c0 += 32) {
                  masked(c0);
                  float top = -INFINITY;
#pragma unroll
                  for (int c = 0; c < 32; c += 2) top = fmaxf(top, fmaxf(__uint_as_float(xa[c]), __uint_as_float(xa[c + 1])));
                  mx = fmaxf(mx, top);
                }
                raise(mx);
                if (__any_sync(0xffffffffu, f != 1.f) && !(alive = rescale(sub))) break;
              }
              const float mu = m == -INFINITY ? 0.f : m;
              float2 acc = make_float2(0.f, 0.f);
              ls = 0.f;
              auto weigh = [&](int c0) {
                masked(c0);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                  float2 p = make_float2(ex2_approx(__fadd_rn(__uint_as_float(xa[2 * c]), -mu)),
                                         ex2_approx(__fadd_rn(__uint_as_float(xa[2 * c + 1]), -mu)));
                  // (a maximum of any size: 48 added to it could be rounded away)
                  if constexpr (!I8) p = make_float2(p.x * kDown, p.y * kDown);
                  acc = __fadd2_rn(acc, p);
                  pk[c0 / 2 + c] = I8 ? pack_f16x2(p.x, p.y) : pack_bf16x2(p.x, p.y);
                  if constexpr (!I8) add_bf16x2(ls, pk[c0 / 2 + c]);
                }
              };
              weigh(0);
              weigh(32);
              es = acc.x + acc.y;
              if constexpr (I8) ls = es;
              if (looked || all(!far(ls))) break;
              looked = true;
            }
            if (!alive) break;
          }
          tmem_st32(tS + col, pk);
          l += ls;
          if constexpr (LSE) le += es;
        }
        if (!alive) break;
        publish(1);
        ++cnt;
      }
      if (!alive) break;
      // --------------------------------------------------------------------------------------- output
      if (it.N > 0) {
        if (!(alive = wait(&sm.pv_done[hf][1], cnt - 1))) break;
        tc_fence_after();
      }
      // O over its sum and, INT8, over c: in two steps, since 1 / (l c) may leave the range of floats
      const float inv = over_sum(l);             // no keys: zeros; NaN stays NaN
      const float up = I8 && cn != 0.f ? 1.f / cn : 1.f;
      const size_t pr = size_t(it.sp) * a.out_rows + (off < 0 ? 0 : off / D);
      if (it.N > 0 || a.nsplit == 1) {           // a split without keys leaves its output part unwritten
        // A thread has a row, and rows lie far apart: 64 bytes of each row of the warp at a time go through shared
        // memory, so that a store instruction writes 8 rows of 64 bytes and not 32 of 16 (4700 cycles an item).
        uint4* stage = sm.stage[warp];
        char* dst[4];                            // rows lane / 4 + 8 i, this lane's 16 bytes
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const long long o = __shfl_sync(0xffffffffu, off, lane / 4 + 8 * i);
          char* p = a.nsplit > 1 ? reinterpret_cast<char*>(a.part_o + size_t(it.sp) * a.out_rows * D + o)
                                 : reinterpret_cast<char*>(a.out + o);
          dst[i] = o < 0 ? nullptr : p + (lane & 3) * 16;
        }
        auto put = [&](const uint4 (&w)[4], int byte) {
#pragma unroll
          for (int c = 0; c < 4; ++c) stage[lane * 4 + (c ^ ((lane >> 1) & 3))] = w[c];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r0 = lane / 4 + 8 * i;
            const uint4 x = stage[r0 * 4 + ((lane & 3) ^ ((r0 >> 1) & 3))];
            if (dst[i]) *reinterpret_cast<uint4*>(dst[i] + byte) = x;
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          if (it.N > 0) {
            tmem_ld32(tO + c0, o);
            tmem_wait_ld(o);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = 0;
          }
          float y[32];
#pragma unroll
          for (int c = 0; c < 32; ++c)           // INT8: columns 4g + 1 and 4g + 2 stand for each other's d value
            y[c] = __uint_as_float(o[I8 ? (c & ~3) | ((c & 1) << 1) | ((c >> 1) & 1) : c]) * inv * up;
          uint4 w[4];
          if (a.nsplit > 1) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                w[c] = make_uint4(__float_as_uint(y[16 * z + 4 * c]), __float_as_uint(y[16 * z + 4 * c + 1]),
                                  __float_as_uint(y[16 * z + 4 * c + 2]), __float_as_uint(y[16 * z + 4 * c + 3]));
              put(w, 4 * c0 + 64 * z);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              w[c] = make_uint4(pack_bf16x2(y[8 * c], y[8 * c + 1]), pack_bf16x2(y[8 * c + 2], y[8 * c + 3]),
                                pack_bf16x2(y[8 * c + 4], y[8 * c + 5]), pack_bf16x2(y[8 * c + 6], y[8 * c + 7]));
            put(w, 2 * c0);
          }
        }
      }
      if (off >= 0) {
        const float down = I8 ? kDown : 1.f;
        if (a.nsplit > 1) a.part_ml[pr] = make_float4(m, l * down, (LSE ? le : l) * down, 0.f);
        else if (a.lse) a.lse[off / D] = l == 0.f ? -INFINITY : (m + log2f((LSE ? le : l) * down * kUp)) * 0.69314718055994531f;
      }
      // the next item's first product writes O: order it after these reads (it waits for this half's weights)
      tc_fence_before();
    }
  } else if (warp >= 12) {
    if constexpr (I8) {
      regs_down<112>();
      // ---------------------------------------------------------------------------- key tiles, INT8 codes
      const int lt = tid - 384;
      constexpr int CPR = D / 16, RP = 128 / CPR, NP = KT / RP;   // 16-byte pieces a row, rows a pass, passes
      // Piece c of row r0 + a pass's. For rows of 128 bytes, eight lanes take four pieces of two rows, whose widened
      // chunks (2 c and 2 c + 1, exclusive-or the row) lie in eight different banks.
      const int c = D == 128 ? (lt & 3) | ((lt >> 1) & 4) : lt % CPR;
      const int r0 = D == 128 ? ((lt >> 2) & 1) | ((lt >> 4) << 1) : lt / CPR;
      static_assert(KT == 128, "a thread looks after key lt of the tile");
      char* const to0 = static_cast<char*>(chunk_at<D>(sm.k[0], r0, 2 * c));       // in the first stage of K
      char* const to1 = static_cast<char*>(chunk_at<D>(sm.k[0], r0, 2 * c + 1));
      constexpr int kStage = KT * D * 2, kPass = RP * 128;                         // RP is a multiple of 8 rows
      const int k_to_v = int(reinterpret_cast<char*>(sm.v[0]) - reinterpret_cast<char*>(sm.k[0]));
      auto arrive = [&](uint64_t* bar) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      Item it;
      uint32_t gt = 0, turn = 0;                 // key tiles and r_full phases so far
      bool ok = true;
      for (uint32_t no = 0; ok && take(it, no); ++no) {
        if (it.N == 0) {
          if (lt == 0) mbar_arrive(&sm.next_go);
          __syncwarp();
          continue;
        }
        // The page table is read once a key, two tiles ahead of the keys, and looked at a tile later: a look at once
        // would wait for it. -1: no key.
        auto key_of = [&](int j) { return (it.t0 + j) * KT + lt; };
        auto live = [&](int j) { return j < it.N && key_of(j) >= it.lo_all && key_of(j) < it.hi_all; };
        auto entry = [&](int j) { return live(j) ? page_entry(a, it.s, key_of(j)) : 0; };
        auto row_of = [&](int j, int e) -> int {   // fits: 2^31 rows would be 275 GB of codes
          return live(j) ? int(kv_row(a, checked_page(a, e), it.h, key_of(j))) : -1;
        };
        uint4 kr[NP], vr[NP];
        auto load = [&](const void* base, uint4 (&x)[NP], uint32_t slot) {
          const char* from = static_cast<const char*>(base) + 16 * c;
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const int row = sm.rows[slot & 1][p * RP + r0];
            x[p] = make_uint4(0, 0, 0, 0);
            if (row >= 0) x[p] = __ldg(reinterpret_cast<const uint4*>(from + (long long)row * D));
          }
        };
        float sk = 0.f, svv = 0.f;
        auto load_scales = [&](int row) {
          sk = svv = 0.f;
          if (row >= 0) {
            sk = __ldg(a.k_scale + row);
            svv = __ldg(a.v_scale + row);
          }
        };
        int ahead = entry(1);
        int next = row_of(0, entry(0));
        sm.rows[gt & 1][lt] = next;
        load_scales(next);
        next = row_of(1, ahead);
        ahead = entry(2);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.r_full);
        if (!(ok = wait(&sm.r_full, turn++))) break;
        load(a.k, kr, gt);
        load(a.v, vr, gt);
        float cn = 0.f;
        for (int j = 0; j < it.N; ++j, ++gt) {
          const int st = gt & 1, ms = gt % MS;
          if (lt == 0 && j == it.N - 1) mbar_arrive(&sm.next_go);
          // k_empty(gt) = QK of tile gt - 2 done, so the softmax of tile gt - 3 is through: stage ms is free
          if (gt >= 2 && !(ok = wait(&sm.k_empty[st], (gt >> 1) - 1))) break;
          const uint32_t top_w = __reduce_max_sync(0xffffffffu, __float_as_uint(svv));
          sm.rows[st ^ 1][lt] = next;
          if (lane == 0) sm.red[st][warp - 12] = top_w;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.r_full);
          if (!(ok = wait(&sm.r_full, turn++))) break;
          const float top = __uint_as_float(max(max(sm.red[st][0], sm.red[st][1]), max(sm.red[st][2], sm.red[st][3])));
          float rs = 1.f;
          if (top * cn >= kTilesFull || (cn == 0.f && top > 0.f)) {
            const float n = scale_norm<kTilesUp>(top);
            if (cn != 0.f) rs = n / cn;
            cn = n;
          }
          sm.fk[ms][lt] = sk * (64.f * a.scale_log2);                           // K enters as code / 64
          sm.sv[st][lt] = pack_f16x2(svv * cn, svv * cn);
          if (lt == 0) {
            sm.rs[ms] = rs;
            sm.cn[ms] = cn;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.m_full[ms]);
          const int at = st * kStage;
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            uint32_t o[8];
            codes_bf16(__byte_perm(kr[p].x, 0, 0x3120), o[0], o[1]);
            codes_bf16(__byte_perm(kr[p].y, 0, 0x3120), o[2], o[3]);
            codes_bf16(__byte_perm(kr[p].z, 0, 0x3120), o[4], o[5]);
            codes_bf16(__byte_perm(kr[p].w, 0, 0x3120), o[6], o[7]);
            *reinterpret_cast<uint4*>(to0 + at + p * kPass) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(to1 + at + p * kPass) = make_uint4(o[4], o[5], o[6], o[7]);
          }
          arrive(&sm.k_full[st]);
          if (j + 1 < it.N) load(a.k, kr, gt + 1);
          load_scales(next);
          next = row_of(j + 2, ahead);
          ahead = entry(j + 3);
          if (gt >= 2 && !(ok = wait(&sm.v_empty[st], (gt >> 1) - 1))) break;
          if (!(ok = wait(&sm.m_full[ms], gt / MS))) break;       // sv of the other warps
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            uint32_t o[8];
            const uint32_t f = sm.sv[st][p * RP + r0];
            values_f16(vr[p].x, f, o[0], o[1]);
            values_f16(vr[p].y, f, o[2], o[3]);
            values_f16(vr[p].z, f, o[4], o[5]);
            values_f16(vr[p].w, f, o[6], o[7]);
            *reinterpret_cast<uint4*>(to0 + k_to_v + at + p * kPass) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(to1 + k_to_v + at + p * kPass) = make_uint4(o[4], o[5], o[6], o[7]);
          }
          arrive(&sm.v_full[st]);
          if (j + 1 < it.N) load(a.v, vr, gt + 1);
        }
      }
    }
  } else {
    regs_down<I8 ? 64 : LSE ? 120 : 136>();
    if (warp == 11) {
      // ------------------------------------------------------------------------------------- next item
      int x = blockIdx.x, y = blockIdx.y, z = blockIdx.z;
      bool more = true;
      for (uint32_t no = 0, asked = 0;; ) {
        Item it{};
        if (more) {
          it.s = z;
          it.h = y;
          // the last rows of a causal chunk have the most keys: they start first
          it.sp = 0;
          it.rb = (int(gridDim.x) - 1 - x) * 256;
          if (a.nsplit > 1) {
            it.sp = x % a.nsplit;
            it.rb = (int(gridDim.x) / a.nsplit - 1 - x / a.nsplit) * 256;
          }
          const SeqView sv = seq_view(a, it.s);
          it.R = sv.n * a.G;
          it.kv = sv.kv;
          it.q0 = sv.q0;
          it.past = sv.kv - sv.n;
          const int rows = min(256, it.R - it.rb);
          if (rows > 0) {
            it.nh = rows > 128 ? 2 : 1;
            it.hi_all = a.causal ? min(sv.kv, it.past + (it.rb + rows - 1) / a.G + 1) : sv.kv;
            it.lo_all = a.window ? max(0, it.past + it.rb / a.G - a.window + 1) : 0;
            it.t0 = it.lo_all / KT;
            if (it.hi_all > it.lo_all) {
              it.N = (it.hi_all + KT - 1) / KT - it.t0;
              if (a.nsplit > 1) {
                const int per = (it.N + a.nsplit - 1) / a.nsplit;
                it.t0 += it.sp * per;
                it.N = max(0, min(per, it.N - it.sp * per));
              }
            }
          }
        }
        if (it.nh > 0 || !more) {
          if (no >= 2 && !wait_idle(&sm.item_empty[no & 1], (no >> 1) - 1)) break;
          if (lane == 0) {
            sm.item[no & 1] = it;
            mbar_arrive(&sm.item_full[no & 1]);
          }
          __syncwarp();
          if (!more) break;
          // the next one is asked for when this one's last key tile is: no sooner, so that none waits here while
          // another SM is idle
          if (!wait_idle(&sm.next_go, no)) break;
          ++no;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.next_full, 16);
          ask_next_cta(&sm.next_cta, &sm.next_full);
        }
        __syncwarp();
        if (!wait(&sm.next_full, asked++)) break;
        more = next_cta(&sm.next_cta, x, y, z);
        // every lane has read the answer before the next one may be written over it: a CTA without rows is followed by
        // the next request at once
        fence_proxy_async_smem();
        __syncwarp();
      }
    } else if (I8 ? warp == 9 || warp == 10 : warp == 10) {
      // --------------------------------------------------------------------------------------------- Q
      constexpr int CPR = D / 8, RP = 32 * kQWarps / CPR;
      const int qt = tid - (I8 ? 288 : 320), c = qt % CPR, r0 = qt / CPR;
      static_assert(RP == 2 || RP == 4 || RP == 8, "rows within a swizzle atom");
      const int dg = RP % a.G;                     // RP rows on: step elements, and wrap more where the heads begin anew
      const long long step = RP / a.G * a.q_tok + dg * a.q_head, wrap = a.q_tok - a.G * a.q_head;
      Item it;
      uint32_t used[2] = {0, 0};
      bool ok = true;
      for (uint32_t no = 0; ok && take(it, no, true); ++no) {
        if (it.N == 0) continue;
        auto ready = [&]() {                     // this warp's rows of the halves that were committed
          fence_proxy_async_smem();
          __syncwarp();
        };
        bool held = false;                       // half 0 is on its way and not reported yet
  #pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (hf >= it.nh || !ok) break;
          if (used[hf] > 0) {
            if (held && !__all_sync(0xffffffffu, mbar_test_wait(&sm.q_empty[hf], (used[hf] - 1) & 1))) {
              asm volatile("cp.async.wait_group 0;" ::: "memory");
              ready();
              if (lane == 0) mbar_arrive(&sm.q_full[0]);
              held = false;
            }
            if (!(ok = wait_idle(&sm.q_empty[hf], used[hf] - 1))) break;
          }
          ++used[hf];
          if (a.q_tma) {                         // a box of G heads and 128 / G tokens a panel, by the first of the warps
            if (lane == 0) {
              if (qt == 0) {
                mbar_arrive_expect_tx(&sm.q_full[hf], 128 * D * 2);
                for (int x = 0; x < D; x += 64)
                  tma_load_4d(sm.q[hf] + x * 128, &maps.q, x, it.h * a.G, it.q0 + (it.rb + hf * 128) / a.G,
                              a.q_start ? 0 : it.s, &sm.q_full[hf]);
              } else {
                mbar_arrive(&sm.q_full[hf]);
              }
            }
            __syncwarp();
            continue;
          }
          const int first = it.rb + hf * 128 + r0;
          int g = first % a.G;
          const __nv_bfloat16* from = a.q + (long long)it.s * a.q_seq + (long long)(it.q0 + first / a.G) * a.q_tok +
                                      (long long)(it.h * a.G + g) * a.q_head + c * 8;
          const uint32_t to = smem_u32(chunk_at<D>(sm.q[hf], r0, c));
  #pragma unroll 8
          for (int n = 0; n < 128 / RP; ++n) {     // row r0 + n RP of the half; zeros behind the last row
            const bool in = first + n * RP < it.R;
            cp_async16((to ^ (n * RP % 8 * 16)) + n * RP * 128, in ? from : a.q, in);
            from += step;
            g += dg;
            if (g >= a.G) {
              g -= a.G;
              from += wrap;
            }
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (hf == 0 && it.nh == 2) {             // half 1 follows before half 0 is waited for
            held = true;
            continue;
          }
          if (held) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            ready();
            if (lane == 0) mbar_arrive(&sm.q_full[0]);
          }
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          ready();
          if (lane == 0) mbar_arrive(&sm.q_full[hf]);
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");   // left over where a wait ran out
    } else if (!I8 && warp == 9) {
      // --------------------------------------------------------------------------- key tiles, bf16 by TMA
      const int box = a.box_rows, nb = KT / box;   // rows of a box, boxes of a panel of the tile
      const int sub = lane % nb, panel = lane / nb;
      if (lane == 0) {
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
      }
      Item it;
      uint32_t gt = 0, raw = 0;
      bool ok = true;
      for (uint32_t no = 0; ok && take(it, no); ++no) {
        auto issue = [&](const CUtensorMap* map, void* tile, int key0, uint64_t* bar) {
          const int key = key0 + sub * box;
          const bool in = panel < D / 64 && key + box > it.lo_all && key < it.kv;
          const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, in));
          if (lane == 0) mbar_arrive_expect_tx(bar, boxes * box * 128);
          __syncwarp();
          if (in) {
            const int off = a.page_table ? key & ((1 << a.page_shift) - 1) : key;
            tma_load_3d(static_cast<char*>(tile) + panel * (128 * 128) + sub * box * 128, map, panel * 64, off,
                        page_of(a, it.s, key) * a.Hkv + it.h, bar);
          }
          __syncwarp();
        };
        if (it.N == 0) {
          if (lane == 0) mbar_arrive(&sm.next_go);
          __syncwarp();
          continue;
        }
        for (int j = 0; j < it.N; ++j, ++gt) {
          const int st = gt & 1, key0 = (it.t0 + j) * KT;
          const int v0 = max(it.lo_all - key0, 0), v1 = min(it.kv - key0, KT);   // rows that some query row may see
          if (gt >= 2 && !(ok = wait(&sm.k_empty[st], (gt >> 1) - 1))) break;
          issue(&maps.k, sm.k[st], key0, &sm.k_full[st]);
          if (lane == 0 && j == it.N - 1) mbar_arrive(&sm.next_go);
          __syncwarp();
          if (gt >= 2 && !(ok = wait(&sm.v_empty[st], (gt >> 1) - 1))) break;
          if (v0 == 0 && v1 == KT) {
            issue(&maps.v, sm.v[st], key0, &sm.v_full[st]);
          } else {                                 // the first tile of a window, the last one of the sequence
            issue(&maps.v, sm.v[st], key0, &sm.v_raw);
            if (!(ok = wait(&sm.v_raw, raw++))) break;
            for (int x = lane; x < (v0 + KT - v1) * (D / 8); x += 32) {
              const int r = x / (D / 8);
              *static_cast<uint4*>(chunk_at<D>(sm.v[st], r < v0 ? r : v1 + r - v0, x % (D / 8))) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.v_full[st]);
          }
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
      Item it;
      uint32_t gt = 0, cnt[2] = {0, 0}, used[2] = {0, 0};   // key tiles; key tiles and items of each half
      bool ok = true;
      for (uint32_t no = 0; ok && take(it, no); ++no) {
        if (it.N == 0) continue;
        auto qk = [&](int hf, int j) {
          const uint64_t dq = dq0 + uint64_t(hf * kTile), dk = dk0 + uint64_t(((gt + j) & 1) * kTile);
          if (elect_one()) {
  #pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t at = (kk / 4) * kPanel + (kk % 4) * 2;
              mma_bf16_ss(tmem + S_COL + hf * KT, dq + at, dk + at, IDESC_QK, kk > 0 ? 1u : 0u);
            }
            tc_commit(&sm.s_full[hf]);
            if (hf == it.nh - 1) tc_commit(&sm.k_empty[(gt + j) & 1]);
            if (j == it.N - 1) tc_commit(&sm.q_empty[hf]);
          }
          __syncwarp();
        };
        auto pv = [&](int hf, int j, int sub) {    // 64 keys
          const uint64_t dv = dv0 + uint64_t(((gt + j) & 1) * kTile) + sub * ((64 * 128) >> 4);
          const uint32_t p = tmem + S_COL + hf * KT + 64 * sub;
          if (elect_one()) {
  #pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ts(tmem + O_COL + hf * D, p + 8 * kk, dv + kk * ((16 * 128) >> 4), IDESC_PV,
                          (j > 0 || sub > 0 || kk > 0) ? 1u : 0u);
            tc_commit(&sm.pv_done[hf][sub]);
            if (sub == 1 && hf == it.nh - 1) tc_commit(&sm.v_empty[(gt + j) & 1]);
          }
          __syncwarp();
        };
        ok = wait(&sm.k_full[gt & 1], gt >> 1);
        for (int hf = 0; ok && hf < it.nh; ++hf) {
          if (!(ok = wait(&sm.q_full[hf], used[hf]++))) break;
          tc_fence_after();
          qk(hf, 0);
        }
        for (int j = 0; ok && j < it.N; ++j) {
          for (int hf = 0; ok && hf < it.nh; ++hf) {
            if (hf == 0 && !(ok = wait(&sm.v_full[(gt + j) & 1], (gt + j) >> 1))) break;
            for (int sub = 0; ok && sub < 2; ++sub) {
              ok = wait(&sm.p_full[hf][sub], cnt[hf]);
              tc_fence_after();
              if (ok) pv(hf, j, sub);
            }
            ++cnt[hf];
            if (ok && j + 1 < it.N) {
              if (hf == 0) {
                ok = wait(&sm.k_full[(gt + j + 1) & 1], (gt + j + 1) >> 1);
                tc_fence_after();
              }
              if (ok) qk(hf, j + 1);
            }
          }
        }
        gt += it.N;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    // after a wait that ran out, copies and products may still be on their way into this CTA's memory: 100 us for them
    if (*abort)
      for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 100000;) __nanosleep(1000);
    tc_fence_after();
    tmem_dealloc(tmem, kTileTmem);
  }
}

template <int D, bool I8, bool LSE>
cudaError_t launch_tiles(const PagedArgs& a, const PagedMaps& maps, cudaStream_t st) {
  // one CTA an SM: its TMEM allocation is the whole of it
  const size_t need = sizeof(TileSmem<D, I8>) + 1024, smem = need > 120 * 1024 ? need : 120 * 1024;
  cudaError_t e =
      cudaFuncSetAttribute(paged_tiles_kernel<D, I8, LSE>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.max_q * a.G;
  const dim3 grid(unsigned((rows + 255) / 256 * a.nsplit), a.Hkv, a.S);
  paged_tiles_kernel<D, I8, LSE><<<grid, kTileThreads<I8>, smem, st>>>(a, maps);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tiles(const PagedArgs& a, const PagedMaps& maps, bool int8, cudaStream_t st) {
  // INT8 sums the unrounded weights in any case
  if (int8) return a.d == 128 ? launch_tiles<128, true, false>(a, maps, st) : launch_tiles<64, true, false>(a, maps, st);
  if (a.lse) return a.d == 128 ? launch_tiles<128, false, true>(a, maps, st) : launch_tiles<64, false, true>(a, maps, st);
  return a.d == 128 ? launch_tiles<128, false, false>(a, maps, st) : launch_tiles<64, false, false>(a, maps, st);
}

}  // namespace bsva

// paged_rows.cu -- attention of few query rows (single tokens, short chunks) over cached keys, split over
// the keys, and the kernel that joins the splits.
//
// o_i = sum_t p_it v_t / sum_t p_it, p_it = 2^(x_it - m_i), x_it = scale * log2(e) * (q_i . k_t), over the
// keys t that row i may see (t <= pos_i when causal, t > pos_i - window); m_i the running maximum.
//
// The query heads of one key head share its keys: row r of (sequence, key head) is token r / G, head
// r % G. One CTA = (row tile of 8 * NT rows, split of the keys, key head, sequence); its four warps take
// 16-key blocks in turn, each with its own running maximum, sum and output, and join at the end. The splits of a row
// tile are then joined by their cluster or by a second kernel.
// Such calls are bound by reading the codes (an INT8 key head's token is 2 d + 8 bytes for 4 d flops a
// row), and what bounds the reading is how many bytes are on their way: each warp keeps a ring of 16-key
// blocks of its own in shared memory, filled by cp.async two or three blocks ahead with no registers held
// and no barrier but the warp's, and both products have the keys' data on the 16-row side, so that 8 rows
// waste nothing:
//   S^T [16 keys x 8 rows] += K [16 x 16] . Q^T [16 x 8]        (f16 for INT8 codes, widened exactly; bf16)
//   O^T [16 d   x 8 rows] += V^T [16 x 16 keys] . P^T [16 x 8]  (f16 for INT8 codes, bf16 for bf16 values)
// A product's inner index may run in any order that both operands share, and so may the d index of O:
//   lane (g = lane / 4, t = lane % 4) reads 16-byte pieces of K's tile rows g and g + 8 and takes four
//   consecutive d values a step; of V it reads 1/8 of the d values of tile rows 2t, 2t+1, 2t+8, 2t+9.
// Tile row g is key g or, odd, key g ^ 4, and pieces of a row are stored exclusive-or its number: eight
// lanes that read together then meet eight different banks, for K and for V.
// Measured, one token of each sequence, heads of 128 (a copy moves 6.54 TB/s): 64 sequences of 8192 keys, 8 key heads,
// bf16 pages 323 us (6.66 TB/s), INT8 pages 196 (5.66; issue slots 56 % taken by widening and the softmax, MUFU 5 %);
// 2 of 131000 keys, 40 key heads, INT8 458 (6.0; with the codes through registers instead of the rings 537).

#include <climits>

#include "paged.cuh"

namespace bsva {
namespace {

constexpr int kRowThreads = 128;
constexpr float kLazy = 8.f;   // the running maximum is raised when some logit passes it by 2^8

template <bool F16>
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit values across the warp: lane (g, t) gives row g, columns 2t, 2t+1.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool in) {   // zeros where !in
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0)
                 : "memory");
}

// A warp's ring: blocks of 16 keys, K, V and (INT8) the scales.
template <int D, bool I8>
constexpr int kStageBytes = 32 * D * (I8 ? 1 : 2) + (I8 ? 128 : 0);
template <int D, bool I8>
constexpr int kStages = D == 128 && !I8 ? 3 : 4;
template <int D, bool I8, int NT>
constexpr int kRowSmem() {
  constexpr int ring = 4 * kStages<D, I8> * kStageBytes<D, I8>, join = 4 * 8 * NT * (D + 4) * 4;
  return ring > join ? ring : join;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Where a variable of this CTA's shared memory lies in that of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(const void* p, int rank) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_u32(p)), "r"(rank));
  return d;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

template <int D, bool I8, int NT>
__global__ void __launch_bounds__(kRowThreads) paged_rows_kernel(const PagedArgs a) {
  constexpr int KS = D / 16;              // steps of 16 d values in q . k
  constexpr int EB = I8 ? 1 : 2;          // bytes of a cached value
  constexpr int KL = D * EB / 64;         // 16-byte loads of a lane from one key row
  constexpr int VB = D / 8 * EB;          // bytes of a lane's d values of one V row (8, 16 or 32)
  constexpr int VW = VB / 4;              // ... in words
  constexpr int MT = D / 16;              // 16-row tiles of O^T
  const int s = blockIdx.z, h = blockIdx.y;
  const int rt = blockIdx.x / a.nsplit, sp = blockIdx.x % a.nsplit;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  const SeqView sv = seq_view(a, s);
  const int R = sv.n * a.G;               // rows of this (sequence, key head)
  const int rb = rt * 8 * NT;             // first row of the tile
  if (rb >= R) return;
  const int i0 = rb / a.G, i1 = (min(rb + 8 * NT, R) - 1) / a.G;   // tokens of the tile's rows
  // keys that some row of the tile sees, and this split's part of them (from a multiple of 16)
  const int past = sv.kv - sv.n;
  const int hi_all = a.causal ? min(sv.kv, past + i1 + 1) : sv.kv;
  const int lo_see = a.window ? max(0, past + i0 - a.window + 1) : 0, lo_all = lo_see & ~15;
  // (a cluster shares what there is: its CTAs wait for one another at the end)
  const int per = a.cluster ? ((max(hi_all - lo_all, 0) + a.nsplit - 1) / a.nsplit + 63) & ~63 : a.split_keys;
  const int lo = min((long long)lo_all + (long long)sp * per, (long long)INT_MAX - 64);
  const int hi = min((long long)hi_all, (long long)lo + per);

  // this lane's rows as columns of the products: 8 nt + 2t and + 1; what each sees
  int see_lo[NT][2], see_hi[NT][2];       // first and last key
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = min(rb + 8 * nt + 2 * t + e, R - 1);
      const int pos = past + r / a.G;
      see_hi[nt][e] = a.causal ? min(pos, sv.kv - 1) : sv.kv - 1;
      see_lo[nt][e] = a.window ? max(0, pos - a.window + 1) : 0;
    }
  // blocks in [full_lo, full_hi) need no mask: every row of the tile sees all of them
  const int full_lo = a.window ? max(0, past + i1 - a.window + 1) : 0;
  const int full_hi = a.causal ? min(sv.kv, past + i0 + 1) : sv.kv;

  float m[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
  }
  float cn = 0.f;                         // INT8: the scales' power of two (0: not set yet)

  extern __shared__ __align__(128) unsigned char smem_rows[];
  constexpr int RB = D * EB, CPR = RB / 16;             // bytes and 16-byte pieces of a cached row
  constexpr int STAGE = kStageBytes<D, I8>, NS = kStages<D, I8>;
  unsigned char* ring = smem_rows + warp * (NS * STAGE);
  // piece c of row r of a block, within a stage's K or V
  auto piece = [](int r, int c) { return r * RB + (CPR == 4 ? c ^ ((r >> 1) & 3) : c ^ (r & 7)) * 16; };
  const int kg = g & 1 ? g ^ 4 : g;       // key of tile row g
  const char* kbase = static_cast<const char*>(a.k);
  const char* vbase = static_cast<const char*>(a.v);
  // Block at `key` into stage st; rows that no row of the tile sees become zeros: what unwritten memory holds must
  // not reach O. Rows of a block lie in one page (pages hold a multiple of 16 tokens), found a block ahead.
  int page = 0;
  auto find = [&](int key) { page = key < hi ? page_of(a, s, key) : 0; };
  // where this lane's pieces go: x = lane + 32 i is row x / CPR, piece x % CPR; a step of i moves 32 / CPR rows, and the
  // swizzle repeats every 8 rows
  constexpr int NI = CPR / 2, RI = 32 / CPR, PER = RI >= 8 ? 1 : 8 / RI;
  uint32_t to[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) to[i] = smem_u32(ring) + piece(lane / CPR + i * RI, lane % CPR);
  const uint32_t to_scale = smem_u32(ring) + 32 * RB + lane * 4;
  const float* scales = I8 ? (lane < 16 ? a.k_scale : a.v_scale) + (lane & 15) : nullptr;
  auto issue = [&](int st, int key) {
    if (key < hi) {
      const size_t row = kv_row(a, page, h, key);
      const bool whole = key >= lo_see && key + 16 <= hi;
      const char* kp = kbase + row * RB + lane * 16;
      const char* vp = vbase + row * RB + lane * 16;
      if (whole) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const uint32_t d = to[i % PER] + st * STAGE + (i / PER) * (PER * RI * RB);
          cp_async<16>(d, kp + i * 512, true);
          cp_async<16>(d + 16 * RB, vp + i * 512, true);
        }
        if constexpr (I8) cp_async<4>(to_scale + st * STAGE, scales + row, true);
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int r = key + lane / CPR + i * RI;
          const bool in = r < hi && r >= lo_see;
          const uint32_t d = to[i % PER] + st * STAGE + (i / PER) * (PER * RI * RB);
          cp_async<16>(d, in ? kp + i * 512 : kbase, in);
          cp_async<16>(d + 16 * RB, in ? vp + i * 512 : vbase, in);
        }
        if constexpr (I8) {               // 16 scales of K, 16 of V
          const int r = key + (lane & 15);
          const bool in = r < hi && r >= lo_see;
          cp_async<4>(to_scale + st * STAGE, in ? scales + row : a.k_scale, in);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  constexpr int STEP = 16 * (kRowThreads / 32);
  int key = lo + 16 * warp;
  find(key);
#pragma unroll
  for (int st = 0; st < NS - 1; ++st) {
    issue(st, key + st * STEP);
    find(key + (st + 1) * STEP);
  }
  // q as the B operand: lane (g, t) holds row 8 nt + g, the d values its key pieces have. With INT8 codes it enters as
  // f16, whose codes widen in fewer instructions than bf16's: a row times 2^-x with its largest value in [2^14, 2^15).
  // That is exact but for values below 2^-29 of the row's largest, which lose at most 2^-39 of it. qf: 2^x times
  // the softmax scale, of the rows that are this lane's columns.
  uint32_t bq[NT][KS][2];
  float qf[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = rb + 8 * nt + g;
    const bool have = r < R;
    const __nv_bfloat16* qp = a.q + (long long)s * a.q_seq + (long long)(sv.q0 + (have ? r / a.G : 0)) * a.q_tok +
                              (long long)(h * a.G + (have ? r % a.G : 0)) * a.q_head;
    float top = 0.f;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      // four consecutive d values: INT8 pieces hold 16 of them, bf16 pieces 8
      const int d0 = I8 ? (kk / 4) * 64 + 16 * t + 4 * (kk % 4) : (kk / 2) * 32 + 8 * t + 4 * (kk % 2);
      const uint2 w = have ? __ldg(reinterpret_cast<const uint2*>(qp + d0)) : make_uint2(0, 0);
      bq[nt][kk][0] = I8 ? __byte_perm(w.x, w.y, 0x5410) : w.x;   // INT8: (d0, d0+2), (d0+1, d0+3)
      bq[nt][kk][1] = I8 ? __byte_perm(w.x, w.y, 0x7632) : w.y;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(bq[nt][kk][e] << 16)),
                               fabsf(__uint_as_float(bq[nt][kk][e] & 0xffff0000u))));
    }
    if constexpr (I8) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int x = min(max(int(__float_as_uint(top) >> 23), 15), 254) - 14;      // biased exponent of 2^x
      const float down = __uint_as_float(uint32_t(254 - x) << 23), up = __uint_as_float(uint32_t(x) << 23);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          bq[nt][kk][e] = pack_f16x2(__uint_as_float(bq[nt][kk][e] << 16) * down,
                                     __uint_as_float(bq[nt][kk][e] & 0xffff0000u) * down);
#pragma unroll
      for (int e = 0; e < 2; ++e) qf[nt][e] = __shfl_sync(0xffffffffu, up, (2 * t + e) * 4) * a.scale_log2;
    }
  }

  for (int st = 0; key < hi; key += STEP, st = st + 1 == NS ? 0 : st + 1) {
    asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
    __syncwarp();                         // every lane's part of this block is in, and the last block is done with
    issue(st == 0 ? NS - 1 : st - 1, key + (NS - 1) * STEP);
    find(key + NS * STEP);
    const unsigned char* stage = ring + st * STAGE;
    uint4 kr[2][KL];
    float ks[2], vs[2];                   // INT8: scales of a key and of its values
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int c = 0; c < KL; ++c) kr[e][c] = *reinterpret_cast<const uint4*>(stage + piece(kg + 8 * e, t + 4 * c));
      if constexpr (I8) {
        ks[e] = reinterpret_cast<const float*>(stage + 32 * RB)[kg + 8 * e];
        vs[e] = reinterpret_cast<const float*>(stage + 32 * RB)[16 + kg + 8 * e];
      }
    }
    // ---- logits of 16 keys, in log2 units: lane holds keys g (e = 0, 1) and g + 8 (e = 2, 3)
    float x[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[nt][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      uint32_t a0, a1, a2, a3;
      if constexpr (I8) {
        const uint32_t* w0 = &kr[0][kk / 4].x + kk % 4;
        const uint32_t* w1 = &kr[1][kk / 4].x + kk % 4;
        widen_f16(*w0, a0, a2);
        widen_f16(*w1, a1, a3);
      } else {
        const uint32_t* w0 = &kr[0][kk / 2].x + 2 * (kk % 2);
        const uint32_t* w1 = &kr[1][kk / 2].x + 2 * (kk % 2);
        a0 = w0[0]; a2 = w0[1];
        a1 = w1[0]; a3 = w1[1];
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_16x8x16<I8>(x[nt], a0, a1, a2, a3, bq[nt][kk][0], bq[nt][kk][1]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // rounded here, not fused with the subtraction of the maximum, which was taken from rounded logits; the query's factor
      // meets the key's first, since codes times a large query may leave fp32 where the logit does not
#pragma unroll
      for (int e = 0; e < 4; ++e) x[nt][e] = __fmul_rn(x[nt][e], I8 ? ks[e >> 1] * qf[nt][e & 1] : a.scale_log2);
    }
    if (key < full_lo || key + 16 > min(full_hi, hi)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int kk = key + kg + 8 * (e >> 1);
          if (kk >= hi || kk < see_lo[nt][e & 1] || kk > see_hi[nt][e & 1]) x[nt][e] = -INFINITY;
        }
    }
    // ---- raise the running maximum where a logit passes it by 2^8 (always at the first block)
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) over = over || fmaxf(x[nt][e], x[nt][e + 2]) > m[nt][e] + kLazy;
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float al[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(x[nt][e], x[nt][e + 2]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
          const float mn = fmaxf(m[nt][e], mx);
          al[e] = mn == -INFINITY ? 1.f : ex2_approx(m[nt][e] - mn);
          m[nt][e] = mn;
          l[nt][e] *= al[e];
        }
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][j][e] *= al[e & 1];
      }
    }
    float c0 = 1.f, c1 = 1.f;             // INT8: weight of a key's codes, s_v * cn
    if constexpr (I8) {
      const float mine = fmaxf(vs[0], vs[1]);
      if (__any_sync(0xffffffffu, mine * cn >= kRowsFull || (cn == 0.f && mine > 0.f))) {
        const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mine)));
        const float c = scale_norm<kRowsUp>(top), f = cn == 0.f ? 1.f : c / cn;
        cn = c;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][j][e] *= f;
      }
      c0 = vs[0] * cn;
      c1 = vs[1] * cn;
    }
    // ---- weights, transposed into the B operand of the second product
    // (bf16 values: the weights enter as two bf16 terms, since one would add as much error as the output's rounding)
    uint32_t bp[NT][2], bl[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float mu = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
        p[e] = ex2_approx(x[nt][e] - mu);
        if constexpr (!I8) p[e] *= kDown;
        l[nt][e & 1] += p[e];
      }
      if constexpr (I8) {
        bp[nt][0] = transpose_8x8(pack_f16x2(p[0] * c0, p[1] * c0));
        bp[nt][1] = transpose_8x8(pack_f16x2(p[2] * c1, p[3] * c1));
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w = pack_bf16x2(p[2 * e], p[2 * e + 1]);
          bp[nt][e] = transpose_8x8(w);
          bl[nt][e] = transpose_8x8(pack_bf16x2(p[2 * e] - __uint_as_float(w << 16),
                                                p[2 * e + 1] - __uint_as_float(w & 0xffff0000u)));
        }
      }
    }
    // ---- O^T: word w of the lane's V pieces gives d values in pairs, tile rows (2t, 2t+1) and (2t+8, 2t+9)
    uint32_t vr[4][VW];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = (e & 1 ? (2 * t + 1) ^ 4 : 2 * t) + 8 * (e >> 1);
      const unsigned char* vst = stage + 16 * RB;
      if constexpr (VB == 8) {
        const uint2 x = *reinterpret_cast<const uint2*>(vst + piece(r, g >> 1) + (g & 1) * 8);
        vr[e][0] = x.x; vr[e][1] = x.y;
      } else {
#pragma unroll
        for (int c = 0; c < VB / 16; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(vst + piece(r, g + 8 * c));
          vr[e][4 * c] = x.x; vr[e][4 * c + 1] = x.y; vr[e][4 * c + 2] = x.z; vr[e][4 * c + 3] = x.w;
        }
      }
    }
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      const uint32_t a_lo = __byte_perm(vr[0][w], vr[1][w], 0x5410), a_hi = __byte_perm(vr[0][w], vr[1][w], 0x7632);
      const uint32_t b_lo = __byte_perm(vr[2][w], vr[3][w], 0x5410), b_hi = __byte_perm(vr[2][w], vr[3][w], 0x7632);
      if constexpr (I8) {                 // d values 4w .. 4w+3: two tiles
        uint32_t a0, a1, a2, a3;
        widen_f16(a_lo, a0, a1);
        widen_f16(b_lo, a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16x8x16<true>(o[nt][2 * w], a0, a1, a2, a3, bp[nt][0], bp[nt][1]);
        widen_f16(a_hi, a0, a1);
        widen_f16(b_hi, a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16x8x16<true>(o[nt][2 * w + 1], a0, a1, a2, a3, bp[nt][0], bp[nt][1]);
      } else {                            // d values 2w, 2w+1: one tile
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16x8x16<false>(o[nt][w], a_lo, a_hi, b_lo, b_hi, bp[nt][0], bp[nt][1]);
          mma_16x8x16<false>(o[nt][w], a_lo, a_hi, b_lo, b_hi, bl[nt][0], bl[nt][1]);
        }
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");

  // ---- join the four warps: each leaves its maximum, sum and output (over the sum and cn) in shared memory
  constexpr int W = kRowThreads / 32, NR = 8 * NT;
  __shared__ float s_m[W][NR], s_l[W][NR];
  __shared__ float2 s_ml[NR];             // of the CTA, for its cluster
  float (*s_o)[NR][D + 4] = reinterpret_cast<float (*)[NR][D + 4]>(smem_rows);   // over the rings, which are through
  __syncthreads();
  const float inv_c = I8 && cn != 0.f ? 1.f / cn : 1.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float ls = l[nt][e];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, d);
      const int r = 8 * nt + 2 * t + e;
      const float inv = over_sum(ls);
      if (g == 0) {
        s_m[warp][r] = m[nt][e];
        s_l[warp][r] = I8 ? ls * kDown : ls;
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        // lane's d values: of each of its pieces, 16 bytes of codes or values, 8 for INT8 rows of 64
        constexpr int PV = VB < 16 ? VB : 16 / EB;
        const int d0 = (2 * j / PV) * 8 * PV + g * PV + 2 * j % PV;
        s_o[warp][r][d0] = o[nt][j][e] * inv * inv_c;
        s_o[warp][r][d0 + 1] = o[nt][j][e + 2] * inv * inv_c;
      }
    }
  __syncthreads();
  for (int x = threadIdx.x; x < NR * (D / 4); x += kRowThreads) {
    const int r = x / (D / 4), c = x % (D / 4);
    const int rr = rb + r;
    if (rr >= R) continue;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) mx = fmaxf(mx, s_m[w][r]);
    float ls = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = (s_m[w][r] == -INFINITY ? 0.f : ex2_approx(s_m[w][r] - mx)) * s_l[w][r];
      const float4 z = *reinterpret_cast<const float4*>(&s_o[w][r][4 * c]);
      ls += f;
      y.x += f * z.x; y.y += f * z.y; y.z += f * z.z; y.w += f * z.w;
    }
    const long long off = (long long)s * a.o_seq + (long long)(sv.q0 + rr / a.G) * a.o_tok +
                          (long long)(h * a.G + rr % a.G) * a.o_head;
    const float inv = over_sum(ls);
    y = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
    if (a.cluster) {
      *reinterpret_cast<float4*>(&s_o[0][r][4 * c]) = y;
      if (c == 0) s_ml[r] = make_float2(mx, ls);
    } else if (a.nsplit > 1) {
      const size_t pr = size_t(sp) * a.out_rows + off / D;
      *reinterpret_cast<float4*>(a.part_o + pr * D + 4 * c) = y;
      if (c == 0) a.part_ml[pr] = make_float4(mx, ls, ls, 0.f);
    } else {
      *reinterpret_cast<uint2*>(a.out + off + 4 * c) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
      if (c == 0 && a.lse) a.lse[off / D] = ls == 0.f ? -INFINITY : (mx + log2f(ls * kUp)) * 0.69314718055994531f;
    }
  }
  if (!a.cluster) return;
  // ---- join the cluster: each of its CTAs takes a share of the outputs and reads the others' parts, in their order
  cluster_sync();
  for (int x = sp * kRowThreads + threadIdx.x; x < NR * (D / 4); x += a.nsplit * kRowThreads) {
    const int r = x / (D / 4), c = x % (D / 4);
    const int rr = rb + r;
    if (rr >= R) continue;
    float mx = -INFINITY, ls = 0.f;
    for (int p = 0; p < a.nsplit; ++p) mx = fmaxf(mx, ld_cluster2(in_cta(&s_ml[r], p)).x);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = 0; p < a.nsplit; ++p) {
      const float2 ml = ld_cluster2(in_cta(&s_ml[r], p));
      const float4 z = ld_cluster4(in_cta(&s_o[0][r][4 * c], p));
      const float f = (ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mx)) * ml.y;
      ls += f;
      y.x += f * z.x; y.y += f * z.y; y.z += f * z.z; y.w += f * z.w;
    }
    const long long off = (long long)s * a.o_seq + (long long)(sv.q0 + rr / a.G) * a.o_tok +
                          (long long)(h * a.G + rr % a.G) * a.o_head;
    const float inv = over_sum(ls);
    *reinterpret_cast<uint2*>(a.out + off + 4 * c) =
        make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
    if (c == 0 && a.lse) a.lse[off / D] = ls == 0.f ? -INFINITY : (mx + log2f(ls * kUp)) * 0.69314718055994531f;
  }
  cluster_sync();                         // no CTA leaves while another reads its parts
}

// Joins the splits of every output row, in an order that the number of splits fixes. PG groups of D/4 lanes a row, 4
// values a lane; group g takes splits g, g + PG, ... and the groups' sums are joined in shared memory.
template <int D, int PG>
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedArgs a) {
  constexpr int LPR = D / 4, RPB = 256 / (LPR * PG);
  // launched while the kernel that writes the parts still runs: from here on its results are there
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = threadIdx.x % LPR, g = threadIdx.x / LPR % PG, rw = threadIdx.x / (LPR * PG);
  const long long x = (long long)blockIdx.x * RPB + rw;   // (token, head) of the sequence
  const int s = blockIdx.y, Hq = a.Hkv * a.G;
  const SeqView sv = seq_view(a, s);
  const bool in = x < (long long)sv.n * Hq;
  const long long off = in ? (long long)s * a.o_seq + (sv.q0 + x / Hq) * a.o_tok + (x % Hq) * a.o_head : 0;
  const size_t row = off / D;
  float mx = -INFINITY, ls = 0.f, le = 0.f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  if (in) {
    for (int p = g; p < a.nsplit; p += PG) mx = fmaxf(mx, a.part_ml[size_t(p) * a.out_rows + row].x);
    for (int p = g; p < a.nsplit; p += PG) {
      const size_t pr = size_t(p) * a.out_rows + row;
      const float4 ml = a.part_ml[pr];
      if (ml.y == 0.f) continue;   // a split without a key of this row: its output part is not written (a NaN goes on)
      const float e = ex2_approx(ml.x - mx), f = e * ml.y;
      const float4 z = *reinterpret_cast<const float4*>(a.part_o + pr * D + 4 * c);
      ls += f;
      le += e * ml.z;
      y.x += f * z.x; y.y += f * z.y; y.z += f * z.z; y.w += f * z.w;
    }
  }
  if constexpr (PG > 1) {
    __shared__ float4 s_y[RPB][PG][LPR], s_ml[RPB][PG];
    s_y[rw][g][c] = y;
    if (c == 0) s_ml[rw][g] = make_float4(mx, ls, le, 0.f);
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int i = 0; i < PG; ++i) mx = fmaxf(mx, s_ml[rw][i].x);
    ls = le = 0.f;
    y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < PG; ++i) {
      const float4 ml = s_ml[rw][i], z = s_y[rw][i][c];
      const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mx);
      ls += f * ml.y;
      le += f * ml.z;
      y.x += f * z.x; y.y += f * z.y; y.z += f * z.z; y.w += f * z.w;
    }
  }
  if (!in) return;
  const float inv = over_sum(ls);
  *reinterpret_cast<uint2*>(a.out + off + 4 * c) =
      make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
  if (c == 0 && a.lse) a.lse[row] = le == 0.f ? -INFINITY : (mx + log2f(le * kUp)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_paged_rows(const PagedArgs& a, bool int8, cudaStream_t st) {
  const long long rows = (long long)a.max_q * a.G;
  const int nr = rows <= 8 ? 8 : 16;
  const dim3 grid(unsigned((rows + nr - 1) / nr * a.nsplit), a.Hkv, a.S);
  cudaError_t e = cudaSuccess;
  auto go = [&](auto f, int smem) {
    if (smem > 40 * 1024) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = unsigned(a.nsplit);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = kRowThreads;
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = a.cluster ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, f, a);
  };
#define BSVA_ROWS(D, I8)                                              \
  nr == 8 ? go(paged_rows_kernel<D, I8, 1>, kRowSmem<D, I8, 1>())     \
          : go(paged_rows_kernel<D, I8, 2>, kRowSmem<D, I8, 2>())
  if (a.d == 128) {
    if (int8) BSVA_ROWS(128, true); else BSVA_ROWS(128, false);
  } else {
    if (int8) BSVA_ROWS(64, true); else BSVA_ROWS(64, false);
  }
#undef BSVA_ROWS
  return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_paged_combine(const PagedArgs& a, cudaStream_t st) {
  const long long rows = (long long)a.max_q * a.Hkv * a.G;
  // Eight groups a row shorten the chain of loads, which is all there is to few rows: 40 rows of 8 splits 13.3 us with
  // the kernel before it (one group 15.4), of 64 splits 19.5 (34), of 222 117 (229). Many rows of few splits
  // keep the GPU busy with one group: 4096 rows of 9 splits, 265 us for 271.
  const int pg = a.nsplit > 16 || (a.nsplit > 2 && rows * a.S <= 2048) ? 8 : 1;
  const long long rpb = 256 / (a.d / 4 * pg);
  // the launch overlaps the end of the kernel before it (the parts' writer); the device waits for that one itself
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned((rows + rpb - 1) / rpb), a.S);
  cfg.blockDim = 256;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto go = [&](auto f) { return cudaLaunchKernelEx(&cfg, f, a); };
  if (a.d == 128) return pg > 1 ? go(paged_combine_kernel<128, 8>) : go(paged_combine_kernel<128, 1>);
  return pg > 1 ? go(paged_combine_kernel<64, 8>) : go(paged_combine_kernel<64, 1>);
}

}  // namespace bsva

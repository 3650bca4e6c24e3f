// paged_kv.cu -- writing new tokens into a paged K/V cache (quantised per token and head, or bf16) and
// reading tokens back as bf16.
//
// Quantiser of a (token, head) row x of d values: s = fl32(amax / 127), code = rint_half_even(fl32(x / s)),
// 0 where s = 0: the library's block quantiser with the block shrunk to one row, so that a token can be
// appended without touching the codes of its neighbours. Reading gives bf16(code * s). A row that holds a NaN gets the
// scale NaN and one that holds an infinity the scale inf with codes 0, so that both read back, and attend, as NaN.
//
// Both kernels move every byte once: writing takes 2 B in and 1 + 4/d B out an element, reading the reverse. A row of
// d values is held by d/8 lanes (16 bytes of bf16 each), so a warp's loads and stores are whole 32-byte sectors; each
// thread has several independent rows in flight. Measured, 2 sequences of 8064 tokens, 40 heads of 128 (d = 64 within
// 5 % for the same bytes): bf16 pages, write 109 us (6.05 TB/s of a measured copy's 6.54), read 106 (6.2); INT8 pages,
// read 84 us (6.0), bound by HBM like those; write 130 us (3.85), bound by the quantiser's instructions.
#include "common.cuh"
#include "paged.cuh"
#include "quant.cuh"

namespace bsva {
namespace {

constexpr int kKvThreads = 256;
constexpr int kWriteRows = 2;   // rows of K and of V that a thread has in flight

// The larger |value| of two pairs of bf16, NaN if one is (signs of the result are meaningless), and of a pair.
__device__ __forceinline__ uint32_t row_max(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float row_max_fold(uint32_t m) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;"
      : "=f"(d)
      : "f"(__uint_as_float((m & 0x7FFFu) << 16)), "f"(__uint_as_float(m & 0x7FFF0000u)));
  return d;
}

// Codes of 8 bf16 values (w) of a row with scale sc, rcp = fl(1 / sc) or 0: the fast step of quant.cuh in pairs.
__device__ __forceinline__ uint2 quant8(const uint32_t (&w)[4], float sc, float rcp) {
  const float2 rc = make_float2(rcp, rcp), mg = make_float2(kMagic, kMagic), nmg = make_float2(-kMagic, -kMagic),
               n1 = make_float2(-1.f, -1.f);
  float2 t[4];
  float dm = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 q = __fmul2_rn(make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u)), rc);
    t[e] = __fadd2_rn(q, mg);
    const float2 d = __ffma2_rn(__fadd2_rn(t[e], nmg), n1, q);   // exact: how far q is from its integer
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(dm) : "f"(dm), "f"(d.x), "f"(d.y));
  }
  // near a half-integer, or a scale below 2^-120 (its reciprocal could overflow): the IEEE division. Half of the warps
  // come here, since half a row's largest value, 63.5 s, is a common one, so the pairs are looked at once more
  // (2 x 8064 tokens, 40 heads: 130 us, all four pairs divided 139, none 107).
  if (dm >= kBand || (sc > 0.f && rcp == 0.f)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = __uint_as_float(w[e] << 16), y = __uint_as_float(w[e] & 0xFFFF0000u);
      if (rcp == 0.f || fabsf(x * rcp - (t[e].x - kMagic)) >= kBand || fabsf(y * rcp - (t[e].y - kMagic)) >= kBand)
        t[e] = make_float2(quant_exact(x, sc), quant_exact(y, sc));
    }
  }
  uint32_t b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = __byte_perm(__float_as_uint(t[e].x), __float_as_uint(t[e].y), 0x0040);
  return make_uint2(__byte_perm(b[0], b[1], 0x5410), __byte_perm(b[2], b[3], 0x5410));
}

// One CTA per (block of 2^shift new tokens, heads that fill its rows up, sequence): a row slot's low bits are the
// token, so that long chunks write whole runs of a head's page and single tokens fill a CTA with their heads, both
// without a division. A thread takes kWriteRows rows of K and the same of V.
template <int D, bool I8>
__global__ void __launch_bounds__(kKvThreads) paged_write_kernel(const PagedArgs a, const __nv_bfloat16* __restrict__ k,
                                                                 const __nv_bfloat16* __restrict__ v,
                                                                 long long k_stride, long long v_stride, int shift) {
  constexpr int LPR = D / 8;                    // lanes of a row
  constexpr int RPP = kKvThreads / LPR;         // rows a pass
  constexpr int N = 2 * kWriteRows;             // K rows, then V rows
  const int s = blockIdx.z;
  const SeqView sv = seq_view(a, s);
  // lengths clamped into their bounds give positions of other tokens: nothing is written over those
  if (sv.bad || int(blockIdx.x << shift) >= sv.n) return;
  const int c = threadIdx.x % LPR;
  uint4 x[N];
  long long dst[kWriteRows];                    // destination row, or -1
#pragma unroll
  for (int u = 0; u < kWriteRows; ++u) {
    const int slot = threadIdx.x / LPR + u * RPP;
    const int i = (blockIdx.x << shift) + (slot & ((1 << shift) - 1));
    const int h = blockIdx.y * ((RPP * kWriteRows) >> shift) + (slot >> shift);
    x[u] = x[u + kWriteRows] = make_uint4(0, 0, 0, 0);
    dst[u] = -1;
    if (i < sv.n && h < a.Hkv) {
      const long long tok = sv.q0 + i;
      x[u] = __ldg(reinterpret_cast<const uint4*>(k + tok * k_stride + h * D) + c);
      x[u + kWriteRows] = __ldg(reinterpret_cast<const uint4*>(v + tok * v_stride + h * D) + c);
      // a position before the sequence (kv_len smaller than the chunk) or a page outside the cache: not written
      const int pos = sv.kv - sv.n + i;
      int page = -1;
      if (pos >= 0) page = __ldg(a.page_table + size_t(s) * a.max_pages + (pos >> a.page_shift));
      if (unsigned(page) < unsigned(a.n_pages)) dst[u] = (long long)kv_row(a, page, h, pos);
      else atomicOr(a.status, kStatusBounds);
    }
  }
  char* kd = static_cast<char*>(const_cast<void*>(a.k));
  char* vd = static_cast<char*>(const_cast<void*>(a.v));
  if constexpr (!I8) {
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (dst[u % kWriteRows] >= 0)
        reinterpret_cast<uint4*>(u < kWriteRows ? kd : vd)[dst[u % kWriteRows] * LPR + c] = x[u];
  } else {
    float m[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      uint32_t p = row_max(row_max(x[u].x, x[u].y), row_max(x[u].z, x[u].w));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) p = row_max(p, __shfl_xor_sync(0xffffffffu, p, o));
      m[u] = row_max_fold(p);
    }
    // the N divisions of a row's lanes, one a lane
    static_assert(N == 4 && LPR >= 4, "four rows a thread");
    const float mine = c & 2 ? (c & 1 ? m[3] : m[2]) : (c & 1 ? m[1] : m[0]);
    const float sc1 = __fdiv_rn(mine, 127.0f), rcp1 = sc1 >= 0x1p-120f ? __frcp_rn(sc1) : 0.f;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const float sc = __shfl_sync(0xffffffffu, sc1, u, LPR), rcp = __shfl_sync(0xffffffffu, rcp1, u, LPR);
      const uint2 q = quant8({x[u].x, x[u].y, x[u].z, x[u].w}, sc, rcp);
      const long long d = dst[u % kWriteRows];
      if (d >= 0) {
        reinterpret_cast<uint2*>(u < kWriteRows ? kd : vd)[d * LPR + c] = q;
        if (c == 0) const_cast<float*>(u < kWriteRows ? a.k_scale : a.v_scale)[d] = sc;
      }
    }
  }
}

constexpr int kReadRows = 4;

// One CTA per (block of output rows, head, sequence): tokens first + r of the sequence, zeros behind its
// last one. Each thread writes 8 values a row of K and of V.
template <int D, bool I8>
__global__ void __launch_bounds__(kKvThreads) paged_read_kernel(const PagedArgs a, const int32_t* __restrict__ first,
                                                                int L, __nv_bfloat16* __restrict__ k_out,
                                                                __nv_bfloat16* __restrict__ v_out) {
  constexpr int LPR = D / 8;
  constexpr int RPP = kKvThreads / LPR;
  const int s = blockIdx.z, h = blockIdx.y;
  const int c = threadIdx.x % LPR;
  const SeqView sv = seq_view(a, s);
  int f = first ? first[s] : 0;
  if (f < 0 || (f < sv.kv && sv.kv - f > L)) {   // a negative start, or more live tokens than the output holds
    atomicOr(a.status, kStatusBounds);
    f = max(f, 0);
  }
  const int live = min(max(sv.kv - f, 0), L);
  const int r0 = blockIdx.x * (RPP * kReadRows) + threadIdx.x / LPR;
  uint4 x[2][kReadRows];
  float sc[2][kReadRows];
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    const int r = r0 + u * RPP;
    x[0][u] = x[1][u] = make_uint4(0, 0, 0, 0);
    sc[0][u] = sc[1][u] = 0.f;
    if (r < live) {
      const size_t row = kv_row(a, page_of(a, s, f + r), h, f + r);
      if constexpr (I8) {
        const uint2 kk = __ldg(reinterpret_cast<const uint2*>(a.k) + row * LPR + c);
        const uint2 vv = __ldg(reinterpret_cast<const uint2*>(a.v) + row * LPR + c);
        x[0][u].x = kk.x; x[0][u].y = kk.y;
        x[1][u].x = vv.x; x[1][u].y = vv.y;
        sc[0][u] = __ldg(a.k_scale + row);
        sc[1][u] = __ldg(a.v_scale + row);
      } else {
        x[0][u] = __ldg(reinterpret_cast<const uint4*>(a.k) + row * LPR + c);
        x[1][u] = __ldg(reinterpret_cast<const uint4*>(a.v) + row * LPR + c);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    const int r = r0 + u * RPP;
    if (r >= L) continue;
    const size_t o = ((size_t(s) * a.Hkv + h) * L + r) * LPR + c;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      uint4 y = x[z][u];
      if constexpr (I8) {
        const uint32_t w[2] = {x[z][u].x, x[z][u].y};
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int lo = int(w[e >> 1] << (e & 1 ? 8 : 24)) >> 24, hi = int(w[e >> 1] << (e & 1 ? 0 : 16)) >> 24;
          p[e] = pack_bf16x2(float(lo) * sc[z][u], float(hi) * sc[z][u]);
        }
        y = make_uint4(p[0], p[1], p[2], p[3]);
      }
      reinterpret_cast<uint4*>(z ? v_out : k_out)[o] = y;
    }
  }
}

}  // namespace

cudaError_t launch_paged_write(const PagedArgs& a, bool int8, const __nv_bfloat16* k, const __nv_bfloat16* v,
                               long long k_stride, long long v_stride, cudaStream_t st) {
  const int rows = kKvThreads / (a.d / 8) * kWriteRows;   // of a CTA
  int shift = 0;
  while ((1 << shift) < rows && (1 << shift) < a.max_q) ++shift;
  const int heads = rows >> shift;
  const dim3 grid((a.max_q + (1 << shift) - 1) >> shift, (a.Hkv + heads - 1) / heads, a.S);
  auto go = [&](auto f) { f<<<grid, kKvThreads, 0, st>>>(a, k, v, k_stride, v_stride, shift); };
  if (a.d == 128) int8 ? go(paged_write_kernel<128, true>) : go(paged_write_kernel<128, false>);
  else int8 ? go(paged_write_kernel<64, true>) : go(paged_write_kernel<64, false>);
  return cudaGetLastError();
}

cudaError_t launch_paged_read(const PagedArgs& a, bool int8, const int32_t* first, int L, __nv_bfloat16* k_out,
                              __nv_bfloat16* v_out, cudaStream_t st) {
  const int rpb = kKvThreads / (a.d / 8) * kReadRows;
  const dim3 grid((L + rpb - 1) / rpb, a.Hkv, a.S);
  auto go = [&](auto f) { f<<<grid, kKvThreads, 0, st>>>(a, first, L, k_out, v_out); };
  if (a.d == 128) int8 ? go(paged_read_kernel<128, true>) : go(paged_read_kernel<128, false>);
  else int8 ? go(paged_read_kernel<64, true>) : go(paged_read_kernel<64, false>);
  return cudaGetLastError();
}

}  // namespace bsva

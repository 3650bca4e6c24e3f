// paged_kv.cu -- writing new tokens into a paged K/V cache (quantised per token and head, or bf16) and
// reading tokens back as bf16.
//
// Quantiser of a (token, head) row x of d values: s = fl32(amax / 127), code = rint_half_even(fl32(x / s)),
// 0 where s = 0: the library's block quantiser with the block shrunk to one row, so that a token can be
// appended without touching the codes of its neighbours. Reading gives bf16(code * s).
//
// Both kernels move every byte once and are bound by HBM: writing takes 2 B in and 1 + 4/d B out an element,
// reading the reverse. A row of d values is held by d/8 lanes (16 bytes of bf16 each), so a warp's loads
// and stores are whole 32-byte sectors; each thread has several independent rows in flight.
#include "common.cuh"
#include "paged.cuh"
#include "quant.cuh"

namespace bsva {
namespace {

constexpr int kKvThreads = 256;
constexpr int kWriteRows = 4;   // rows a thread has in flight

// One CTA per (block of rows of a sequence's new tokens, K or V, sequence); rows are (token, head) pairs,
// head fastest, as the source has them.
template <int D, bool I8>
__global__ void __launch_bounds__(kKvThreads) paged_write_kernel(const PagedArgs a, const __nv_bfloat16* __restrict__ k,
                                                                 const __nv_bfloat16* __restrict__ v,
                                                                 long long k_stride, long long v_stride) {
  constexpr int LPR = D / 8;                    // lanes of a row
  constexpr int RPP = kKvThreads / LPR;         // rows a pass
  const int s = blockIdx.z;
  const bool isV = blockIdx.y == 1;
  const SeqView sv = seq_view(a, s);
  const long long rows = (long long)sv.n * a.Hkv;
  const long long row0 = (long long)blockIdx.x * (RPP * kWriteRows) + threadIdx.x / LPR;
  const int c = threadIdx.x % LPR;
  const __nv_bfloat16* src = isV ? v : k;
  const long long stride = isV ? v_stride : k_stride;

  uint4 x[kWriteRows];
  long long dst[kWriteRows];                    // destination row, or -1
#pragma unroll
  for (int u = 0; u < kWriteRows; ++u) {
    const long long r = row0 + (long long)u * RPP;
    x[u] = make_uint4(0, 0, 0, 0);
    dst[u] = -1;
    if (r < rows) {
      const int i = int(r / a.Hkv), h = int(r % a.Hkv);
      const int pos = sv.kv - sv.n + i;         // negative where kv_len is smaller than the chunk: not written
      if (pos >= 0) {
        const int page = __ldg(a.page_table + size_t(s) * a.max_pages + (pos >> a.page_shift));
        if (unsigned(page) < unsigned(a.n_pages)) {
          dst[u] = (long long)kv_row(a, page, h, pos);
          x[u] = __ldg(reinterpret_cast<const uint4*>(src + (long long)(sv.q0 + i) * stride + (long long)h * D) + c);
        } else {
          atomicOr(a.status, kStatusBounds);
        }
      } else {
        atomicOr(a.status, kStatusBounds);
      }
    }
  }
  if constexpr (!I8) {
    uint4* out = reinterpret_cast<uint4*>(const_cast<void*>(isV ? a.v : a.k));
#pragma unroll
    for (int u = 0; u < kWriteRows; ++u)
      if (dst[u] >= 0) out[dst[u] * LPR + c] = x[u];
  } else {
    uint2* out = reinterpret_cast<uint2*>(const_cast<void*>(isV ? a.v : a.k));
    float* scale = const_cast<float*>(isV ? a.v_scale : a.k_scale);
#pragma unroll
    for (int u = 0; u < kWriteRows; ++u) {
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float m = bmax_fold(bmax_abs(bmax_abs(w[0], w[1]), bmax_abs(w[2], w[3])));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float sc = __fdiv_rn(m, 127.0f);
      // below 2^-120 the reciprocal could overflow: those rows take the IEEE division
      const bool slow = sc > 0.f && sc < 0x1p-120f;
      const float rcp = sc >= 0x1p-120f ? __frcp_rn(sc) : 0.f;
      float t[8], dm = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xe = __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
        const float q = xe * rcp;
        t[e] = __fadd_rn(q, kMagic);
        dm = fmaxf(dm, fabsf(__fsub_rn(q, __fsub_rn(t[e], kMagic))));
      }
      if (dm >= kBand || slow) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          t[e] = quant_exact(__uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16), sc);
      }
      if (dst[u] >= 0) {
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = __byte_perm(__float_as_uint(t[2 * e]), __float_as_uint(t[2 * e + 1]), 0x0040);
        out[dst[u] * LPR + c] = make_uint2(__byte_perm(b[0], b[1], 0x5410), __byte_perm(b[2], b[3], 0x5410));
        if (c == 0) scale[dst[u]] = sc;
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
  const long long rpb = kKvThreads / (a.d / 8) * kWriteRows;
  const dim3 grid(unsigned(((long long)a.max_q * a.Hkv + rpb - 1) / rpb), 2, a.S);
  auto go = [&](auto f) { f<<<grid, kKvThreads, 0, st>>>(a, k, v, k_stride, v_stride); };
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

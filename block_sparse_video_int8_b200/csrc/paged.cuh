// paged.cuh -- what the paged-cache kernels share: the description of a call (pages, sequences, query
// rows), the checked view of one sequence, the address of a cached key, and the exact widening of
// INT8 codes to 16-bit floats.
#pragma once

#include "common.cuh"

namespace bsva {

// One call. Two sources of keys go through the same kernels:
//  - pages: row (page, head, offset) of k and v, found through page_table (page_shift = log2(page_size));
//  - contiguous [S, Hkv, max_kv, d] tensors (cross attention): page_table null, sequence s is "page" s.
// q_start null: every sequence has max_q query rows; kv_len null: max_kv keys.
struct PagedArgs {
  const void* k;
  const void* v;                // int8 codes or bf16
  const float* k_scale;         // [n_pages, Hkv, page_size], INT8 only
  const float* v_scale;
  const int32_t* q_start;       // [S + 1]
  const int32_t* kv_len;        // [S]
  const int32_t* page_table;    // [S, max_pages]
  const __nv_bfloat16* q;       // element strides below
  __nv_bfloat16* out;
  float* lse;                   // [out rows], nullable
  float* part_o;                // [nsplit, out rows, d] outputs of the splits, each divided by its sum
  float4* part_ml;              // [nsplit, out rows] (running max in log2 units, sum that divides O, sum of the
                                // unrounded weights, unused); sums times kDown
  uint32_t* status;
  long long q_seq, q_tok, q_head;   // q strides (q_seq: contiguous source only)
  long long o_seq, o_tok, o_head;   // out strides; out row index = offset / d
  long long out_rows;
  float scale_log2;             // softmax scale * log2(e)
  int n_pages, page_shift, max_pages, page_rows;   // page_rows: rows a page holds
  int box_rows;                 // rows of a TMA box of bf16 pages: a page's, at most a key tile's
  int S, T, Hkv, G, d;
  int max_q, max_kv;
  int causal, window;
  int q_tma;                    // tile kernel: Q by TMA (G divides 128)
  int nsplit, split_keys;       // rows kernel: keys of a split; tile kernel: splits share a row tile's key tiles
  int cluster;                  // rows kernel: the splits of a row tile are a cluster of CTAs, which joins them
  uint64_t wait_limit_ns;
};

// bf16 keys and values for the tile kernel, [heads of all pages][rows][d]; boxes of box_rows rows x 64 values.
// Queries (q_tma) [sequences][tokens][heads][d], boxes of 128 rows x 64 values.
struct PagedMaps {
  CUtensorMap k, v, q;
};

// A sequence as the kernels use it. Values that the caller's device arrays hold are clamped into the
// ranges that the host checked the buffers for, and a value outside records kStatusBounds: no access
// leaves its buffer whatever the arrays say.
struct SeqView {
  int n;     // new tokens (query rows a head)
  int kv;    // keys
  int q0;    // first row of the sequence in the packed tensors
  bool bad;  // a value was outside its range
};

__device__ __forceinline__ SeqView seq_view(const PagedArgs& a, int s) {
  SeqView r;
  r.bad = false;
  if (a.q_start) {
    const int lo = a.q_start[s], hi = a.q_start[s + 1];
    r.q0 = min(max(lo, 0), a.T);
    r.n = min(min(max(hi, r.q0), a.T) - r.q0, a.max_q);
    r.bad = r.q0 != lo || r.n != hi - lo;
  } else {
    r.q0 = 0;
    r.n = a.max_q;
  }
  if (a.kv_len) {
    const int kv = a.kv_len[s];
    r.kv = min(max(kv, 0), a.max_kv);
    r.bad = r.bad || kv != r.kv;
  } else {
    r.kv = a.max_kv;
  }
  if (r.bad) atomicOr(a.status, kStatusBounds);
  return r;
}

// The page table's entry for token t of sequence s, and the page that it names: one outside [0, n_pages) is recorded
// and read as page 0.
__device__ __forceinline__ int page_entry(const PagedArgs& a, int s, int t) {
  return __ldg(a.page_table + size_t(s) * a.max_pages + (t >> a.page_shift));
}
__device__ __forceinline__ int checked_page(const PagedArgs& a, int entry) {
  if (unsigned(entry) < unsigned(a.n_pages)) return entry;
  atomicOr(a.status, kStatusBounds);
  return 0;
}
__device__ __forceinline__ int page_of(const PagedArgs& a, int s, int t) {
  return a.page_table ? checked_page(a, page_entry(a, s, t)) : s;
}

// Row index (of d elements, or of one scale) of token t of a head, in the page that page_of gave.
__device__ __forceinline__ size_t kv_row(const PagedArgs& a, int page, int head, int t) {
  const int off = a.page_table ? t & ((1 << a.page_shift) - 1) : t;
  return (size_t(page) * a.Hkv + head) * a.page_rows + off;
}

// ---- widening: each 32-bit word holds four INT8 codes b0..b3; the two results hold the pairs (b0, b2)
// and (b1, b3). Callers choose which element sits in which byte, or which order the pairs stand for.
__device__ __forceinline__ uint32_t lop_and_xor(uint32_t x, uint32_t m, uint32_t o) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(x), "r"(m), "r"(o));   // (x & m) ^ o
  return r;
}
// f16: 0x6400 | (b + 128) = 1024 + 128 + b, minus 1152.
__device__ __forceinline__ void widen_f16(uint32_t w, uint32_t& even, uint32_t& odd) {
  auto half = [](uint32_t x) {
    uint32_t v = lop_and_xor(x, 0x00ff00ffu, 0x64806480u);
    __half2 d = __hsub2(*reinterpret_cast<__half2*>(&v), __floats2half2_rn(1152.f, 1152.f));
    return *reinterpret_cast<uint32_t*>(&d);
  };
  even = half(w);
  odd = half(w >> 8);
}

// 1 / sum, 0 for the sum of no weights. Within 2 units of the last place, for sums in [2^-126, 2^126].
__device__ __forceinline__ float over_sum(float x) { return x == 0.f ? 0.f : __fdividef(1.f, x); }

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Sums of weights are kept times 2^-48, those of bf16 values as sums of weights times 2^-48, and outputs are divided by
// their sum before they are joined: the sums of 2^30 keys' weights stay below one, and so every weighted sum of values
// below the largest of them, whatever its size. (The price: a weighted value below 2^-126 loses bits, so values below 2^-54
// have less than fp32's precision, and weights below 2^-78 of the largest are lost.)
constexpr float kDown = 0x1p-48f, kUp = 0x1p48f, kDownLog2 = 48.f;

// ---- INT8 values in an f16 product: the scale s_v of a key's values enters as s_v * c with c a power of two, so that it
// fits f16 whatever the scales' range. c is set by the largest scale S of the keys met so far that some row of the tile
// sees, and set anew (the output so far rescaled) when a scale comes that would leave f16; it never falls.
// Few rows: the weight is p * s_v * c, p <= 2^8 by the lazy running maximum, 2^6 <= S c < 2^7. Tiles: the value is
// code * (s_v * c), 2^5 <= S c < 2^8. Both are rounded within 2^-11 (tiles: the product and its factor), as far as they
// are normal in f16, 2^-14: that is so for keys with s_v >= 2^-19 S (few rows, those that weigh at least 1: 2^-20 S),
// and below each halving costs a bit of what such a key adds. The sum of the weights takes p itself, in fp32.
constexpr int kRowsUp = 6, kTilesUp = 5;                       // log2 of S c when c is set, rounded down
constexpr float kRowsFull = 128.f, kTilesFull = 256.f;         // s_v * c reaches this: c is set anew
// 2^UP * 2^-floor(log2 s), it and its reciprocal in the normal range
template <int UP>
__device__ __forceinline__ float scale_norm(float s) {
  const int e = min(max(int(__float_as_uint(s) >> 23), UP + 1), 253);
  return __uint_as_float(uint32_t(254 + UP - e) << 23);
}

cudaError_t launch_paged_write(const PagedArgs& a, bool int8, const __nv_bfloat16* k, const __nv_bfloat16* v,
                               long long k_stride, long long v_stride, cudaStream_t st);
cudaError_t launch_paged_read(const PagedArgs& a, bool int8, const int32_t* first, int L, __nv_bfloat16* k_out,
                              __nv_bfloat16* v_out, cudaStream_t st);
cudaError_t launch_paged_rows(const PagedArgs& a, bool int8, cudaStream_t st);
cudaError_t launch_paged_tiles(const PagedArgs& a, const PagedMaps& maps, bool int8, cudaStream_t st);
cudaError_t launch_paged_combine(const PagedArgs& a, cudaStream_t st);

}  // namespace bsva

// paged_api.cu -- the C entries of the paged K/V cache and of cross attention (include/bsva.h): argument
// checks, the split of a call over the GPU, workspace carving and launches.
#include <cmath>

#include "api.cuh"
#include "paged.cuh"

using namespace bsva;

namespace {

constexpr int kMaxSplits = 256;

int ilog2(int x) {
  int r = 0;
  while ((1 << r) < x) ++r;
  return r;
}

int check_cache(const bsva_paged_kv* c) {
  if (c == nullptr) return fail(BSVA_ERR_INVALID_ARG, "cache is NULL");
  if (c->d != 64 && c->d != 128) return fail(BSVA_ERR_UNSUPPORTED, "head dim d = %d; supported: 64, 128", c->d);
  if (c->H < 1 || c->H > 65535) return fail(BSVA_ERR_INVALID_ARG, "cache: H = %d", c->H);
  if (c->n_pages < 1) return fail(BSVA_ERR_INVALID_ARG, "cache: n_pages = %d", c->n_pages);
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return fail(BSVA_ERR_INVALID_ARG, "page_size = %d; supported: 16, 32, 64, 128, 256", c->page_size);
  if (c->dtype != BSVA_KV_INT8 && c->dtype != BSVA_KV_BF16)
    return fail(BSVA_ERR_INVALID_ARG, "cache dtype = %d; use BSVA_KV_INT8 (0) or BSVA_KV_BF16 (1)", c->dtype);
  if ((long long)c->n_pages * c->H >= (1ll << 31) / c->page_size)   // the kernels keep a row's number in an int
    return fail(BSVA_ERR_INVALID_ARG, "cache: n_pages * H * page_size = %d * %d * %d is not below 2^31", c->n_pages, c->H,
                c->page_size);
  return BSVA_OK;
}

int check_cache_ptrs(const bsva_paged_kv* c) {
  REQUIRE_PTR(c->k, 16); REQUIRE_PTR(c->v, 16);
  if (c->dtype == BSVA_KV_INT8) { REQUIRE_PTR(c->k_scale, 4); REQUIRE_PTR(c->v_scale, 4); }
  return BSVA_OK;
}

int check_batch(const bsva_paged_kv* c, const bsva_paged_batch* b) {
  if (b == nullptr) return fail(BSVA_ERR_INVALID_ARG, "batch is NULL");
  if (b->S < 1 || b->S > 65535) return fail(BSVA_ERR_INVALID_ARG, "batch: S = %d outside [1, 65535]", b->S);
  if (b->T < 0 || b->max_q < 1 || b->max_q > (1 << 24))
    return fail(BSVA_ERR_INVALID_ARG, "batch: T = %d, max_q = %d (T >= 0, 1 <= max_q <= 2^24)", b->T, b->max_q);
  if (b->max_kv < 1 || b->max_kv > (1 << 30)) return fail(BSVA_ERR_INVALID_ARG, "batch: max_kv = %d", b->max_kv);
  if (b->max_pages < 1 || (long long)b->max_pages * c->page_size < b->max_kv)
    return fail(BSVA_ERR_INVALID_ARG, "batch: max_pages = %d pages of %d tokens hold less than max_kv = %d", b->max_pages,
                c->page_size, b->max_kv);
  return BSVA_OK;
}

int check_heads(int Hq, int Hkv, long long max_q) {
  if (Hkv < 1 || Hq < 1 || Hq > 65535 || Hq % Hkv)
    return fail(BSVA_ERR_INVALID_ARG, "Hq = %d is not a positive multiple of %d key heads", Hq, Hkv);
  if (max_q * (Hq / Hkv) > (1ll << 30))
    return fail(BSVA_ERR_INVALID_ARG, "%lld query rows of %d heads a key head are too many for one call", max_q, Hq / Hkv);
  return BSVA_OK;
}

// How a call is laid over the GPU. Few rows leave few CTAs, so their keys are split and joined by a second
// kernel; the number of splits follows from the host bounds alone.
struct Plan {
  bool tiles = false;   // tensor-core tiles of 256 rows, or 8 or 16 rows a CTA
  int nsplit = 1, split_keys = 0;
  bool cluster = false;   // the splits of a row tile are a cluster of CTAs, which joins them without a second kernel
  int cap = 1;   // >= nsplit, and no smaller for more keys: workspaces are sized by it
};

Plan make_plan(int S, int Hkv, int G, int max_q, int keys, int d, bool int8) {
  Plan p;
  const long long rows = (long long)max_q * G;
  // Tiles of 256 rows pay from some rows on; below, row tiles of 16 that read the keys again are faster. 8 sequences of
  // 8192 keys, 8 key heads, tiles / rows, us: INT8 24 rows 113 / 65, 48 rows 117 / 80, 100 rows 123 / 115 (one sequence
  // of 30000 keys 72 / 117), 200 rows 142 / 197; bf16 24 rows 73 / 68, 48 rows 74 / 80, 100 rows 75 / 117.
  p.tiles = rows > (int8 ? 64 : 32);
  if (p.tiles) {
    // An item is 256 rows over all keys, one at a time an SM. Splitting the keys n ways levels the last round (and
    // fills the SMs where there are few items), and costs writing and joining n partial outputs. The time of each n
    // from measured rates: 128 keys take an item 3.2 us with INT8 codes, 1.95 us with bf16 (head dim 64: 0.6 of it),
    // partial outputs move at 5.5 TB/s, the second kernel costs 4 us. (2048 x 32760 tokens, 320 items: n = 1 2486 us.)
    const long long items = (rows + 255) / 256 * Hkv * S, tiles = (keys + 127) / 128;
    const long long most = tiles / 2, room = 148 * 9 / items;   // splits of two key tiles at least
    long long cap = most < room ? most : room;
    cap = cap < kMaxSplits ? cap : kMaxSplits;
    p.cap = int(cap < 1 ? 1 : cap);
    const double step = (int8 ? 3.2 : 1.95) * (d == 64 ? 0.6 : 1.0);
    double best = 0;
    for (int n = 1; n <= p.cap; ++n) {
      const double t = double((items * n + 147) / 148) * double((tiles + n - 1) / n) * step +
                       (n > 1 ? 4.0 + double(n) * rows * Hkv * S * (8.0 * d + 32.0) / 5.5e6 : 0.0);
      if (n == 1 || t < best) {
        best = t;
        p.nsplit = n;
      }
    }
    return p;
  }
  const long long nr = rows <= 8 ? 8 : 16, items = (rows + nr - 1) / nr * Hkv * S;
  // Three CTAs an SM run at once. Splits of 128 keys (two blocks a warp) until they are filled once, of 1024 keys until
  // four times: short ends and unequal sequences then leave few SMs idle, and joining costs little beside 1024 keys.
  // (One, four, eight times, us: 2 x 131000 keys, 40 key heads 550, 433, 443; 16 sequences of up to 1500 keys 21, 24.6,
  // 26.7. Least keys 512, 1024: 32768 keys, 8 key heads 34, 30; 131000 86, 82; 4 x 5000 23.3, 21.8.)
  auto splits = [&](long long ctas, long long least) {
    const long long want = (ctas + items - 1) / items, most = (keys + least - 1) / least;
    return want < most ? want : most;
  };
  long long n = splits(148 * 3, 128), n4 = splits(148 * 12, 1024);
  n = n > n4 ? n : n4;
  n = n < kMaxSplits ? n : kMaxSplits;
  n = n < 1 ? 1 : n;
  p.cap = int(n);
  const long long per = ((keys + n - 1) / n + 63) / 64 * 64;
  p.split_keys = int(per);
  p.nsplit = int((keys + per - 1) / per);
  // A cluster of 8 at most joins its splits itself where each CTA has an SM to itself: one launch less, 1003 keys, 8 key
  // heads (64 CTAs) 8.3 us a call in a loop for 9.8. Where SMs hold several CTAs, those that wait for their cluster
  // keep others out: 16 sequences of 1500 keys, 12 heads (576 CTAs) 16.5 us for 14.5; 8 x 3000 keys, 8 heads 32.8 for 27.6.
  p.cluster = p.nsplit > 1 && p.nsplit <= 8 && items * p.nsplit <= 148;
  return p;
}

size_t align256z(size_t x) { return (x + 255) & ~size_t(255); }

// Status word, then the partial outputs and their maxima and sums.
struct PagedWs {
  size_t part_o = 256, part_ml = 0, total = 256;
  PagedWs(int cap, size_t out_rows, int d) {
    if (cap < 2) return;
    part_ml = align256z(part_o + size_t(cap) * out_rows * d * 4);
    total = align256z(part_ml + size_t(cap) * out_rows * 16);
  }
};

void fill_cache(PagedArgs& a, const bsva_paged_kv* c, const bsva_paged_batch* b) {
  a.k = c->k; a.v = c->v; a.k_scale = c->k_scale; a.v_scale = c->v_scale;
  a.q_start = b->q_start; a.kv_len = b->kv_len; a.page_table = b->page_table;
  a.n_pages = c->n_pages; a.page_shift = ilog2(c->page_size); a.page_rows = c->page_size; a.max_pages = b->max_pages;
  a.S = b->S; a.T = b->T; a.Hkv = c->H; a.G = 1; a.d = c->d; a.max_q = b->max_q; a.max_kv = b->max_kv;
  a.wait_limit_ns = kWaitLimitNs;
}

int run_paged(PagedArgs& a, bool int8, const Plan& p, const PagedWs& w, void* workspace, cudaStream_t st) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.nsplit = p.nsplit;
  a.split_keys = p.split_keys;
  a.cluster = p.cluster;
  a.part_o = p.nsplit > 1 ? reinterpret_cast<float*>(ws + w.part_o) : nullptr;
  a.part_ml = p.nsplit > 1 ? reinterpret_cast<float4*>(ws + w.part_ml) : nullptr;
  PagedMaps maps{};
  if (p.tiles) {
    int rc;
    a.box_rows = a.page_table && a.page_rows < 128 ? a.page_rows : 128;
    if ((rc = get_encoder())) return rc;
    for (int z = 0; z < 2 && !int8; ++z)
      if ((rc = encode_map(z ? &maps.v : &maps.k, z ? a.v : a.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.d, a.page_rows,
                           uint64_t(a.n_pages) * a.Hkv, 64, a.box_rows, CU_TENSOR_MAP_SWIZZLE_128B, z ? "v" : "k")))
        return rc;
    a.q_tma = 128 % a.G == 0;
    if (a.q_tma) {
      const uint64_t tokens = a.q_start ? a.T : a.max_q, seqs = a.q_start ? 1 : a.S;
      const uint64_t stride[3] = {uint64_t(a.q_head) * 2, uint64_t(a.q_tok) * 2,
                                  uint64_t(a.q_start ? tokens * a.q_tok : a.q_seq) * 2};
      if ((rc = encode_map_4d(&maps.q, a.q, a.d, uint64_t(a.Hkv) * a.G, tokens, seqs, stride, 64, a.G, 128 / a.G, "q")))
        return rc;
    }
  }
  cudaError_t e = p.tiles ? launch_paged_tiles(a, maps, int8, st) : launch_paged_rows(a, int8, st);
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  if (p.nsplit > 1 && !a.cluster) {
    e = launch_paged_combine(a, st);
    if (e != cudaSuccess) return cuda_fail(e, "split combination launch");
  }
  return ok();
}

}  // namespace

extern "C" {

size_t bsva_paged_workspace_bytes(const bsva_paged_kv* c, const bsva_paged_batch* b, int Hq) {
  if (check_cache(c) || check_batch(c, b) || check_heads(Hq, c->H, b->max_q)) return 0;
  return PagedWs(make_plan(b->S, c->H, Hq / c->H, b->max_q, b->max_kv, c->d, c->dtype == BSVA_KV_INT8).cap, size_t(b->T) * Hq, c->d).total;
}

int bsva_paged_kv_write(const bsva_paged_kv* c, const bsva_paged_batch* b, const void* k, const void* v,
                        long long k_stride, long long v_stride, void* workspace, size_t workspace_bytes,
                        bsva_stream_t stream) {
  BSVA_RANGE("bsva_paged_kv_write");
  int rc;
  if ((rc = check_cache(c)) || (rc = check_cache_ptrs(c)) || (rc = check_batch(c, b))) return rc;
  REQUIRE_PTR(b->q_start, 4); REQUIRE_PTR(b->kv_len, 4); REQUIRE_PTR(b->page_table, 4);
  if ((rc = check_heads(c->H, c->H, (long long)b->max_q * c->H))) return rc;
  if (k_stride < (long long)c->H * c->d || v_stride < (long long)c->H * c->d || k_stride % 8 || v_stride % 8)
    return fail(BSVA_ERR_INVALID_ARG, "token strides %lld, %lld must be multiples of 8 and at least H*d = %d", k_stride,
                v_stride, c->H * c->d);
  if (b->T > 0) { REQUIRE_PTR(k, 16); REQUIRE_PTR(v, 16); }
  if ((rc = check_workspace(workspace, workspace_bytes, 256))) return rc;
  if ((rc = check_device())) return rc;
  if (b->T == 0) return ok();
  PagedArgs a{};
  fill_cache(a, c, b);
  a.status = static_cast<uint32_t*>(workspace);
  cudaError_t e = launch_paged_write(a, c->dtype == BSVA_KV_INT8, static_cast<const __nv_bfloat16*>(k),
                                     static_cast<const __nv_bfloat16*>(v), k_stride, v_stride,
                                     reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged write launch");
  return ok();
}

int bsva_paged_kv_read(const bsva_paged_kv* c, const bsva_paged_batch* b, const int32_t* first, int L, void* k_out,
                       void* v_out, void* workspace, size_t workspace_bytes, bsva_stream_t stream) {
  BSVA_RANGE("bsva_paged_kv_read");
  int rc;
  if ((rc = check_cache(c)) || (rc = check_cache_ptrs(c)) || (rc = check_batch(c, b))) return rc;
  REQUIRE_PTR(b->kv_len, 4); REQUIRE_PTR(b->page_table, 4);
  if (first && !aligned(first, 4)) return fail(BSVA_ERR_INVALID_ARG, "first is not 4-byte aligned");
  if (L < 1 || L > (1 << 30)) return fail(BSVA_ERR_INVALID_ARG, "L = %d", L);
  REQUIRE_PTR(k_out, 16); REQUIRE_PTR(v_out, 16);
  if ((rc = check_workspace(workspace, workspace_bytes, 256))) return rc;
  if ((rc = check_device())) return rc;
  PagedArgs a{};
  fill_cache(a, c, b);
  a.q_start = nullptr;
  a.status = static_cast<uint32_t*>(workspace);
  cudaError_t e = launch_paged_read(a, c->dtype == BSVA_KV_INT8, first, L, static_cast<__nv_bfloat16*>(k_out),
                                    static_cast<__nv_bfloat16*>(v_out), reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged read launch");
  return ok();
}

int paged_attn_fwd(const bsva_paged_kv* c, const bsva_paged_batch* b, const void* q, long long q_stride, int Hq,
                   int causal, int window, float softmax_scale, void* out, float* lse, void* workspace,
                   size_t workspace_bytes, bsva_stream_t stream) {
  BSVA_RANGE("paged_attn_fwd");
  int rc;
  if ((rc = check_cache(c)) || (rc = check_cache_ptrs(c)) || (rc = check_batch(c, b))) return rc;
  REQUIRE_PTR(b->q_start, 4); REQUIRE_PTR(b->kv_len, 4); REQUIRE_PTR(b->page_table, 4);
  if ((rc = check_heads(Hq, c->H, b->max_q))) return rc;
  if (q_stride < (long long)Hq * c->d || q_stride % 8)
    return fail(BSVA_ERR_INVALID_ARG, "token stride %lld must be a multiple of 8 and at least Hq*d = %d", q_stride,
                Hq * c->d);
  if (causal != 0 && causal != 1) return fail(BSVA_ERR_INVALID_ARG, "causal = %d; use 0 or 1", causal);
  if (window < 0 || (window > 0 && !causal))
    return fail(BSVA_ERR_INVALID_ARG, "window = %d must be >= 0, and 0 without causal", window);
  if (std::isnan(softmax_scale) || std::isinf(softmax_scale))
    return fail(BSVA_ERR_INVALID_ARG, "softmax_scale must be finite");
  if (lse && !aligned(lse, 4)) return fail(BSVA_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  if (b->T > 0) { REQUIRE_PTR(q, 16); REQUIRE_PTR(out, 16); }
  const size_t rows = size_t(b->T) * Hq;
  const PagedWs w(make_plan(b->S, c->H, Hq / c->H, b->max_q, b->max_kv, c->d, c->dtype == BSVA_KV_INT8).cap, rows, c->d);
  if ((rc = check_workspace(workspace, workspace_bytes, w.total))) return rc;
  if ((rc = check_device())) return rc;
  if (b->T == 0) return ok();
  PagedArgs a{};
  fill_cache(a, c, b);
  a.G = Hq / c->H;
  a.q = static_cast<const __nv_bfloat16*>(q); a.q_tok = q_stride; a.q_head = c->d;
  a.out = static_cast<__nv_bfloat16*>(out); a.o_tok = (long long)Hq * c->d; a.o_head = c->d;
  a.lse = lse;
  a.out_rows = (long long)rows;
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf(float(c->d));
  a.scale_log2 = scale * 1.4426950408889634f;
  a.causal = causal;
  a.window = window >= b->max_kv ? 0 : window;   // one that hides no key is none
  // keys a sequence's rows can see: with a window, its width and the chunk's length (from a multiple of 16)
  const long long reach = a.window ? (long long)a.window + b->max_q + 15 : b->max_kv;
  const Plan p = make_plan(b->S, c->H, a.G, b->max_q, reach < b->max_kv ? int(reach) : b->max_kv, c->d, c->dtype == BSVA_KV_INT8);
  return run_paged(a, c->dtype == BSVA_KV_INT8, p, w, workspace,
                   reinterpret_cast<cudaStream_t>(stream));
}

static int check_cross(const bsva_shape& s, int Hkv) {
  int rc;
  if ((rc = check_shape(s))) return rc;
  return check_heads(s.H, Hkv, s.Lq);
}

size_t bsva_cross_attn_workspace_bytes(bsva_shape s, int Hkv) {
  s.n_prefix = 0;
  if (check_cross(s, Hkv)) return 0;
  return PagedWs(make_plan(s.B, Hkv, s.H / Hkv, s.Lq, s.Lk, s.d, false).cap, size_t(s.B) * s.H * s.Lq, s.d).total;
}

int cross_attn_fwd(bsva_shape s, int Hkv, const void* q, const void* k, const void* v, const int32_t* k_len,
                   float softmax_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                   bsva_stream_t stream) {
  BSVA_RANGE("cross_attn_fwd");
  int rc;
  s.n_prefix = 0;
  if ((rc = check_cross(s, Hkv))) return rc;
  if (std::isnan(softmax_scale) || std::isinf(softmax_scale))
    return fail(BSVA_ERR_INVALID_ARG, "softmax_scale must be finite");
  REQUIRE_PTR(q, 16); REQUIRE_PTR(k, 16); REQUIRE_PTR(v, 16); REQUIRE_PTR(out, 16);
  if (k_len && !aligned(k_len, 4)) return fail(BSVA_ERR_INVALID_ARG, "k_len is not 4-byte aligned");
  if (lse && !aligned(lse, 4)) return fail(BSVA_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  const Plan p = make_plan(s.B, Hkv, s.H / Hkv, s.Lq, s.Lk, s.d, false);
  const size_t rows = size_t(s.B) * s.H * s.Lq;
  const PagedWs w(p.cap, rows, s.d);
  if ((rc = check_workspace(workspace, workspace_bytes, w.total))) return rc;
  if ((rc = check_device())) return rc;
  PagedArgs a{};
  a.k = k; a.v = v; a.kv_len = k_len;
  a.n_pages = s.B; a.page_rows = s.Lk;
  a.S = s.B; a.Hkv = Hkv; a.G = s.H / Hkv; a.d = s.d; a.max_q = s.Lq; a.max_kv = s.Lk;
  a.wait_limit_ns = kWaitLimitNs;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.q_seq = a.o_seq = (long long)s.H * s.Lq * s.d;
  a.q_tok = a.o_tok = s.d;
  a.q_head = a.o_head = (long long)s.Lq * s.d;
  a.lse = lse;
  a.out_rows = (long long)rows;
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf(float(s.d));
  a.scale_log2 = scale * 1.4426950408889634f;
  return run_paged(a, false, p, w, workspace, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

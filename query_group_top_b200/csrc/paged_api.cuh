// Host side of the serving step over a paged cache: argument checks, the split
// of the key axis and the launches of pivot_qk_rope, pivot_paged_append,
// pivot_paged_attention and pivot_sparse_attention_paged.  Part of pivot.cu,
// whose helpers it uses.
#pragma once

namespace {

size_t dtype_bytes(int t) { return t == PIVOT_FP32 ? 4 : 2; }

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

// Opts a kernel into its dynamic shared memory, once per device.
template <auto Kernel>
int allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};   // a bit a device
  int dev = 0;
  CUDA_TRY(cudaGetDevice(&dev));
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return PIVOT_OK;
  CUDA_TRY(cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  done.fetch_or(bit, std::memory_order_relaxed);
  return PIVOT_OK;
}

// Heads that rope_kernel reads: 16-byte rows of d channels at strides that keep them aligned.
int head_rows(const char* name, const pivot_heads_t* h, int dtype, HeadRows* out) {
  *out = HeadRows{};
  if (!h) return PIVOT_OK;
  if (!h->data || h->heads < 1) return fail(PIVOT_ERR_INVALID_ARG, "%s: null data or no heads", name);
  const long long step = 16 / static_cast<long long>(dtype_bytes(dtype));
  if (!aligned16(h->data) || (h->weight && !aligned16(h->weight)) || h->token_stride % step || h->head_stride % step)
    return fail(PIVOT_ERR_INVALID_ARG, "%s: rows must start on 16-byte boundaries", name);
  *out = HeadRows{h->data, h->weight, h->token_stride, h->head_stride, h->heads};
  return PIVOT_OK;
}

int paged_rows(const int32_t* block_table, const int32_t* seqlens, const int32_t* cu, int T, int B, int g,
               int num_pages, int page_size, int max_pages, int max_seqlen, PagedRows* out) {
  if (!block_table || !seqlens) return fail(PIVOT_ERR_INVALID_ARG, "null block_table or seqlens");
  if (T < 1 || B < 1) return fail(PIVOT_ERR_INVALID_ARG, "need T >= 1 and B >= 1");
  if (!cu && (g < 1 || static_cast<long long>(B) * g != T))
    return fail(PIVOT_ERR_INVALID_ARG, "without cu offsets every sequence has g >= 1 new tokens and T = B * g");
  if (page_size < 1 || page_size > (1 << 24) || (page_size & (page_size - 1)) != 0)
    return fail(PIVOT_ERR_INVALID_ARG, "page_size must be a power of two (got %d)", page_size);
  if (static_cast<long long>(num_pages) * page_size >= (1ll << 31))
    return fail(PIVOT_ERR_INVALID_ARG, "the cache has too many rows");
  if (num_pages < 1 || max_pages < 1 || max_seqlen < 1)
    return fail(PIVOT_ERR_INVALID_ARG, "need num_pages, max_pages, max_seqlen >= 1");
  const int lg = log2_of(page_size);
  *out = PagedRows{block_table, seqlens, cu, B, T, g, max_pages, num_pages, lg, paged_max_len(max_pages, lg, max_seqlen)};
  return PIVOT_OK;
}

template <int D, class T>
int launch_rope(const RopeParams& rp, bool half, int grid, cudaStream_t st) {
  TraceScope tr(rp.kpages ? "paged_append" : "qk_rope", st);
  const size_t smem = static_cast<size_t>(rp.tokens_per_block) * (rp.rot / 2) * sizeof(float2);
  if (half)
    rope_kernel<D, true, T><<<grid, kRopeNT, smem, st>>>(rp);
  else
    rope_kernel<D, false, T><<<grid, kRopeNT, smem, st>>>(rp);
  CUDA_TRY(cudaGetLastError());
  return PIVOT_OK;
}

int run_rope(RopeParams rp, int dtype, const pivot_rope_t* rope, int d, cudaStream_t st) {
  if (d != 64 && d != 128) return fail(PIVOT_ERR_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", d);
  const bool turned = rope && rope->freqs;
  rp.rot = turned ? rope->rot_dim : 0;
  if (turned && (rp.rot < 16 || rp.rot > d || rp.rot % 16))
    return fail(PIVOT_ERR_INVALID_ARG, "rot_dim must be a multiple of 16 in [16, d] (got %d)", rp.rot);
  if (turned && rope->layout != PIVOT_ROPE_HALF && rope->layout != PIVOT_ROPE_INTERLEAVED)
    return fail(PIVOT_ERR_INVALID_ARG, "layout must be PIVOT_ROPE_HALF or PIVOT_ROPE_INTERLEAVED");
  if (turned && (reinterpret_cast<uintptr_t>(rope->freqs) & 7))
    return fail(PIVOT_ERR_INVALID_ARG, "freqs must be 8-byte aligned");
  rp.amplitude = turned ? static_cast<float>(rope->amplitude) : 1.f;
  rp.eps = rope ? static_cast<float>(rope->eps) : 0.f;
  rp.freqs = turned ? rope->freqs : nullptr;
  DeviceInfo* dev = nullptr;
  if (int rc = device_info(&dev)) return rc;
  rp.status = dev->status;
  // Tokens a block: its groups of d/16 lanes are dealt out to them, so that each
  // group finds some eight rows of a kind at its token.  Fewer tokens a block where
  // there are not enough for two blocks an SM: then latency counts, and a token's
  // heads go to as many groups as there are.
  const int most = std::max(rp.q.n, std::max(rp.k.n, rp.v.n)), groups = kRopeNT / (d / 16);
  int tb = 1;
  while (tb < 16 && tb < groups && 2 * tb * most <= 8 * groups) tb *= 2;
  while (tb > 1 && (rp.T + tb - 1) / tb < 2 * dev->sms) tb >>= 1;
  rp.tokens_per_block = tb;
  const int grid = (rp.T + tb - 1) / tb;
  const bool half = !turned || rope->layout == PIVOT_ROPE_HALF;
  if (dtype == PIVOT_BF16)
    return d == 128 ? launch_rope<128, __nv_bfloat16>(rp, half, grid, st) : launch_rope<64, __nv_bfloat16>(rp, half, grid, st);
  if (dtype == PIVOT_FP16)
    return d == 128 ? launch_rope<128, __half>(rp, half, grid, st) : launch_rope<64, __half>(rp, half, grid, st);
  return d == 128 ? launch_rope<128, float>(rp, half, grid, st) : launch_rope<64, float>(rp, half, grid, st);
}

int check_dtype(int dtype) {
  if (dtype != PIVOT_BF16 && dtype != PIVOT_FP16 && dtype != PIVOT_FP32)
    return fail(PIVOT_ERR_INVALID_ARG, "dtype must be PIVOT_BF16, PIVOT_FP16 or PIVOT_FP32");
  return PIVOT_OK;
}

// How many parts to cut `units` equal pieces of work of `len` keys into, where
// the device takes `slots` at a time: the rounds it takes times a part's time
// (its keys and a fixed part), and the join's (its launch, and the parts' rows
// through memory).  Times in ns.  A cut that leaves a last round nearly empty
// costs that round (64 sequences, 8 key heads, 8192 keys in 2 parts: 396 us; in
// 4: 350); a cut of many rows costs their parts' bytes.
struct PartCost {
  double per_key, fixed, join, join_per_part;
};
int best_parts(long long units, long long slots, long long len, const PartCost& c, long long most) {
  if (most <= 1) return 1;
  long long best = 1;
  double least = -1;
  // the least is at one part or at the most parts of some number of rounds
  for (long long r = 0; r <= 16; ++r) {
    const long long n = r == 0 ? 1 : std::min(most, r * slots / units);
    if (n < 1) continue;
    const double cost = static_cast<double>((units * n + slots - 1) / slots) *
                            (static_cast<double>((len + n - 1) / n) * c.per_key + c.fixed) +
                        (n > 1 ? c.join + static_cast<double>(n) * c.join_per_part : 0.0);
    if (least < 0 || cost < least) least = cost, best = n;
    if (n == most && r > 0) break;
  }
  return static_cast<int>(best);
}

// Which kernel takes a call of paged attention, and how the key axis is split.
struct AttendPlan {
  bool tiles;               // attend_tiles_kernel, else attend_rows_kernel
  int rows;                 // packed rows of a CTA
  int nsplit, min_chunk;
  int nsplit_many;          // of the sequences of many rows among those of few
  size_t part_lse, total;   // workspace: the parts' rows at 0, their lse at part_lse
};

constexpr int kMixedRows = 512;   // packed rows of a batch above which a long chunk in it is looked for
constexpr int kFewRows = 16;   // packed rows of a sequence up to which attend_rows_kernel takes it

AttendPlan plan_attend(int T, int B, int Hq, int Hk, int d, int max_seqlen, int sms) {
  AttendPlan a{};
  const long long rows = static_cast<long long>(T) * (Hq / Hk);
  // Up to 16 rows a sequence the matrix tiles gain nothing (two sequences of
  // 32000, 8 key heads: 56 us either way); at 24 they take 34 us for 61 (16
  // sequences of 2000).  Many short sequences cost either kernel its CTAs (1500
  // of 120 keys, 20 rows, 8 key heads of 64: 571 us by tiles, 728 by rows).
  a.tiles = rows > static_cast<long long>(kFewRows) * B;
  // The fewest keys that a part is worth: two key tiles (one: 24 us for 20 at some
  // sizes, 10 for 12 at others), or two steps of each of the few-row kernel's
  // warps (4 sequences of 640 keys, 128 heads over 16: 10.3 us; 256 keys: 11.9).
  a.min_chunk = a.tiles ? 256 : 128;
  const long long most = (max_seqlen + a.min_chunk - 1) / a.min_chunk;
  const double part_time = static_cast<double>(T) * Hq * d * 8 / 5000;   // a part of every row written and read
  auto units = [&](long long per_cta) { return (rows + B * per_cta - 1) / (B * per_cta) * B * Hk; };
  if (a.tiles) {
    // 1.4 us a key tile of both row tiles (1.1 at 64 channels), some 6 us before and after
    a.rows = 256;
    a.nsplit = best_parts(units(256), sms, max_seqlen,
                          PartCost{(d == 128 ? 1400. : 1100.) / 128, 6000, 4000, part_time}, most);
  } else {
    // a key's and its value's bytes at an SM's share of the memory's rate (41 bytes a ns of 6.1 TB/s), among its CTAs;
    // some 3 us before and after
    constexpr double kSmBytesPerNs = 41;
    a.rows = rows <= 8ll * B ? 8 : 16;
    const int per_sm = d == 128 ? KvRing<128>::PER_SM : KvRing<64>::PER_SM;
    a.nsplit = best_parts(units(a.rows), static_cast<long long>(per_sm) * sms, max_seqlen,
                          PartCost{4. * d / kSmBytesPerNs * per_sm, 3300, 4500, part_time}, most);
  }
  // the matrix tiles' launch for long chunks among single tokens, which may find
  // none: two parts at most, so that it is over soon
  a.nsplit_many = a.tiles ? a.nsplit : std::min(a.nsplit, 2);
  if (a.nsplit > 1) {
    const size_t parts = static_cast<size_t>(a.nsplit) * T * Hq;
    a.part_lse = up(parts * d * sizeof(float));
    a.total = a.part_lse + up(parts * sizeof(float));
  }
  return a;
}

template <int D>
int launch_attend_kernel(PagedAttendParams ap, bool tiles, int rows_per_cta, long long row_tiles, cudaStream_t st) {
  const long long ctas = row_tiles * ap.Hk * (tiles ? ap.nsplit_many : ap.nsplit);
  if (ctas >= (1ll << 31)) return fail(PIVOT_ERR_INVALID_ARG, "too many rows");
  ap.tiles = static_cast<int>(row_tiles);
  const unsigned grid = static_cast<unsigned>(ctas);
  if (tiles) {
    CUtensorMap mk{}, mv{};
    TraceScope tr("attend_tiles", st);
    if (ap.rows.log2_page < 3) {
      if (int rc = allow_smem<attend_tiles_kernel<D, true>>(TcCfg<D>::SMEM)) return rc;
      attend_tiles_kernel<D, true><<<grid, TcCfg<D>::THREADS, TcCfg<D>::SMEM, st>>>(mk, mv, ap);
    } else {
      const int rows = ap.rows.num_pages << ap.rows.log2_page, box_rows = std::min(1 << ap.rows.log2_page, 128);
      if (int rc = make_rows_map(&mk, ap.kpages, rows, ap.Hk, ap.Hk, D, box_rows)) return rc;
      if (int rc = make_rows_map(&mv, ap.vpages, rows, ap.Hk, ap.Hk, D, box_rows)) return rc;
      if (int rc = allow_smem<attend_tiles_kernel<D, false>>(TcCfg<D>::SMEM)) return rc;
      attend_tiles_kernel<D, false><<<grid, TcCfg<D>::THREADS, TcCfg<D>::SMEM, st>>>(mk, mv, ap);
    }
  } else {
    TraceScope tr("attend_rows", st);
    if (rows_per_cta == 8) {
      if (int rc = allow_smem<attend_rows_kernel<D, 1>>(KvRing<D>::SMEM)) return rc;
      attend_rows_kernel<D, 1><<<grid, 128, KvRing<D>::SMEM, st>>>(ap);
    } else {
      if (int rc = allow_smem<attend_rows_kernel<D, 2>>(KvRing<D>::SMEM)) return rc;
      attend_rows_kernel<D, 2><<<grid, 128, KvRing<D>::SMEM, st>>>(ap);
    }
  }
  CUDA_TRY(cudaGetLastError());
  return PIVOT_OK;
}

// most_new: with cu, a bound on a sequence's new tokens, 0 unknown.
template <int D>
int launch_attend(PagedAttendParams ap, const AttendPlan& pl, int most_new, cudaStream_t st) {
  const long long packed = static_cast<long long>(ap.rows.T) * ap.grp, B = ap.rows.B;
  ap.over = 0;
  ap.upto = 0x7FFFFFFF;
  ap.many = pl.tiles ? -1 : 0x7FFFFFFF;   // one kernel takes every sequence
  if (!ap.rows.cu) {
    const long long per = (static_cast<long long>(ap.rows.g) * ap.grp + pl.rows - 1) / pl.rows;
    if (int rc = launch_attend_kernel<D>(ap, pl.tiles, pl.rows, B * per, st)) return rc;
  } else {
    // Few rows a sequence on average may still be one long chunk among many
    // single tokens: then the sequences are dealt out by their own rows, and
    // those of many go to the matrix tiles (a chunk of 512 tokens among 200
    // single ones over 4000 keys, 32 heads over 8: 632 us for 822; where there
    // is none, the launch costs some 4 us, which a bound on the tokens spares).
    // Below kMixedRows no chunk is long enough to need it.
    if (!pl.tiles && packed > kMixedRows && (most_new == 0 || static_cast<long long>(most_new) * ap.grp > kFewRows)) {
      ap.over = ap.many = kFewRows;
      if (int rc = launch_attend_kernel<D>(ap, true, 256, packed / 256 + std::min(B, packed / (kFewRows + 1)), st)) return rc;
      ap.over = 0;
      ap.upto = kFewRows;
    }
    if (int rc = launch_attend_kernel<D>(ap, pl.tiles, pl.rows, (packed + pl.rows - 1) / pl.rows + B, st)) return rc;
  }
  if (ap.nsplit > 1) {
    TraceScope tr("attend_join", st);
    cudaLaunchConfig_t cfg{};
    const long long rows = static_cast<long long>(ap.rows.T) * ap.Hq;
    // four warps a row only where the rows leave the device room (1694 tokens of
    // 3 heads of 64 over 5882 keys: 31.6 us with them, 25.2 without)
    const bool wide = ap.nsplit > 4 && rows <= 1024;
    cfg.gridDim = dim3(static_cast<unsigned>(wide ? rows : (rows + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    CUDA_TRY(wide ? cudaLaunchKernelEx(&cfg, attend_join_kernel<D, true>, ap)
                  : cudaLaunchKernelEx(&cfg, attend_join_kernel<D, false>, ap));
  }
  CUDA_TRY(cudaGetLastError());
  return PIVOT_OK;
}

template <int D>
int launch_sparse_paged(AttendPagedParams ap, int B, int sms, cudaStream_t st) {
  const long long units = static_cast<long long>(B) * ap.g * ap.H, slots = static_cast<long long>(KvRing<D>::PER_SM) * sms;
  // CTAs that share a row's indices: the cluster of 1, 2, 4 or 8 with the least
  // rounds times length, a part's fixed cost being some 150 indices, and 100
  // more for the cluster's two barriers
  int parts = 1;
  long long least = -1;
  for (int n = 1; n <= 8; n *= 2) {
    const long long cost = (units * n + slots - 1) / slots * ((ap.top_k + n - 1) / n + 150) + (n > 1 ? 100 : 0);
    if (least < 0 || cost < least) least = cost, parts = n;
  }
  if (units * parts >= (1ll << 31)) return fail(PIVOT_ERR_INVALID_ARG, "B * g * H too large");
  ap.parts = parts;
  if (int rc = allow_smem<sparse_attention_paged_kernel<D>>(KvRing<D>::SMEM)) return rc;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(units * parts));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = KvRing<D>::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(parts);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = parts > 1 ? 1 : 0;
  TraceScope tr("sparse_attention_paged", st);
  CUDA_TRY(cudaLaunchKernelEx(&cfg, sparse_attention_paged_kernel<D>, ap));
  return PIVOT_OK;
}

}  // namespace

extern "C" {

int pivot_qk_rope(const pivot_heads_t* q, const pivot_heads_t* k, int dtype, const int32_t* positions,
                  const pivot_rope_t* rope, int T, int d, void* out_q, void* out_k, void* stream) {
  RopeParams rp{};
  if (int rc = check_dtype(dtype)) return rc;
  if (int rc = head_rows("q", q, dtype, &rp.q)) return rc;
  if (int rc = head_rows("k", k, dtype, &rp.k)) return rc;
  if (T < 1) return fail(PIVOT_ERR_INVALID_ARG, "T must be >= 1");
  if ((!q && !k) || (q && !out_q) || (k && !out_k)) return fail(PIVOT_ERR_INVALID_ARG, "null tensor pointer");
  if (!aligned16(out_q) || !aligned16(out_k)) return fail(PIVOT_ERR_INVALID_ARG, "outputs must be 16-byte aligned");
  if (rope && rope->freqs && !positions) return fail(PIVOT_ERR_INVALID_ARG, "a rotation needs positions");
  rp.positions = positions;
  rp.out_q = static_cast<uint16_t*>(out_q);
  rp.out_k = static_cast<uint16_t*>(out_k);
  rp.T = T;
  return run_rope(rp, dtype, rope, d, static_cast<cudaStream_t>(stream));
}

int pivot_paged_append(const pivot_heads_t* k, const pivot_heads_t* v, const pivot_heads_t* q, int dtype,
                       const pivot_rope_t* rope, const int32_t* block_table, const int32_t* seqlens,
                       const int32_t* cu_new, int T, int B, int d, int g, int num_pages, int page_size, int max_pages,
                       void* kpages, void* vpages, void* out_q, void* stream) {
  RopeParams rp{};
  rp.clear = (dtype & PIVOT_CLEAR_LEFT_OUT) != 0;
  dtype &= ~PIVOT_CLEAR_LEFT_OUT;
  if (int rc = check_dtype(dtype)) return rc;
  if (!k || !kpages || (v && !vpages) || (q && !out_q)) return fail(PIVOT_ERR_INVALID_ARG, "null tensor pointer");
  if (int rc = head_rows("k", k, dtype, &rp.k)) return rc;
  if (int rc = head_rows("v", v, dtype, &rp.v)) return rc;
  if (int rc = head_rows("q", q, dtype, &rp.q)) return rc;
  if (v && v->heads != k->heads) return fail(PIVOT_ERR_INVALID_ARG, "k and v must have the same heads");
  if (v && v->weight) return fail(PIVOT_ERR_INVALID_ARG, "values take no norm weight");
  if (!aligned16(kpages) || !aligned16(vpages) || !aligned16(out_q))
    return fail(PIVOT_ERR_INVALID_ARG, "outputs must be 16-byte aligned");
  if (int rc = paged_rows(block_table, seqlens, cu_new, T, B, g, num_pages, page_size, max_pages, 0x7FFFFFFF, &rp.rows))
    return rc;
  rp.out_q = static_cast<uint16_t*>(out_q);
  rp.kpages = static_cast<uint16_t*>(kpages);
  rp.vpages = static_cast<uint16_t*>(vpages);
  rp.T = T;
  return run_rope(rp, dtype, rope, d, static_cast<cudaStream_t>(stream));
}

size_t pivot_paged_attention_workspace_size(int T, int B, int Hq, int Hk, int d, int max_seqlen) {
  if (T < 1 || B < 1 || Hk < 1 || Hq < Hk || d < 1 || max_seqlen < 1) return 0;
  return plan_attend(T, B, Hq, Hk, d, max_seqlen, device_sms()).total;
}

int pivot_paged_attention(const void* q, const void* kpages, const void* vpages, const int32_t* block_table,
                          const int32_t* seqlens, const int32_t* cu_q, const pivot_attend_t* options, int T, int B,
                          int Hq, int Hk, int d, int g, int num_pages, int page_size, int max_pages, int max_seqlen,
                          void* out, float* out_lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !kpages || !vpages || !out) return fail(PIVOT_ERR_INVALID_ARG, "null tensor pointer");
  if (out == q) return fail(PIVOT_ERR_INVALID_ARG, "out must not be q");
  if (!aligned16(q) || !aligned16(kpages) || !aligned16(vpages) || !aligned16(out))
    return fail(PIVOT_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  if (d != 64 && d != 128) return fail(PIVOT_ERR_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", d);
  if (Hk < 1 || Hq < Hk || Hq % Hk)
    return fail(PIVOT_ERR_INVALID_ARG, "query heads must be a multiple of the key heads (Hq=%d, Hk=%d)", Hq, Hk);
  PagedAttendParams ap{};
  if (int rc = paged_rows(block_table, seqlens, cu_q, T, B, g, num_pages, page_size, max_pages, max_seqlen, &ap.rows))
    return rc;
  if (cu_q && g < 0) return fail(PIVOT_ERR_INVALID_ARG, "with cu_q, g bounds a sequence's new tokens (0: unknown)");
  if (max_seqlen >= (1 << 30)) return fail(PIVOT_ERR_INVALID_ARG, "max_seqlen too large");
  const double scale = options ? options->scale : 1.0 / sqrt(static_cast<double>(d));
  if (!(scale > 0.0) || !(scale < 1e30)) return fail(PIVOT_ERR_INVALID_ARG, "scale must be positive and finite");
  // rows of q are counted in 32 bits (more than 180 GB of them would pass that)
  if (static_cast<long long>(T) * Hq >= (1ll << 31) - 512) return fail(PIVOT_ERR_INVALID_ARG, "too many rows");
  DeviceInfo* dev = nullptr;
  if (int rc = device_info(&dev)) return rc;
  const AttendPlan pl = plan_attend(T, B, Hq, Hk, d, max_seqlen, dev->sms);
  if (pl.total > workspace_bytes || (pl.total && !workspace))
    return fail(PIVOT_ERR_WORKSPACE, "workspace too small: need %zu bytes, got %zu", pl.total, workspace_bytes);
  if (pl.total && (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0)
    return fail(PIVOT_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  ap.q = static_cast<const uint16_t*>(q);
  ap.kpages = static_cast<const uint16_t*>(kpages);
  ap.vpages = static_cast<const uint16_t*>(vpages);
  ap.Hq = Hq;
  ap.Hk = Hk;
  ap.grp = Hq / Hk;
  ap.self_key = options ? (options->include_self != 0) : 1;
  ap.nsplit = pl.nsplit;
  ap.nsplit_many = pl.nsplit_many;
  ap.min_chunk = pl.min_chunk;
  ap.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  ap.out = static_cast<uint16_t*>(out);
  ap.lse = out_lse;
  ap.part_o = pl.total ? static_cast<float*>(workspace) : nullptr;
  ap.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.part_lse);
  ap.status = dev->status;
  ap.wait_ns = wait_limit_ns();
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 128 ? launch_attend<128>(ap, pl, g, st) : launch_attend<64>(ap, pl, g, st);
}

int pivot_sparse_attention_paged(const void* q, const void* kpages, const void* vpages, const int32_t* block_table,
                                 const int32_t* seqlens, const int32_t* idx, int B, int H, int d, int g, int num_pages,
                                 int page_size, int max_pages, int top_k, float* out, void* stream) {
  if (!q || !kpages || !vpages || !idx || !out) return fail(PIVOT_ERR_INVALID_ARG, "null tensor pointer");
  if (!aligned16(q) || !aligned16(kpages) || !aligned16(vpages) || !aligned16(idx) || !aligned16(out))
    return fail(PIVOT_ERR_INVALID_ARG, "tensor pointers must be 16-byte aligned");
  if (d != 64 && d != 128) return fail(PIVOT_ERR_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", d);
  if (B < 1 || g < 1 || H < 1 || top_k < 1) return fail(PIVOT_ERR_INVALID_ARG, "need B, g, H, top_k >= 1");
  // places in a row are counted in 32 bits, a CTA's stride past the last one included
  if (top_k > (1 << 30)) return fail(PIVOT_ERR_INVALID_ARG, "top_k must be at most 2^30 (got %d)", top_k);
  if (static_cast<double>(B) * g * H >= 2147483648.0) return fail(PIVOT_ERR_INVALID_ARG, "B * g * H too large");
  AttendPagedParams ap{};
  if (int rc = paged_rows(block_table, seqlens, nullptr, B * g, B, g, num_pages, page_size, max_pages, 0x7FFFFFFF, &ap.rows))
    return rc;
  DeviceInfo* dev = nullptr;
  if (int rc = device_info(&dev)) return rc;
  ap.q = static_cast<const uint16_t*>(q);
  ap.kpages = static_cast<const uint16_t*>(kpages);
  ap.vpages = static_cast<const uint16_t*>(vpages);
  ap.idx = idx;
  ap.out = out;
  ap.H = H;
  ap.g = g;
  ap.top_k = top_k;
  ap.scale_log2 = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(d)));
  ap.status = dev->status;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 128 ? launch_sparse_paged<128>(ap, B, dev->sms, st) : launch_sparse_paged<64>(ap, B, dev->sms, st);
}

}  // extern "C"

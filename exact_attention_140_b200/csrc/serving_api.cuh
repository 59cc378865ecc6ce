// serving_api.cuh -- host side of the serving operators: argument checks,
// choice of kernel and of the key windows, launches.  Part of attn_api.cu (it
// uses that file's device state, map cache and log).
#pragma once

namespace attn {
namespace {

bool head_size_ok(int d) { return d == 64 || d == 128 || d == 256; }

// Checks of a cache description; its pointers only where it has pages.
int check_cache(const attn_kv_cache_t* c) {
  if (c == nullptr || c->n_pages < 0 || c->Hkv < 1) return ATTN_ERR_INVALID_ARG;
  if (c->dtype != ATTN_BF16 && c->dtype != ATTN_FP8_E4M3) return ATTN_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)) != 0) return ATTN_ERR_INVALID_ARG;
  if (!head_size_ok(c->d) || c->Hkv > 65535) return ATTN_ERR_UNSUPPORTED;
  if (c->n_pages == 0) return ATTN_OK;
  if (c->k_pages == nullptr || c->v_pages == nullptr) return ATTN_ERR_INVALID_ARG;
  const bool e4m3 = c->dtype == ATTN_FP8_E4M3;
  if (e4m3 != (c->k_exp != nullptr) || e4m3 != (c->v_exp != nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}
int page_shift(const attn_kv_cache_t* c) {
  int s = 0;
  while ((1 << s) < c->page_size) ++s;
  return s;
}

// A [T, H, d] tensor with a token stride.
int check_rows(const void* x, int H, int d, long long stride) {
  if (x == nullptr || stride < (long long)H * d) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(x) || stride % 8 != 0) return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

int check_rope(const attn_rope_t* r, int d, const long long* positions) {
  if (r == nullptr || !std::isfinite(r->eps) || r->eps < 0.f || !std::isfinite(r->amplitude)) return ATTN_ERR_INVALID_ARG;
  if (r->interleaved != 0 && r->interleaved != 1) return ATTN_ERR_INVALID_ARG;
  if (r->rot_dim < 0 || r->rot_dim > d || r->rot_dim % 16 != 0) return ATTN_ERR_INVALID_ARG;
  if (r->rot_dim > 0 && (r->freqs == nullptr || positions == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(r->q_weight) || !aligned16(r->k_weight)) return ATTN_ERR_MISALIGNED;
  if (r->rot_dim > 0 && ((reinterpret_cast<uintptr_t>(r->freqs) | reinterpret_cast<uintptr_t>(positions)) & 7u) != 0)
    return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

void fill_rope(HeadRowsParams* p, const attn_rope_t* r, const long long* positions) {
  p->q_weight = static_cast<const __nv_bfloat16*>(r->q_weight);
  p->k_weight = static_cast<const __nv_bfloat16*>(r->k_weight);
  p->eps = r->eps;
  p->amplitude = r->amplitude;
  p->freqs = r->freqs;
  p->rot = r->rot_dim;
  p->interleaved = r->interleaved != 0;
  p->positions = positions;
}

// Tokens of a block: several in a long call (their weights, pointers and cosines
// are shared), one in a short one, whose rows are spread over blocks instead.
template <int D, bool INTERLEAVED>
int launch_head_rows_d(const HeadRowsParams& p, int mode, DeviceState* st, cudaStream_t s) {
  constexpr int NG = 256 / (D / 8);
  const int rows = p.Hq + p.Hkv + (mode != kRowsDense ? p.Hkv : 0), sets = (rows + NG - 1) / NG;
  const long long fill = (long long)kHeadRowsBps * st->num_sms;  // blocks the GPU holds at once
  // the count whose blocks come out nearest to whole rounds of the GPU
  long long tokens = 1;
  double best = 0.0;
  for (long long n = kHeadRowsMaxTokens; n >= 1; --n) {
    const long long b = (p.T + n - 1) / n;
    const double even = (double)p.T / (double)(n * ((b + fill - 1) / fill) * fill);
    if (even > best + 0.02) {
      best = even;
      tokens = n;
    }
  }
  const long long gx = (p.T + tokens - 1) / tokens;
  long long gy = fill / gx;
  gy = gy < 1 ? 1 : (gy > sets ? sets : gy);
  const dim3 grid((unsigned)gx, (unsigned)gy);
  ATTN_LOGF("attn: head_rows_kernel<%d, %s, %d> grid=(%u,%u) block=256 T=%lld tokens=%lld Hq=%d Hkv=%d rot=%d\n", D,
            INTERLEAVED ? "interleaved" : "half", mode, grid.x, grid.y, p.T, tokens, p.Hq, p.Hkv, p.rot);
  switch (mode) {
    case kRowsDense: head_rows_kernel<D, INTERLEAVED, kRowsDense><<<grid, 256, 0, s>>>(p, (int)tokens); break;
    case kRowsBf16Cache: head_rows_kernel<D, INTERLEAVED, kRowsBf16Cache><<<grid, 256, 0, s>>>(p, (int)tokens); break;
    default: head_rows_kernel<D, INTERLEAVED, kRowsE4m3Cache><<<grid, 256, 0, s>>>(p, (int)tokens); break;
  }
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
int launch_head_rows(HeadRowsParams& p, int d, long long T, int mode, DeviceState* st, cudaStream_t s) {
  if (p.Hq + p.Hkv == 0) return ATTN_OK;
  p.T = T;
  switch (d) {
    case 64: return p.interleaved ? launch_head_rows_d<64, true>(p, mode, st, s) : launch_head_rows_d<64, false>(p, mode, st, s);
    case 128: return p.interleaved ? launch_head_rows_d<128, true>(p, mode, st, s) : launch_head_rows_d<128, false>(p, mode, st, s);
    default: return p.interleaved ? launch_head_rows_d<256, true>(p, mode, st, s) : launch_head_rows_d<256, false>(p, mode, st, s);
  }
}

template <int D, bool E4M3>
int launch_kv_read(const KvReadParams& p, cudaStream_t s) {
  const long long blocks = (p.T + 7) / 8;  // a warp per token
  if (blocks > 0x7FFFFFFFll) return ATTN_ERR_UNSUPPORTED;
  ATTN_LOGF("attn: kv_read_kernel<%d, %s> grid=(%lld) block=256 T=%lld Hkv=%d\n", D, E4M3 ? "e4m3" : "bf16", blocks, p.T,
            p.Hkv);
  kv_read_kernel<D, E4M3><<<(unsigned)blocks, 256, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int launch_kv_read_cache(KvReadParams& p, const attn_kv_cache_t* cache, const int* table, int table_width, int n_seqs,
                         void* k, void* v, DeviceState* st, cudaStream_t s) {
  p.k_pages = cache->k_pages;
  p.v_pages = cache->v_pages;
  p.k_exp = cache->k_exp;
  p.v_exp = cache->v_exp;
  p.n_pages = cache->n_pages;
  p.page_shift = page_shift(cache);
  p.Hkv = cache->Hkv;
  p.n_seqs = n_seqs;
  p.table_width = table_width;
  p.table = table;
  p.k = static_cast<__nv_bfloat16*>(k);
  p.v = static_cast<__nv_bfloat16*>(v);
  p.err = st->err;
  const bool e4m3 = cache->dtype == ATTN_FP8_E4M3;
  switch (cache->d) {
    case 64: return e4m3 ? launch_kv_read<64, true>(p, s) : launch_kv_read<64, false>(p, s);
    case 128: return e4m3 ? launch_kv_read<128, true>(p, s) : launch_kv_read<128, false>(p, s);
    default: return e4m3 ? launch_kv_read<256, true>(p, s) : launch_kv_read<256, false>(p, s);
  }
}

// ---------------------------------------------------------------- paged attention
// How a paged call runs.  Few rows per sequence: paged_fwd_kernel, `size` its
// block configuration, `blocks` its grid.  More (items > 0): the tcgen05 kernel
// over items, each sequence's keys cut into n_windows windows where the items are
// few, or over pieces of items of equal cost in sum.
// expand > 0: an e4m3 cache read back into bf16 rows first, `expand` of them for each
// sequence.
struct PagedPlan {
  int size, block_rows, unit, row_tiles, blocks;
  bool cluster, pieces;
  long long items;
  int window, n_windows, expand;
};
long long ragged_max_items(long long Tq, long long n_seqs, int Hq, int Hkv, int block_rows);
int ragged_block_rows(int d, bool prompts);
int ragged_rows_per_token(int Hq, int Hkv);
long long ragged_plan_bytes(long long n_seqs, long long items, int nh);

constexpr int kSms = 148;  // SMs of a B200: the grids and their workspace go by it
constexpr int kPieceBlocks = 2 * kSms;  // with more blocks than that whole items are as good
// Rows of a block: one tile of 8 rows a warp, then two where the accumulators fit
// (d = 256: one), then more warps along the rows.
constexpr int kPagedSizes = 4;
int paged_block_rows(int d, int size) { return size == 0 ? 8 : (d == 256 ? 8 : 16) << (size - 1); }
template <int D, bool E4M3, int SIZE>
using PagedCfgOf = PagedCfg<D, E4M3, (SIZE == 0 || D == 256) ? 1 : 2, SIZE <= 1 ? 1 : (SIZE == 2 ? 2 : 4)>;
struct PagedGeometry {
  int unit, blocks_per_sm;  // keys of a unit; blocks that share an SM
};
template <int D, bool E4M3>
PagedGeometry paged_geometry(int size) {
  constexpr PagedGeometry b[kPagedSizes] = {{PagedCfgOf<D, E4M3, 0>::TK, PagedCfgOf<D, E4M3, 0>::BPS},
                                            {PagedCfgOf<D, E4M3, 1>::TK, PagedCfgOf<D, E4M3, 1>::BPS},
                                            {PagedCfgOf<D, E4M3, 2>::TK, PagedCfgOf<D, E4M3, 2>::BPS},
                                            {PagedCfgOf<D, E4M3, 3>::TK, PagedCfgOf<D, E4M3, 3>::BPS}};
  return b[size];
}
PagedGeometry paged_geometry(int d, bool e4m3, int size) {
  switch (d) {
    case 64: return e4m3 ? paged_geometry<64, true>(size) : paged_geometry<64, false>(size);
    case 128: return e4m3 ? paged_geometry<128, true>(size) : paged_geometry<128, false>(size);
    default: return e4m3 ? paged_geometry<256, true>(size) : paged_geometry<256, false>(size);
  }
}

constexpr long long kExpandBytes = 1ll << 30;  // of workspace for expanded keys and values, at most

// Whole items, key windows or pieces, by an estimate in us from what the host
// knows.  A block takes 16 ns a key (21 at d = 256) and 9.6 us besides.  Windows
// (one: whole items): the waves of blocks, and writing and merging the partial
// rows (4 TB/s, 5 us to begin with); with equal lengths they fit, and need no list.
// Pieces: the mean of an SM, 24 us of fixed costs and the list, two partial blocks an
// SM, and the look-ups of the merge.  From two waves on the mean of a causal chunk
// counts; the sequences of a batch differ, so less than the longest on average is
// assumed, and that long and short blocks pair off in part.
// Measured, us by windows / by pieces / by the estimates (32/8 heads of 128, bf16,
// one call after another): 1 x 8192 keys, 2048 new tokens 240 / 287 / 248, 272; 4 x up
// to 12000, 256 tokens 204 / 148 / 202, 172; the same, 512 tokens 302 / 272 / 340, 283;
// 1 x 32768, 256 tokens 156 / 155 / 154, 160; the same, 2048 tokens 991 / 950 / 1035, 952.
// With many items pieces gain nothing, and those of one head drift apart and read its
// keys from HBM more often: 4 x up to 8192, 2048 tokens 501 / 571.
void plan_long(PagedPlan* pl, long long blocks, int Tq, int n_seqs, int max_q, int Hq, int max_kv, int block_rows, int d) {
  const double ns = d == 256 ? 0.021 : 0.016, mean_kv = max_kv - 0.5 * (max_q < max_kv ? max_q : max_kv);
  long long want = 1;
  double best = 0.0;
  for (long long n = 1; n <= 16 && (n == 1 || max_kv / n >= 512); ++n) {
    const long long waves = (blocks * n + kSms - 1) / kSms;
    const double keys = (waves == 1 ? max_kv : mean_kv * (n_seqs > 1 ? 0.85 : 1.0)) / (double)n;
    const double t = waves * (keys * ns + 9.6) + (n == 1 ? 0.0 : 5.0 + 2.0 * n * Tq * Hq * d * 4 / 4e6);
    if (n == 1 || t < best) {
      best = t;
      want = n;
    }
  }
  const double mean = blocks * mean_kv * (n_seqs > 1 ? 0.75 : 1.0) / kSms;
  const double pieces = (mean < 512.0 ? 512.0 : mean) * ns + 24.0 + 2.0 * 2 * kSms * block_rows * d * 4 / 4e6 +
                        5e-4 * Tq * Hq;
  pl->n_windows = 1;
  if (blocks <= kPieceBlocks && pl->items <= kPieceItems && n_seqs <= kPieceSeqs && pieces < best) {
    pl->pieces = true;
    return;
  }
  const long long w = (((long long)max_kv + want - 1) / want + 127) / 128 * 128;
  pl->window = (int)(w < 128 ? 128 : w);
  if (max_kv > pl->window) pl->n_windows = (int)(((long long)max_kv + pl->window - 1) / pl->window);
}
PagedPlan paged_plan(const attn_kv_cache_t* c, int Tq, int n_seqs, int max_q, int Hq, int max_kv) {
  PagedPlan pl = {};
  const int Hkv = c->Hkv;
  const long long rows = (long long)max_q * (Hq / Hkv);
  if (rows > 64 && c->n_pages > 0) {
    pl.items = ragged_max_items(Tq, n_seqs, Hq, Hkv, ragged_block_rows(c->d, false));
    const int g = ragged_rows_per_token(Hq, Hkv), rows_block = ragged_block_rows(c->d, false);
    // blocks: known where every sequence has max_q tokens
    long long n_items = (long long)n_seqs * max_q == Tq ? (long long)n_seqs * (((long long)max_q * g + rows_block - 1) / rows_block)
                                                        : (long long)Tq * g / rows_block + (n_seqs + 1) / 2;
    n_items = n_items < n_seqs ? n_seqs : (n_items > pl.items ? pl.items : n_items);
    plan_long(&pl, n_items * (g > 1 ? Hkv : Hq), Tq, n_seqs, max_q, Hq, max_kv, rows_block, c->d);
    // Codes expanded once for all query blocks, or by every block for itself, by the
    // rows of a sequence.  Measured on 4 sequences of up to 8192 keys, us by blocks /
    // with the pass: d = 128 (32/8 heads) 512 rows 114 / 128, 1024 rows 182 / 179,
    // 4096 rows 464 / 394; d = 256 (16/8) 256 rows 167 / 170, 512 rows 297 / 230;
    // d = 64 (12/12) 2048 rows 237 / 261.  2048 tokens over 32768 of 32/8 x 128: 1339 /
    // 1029.
    const int expand_from = c->d == 64 ? INT_MAX : (c->d == 128 ? 1024 : 512);
    const long long pad = ((long long)max_kv + 127) / 128 * 128;
    if (c->dtype == ATTN_FP8_E4M3 && rows >= expand_from &&
        n_seqs * pad * Hkv * c->d * 4 <= kExpandBytes && n_seqs * pad <= 0x7FFFFFFFll)
      pl.expand = (int)pad;
    return pl;
  }
  while (pl.size < kPagedSizes - 1 && paged_block_rows(c->d, pl.size) < rows) ++pl.size;
  pl.block_rows = paged_block_rows(c->d, pl.size);
  const PagedGeometry ge = paged_geometry(c->d, c->dtype == ATTN_FP8_E4M3, pl.size);
  pl.unit = ge.unit;
  pl.row_tiles = (int)((rows + pl.block_rows - 1) / pl.block_rows);
  const long long units = max_kv > pl.unit ? ((long long)max_kv + pl.unit - 1) / pl.unit : 1;  // of a segment
  const long long segments = (long long)n_seqs * pl.row_tiles * Hkv, most = (long long)kSms * ge.blocks_per_sm;
  // a cluster per segment where the clusters fit the GPU at once and their blocks
  // have no more than a few units each
  pl.cluster = units > 1 && units <= 4 * kPagedCluster && segments * kPagedCluster <= most;
  if (pl.cluster)
    pl.blocks = (int)segments * kPagedCluster;
  else
    pl.blocks = (int)(segments * units < most ? segments * units : most);
  return pl;
}
// The list of pieces and what long_combine_kernel finds them by.
struct PieceSpace {
  long long pieces, list, lin, first;  // entries of the list; bytes
};
PieceSpace piece_space(long long n_seqs, long long items, int nh) {
  PieceSpace s;
  s.pieces = items * nh + kSms;  // (every cut adds one)
  s.list = (4 * kPlanPiece * s.pieces + 15) / 16 * 16;
  s.lin = 8 * (items + 2);
  s.first = 4 * (n_seqs + 1);
  return s;
}
// Workspace.  paged_fwd_kernel: a long long per sequence and one, the partial
// rows, their LSE (nothing for clusters).  tcgen05: the list of items or pieces (and
// the places of their tiles), the pieces' or windows' partial rows, their LSE.
struct PagedSpace {
  long long head, o, lse, kv;  // bytes of each (kv: keys, and as much again for values)
  long long all() const { return head + o + lse + 2 * kv; }
};
PagedSpace paged_space(const PagedPlan& pl, long long Tq, long long n_seqs, long long Hq, long long Hkv, long long d) {
  auto round = [](long long b) { return (b + 255) / 256 * 256; };
  PagedSpace s = {};
  if (pl.items > 0) {
    const int nh = (int)(ragged_rows_per_token((int)Hq, (int)Hkv) > 1 ? Hkv : Hq);
    if (pl.pieces) {
      const PieceSpace ps = piece_space(n_seqs, pl.items, nh);
      s.head = round(ps.list + ps.lin + ps.first);
      s.o = 2ll * kSms * ragged_block_rows((int)d, false) * d * 4;
      s.lse = round(2ll * kSms * ragged_block_rows((int)d, false) * 4);
    } else {
      s.head = ragged_plan_bytes(n_seqs, pl.items, nh);
      if (pl.n_windows > 1) {
        s.o = round(pl.n_windows * Tq * Hq * d * 4);
        s.lse = round(pl.n_windows * Tq * Hq * 4);
      }
    }
    s.kv = n_seqs * pl.expand * Hkv * d * 2;
    return s;
  }
  if (pl.cluster) return s;
  s.head = round((n_seqs + 1) * 8);
  s.o = 2ll * pl.blocks * pl.block_rows * d * 4;
  s.lse = round(2ll * pl.blocks * pl.block_rows * 4);
  return s;
}

template <class Cfg>
int launch_paged_cfg(const PagedParams& p, const PagedPlan& pl, const attn_kv_cache_t* c, DeviceState* st, cudaStream_t s) {
  static std::atomic<unsigned> attr_set[kMaxDevices], attr_set_cluster[kMaxDevices];
  int rc = pl.cluster ? set_smem_once(paged_fwd_kernel<Cfg, true>, (int)Cfg::SMEM, attr_set_cluster, st)
                      : set_smem_once(paged_fwd_kernel<Cfg, false>, (int)Cfg::SMEM, attr_set, st);
  if (rc != ATTN_OK) return rc;
  CUtensorMap tk, tv;
  std::memset(&tk, 0, sizeof(tk));
  std::memset(&tv, 0, sizeof(tv));
  if (p.max_kv > 0) {  // (without a key the maps are never used)
    const auto encode = Cfg::E4M3 ? encode_pages_e4m3 : encode_pages;
    const int rows = c->page_size < Cfg::TK ? c->page_size : Cfg::TK;
    if (encode(&tk, c->k_pages, c->n_pages, c->page_size, c->Hkv, c->d, rows) != ATTN_OK ||
        encode(&tv, c->v_pages, c->n_pages, c->page_size, c->Hkv, c->d, rows) != ATTN_OK)
      return ATTN_ERR_CUDA;
  }
  ATTN_LOGF("attn: paged_fwd_kernel<%d, %s, NT=%d RW=%d%s> grid=(%d) block=%d smem=%u seqs=%d max_q=%d Hq=%d Hkv=%d\n",
            Cfg::D, Cfg::E4M3 ? "e4m3" : "bf16", Cfg::NT, Cfg::RW, pl.cluster ? " clusters" : "", pl.blocks, Cfg::NTHREADS,
            (unsigned)Cfg::SMEM, p.n_seqs, p.max_q, p.Hq, p.Hkv);
  if (!pl.cluster) {
    paged_fwd_kernel<Cfg, false><<<(unsigned)pl.blocks, Cfg::NTHREADS, Cfg::SMEM, s>>>(tk, tv, p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
  }
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = kPagedCluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)pl.blocks);
  cfg.blockDim = dim3(Cfg::NTHREADS);
  cfg.dynamicSmemBytes = Cfg::SMEM;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_fwd_kernel<Cfg, true>, tk, tv, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
template <int D, bool E4M3>
int launch_paged_size(const PagedParams& p, const PagedPlan& pl, const attn_kv_cache_t* c, DeviceState* st, cudaStream_t s) {
  switch (pl.size) {
    case 0: return launch_paged_cfg<PagedCfgOf<D, E4M3, 0>>(p, pl, c, st, s);
    case 1: return launch_paged_cfg<PagedCfgOf<D, E4M3, 1>>(p, pl, c, st, s);
    case 2: return launch_paged_cfg<PagedCfgOf<D, E4M3, 2>>(p, pl, c, st, s);
    default: return launch_paged_cfg<PagedCfgOf<D, E4M3, 3>>(p, pl, c, st, s);
  }
}
// A kernel that is launched while the one before it in the stream still runs and
// waits for that one's results on the device, so its launch overlaps it.
template <class... Args>
int launch_dependent(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
template <int D>
int launch_paged(const PagedParams& p, const PagedPlan& pl, const attn_kv_cache_t* c, DeviceState* st, cudaStream_t s) {
  const int rc = c->dtype == ATTN_FP8_E4M3 ? launch_paged_size<D, true>(p, pl, c, st, s)
                                           : launch_paged_size<D, false>(p, pl, c, st, s);
  if (rc != ATTN_OK || pl.cluster || p.max_kv <= pl.unit) return rc;  // (a segment of one unit is never shared)
  const long long blocks = ((long long)p.Tq * p.Hq + 7) / 8;
  ATTN_LOGF("attn: paged_combine_kernel<%d> grid=(%lld) block=256 Tq=%d Hq=%d\n", D, blocks, p.Tq, p.Hq);
  if (blocks > 0x7FFFFFFFll) return ATTN_ERR_UNSUPPORTED;
  return launch_dependent(paged_combine_kernel<D>, dim3((unsigned)blocks), 256, 0, s, p, pl.block_rows, pl.unit, pl.blocks);
}

// ---------------------------------------------------------------- packed sequences on tcgen05
// The long-range configurations over packed sequences (1) or a paged cache (2
// bf16, 3 e4m3).  All exponentials on the hardware unit: the software share's 1e-4
// would show in the LSE of a short sequence, and it loses a NaN score (4 x 4096
// tokens of 32/8 heads, causal: 568 us, with the share 555).
// The heads of a group are always stacked where the group divides the tile: a
// block then covers fewer tokens, which wastes less of a causal block's diagonal
// and of a short sequence, and a key tile is read once per group.
// Causal packed prompts at d = 64: blocks of one query tile, two sharing an SM,
// whose starts and ends overlap each other's work (prompts up to 1024, 12 heads: 32.5
// -> 29.9 us, up to 4096: 115 -> 107; not causal 167 -> 169, over a cache 136 -> 140).
template <bool C, int R> using CfgRagD64 = std::conditional_t<C && R == 1, FwdCfg<64, 128, 1, 2, 2, C, false, 0, 1, false, 1, true, false, R>,
                                                              FwdCfg<64, 128, 2, 3, 3, C, false, 0, 1, false, 1, true, false, R>>;
template <bool C, int R> using CfgRagD128 = FwdCfg<128, 128, 2, 2, 2, C, false, 0, 1, false, 1, true, false, R>;
template <bool C, int R> using CfgRagD256 = FwdCfg<256, 64, 1, 2, 2, C, false, 0, 2, false, 1, true, false, R>;

// Rows of a block (packed prompts: at least).
int ragged_block_rows(int d, bool prompts) { return d == 256 || (d == 64 && prompts) ? 128 : 256; }
int ragged_rows_per_token(int Hq, int Hkv) { return pack_factor(Hq, Hkv); }
// Items at most: every sequence may end in a block of one row.
long long ragged_max_items(long long Tq, long long n_seqs, int Hq, int Hkv, int block_rows) {
  const long long n = n_seqs < Tq ? n_seqs : Tq;
  return (Tq * ragged_rows_per_token(Hq, Hkv) + n * (block_rows - 1)) / block_rows;
}
constexpr long long kMaxItems = 1ll << 26;  // (item numbers times the ints of an item stay within 32 bits)
// Whether the items are listed ahead: with many sequences, or where an SM has more
// than one block to start (finding its item takes a block about 1 us, the list 5 us
// and a launch: 4 prompts of up to 100 tokens 26 -> 18 us a call without it).
bool ragged_listed(long long n_seqs, long long items, int nh) { return n_seqs > kPickSeqs || items * nh > kSms; }
long long ragged_plan_bytes(long long n_seqs, long long items, int nh) {
  return ragged_listed(n_seqs, items, nh) ? (4 * kPlanItem * items + 255) / 256 * 256 : 0;
}

struct RaggedCall {
  const void *q, *k, *v;
  void* o;
  float* lse;
  int Tq, Tk, n_seqs, max_q, Hq, Hkv, d;
  const int *cu_q, *cu_k, *kv_lens, *table;
  int table_width, max_kv;
  int seq_stride;  // packed keys whose sequence s starts at row s * seq_stride (kv_lens of them)
  long long q_stride, k_stride, v_stride;
  const attn_kv_cache_t* cache;  // paged
  bool causal;
  float scale;
  bool pieces;
  int n_windows, window;
  float *o_part, *lse_part;
  int* plan;
};

template <class Cfg>
int launch_ragged(const RaggedCall& c, DeviceState* st, cudaStream_t s) {
  static std::atomic<unsigned> attr_set[kMaxDevices];
  int rc = set_smem_once(attn_fwd_kernel<Cfg>, (int)Cfg::SMEM_BYTES, attr_set, st);
  if (rc != ATTN_OK) return rc;
  const int g = ragged_rows_per_token(c.Hq, c.Hkv);
  const long long items = ragged_max_items(c.Tq, c.n_seqs, c.Hq, c.Hkv, Cfg::BM * Cfg::NQT);
  const int nh = g > 1 ? c.Hkv : c.Hq;
  const PieceSpace ps = piece_space(c.n_seqs, items, nh);
  const long long blocks = c.pieces ? ps.pieces : items * nh * c.n_windows;
  if (blocks > 0x7FFFFFFFll) return ATTN_ERR_UNSUPPORTED;
  CUtensorMap tq, tk, tv;
  rc = g > 1 ? encode_packed_groups(&tq, c.q, c.Tq, c.Hq, g, c.d, c.q_stride, Cfg::BM)
             : encode_packed(&tq, c.q, c.Tq, c.Hq, c.d, c.q_stride, Cfg::BM);
  if (rc != ATTN_OK) return rc;
  if (Cfg::RAGGED == 1) {
    // (no key anywhere: the maps are never used, and a map of no rows cannot be made)
    if (c.Tk == 0) {
      tk = tv = tq;
    } else if (encode_packed(&tk, c.k, c.Tk, c.Hkv, c.d, c.k_stride, Cfg::BN) != ATTN_OK ||
               encode_packed(&tv, c.v, c.Tk, c.Hkv, c.d, c.v_stride, Cfg::BN) != ATTN_OK) {
      return ATTN_ERR_CUDA;
    }
  } else {
    const attn_kv_cache_t* ch = c.cache;
    const int rows = ch->page_size < Cfg::BN ? ch->page_size : Cfg::BN;
    const auto encode = Cfg::KV8 ? encode_pages_e4m3 : encode_pages;
    if (encode(&tk, ch->k_pages, ch->n_pages, ch->page_size, ch->Hkv, ch->d, rows) != ATTN_OK ||
        encode(&tv, ch->v_pages, ch->n_pages, ch->page_size, ch->Hkv, ch->d, rows) != ATTN_OK)
      return ATTN_ERR_CUDA;
  }
  PlanParams pp;
  pp.plan = c.pieces || ragged_listed(c.n_seqs, items, nh) ? c.plan : nullptr;
  pp.max_items = (int)items;
  pp.n_seqs = c.n_seqs;
  pp.Tq = c.Tq;
  pp.Tk = c.Tk;
  pp.max_q = c.max_q;
  pp.max_kv = c.max_kv;
  pp.cu_q = c.cu_q;
  pp.cu_k = c.cu_k;
  pp.kv_lens = c.kv_lens;
  pp.k_stride = c.seq_stride;
  pp.rows_per_token = g;
  pp.block_rows = Cfg::BM * Cfg::NQT;
  pp.bn = Cfg::BN;
  pp.causal = c.causal;
  pp.err = st->err;
  if (c.pieces) {
    PiecePlanParams pc;
    pc.seqs = pp;
    pc.max_pieces = (int)ps.pieces;
    pc.nh = nh;
    pc.runs = kSms;
    pc.min_share = 512 / Cfg::BN;
    pc.lin = reinterpret_cast<long long*>(reinterpret_cast<char*>(c.plan) + ps.list);
    pc.first = reinterpret_cast<int*>(reinterpret_cast<char*>(c.plan) + ps.list + ps.lin);
    ATTN_LOGF("attn: piece_plan_kernel grid=(1) block=%d seqs=%d items<=%lld\n", kPlanThreads, c.n_seqs, items);
    piece_plan_kernel<<<1, kPlanThreads, 0, s>>>(pc);
    if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  } else if (pp.plan != nullptr) {
    ATTN_LOGF("attn: ragged_plan_kernel grid=(1) block=%d seqs=%d items<=%lld\n", kPlanThreads, c.n_seqs, items);
    ragged_plan_kernel<<<1, kPlanThreads, 0, s>>>(pp);
    if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  }

  RaggedFwdParams p = {};
  p.o = c.o;
  p.lse = c.lse;
  p.B = 1;
  p.Hq = c.Hq;
  p.Hkv = c.Hkv;
  p.Nq = c.Tq;
  p.Nk = c.Tk;
  p.group = c.Hq / c.Hkv;
  p.nb = 1;
  p.nh = nh;
  p.pack = g;
  p.sl2 = c.scale * 1.4426950408889634f;
  p.n_splits = c.n_windows;
  p.kv_chunk = c.n_windows > 1 ? c.window : 0x7FFFFFFF;
  p.o_part = c.o_part;
  p.lse_part = c.lse_part;
  p.err = st->err;
  p.timeout_ns = timeout_ns();
  // heads whose keys and values fit about 48 MB of L2 run together, as causal attn_fwd launches
  const long long kv_head = 4ll * c.Tk * c.d / (g > 1 ? 1 : p.group);
  long long band = (48ll << 20) / (kv_head > 0 ? kv_head : 1);
  p.band = (int)(band < 1 ? 1 : (band > nh ? nh : band));
  p.rg.seqs = pp;
  p.rg.pieces = c.pieces;
  p.rg.table = c.table;
  p.rg.table_width = c.table_width;
  p.rg.page_shift = c.cache != nullptr ? page_shift(c.cache) : 0;
  p.rg.n_pages = c.cache != nullptr ? c.cache->n_pages : 0;
  p.rg.k_exp = c.cache != nullptr ? c.cache->k_exp : nullptr;
  p.rg.v_exp = c.cache != nullptr ? c.cache->v_exp : nullptr;
  const dim3 grid((unsigned)blocks);
  if (log_on()) {
    char extra[96];
    std::snprintf(extra, sizeof extra, " packed sequences%s%s windows=%d pack=%d band=%d",
                  Cfg::RAGGED == 1 ? "" : (Cfg::KV8 ? " (paged e4m3)" : " (paged)"), c.pieces ? " pieces" : "",
                  c.n_windows, g, p.band);
    log_launch<Cfg>("attn_fwd_kernel", grid, c.n_seqs, c.Hq, c.Hkv, c.Tq, c.Tk, extra);
  }
  if (pp.plan == nullptr) {
    attn_fwd_kernel<Cfg><<<grid, Cfg::NTHREADS, Cfg::SMEM_BYTES, s>>>(tq, tk, tv, p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
  }
  // (the launch overlaps the list's kernel, which the attention kernel waits for)
  return launch_dependent(attn_fwd_kernel<Cfg>, grid, Cfg::NTHREADS, Cfg::SMEM_BYTES, s, tq, tk, tv, (const RaggedFwdParams)p);
}
template <int R>
int launch_ragged_d(const RaggedCall& c, DeviceState* st, cudaStream_t s) {
  switch (c.d) {
    case 64: return c.causal ? launch_ragged<CfgRagD64<true, R>>(c, st, s) : launch_ragged<CfgRagD64<false, R>>(c, st, s);
    case 128:
      return c.causal ? launch_ragged<CfgRagD128<true, R>>(c, st, s) : launch_ragged<CfgRagD128<false, R>>(c, st, s);
    default:
      return c.causal ? launch_ragged<CfgRagD256<true, R>>(c, st, s) : launch_ragged<CfgRagD256<false, R>>(c, st, s);
  }
}

int check_paged_sizes(const attn_kv_cache_t* c, int Tq, int n_seqs, int max_q, int Hq, int max_kv) {
  int rc = check_cache(c);
  if (rc != ATTN_OK) return rc;
  if (Tq < 0 || n_seqs < 0 || Hq < 0 || max_kv < 0 || Hq % c->Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (Tq == 0 || n_seqs == 0 || Hq == 0) return -1;  // nothing to compute
  if (max_q < 1 || max_q > Tq) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

}  // namespace
}  // namespace attn

extern "C" {

int attn_rope_freqs(double* freqs, int rot_dim, double base, int kind, double factor, double trained_len,
                    double fast_turns, double slow_turns, float* amplitude) {
  if (freqs == nullptr || rot_dim < 2 || rot_dim > 65536 || rot_dim % 2 != 0) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(base) || !(base > 1.0) || !std::isfinite(factor) || !(factor >= 1.0)) return ATTN_ERR_INVALID_ARG;
  if (kind < ATTN_ROPE_PLAIN || kind > ATTN_ROPE_BANDS) return ATTN_ERR_INVALID_ARG;
  if (kind == ATTN_ROPE_NTK && rot_dim == 2 && factor > 1.0) return ATTN_ERR_INVALID_ARG;  // one pair: no slowest to stretch
  double low = 0.0, high = 0.0;  // BANDS: the pair indexes between which the frequencies are blended
  const double two_pi = 6.283185307179586476925;
  if (kind == ATTN_ROPE_BANDS) {
    if (!std::isfinite(trained_len) || !(trained_len > 0.0) || !std::isfinite(fast_turns) || !(slow_turns > 0.0) ||
        !(fast_turns > slow_turns))
      return ATTN_ERR_INVALID_ARG;
    // pair i turns trained_len * base^(-2i / rot_dim) / 2 pi times
    auto index_of = [&](double turns) {
      return rot_dim * std::log(trained_len / (turns * two_pi)) / (2.0 * std::log(base));
    };
    low = std::floor(index_of(fast_turns));
    high = std::ceil(index_of(slow_turns));
    low = low < 0.0 ? 0.0 : low;
    high = high > rot_dim / 2 - 1 ? rot_dim / 2 - 1 : high;
    if (high <= low) high = low + 1e-3;
  }
  const double b = kind == ATTN_ROPE_NTK && factor > 1.0 ? base * std::pow(factor, rot_dim / (rot_dim - 2.0)) : base;
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(b, -2.0 * i / rot_dim);
    if (kind == ATTN_ROPE_LINEAR) {
      freqs[i] = f / factor;
    } else if (kind == ATTN_ROPE_BANDS) {
      double slow = (i - low) / (high - low);  // share of the stretched frequency
      slow = slow < 0.0 ? 0.0 : (slow > 1.0 ? 1.0 : slow);
      freqs[i] = f - (f - f / factor) * slow;
    } else {
      freqs[i] = f;
    }
  }
  if (amplitude != nullptr) *amplitude = kind == ATTN_ROPE_BANDS ? (float)(1.0 + 0.1 * std::log(factor)) : 1.f;
  return ATTN_OK;
}

int attn_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, long long T, int Hq, int Hkv, int d,
                      long long q_stride, long long k_stride, long long q_out_stride, long long k_out_stride,
                      const long long* positions, const attn_rope_t* rope, void* stream) {
  if (T < 0 || Hq < 0 || Hkv < 0) return ATTN_ERR_INVALID_ARG;
  if (!head_size_ok(d) || T > 0x7FFFFFFFll || Hq > 65535 || Hkv > 65535) return ATTN_ERR_UNSUPPORTED;
  int rc = check_rope(rope, d, positions);
  if (rc != ATTN_OK) return rc;
  if (T == 0 || (Hq == 0 && Hkv == 0)) return ATTN_OK;
  if (Hq > 0 && ((rc = check_rows(q, Hq, d, q_stride)) != ATTN_OK || (rc = check_rows(q_out, Hq, d, q_out_stride)) != ATTN_OK))
    return rc;
  if (Hkv > 0 &&
      ((rc = check_rows(k, Hkv, d, k_stride)) != ATTN_OK || (rc = check_rows(k_out, Hkv, d, k_out_stride)) != ATTN_OK))
    return rc;
  int dev = 0;
  DeviceState* st = nullptr;
  if ((rc = device_state(&dev, &st)) != ATTN_OK) return rc;
  HeadRowsParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.Hq = Hq;
  p.Hkv = Hkv;
  fill_rope(&p, rope, positions);
  p.err = st->err;
  return launch_head_rows(p, d, T, kRowsDense, st, static_cast<cudaStream_t>(stream));
}

int attn_kv_write(const attn_kv_cache_t* cache, const void* k, const void* v, long long T, long long k_stride,
                  long long v_stride, const long long* slots, const attn_rope_t* rope, const long long* positions,
                  const void* q, void* q_out, int Hq, long long q_stride, long long q_out_stride, void* stream) {
  int rc = check_cache(cache);
  if (rc != ATTN_OK) return rc;
  if (T < 0 || Hq < 0) return ATTN_ERR_INVALID_ARG;
  if (T > 0x7FFFFFFFll || Hq > 65535) return ATTN_ERR_UNSUPPORTED;
  const int d = cache->d, Hkv = cache->Hkv;
  if (rope != nullptr && (rc = check_rope(rope, d, positions)) != ATTN_OK) return rc;
  if (rope == nullptr && Hq > 0) return ATTN_ERR_INVALID_ARG;  // queries only take part in the norm and rotation
  if (T == 0) return ATTN_OK;
  if ((rc = check_rows(k, Hkv, d, k_stride)) != ATTN_OK || (rc = check_rows(v, Hkv, d, v_stride)) != ATTN_OK) return rc;
  if (Hq > 0 && ((rc = check_rows(q, Hq, d, q_stride)) != ATTN_OK || (rc = check_rows(q_out, Hq, d, q_out_stride)) != ATTN_OK))
    return rc;
  if (slots == nullptr) return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(slots) & 7u) != 0) return ATTN_ERR_MISALIGNED;
  int dev = 0;
  DeviceState* st = nullptr;
  if ((rc = device_state(&dev, &st)) != ATTN_OK) return rc;
  HeadRowsParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.slots = slots;
  p.n_slots = (long long)cache->n_pages * cache->page_size;
  p.k_pages = cache->k_pages;
  p.v_pages = cache->v_pages;
  p.k_exp = cache->k_exp;
  p.v_exp = cache->v_exp;
  if (rope != nullptr) fill_rope(&p, rope, positions);
  p.err = st->err;
  return launch_head_rows(p, d, T, cache->dtype == ATTN_FP8_E4M3 ? kRowsE4m3Cache : kRowsBf16Cache, st,
                          static_cast<cudaStream_t>(stream));
}

int attn_kv_read(const attn_kv_cache_t* cache, const int* table, int table_width, const int* cu, int n_seqs, void* k,
                 void* v, long long T, void* stream) {
  int rc = check_cache(cache);
  if (rc != ATTN_OK) return rc;
  if (T < 0 || n_seqs < 0 || table_width < 0) return ATTN_ERR_INVALID_ARG;
  if (T == 0 || n_seqs == 0) return ATTN_OK;
  if (T > 0x7FFFFFFFll) return ATTN_ERR_UNSUPPORTED;
  if (cu == nullptr || k == nullptr || v == nullptr || (table_width > 0 && table == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) ||
      ((reinterpret_cast<uintptr_t>(cu) | reinterpret_cast<uintptr_t>(table)) & 3u) != 0)
    return ATTN_ERR_MISALIGNED;
  int dev = 0;
  DeviceState* st = nullptr;
  if ((rc = device_state(&dev, &st)) != ATTN_OK) return rc;
  KvReadParams p = {};
  p.cu = cu;
  p.T = T;
  return launch_kv_read_cache(p, cache, table, table_width, n_seqs, k, v, st, static_cast<cudaStream_t>(stream));
}

long long attn_fwd_varlen_workspace_bytes(int Tq, int n_seqs, int Hq, int Hkv, int d) {
  if (Tq < 0 || n_seqs < 0 || Hq < 0 || Hkv < 1 || Hq % Hkv != 0 || !head_size_ok(d)) return -1;
  if (Tq == 0 || n_seqs == 0 || Hq == 0) return 0;
  const long long items = ragged_max_items(Tq, n_seqs, Hq, Hkv, ragged_block_rows(d, true));
  const int nh = ragged_rows_per_token(Hq, Hkv) > 1 ? Hkv : Hq;
  return items > kMaxItems ? -1 : ragged_plan_bytes(n_seqs, items, nh);
}

int attn_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse, int Tq, int Tk, int n_seqs,
                    const int* cu_q, const int* cu_k, int Hq, int Hkv, int d, long long q_stride, long long k_stride,
                    long long v_stride, int causal, float scale, void* workspace, long long workspace_bytes,
                    void* stream) {
  if (Tq < 0 || Tk < 0 || n_seqs < 0 || Hq < 0 || Hkv < 0) return ATTN_ERR_INVALID_ARG;
  if ((causal != 0 && causal != 1) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (Tq == 0 || n_seqs == 0 || Hq == 0) return ATTN_OK;
  if (Hkv == 0 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (!head_size_ok(d) || Hq > 65535) return ATTN_ERR_UNSUPPORTED;
  if (cu_q == nullptr || cu_k == nullptr || o == nullptr) return ATTN_ERR_INVALID_ARG;
  int rc;
  if ((rc = check_rows(q, Hq, d, q_stride)) != ATTN_OK) return rc;
  if (Tk > 0 && ((rc = check_rows(k, Hkv, d, k_stride)) != ATTN_OK || (rc = check_rows(v, Hkv, d, v_stride)) != ATTN_OK))
    return rc;
  if (!aligned16(o) || ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(cu_q) |
                         reinterpret_cast<uintptr_t>(cu_k)) & 3u) != 0)
    return ATTN_ERR_MISALIGNED;
  const long long need = attn_fwd_varlen_workspace_bytes(Tq, n_seqs, Hq, Hkv, d);
  if (need < 0) return ATTN_ERR_UNSUPPORTED;
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return ATTN_ERR_MISALIGNED;
  }
  int dev = 0;
  DeviceState* st = nullptr;
  if ((rc = device_state(&dev, &st)) != ATTN_OK) return rc;
  RaggedCall c = {};
  c.q = q;
  c.k = k;
  c.v = v;
  c.o = o;
  c.lse = lse;
  c.Tq = Tq;
  c.Tk = Tk;
  c.n_seqs = n_seqs;
  c.max_q = Tq;
  c.Hq = Hq;
  c.Hkv = Hkv;
  c.d = d;
  c.cu_q = cu_q;
  c.cu_k = cu_k;
  c.q_stride = q_stride;
  c.k_stride = k_stride;
  c.v_stride = v_stride;
  c.causal = causal != 0;
  c.scale = scale;
  c.n_windows = 1;
  c.plan = static_cast<int*>(workspace);
  return launch_ragged_d<1>(c, st, static_cast<cudaStream_t>(stream));
}

long long attn_fwd_paged_workspace_bytes(const attn_kv_cache_t* cache, int Tq, int n_seqs, int max_q, int Hq,
                                         int max_kv) {
  const int rc = check_paged_sizes(cache, Tq, n_seqs, max_q, Hq, max_kv);
  if (rc == -1) return 0;
  if (rc != ATTN_OK) return -1;
  if (cache->n_pages == 0) max_kv = 0;
  const PagedPlan pl = paged_plan(cache, Tq, n_seqs, max_q, Hq, max_kv);
  if (pl.items > kMaxItems) return -1;
  return paged_space(pl, Tq, n_seqs, Hq, cache->Hkv, cache->d).all();
}

int attn_fwd_paged(const void* q, const attn_kv_cache_t* cache, void* o, float* lse, int Tq, int n_seqs, int max_q,
                   const int* cu_q, const int* table, int table_width, const int* kv_lens, int max_kv, int Hq,
                   long long q_stride, int causal, float scale, void* workspace, long long workspace_bytes,
                   void* stream) {
  int rc = check_paged_sizes(cache, Tq, n_seqs, max_q, Hq, max_kv);
  if (rc > 0) return rc;
  if ((causal != 0 && causal != 1) || !std::isfinite(scale) || table_width < 0) return ATTN_ERR_INVALID_ARG;
  if (rc == -1) return ATTN_OK;
  const int d = cache->d;
  if ((long long)table_width * cache->page_size < max_kv) return ATTN_ERR_INVALID_ARG;
  if (cu_q == nullptr && (long long)n_seqs * max_q != Tq) return ATTN_ERR_INVALID_ARG;
  if (kv_lens == nullptr || o == nullptr || (max_kv > 0 && table == nullptr)) return ATTN_ERR_INVALID_ARG;
  if ((rc = check_rows(q, Hq, d, q_stride)) != ATTN_OK) return rc;
  if (!aligned16(o) || ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(cu_q) |
                         reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(kv_lens)) & 3u) != 0)
    return ATTN_ERR_MISALIGNED;
  if (cache->n_pages == 0) max_kv = 0;  // there is nothing to read
  const PagedPlan pl = paged_plan(cache, Tq, n_seqs, max_q, Hq, max_kv);
  if (pl.items > kMaxItems) return ATTN_ERR_UNSUPPORTED;
  const PagedSpace sp = paged_space(pl, Tq, n_seqs, Hq, cache->Hkv, d);
  if (sp.all() > 0) {
    if (workspace == nullptr || workspace_bytes < sp.all()) return ATTN_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return ATTN_ERR_MISALIGNED;
  }
  int dev = 0;
  DeviceState* st = nullptr;
  if ((rc = device_state(&dev, &st)) != ATTN_OK) return rc;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  float* o_part = sp.o > 0 ? reinterpret_cast<float*>(ws + sp.head) : nullptr;
  float* lse_part = sp.o > 0 ? reinterpret_cast<float*>(ws + sp.head + sp.o) : nullptr;
  PagedSeqs seqs;
  seqs.Tq = Tq;
  seqs.n_seqs = n_seqs;
  seqs.max_q = max_q;
  seqs.max_kv = max_kv;
  seqs.cu_q = cu_q;
  seqs.kv_lens = kv_lens;
  if (pl.items > 0) {
    RaggedCall c = {};
    c.q = q;
    c.o = o;
    c.lse = lse;
    c.Tq = Tq;
    const long long cached = (long long)cache->n_pages * cache->page_size, reach = (long long)n_seqs * max_kv;
    c.Tk = (int)std::min<long long>(std::min(cached, reach), 0x7FFFFFFF);  // (for the L2 bands only)
    c.n_seqs = n_seqs;
    c.max_q = max_q;
    c.Hq = Hq;
    c.Hkv = cache->Hkv;
    c.d = d;
    c.cu_q = cu_q;
    c.kv_lens = kv_lens;
    c.table = table;
    c.table_width = table_width;
    c.max_kv = max_kv;
    c.q_stride = q_stride;
    c.cache = cache;
    c.causal = causal != 0;
    c.scale = scale;
    c.pieces = pl.pieces;
    c.n_windows = pl.n_windows;
    c.window = pl.window;
    c.o_part = o_part;
    c.lse_part = lse_part;
    c.plan = static_cast<int*>(workspace);
    if (pl.expand > 0) {
      char* kv = ws + sp.head + sp.o + sp.lse;
      KvReadParams rp = {};
      rp.lens = kv_lens;
      rp.stride = pl.expand;
      rp.T = (long long)n_seqs * pl.expand;
      if ((rc = launch_kv_read_cache(rp, cache, table, table_width, n_seqs, kv, kv + sp.kv, st, s)) != ATTN_OK) return rc;
      c.k = kv;
      c.v = kv + sp.kv;
      c.k_stride = c.v_stride = (long long)cache->Hkv * d;
      c.Tk = n_seqs * pl.expand;
      c.seq_stride = pl.expand;
      c.cache = nullptr;
      rc = launch_ragged_d<1>(c, st, s);
    } else {
      rc = cache->dtype == ATTN_FP8_E4M3 ? launch_ragged_d<3>(c, st, s) : launch_ragged_d<2>(c, st, s);
    }
    if (rc != ATTN_OK || (!pl.pieces && pl.n_windows == 1)) return rc;
    LongParams wp;
    static_cast<PagedSeqs&>(wp) = seqs;
    wp.o = static_cast<__nv_bfloat16*>(o);
    wp.lse = lse;
    wp.Hq = Hq;
    wp.window = pl.pieces ? 0 : pl.window;
    wp.rows_per_token = ragged_rows_per_token(Hq, cache->Hkv);
    wp.block_rows = ragged_block_rows(d, false);
    wp.nh = wp.rows_per_token > 1 ? cache->Hkv : Hq;
    wp.max_items = (int)pl.items;
    const PieceSpace ps = piece_space(n_seqs, pl.items, wp.nh);
    wp.lin = reinterpret_cast<const long long*>(ws + ps.list);
    wp.first = reinterpret_cast<const int*>(ws + ps.list + ps.lin);
    wp.o_part = o_part;
    wp.lse_part = lse_part;
    // a block per token, or more in a short call, whose heads are spread
    const int sets = (Hq + 7) / 8, spread = 4 * kSms / Tq;
    const dim3 grid((unsigned)Tq, (unsigned)(spread < 1 ? 1 : (spread > sets ? sets : spread)));
    ATTN_LOGF("attn: long_combine_kernel<%d> grid=(%u,%u) block=256 Tq=%d Hq=%d\n", d, grid.x, grid.y, Tq, Hq);
    switch (d) {
      case 64: return launch_dependent(long_combine_kernel<64>, grid, 256, 0, s, (const LongParams)wp);
      case 128: return launch_dependent(long_combine_kernel<128>, grid, 256, 0, s, (const LongParams)wp);
      default: return launch_dependent(long_combine_kernel<256>, grid, 256, 0, s, (const LongParams)wp);
    }
  }
  PagedParams p;
  static_cast<PagedSeqs&>(p) = seqs;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.Hq = Hq;
  p.Hkv = cache->Hkv;
  p.group = Hq / cache->Hkv;
  p.table = table;
  p.table_width = table_width;
  p.k_exp = cache->k_exp;
  p.v_exp = cache->v_exp;
  p.n_pages = cache->n_pages;
  p.page_shift = page_shift(cache);
  p.causal = causal;
  p.row_tiles = pl.row_tiles;
  p.sl2 = scale * 1.4426950408889634f;
  p.base = static_cast<long long*>(workspace);
  p.o_part = o_part;
  p.lse_part = lse_part;
  p.err = st->err;
  p.timeout_ns = timeout_ns();
  switch (d) {
    case 64: return launch_paged<64>(p, pl, cache, st, s);
    case 128: return launch_paged<128>(p, pl, cache, st, s);
    default: return launch_paged<256>(p, pl, cache, st, s);
  }
}

}  // extern "C"

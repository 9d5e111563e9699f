// train_ops.cuh -- C entry points of the standalone training operators on the
// caller's tensors: block-scaled FP8 quantization and product, cross entropy
// over a large vocabulary with its gradient, and gradient clipping over many
// tensors.  Included once, by gpt.cu, whose helpers
// (status codes, tensor maps, launches, GEMM dispatch) it uses.  Documented in
// include/gpt.h.
#pragma once
#include "clip.cuh"
#include "fp8_block.cuh"
#include "linear_ce.cuh"

// ======================================================================== device of a call
// A call runs on the device of its tensors, made current for the call and
// restored after; a stream of another device is refused by the launch.  (The
// stream itself cannot be asked for its device while it is being captured.)
// Every tensor has to be device memory of that device: a host pointer or
// another GPU's would fault in the kernel.
struct DeviceScope {
  int prev = -1, dev = -1;
  int enter(const char* fn, const void* p) {
    CUDA_TRY(cudaGetDevice(&prev));
    cudaPointerAttributes a;
    CUDA_TRY(cudaPointerGetAttributes(&a, p));
    if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged)
      return fail(GPT_ERR_ARG, "%s: a tensor is no device memory", fn);
    dev = a.type == cudaMemoryTypeDevice ? a.device : prev;
    if (dev != prev) CUDA_TRY(cudaSetDevice(dev));
    return GPT_OK;
  }
  int check(const char* fn, const char* what, const void* p) const {
    if (!p) return GPT_OK;
    cudaPointerAttributes a;
    CUDA_TRY(cudaPointerGetAttributes(&a, p));
    if (a.type == cudaMemoryTypeManaged) return GPT_OK;
    if (a.type != cudaMemoryTypeDevice || a.device != dev)
      return fail(GPT_ERR_ARG, "%s: %s is no memory of device %d", fn, what, dev);
    return GPT_OK;
  }
  ~DeviceScope() {
    if (dev >= 0 && dev != prev) cudaSetDevice(prev);
  }
};
#define ON_DEVICE_OF(fn, p) \
  DeviceScope scope_;       \
  TRY(scope_.enter(fn, p))
#define CHECK_PTR(fn, p) TRY(scope_.check(fn, #p, p))

// SMs of the device that p lies on (of the current one if p is no device memory,
// which ON_DEVICE_OF then refuses): a call's tile forms and its workspace are planned
// once, for the device that it will run on.
static int sms_of(const void* p) {
  cudaPointerAttributes a;
  int sms = 0;
  if (p && cudaPointerGetAttributes(&a, p) == cudaSuccess && a.type == cudaMemoryTypeDevice &&
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, a.device) == cudaSuccess)
    return sms;
  cudaGetLastError();
  return device_sms();
}

// A strided block of rows in memory, for the checks that a call's outputs do not
// overlap what it reads or writes elsewhere.
struct Span {
  const char* name;
  const void* p;
  long long rows;
  unsigned long long row_bytes, pitch;
};
static bool spans_overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || !a.row_bytes || !b.row_bytes) return false;
  const unsigned long long a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const unsigned long long a1 = a0 + (a.rows - 1) * a.pitch + a.row_bytes, b1 = b0 + (b.rows - 1) * b.pitch + b.row_bytes;
  if (a1 <= b0 || b1 <= a0) return false;
  // columns side by side in rows of one pitch do not touch
  if (a.pitch == b.pitch && a.pitch > 0) {
    const unsigned long long shift = b0 >= a0 ? (b0 - a0) % a.pitch : (a.pitch - (a0 - b0) % a.pitch) % a.pitch;
    if (shift >= a.row_bytes && shift + b.row_bytes <= a.pitch) return false;
  }
  return true;
}
// outputs first: each against everything behind it
static int check_spans(const char* fn, const Span* s, int outputs, int n) {
  for (int i = 0; i < outputs; ++i)
    for (int j = i + 1; j < n; ++j)
      if (spans_overlap(s[i], s[j])) return fail(GPT_ERR_ARG, "%s: %s overlaps %s", fn, s[i].name, s[j].name);
  return GPT_OK;
}

static bool misaligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }
static size_t dtype_size(int dtype) { return dtype == GPT_DTYPE_BF16 ? 2 : 4; }

// ======================================================================== block-scaled FP8
constexpr long long MAX_ROWS = 1LL << 30;  // rows or columns: tile coordinates stay in 32 bits
static long long scale_atoms(long long rows, long long cols) { return cdiv_ll(rows, 128) * cdiv_ll(cols, 512); }

extern "C" int fp8_block_scale_bytes(long long rows, long long cols, size_t* bytes) {
  if (!bytes || rows < 1 || cols < 1 || rows > MAX_ROWS || cols > MAX_ROWS)
    return fail(GPT_ERR_ARG, "fp8_block_scale_bytes: bad argument");
  *bytes = (size_t)scale_atoms(rows, cols) * 512;
  return GPT_OK;
}

template <typename T>
static int quantize_launch(const T* x, const QuantArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)std::min(a.tiles, QUANT_BLOCKS * device_sms());
  CUtensorMap map = {};
  ++g_launches;
  if (!misaligned(x, 16) && (a.ldx * sizeof(T)) % 16 == 0) {
    const uint64_t dims[2] = {(uint64_t)a.cols, (uint64_t)a.rows}, str[1] = {(uint64_t)a.ldx * sizeof(T)};
    const uint32_t box[2] = {128, 128};
    TRY(make_tmap_gen(&map, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, x,
                      dims, str, box, CU_TENSOR_MAP_SWIZZLE_NONE));
    TRY(allow_smem(fp8_block_quantize_kernel<T, true>, quant_smem<T>()));
    launch_pdl(fp8_block_quantize_kernel<T, true>, grid, QUANT_THREADS, quant_smem<T>(), st, map, x, a);
  } else {
    TRY(allow_smem(fp8_block_quantize_kernel<T, false>, quant_smem<T>()));
    launch_pdl(fp8_block_quantize_kernel<T, false>, grid, QUANT_THREADS, quant_smem<T>(), st, map, x, a);
  }
  LAUNCH_CHECK();
  return GPT_OK;
}

extern "C" int fp8_block_quantize(const void* x, int dtype, long long rows, long long cols, long long ldx, int square,
                                  uint8_t* q, long long ldq, uint8_t* scales, uint8_t* qt, long long ldqt,
                                  uint8_t* scales_t, void* stream) {
  const char* fn = "fp8_block_quantize";
  if (rows < 0 || cols < 0 || rows > MAX_ROWS || cols > MAX_ROWS || ldx < cols)
    return fail(GPT_ERR_ARG, "%s: bad argument", fn);
  if (dtype != GPT_DTYPE_F32 && dtype != GPT_DTYPE_BF16) return fail(GPT_ERR_ARG, "%s: bad dtype", fn);
  if (rows == 0 || cols == 0) return GPT_OK;  // whatever the addresses: an empty tensor has none
  if (!x || (!q && !qt)) return fail(GPT_ERR_ARG, "%s: bad argument", fn);
  if ((q && (!scales || ldq < cols || ldq % 16 || misaligned(q, 16) || misaligned(scales, 16))) ||
      (qt && (!scales_t || ldqt < rows || ldqt % 16 || misaligned(qt, 16) || misaligned(scales_t, 16))))
    return fail(GPT_ERR_ARG, "%s: codes need scales, a row pitch that covers a row in a multiple of 16 bytes, "
                             "and 16-byte aligned addresses", fn);
  if (misaligned(x, dtype_size(dtype))) return fail(GPT_ERR_ARG, "%s: x is not aligned to its elements", fn);
  const long long tiles = cdiv_ll(rows, 128) * cdiv_ll(cols, 128);
  const unsigned long long sb = scale_atoms(rows, cols) * 512, sbt = scale_atoms(cols, rows) * 512;
  const Span spans[] = {{"q", q, rows, (unsigned long long)cols, (unsigned long long)ldq}, {"scales", q ? scales : nullptr, 1, sb, 0},
                        {"qt", qt, cols, (unsigned long long)rows, (unsigned long long)ldqt},
                        {"scales_t", qt ? scales_t : nullptr, 1, sbt, 0},
                        {"x", x, rows, cols * dtype_size(dtype), ldx * dtype_size(dtype)}};
  TRY(check_spans(fn, spans, 4, 5));
  if (tiles > 0x7fffffffLL) return fail(GPT_ERR_ARG, "%s: too many elements", fn);
  cudaStream_t st = (cudaStream_t)stream;
  ON_DEVICE_OF(fn, x);
  CHECK_PTR(fn, q); CHECK_PTR(fn, scales); CHECK_PTR(fn, qt); CHECK_PTR(fn, scales_t);
  unsigned* err = nullptr;
  CUDA_TRY(cudaGetSymbolAddress((void**)&err, g_ngram_err));
  const QuantArgs a{rows, cols, ldx, q, ldq, scales, qt, ldqt, scales_t, square != 0, (int)tiles, err};
  if (dtype == GPT_DTYPE_BF16) return quantize_launch((const bf16*)x, a, st);
  return quantize_launch((const float*)x, a, st);
}

// Tile shape (256 or 128 columns, one SM or a pair) and K split of a
// block-scaled product: the form with the least estimated time,
//   fixed + waves * (k-blocks * c + e) + split,
// in microseconds measured on B200 (launch to launch, over 23 shapes from 1 x 8 x
// 16 to 8192 x 2048 x 16384; the choice is within 8% of the best form on each).  A
// pair costs 1 us more to start and, with its one accumulator, more between
// tiles, but moves fewer bytes per product once all SMs pull on L2: short
// products run on one SM per tile (4096 x 4096 x 128: 9.4 us against 10.6 on
// pairs, 200 x 768 x 768: 5.4 against 6.4), long ones on pairs (8192 x 2048 x 16384:
// 207 against 252).  A split adds its second launch and the partials' way
// through L2; K is split in whole scale atoms (4 k-blocks).
struct F8bPlan { int bn, cg, splits; };
static F8bPlan f8b_plan(int M, int N, int K, int sms) {
  const int quads = cdiv(K, 512), kb = cdiv(K, 128);
  F8bPlan best{128, 1, 1};
  double best_t = 1e300;
  for (int cg = 1; cg <= (M > 128 && gemm_pairs_enabled() ? 2 : 1); ++cg)
    for (int bn : {128, 256}) {
      if (bn == 256 ? N <= 128 : cg == 2) continue;  // pairs of 128 columns start later and load no less
      const long long tiles = (long long)cdiv(M, 128 * cg) * cdiv(N, bn), units = sms / cg;
      for (int s = 1; s <= (N % 4 == 0 && tiles < units ? std::min(32, quads) : 1); ++s) {
        const int share = cdiv(quads, s);
        if (cdiv(quads, share) != s) continue;  // the same shares as a smaller split
        const double busy = std::min(1.0, (double)(tiles * s) / units);  // share of the SMs that load
        const double c = cg == 2 ? 0.345 : bn == 256 ? 0.31 + 0.16 * busy : 0.30;
        const double e = cg == 2 ? 1.45 : bn == 256 ? 1.17 : 0.65;
        const double waves = (double)((tiles * s + units - 1) / units);
        const double t = (cg == 2 ? 4.2 : 3.2) + waves * (std::min(kb, 4 * share) * c + e) +
                         (s > 1 ? 1.5 + (double)s * M * N * 8e-7 : 0.0);
        if (t < best_t) { best = F8bPlan{bn, cg, s}; best_t = t; }
      }
    }
  return best;
}

template <int BN, int CG>
static int gemm_f8b_launch(int M, int N, int K, const uint8_t* A, long long lda, const uint8_t* sa, const uint8_t* B,
                           long long ldb, const uint8_t* sb, GemmEpilogue e, int splits, float* partial, unsigned* err,
                           cudaStream_t st) {
  CUtensorMap ta, tb, tcm;
  tc::Params p;
  const uint64_t da[2] = {(uint64_t)K, (uint64_t)M}, la[1] = {(uint64_t)lda};
  const uint32_t ba[2] = {128, tc::BM};
  TRY(make_tmap_gen(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, A, da, la, ba));
  const uint64_t db[2] = {(uint64_t)K, (uint64_t)N}, lb[1] = {(uint64_t)ldb};
  const uint32_t bb[2] = {128, (uint32_t)(BN / CG)};
  TRY(make_tmap_gen(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, B, db, lb, bb));
  const uint64_t dsa[2] = {128, (uint64_t)scale_atoms(M, K)}, dsb[2] = {128, (uint64_t)scale_atoms(N, K)}, ls[1] = {512};
  const uint32_t bsa[2] = {128, 1}, bsb[2] = {128, (BN + 127) / 128};
  TRY(make_tmap_gen(&p.tm_sfa, CU_TENSOR_MAP_DATA_TYPE_INT32, 2, sa, dsa, ls, bsa, CU_TENSOR_MAP_SWIZZLE_NONE));
  TRY(make_tmap_gen(&p.tm_sfb, CU_TENSOR_MAP_DATA_TYPE_INT32, 2, sb, dsb, ls, bsb, CU_TENSOR_MAP_SWIZZLE_NONE));
  p.a_atoms = cdiv(M, 128); p.b_atoms = cdiv(N, 128);
  p.a_skip = 0;
  p.M = M; p.N = N; p.K = K; p.batch = 1;
  p.a_kmajor = 1; p.b_kmajor = 1;
  p.m_tiles = cdiv(M, CG * tc::BM);
  p.n_tiles = cdiv(N, BN);
  p.group_m = (double)N * K > 32.0 * (1 << 20) ? std::min(p.m_tiles, 16) : 1;
  p.kb_total = cdiv(K, 128);
  p.kb_per_split = 4 * cdiv(cdiv(p.kb_total, 4), splits);
  p.splits = cdiv(p.kb_total, p.kb_per_split);
  p.k_chunk = cdiv(p.kb_per_split, cdiv(p.kb_per_split, 16));  // at most 2048 of K
  p.epi = e; p.partial = partial; p.err = err;
  const bool f32 = e.mode != EPI_STORE;
  if (p.splits > 1) {
    const uint64_t dims[3] = {(uint64_t)N, (uint64_t)M, (uint64_t)p.splits};
    const uint64_t str[2] = {(uint64_t)N * 4, (uint64_t)M * N * 4};
    const uint32_t box[3] = {32, 32, 1};
    TRY(make_tmap_gen(&tcm, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, partial, dims, str, box));
    TRY((gemm_tc_launch_k<BN, tc::K_PARTIAL, CG, 2>(ta, tb, tcm, tcm, p, st)));
    const long long total = (long long)M * N;
    const int blocks = (int)std::min<long long>((total + 255) / 256, 4LL * device_sms());
    ++g_launches; launch_pdl(splitk_reduce_kernel<bf16>, blocks, 256, 0, st, partial, p.splits, M, N, e);
    LAUNCH_CHECK();
    return GPT_OK;
  }
  const uint64_t dims[2] = {(uint64_t)N, (uint64_t)M}, str[1] = {(uint64_t)e.ldc * (f32 ? 4 : 2)};
  const uint32_t box[2] = {f32 ? 32u : 64u, 32};
  TRY(make_tmap_gen(&tcm, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, e.C, dims, str, box));
  if (!f32) return gemm_tc_launch_k<BN, tc::K_STORE, CG, 2>(ta, tb, tcm, tcm, p, st);
  if (e.beta) return gemm_tc_launch_k<BN, tc::K_REDUCE_F32, CG, 2>(ta, tb, tcm, tcm, p, st);
  return gemm_tc_launch_k<BN, tc::K_STORE_F32, CG, 2>(ta, tb, tcm, tcm, p, st);
}

extern "C" int gptx_gemm_fp8_block_workspace_bytes(int M, int N, int K, size_t* bytes) {
  if (!bytes || M < 1 || N < 1 || K < 1 || M > MAX_ROWS || N > MAX_ROWS || K > MAX_ROWS)
    return fail(GPT_ERR_ARG, "gptx_gemm_fp8_block_workspace_bytes: bad argument");
  const F8bPlan pl = f8b_plan(M, N, K, device_sms());
  *bytes = pl.splits > 1 ? (size_t)pl.splits * M * N * 4 : 0;
  return GPT_OK;
}

extern "C" int gptx_gemm_fp8_block_plan(int M, int N, int K, int* plan) {
  if (!plan || M < 1 || N < 1 || K < 1 || M > MAX_ROWS || N > MAX_ROWS || K > MAX_ROWS)
    return fail(GPT_ERR_ARG, "gptx_gemm_fp8_block_plan: bad argument");
  const F8bPlan pl = f8b_plan(M, N, K, device_sms());
  plan[0] = pl.bn; plan[1] = pl.cg; plan[2] = pl.splits;
  return GPT_OK;
}

extern "C" int gptx_gemm_fp8_block(int M, int N, int K, const uint8_t* A, long long lda, const uint8_t* scales_a,
                                   const uint8_t* B, long long ldb, const uint8_t* scales_b, int out_dtype, void* C,
                                   long long ldc, int beta, void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "gptx_gemm_fp8_block";
  if (M < 1 || N < 1 || K < 1 || M > MAX_ROWS || N > MAX_ROWS || K > MAX_ROWS || !A || !B || !C || !scales_a ||
      !scales_b || ldc < N || lda < K || ldb < K)
    return fail(GPT_ERR_ARG, "%s: bad argument", fn);
  if (out_dtype != GPT_DTYPE_F32 && out_dtype != GPT_DTYPE_BF16) return fail(GPT_ERR_ARG, "%s: bad out_dtype", fn);
  if (beta && out_dtype != GPT_DTYPE_F32) return fail(GPT_ERR_ARG, "%s: beta needs an fp32 output", fn);
  if ((lda | ldb) % 16 || (ldc * (long long)dtype_size(out_dtype)) % 16 || misaligned(A, 16) || misaligned(B, 16) ||
      misaligned(C, 16) || misaligned(scales_a, 16) || misaligned(scales_b, 16))
    return fail(GPT_ERR_ARG, "%s: addresses and row pitches must be multiples of 16 bytes", fn);
  cudaStream_t st = (cudaStream_t)stream;
  const F8bPlan pl = f8b_plan(M, N, K, sms_of(A));
  const size_t need = pl.splits > 1 ? (size_t)pl.splits * M * N * 4 : 0;
  if (need && (!workspace || ws_bytes < need))
    return fail(GPT_ERR_WORKSPACE, "%s: needs %zu bytes of workspace", fn, need);
  if (need && misaligned(workspace, 256)) return fail(GPT_ERR_ARG, "workspace not 256-byte aligned");
  const Span spans[] = {{"C", C, M, N * dtype_size(out_dtype), ldc * dtype_size(out_dtype)},
                        {"the workspace", need ? workspace : nullptr, 1, need, 0},
                        {"A", A, M, (unsigned long long)K, (unsigned long long)lda}, {"B", B, N, (unsigned long long)K, (unsigned long long)ldb},
                        {"scales_a", scales_a, 1, scale_atoms(M, K) * 512ull, 0}, {"scales_b", scales_b, 1, scale_atoms(N, K) * 512ull, 0}};
  TRY(check_spans(fn, spans, 2, 6));
  ON_DEVICE_OF(fn, A);
  CHECK_PTR(fn, B); CHECK_PTR(fn, C); CHECK_PTR(fn, scales_a); CHECK_PTR(fn, scales_b);
  if (need) CHECK_PTR(fn, workspace);
  unsigned* err = nullptr;
  CUDA_TRY(cudaGetSymbolAddress((void**)&err, g_ngram_err));
  const GemmEpilogue e = epi(out_dtype == GPT_DTYPE_BF16 ? EPI_STORE : EPI_ACCUM_F32, C, ldc, beta != 0);
  float* part = static_cast<float*>(workspace);
#define F8B(BN, CG) \
  gemm_f8b_launch<BN, CG>(M, N, K, A, lda, scales_a, B, ldb, scales_b, e, pl.splits, part, err, st)
  if (pl.bn == 256) return pl.cg == 2 ? F8B(256, 2) : F8B(256, 1);
  return F8B(128, 1);
#undef F8B
}

// ======================================================================== cross entropy without stored logits
// Columns of the vocabulary that the backward pass (and the fp32 forward pass)
// takes at a time.  bf16: as many 256-column tiles as keep the piece's dz
// [N, width] within 512 MB, but no fewer than half of that, chosen so that the
// tiles of the weight gradient (width x d) and of the logits (N x width) fill
// whole waves of SM pairs over all pieces.  More pieces cost a pass over the
// fp32 dx each, fewer cost memory.
static int ce_piece(int N, int V, int d, int dtype, int asked, int sms) {
  const int tiles = cdiv(V, 256);
  if (asked > 0) return std::min(V, 64 * cdiv(std::min(asked, V), 64));
  const long long budget = 512LL << 20, col_bytes = std::max(N, 1) * (long long)(dtype == GPT_DTYPE_BF16 ? 2 : 4) * 256;
  const int most = (int)std::max<long long>(1, std::min<long long>(tiles, budget / col_bytes));
  if (most >= tiles || dtype != GPT_DTYPE_BF16) return std::min(V, most * 256);
  const int units = std::max(1, sms / 2);
  auto waves = [&](long long t) { return (double)((t + units - 1) / units); };
  int best = most;
  double best_cost = 1e300;
  auto products = [&](int n) { return n ? waves((long long)n * cdiv(N, 256)) * d + waves((long long)n * cdiv(d, 256)) * N : 0.0; };
  // every width of up to 512 tiles, at most 256 of more (the choice runs with every call)
  const int step = std::max(1, most / 512);
  for (int w = most; w >= (most + 1) / 2; w -= step) {
    double cost = tiles / w * products(w) + products(tiles % w);
    cost += cdiv(tiles, w) * (waves((long long)cdiv(N, 256) * cdiv(d, 256)) * 0.04 * 256 * w);  // dx read and written
    if (cost < best_cost) { best_cost = cost; best = w; }
  }
  return std::min(V, best * 256);
}

// More rows than these: the targets are counted by a launch of their own instead of
// inside the gradient's first product.  There bf16 counts them in one CTA, beside its
// first tile; fp32 in every block, which costs N^2 V / 1024 reads (B200, a launch
// aside against in every block: 600 x 4096 x 64 61.0 and 63.7 us, 4096 x 4096 x 64 344 and
// 377, 65536 x 4096 x 16 4.0 and 12.2 ms).
constexpr int CE_COUNT_ROWS_BF16 = 4096, CE_COUNT_ROWS_F32 = 512;

// Byte offsets of the operator's scratch inside the caller's workspace.
struct CeWs {
  size_t stats, ztgt, part, counter, base, dz, dx, splitk, total;
  int piece, n_tiles;
  TilePlan lse;  // bf16 forward: the product's form, which n_tiles follows
  long long splitk_elems;
};
static CeWs ce_ws_plan(int N, int V, int d, int dtype, int backward, int asked, int sms) {
  CeWs w = {};
  Carver cv;
  const bool lp = dtype == GPT_DTYPE_BF16;
  w.piece = ce_piece(N, V, d, dtype, asked, sms);
  if (!backward) {
    if (lp) w.lse = lse_plan(N, V, d, sms);
    w.n_tiles = lp ? lse_pairs(V, w.lse) : 1;
    w.stats = cv.take((size_t)w.n_tiles * N * 8);
    w.ztgt = cv.take((size_t)N * 4);
    w.part = cv.take((size_t)cdiv(N, 32) * 16);
    w.counter = cv.take(4);
    if (!lp) w.dz = cv.take((size_t)N * w.piece * 4);
  } else {
    w.base = cv.take(4);
    w.dz = cv.take((size_t)N * (lp ? 64 * cdiv(w.piece, 64) : w.piece) * (lp ? 2 : 4));
    if (lp) {
      if (w.piece < V) w.dx = cv.take((size_t)N * d * 4);
      // split-K partials, for products of few output tiles
      w.splitk_elems = std::min<long long>(16LL * std::max<long long>(N, w.piece) * d, 32LL << 20);
      w.splitk = cv.take((size_t)w.splitk_elems * 4);
    } else {
      w.splitk = cv.take((size_t)CEP_SLOTS * 1024 * 4);
      w.counter = cv.take((size_t)CEP_TILES * 4);
    }
  }
  w.total = cv.take(0);
  return w;
}

static CeProduct ce_product(const float* A, long long lda, int a_kmajor, const float* B, long long ldb, int b_kmajor,
                            float* C, long long ldc, int M, int N, int K, int beta) {
  return CeProduct{A, lda, a_kmajor, B, ldb, b_kmajor, C, ldc, M, N, K, beta, cdiv(M, 32) * cdiv(N, 32), 1, nullptr, nullptr};
}
// Shares of K for products of fewer tiles than SMs: about two blocks per SM,
// at least one chunk for every warp of a block.  `part` has room for CEP_SLOTS
// partial tiles, `counter` for CEP_TILES tiles.
static void ce_split(CeProduct& p0, CeProduct& p1, float* part, unsigned* counter) {
  for (CeProduct* p : {&p0, &p1}) {
    if (p->tiles < 1 || p->tiles > CEP_TILES / 2) continue;
    p->splits = std::max(1, std::min(CEP_TILES / p->tiles, cdiv(p->K, CEP_WARPS * CEP_KC)));
    p->part = part;
    p->counter = counter;
    part += (size_t)p->tiles * p->splits * 1024;
    counter += p->tiles;
  }
}
static int ce_products(const CeProduct& p0, const CeProduct& p1, const CeGrad& gr, cudaStream_t st) {
  ++g_launches;
  launch_pdl(ce_product_kernel, p0.tiles * p0.splits + p1.tiles * p1.splits, CEP_WARPS * 32, 0, st, p0, p1, gr);
  LAUNCH_CHECK();
  return GPT_OK;
}

static const CeProduct ce_no_product = ce_product(nullptr, 0, 0, nullptr, 0, 0, nullptr, 0, 0, 0, 0, 0);

static int ce_check(const char* fn, const void* x, long long ldx, const void* w, long long ldw, int dtype, int N, int V,
                    int d, const int32_t* targets, float softcap) {
  if (N < 0 || V < 1 || d < 1 || N > MAX_ROWS || V > MAX_ROWS || d > MAX_ROWS || !w || (N > 0 && (!x || !targets)) || ldx < d || ldw < d || !(softcap >= 0.f) ||
      std::isinf(softcap))
    return fail(GPT_ERR_ARG, "%s: bad argument", fn);
  if (dtype != GPT_DTYPE_F32 && dtype != GPT_DTYPE_BF16) return fail(GPT_ERR_ARG, "%s: bad dtype", fn);
  if (dtype == GPT_DTYPE_BF16 && (d % 8 || ldx % 8 || ldw % 8 || misaligned(x, 16) || misaligned(w, 16)))
    return fail(GPT_ERR_ARG, "%s: bf16 rows must be 16-byte aligned: d, ldx and ldw multiples of 8", fn);
  if (dtype == GPT_DTYPE_F32 && (misaligned(x, 4) || misaligned(w, 4)))
    return fail(GPT_ERR_ARG, "%s: x or w is not aligned to its elements", fn);
  if (misaligned(targets, 4)) return fail(GPT_ERR_ARG, "%s: targets are not aligned to their elements", fn);
  return GPT_OK;
}

extern "C" int linear_ce_workspace_bytes(int N, int V, int d, int dtype, int backward, int vocab_piece, size_t* bytes) {
  if (!bytes || N < 0 || V < 1 || d < 1 || N > MAX_ROWS || V > MAX_ROWS || d > MAX_ROWS || vocab_piece < 0 || (dtype != GPT_DTYPE_F32 && dtype != GPT_DTYPE_BF16))
    return fail(GPT_ERR_ARG, "linear_ce_workspace_bytes: bad argument");
  *bytes = ce_ws_plan(N, V, d, dtype, backward != 0, vocab_piece, device_sms()).total;
  return GPT_OK;
}

extern "C" int linear_ce_plan(int N, int V, int d, int dtype, int backward, int vocab_piece, int* plan) {
  if (!plan || N < 1 || V < 1 || d < 1 || N > MAX_ROWS || V > MAX_ROWS || d > MAX_ROWS || vocab_piece < 0 ||
      (dtype != GPT_DTYPE_F32 && dtype != GPT_DTYPE_BF16))
    return fail(GPT_ERR_ARG, "linear_ce_plan: bad argument");
  const int sms = device_sms();
  const CeWs w = ce_ws_plan(N, V, d, dtype, backward != 0, vocab_piece, sms);
  const TilePlan none{0, 0, 0, 0};
  TilePlan logits = w.lse, dx = none, dw = none;
  if (dtype == GPT_DTYPE_F32) {
    logits = none;
  } else if (backward) {
    logits = tile_plan(N, w.piece, d, 0, sms);
    dx = tile_plan(N, d, w.piece, w.splitk_elems, sms);
    dw = tile_plan(w.piece, d, N, w.splitk_elems, sms);
  }
  const int out[] = {!backward && dtype == GPT_DTYPE_BF16 ? V : w.piece, logits.bn, logits.cg, logits.n_run,
                     dx.bn, dx.cg, dx.splits, dw.bn, dw.cg, dw.splits};
  for (int i = 0; i < 10; ++i) plan[i] = out[i];
  return GPT_OK;
}

extern "C" int linear_ce_forward(const void* x, long long ldx, const void* w, long long ldw, int dtype, int N, int V,
                                 int d, const int32_t* targets, float softcap, float* loss, float* tok_loss, float* lse,
                                 int vocab_piece, void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "linear_ce_forward";
  TRY(ce_check(fn, x, ldx, w, ldw, dtype, N, V, d, targets, softcap));
  if (N > 0 && !loss && !tok_loss && !lse) return fail(GPT_ERR_ARG, "%s: no output", fn);
  if (vocab_piece < 0) return fail(GPT_ERR_ARG, "%s: bad argument", fn);
  if (misaligned(loss, 4) || misaligned(tok_loss, 4) || misaligned(lse, 4))
    return fail(GPT_ERR_ARG, "%s: an output is not aligned to its elements", fn);
  const CeWs p = ce_ws_plan(N, V, d, dtype, 0, vocab_piece, sms_of(workspace));
  if (!workspace || ws_bytes < p.total) return fail(GPT_ERR_WORKSPACE, "%s: needs %zu bytes of workspace", fn, p.total);
  if (misaligned(workspace, 256)) return fail(GPT_ERR_ARG, "workspace not 256-byte aligned");
  const size_t fes = dtype_size(dtype);
  const Span spans[] = {{"loss", loss, 1, 4, 0}, {"tok_loss", tok_loss, 1, N * 4ull, 0}, {"lse", lse, 1, N * 4ull, 0},
                        {"the workspace", workspace, 1, p.total, 0}, {"x", x, N, d * fes, ldx * fes}, {"w", w, V, d * fes, ldw * fes},
                        {"targets", targets, 1, N * 4ull, 0}};
  TRY(check_spans(fn, spans, 4, 7));
  cudaStream_t st = (cudaStream_t)stream;
  ON_DEVICE_OF(fn, workspace);
  CHECK_PTR(fn, x); CHECK_PTR(fn, w); CHECK_PTR(fn, targets); CHECK_PTR(fn, loss); CHECK_PTR(fn, tok_loss); CHECK_PTR(fn, lse);
  if (N == 0) {
    if (loss) CUDA_TRY(cudaMemsetAsync(loss, 0, 4, st));
    return GPT_OK;
  }
  unsigned* err = nullptr;
  CUDA_TRY(cudaGetSymbolAddress((void**)&err, g_ngram_err));
  uint8_t* b = static_cast<uint8_t*>(workspace);
  float2* stats = reinterpret_cast<float2*>(b + p.stats);
  float* ztgt = reinterpret_cast<float*>(b + p.ztgt);
  double2* part = reinterpret_cast<double2*>(b + p.part);
  unsigned* counter = reinterpret_cast<unsigned*>(b + p.counter);
  if (dtype == GPT_DTYPE_BF16) {
    const GemmCtx g{true, nullptr, 0, err, st, nullptr};
    GemmEpilogue e = epi(EPI_LSE, nullptr, V);
    e.softcap = softcap; e.stats = stats; e.targets = targets; e.ztgt = ztgt; e.counter = counter;
    TRY(gemm_planned(g, p.lse, N, V, d, op_k(x, ldx), op_k(w, ldw), e));
  } else {
    float* z = reinterpret_cast<float*>(b + p.dz);
    for (int v0 = 0; v0 < V; v0 += p.piece) {
      const int width = std::min(p.piece, V - v0);
      TRY(ce_products(ce_product(static_cast<const float*>(x), ldx, 1, static_cast<const float*>(w) + v0 * ldw, ldw, 1, z,
                                 width, N, width, d, 0),
                      ce_no_product, CeGrad{}, st));
      ++g_launches; launch_pdl(ce_piece_stats_kernel, N, 256, 0, st, (const float*)z, width, v0, v0 == 0 ? 1 : 0, softcap,
                               targets, N, stats, ztgt, counter);
      LAUNCH_CHECK();
    }
  }
  const int blocks = cdiv(N, 32);
  const bool few = blocks <= device_sms();
  ++g_launches; launch_pdl(few ? ce_combine_kernel<32> : ce_combine_kernel<8>, blocks, few ? 1024 : 256, 0, st,
                           (const float2*)stats, p.n_tiles, N, V, targets, (const float*)ztgt, lse, tok_loss, part,
                           counter, loss, err);
  LAUNCH_CHECK();
  return GPT_OK;
}

extern "C" int linear_ce_backward(const void* x, long long ldx, const void* w, long long ldw, int dtype, int N, int V,
                                  int d, const int32_t* targets, float softcap, const float* lse, const float* dloss,
                                  const float* dtok, void* dx, long long lddx, void* dw, long long lddw, int dw_dtype,
                                  int dw_beta, int vocab_piece, void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "linear_ce_backward";
  TRY(ce_check(fn, x, ldx, w, ldw, dtype, N, V, d, targets, softcap));
  const bool lp = dtype == GPT_DTYPE_BF16;
  if ((N > 0 && (!lse || (!dx && !dw))) || (dx && lddx < d) || (dw && lddw < d) || (dloss && dtok) || vocab_piece < 0)
    return fail(GPT_ERR_ARG, "%s: bad argument", fn);
  if (dw && ((dw_dtype != GPT_DTYPE_F32 && dw_dtype != GPT_DTYPE_BF16) || (!lp && dw_dtype != GPT_DTYPE_F32) ||
             (dw_beta && dw_dtype != GPT_DTYPE_F32)))
    return fail(GPT_ERR_ARG, "%s: bad dw_dtype (bf16 only with bf16 inputs, accumulation only in fp32)", fn);
  if (lp && ((dx && (misaligned(dx, 16) || lddx % 8)) ||
             (dw && (misaligned(dw, 16) || (lddw * (long long)dtype_size(dw_dtype)) % 16))))
    return fail(GPT_ERR_ARG, "%s: gradient rows must be 16-byte aligned", fn);
  if (!lp && (misaligned(dx, 4) || misaligned(dw, 4))) return fail(GPT_ERR_ARG, "%s: a gradient is not aligned to its elements", fn);
  if (misaligned(lse, 4) || misaligned(dloss, 4) || misaligned(dtok, 4))
    return fail(GPT_ERR_ARG, "%s: lse, dloss or dtok is not aligned to its elements", fn);
  const int sms = sms_of(workspace);
  const CeWs p = ce_ws_plan(N, V, d, dtype, 1, vocab_piece, sms);
  if (!workspace || ws_bytes < p.total) return fail(GPT_ERR_WORKSPACE, "%s: needs %zu bytes of workspace", fn, p.total);
  if (misaligned(workspace, 256)) return fail(GPT_ERR_ARG, "workspace not 256-byte aligned");
  const size_t bes = dtype_size(dtype), wes = dtype_size(dw_dtype);
  const Span spans[] = {{"dx", dx, N, d * bes, lddx * bes}, {"dw", dw, V, d * wes, lddw * wes}, {"the workspace", workspace, 1, p.total, 0},
                        {"x", x, N, d * bes, ldx * bes}, {"w", w, V, d * bes, ldw * bes}, {"targets", targets, 1, N * 4ull, 0},
                        {"lse", lse, 1, N * 4ull, 0}, {"dtok", dtok, 1, N * 4ull, 0}, {"dloss", dloss, 1, 4, 0}};
  TRY(check_spans(fn, spans, 3, 9));
  cudaStream_t st = (cudaStream_t)stream;
  ON_DEVICE_OF(fn, workspace);
  CHECK_PTR(fn, x); CHECK_PTR(fn, w); CHECK_PTR(fn, targets); CHECK_PTR(fn, lse); CHECK_PTR(fn, dloss); CHECK_PTR(fn, dtok);
  CHECK_PTR(fn, dx); CHECK_PTR(fn, dw);
  if (N == 0) {  // no rows: nothing but a weight gradient of zero
    if (dw && !dw_beta)
      CUDA_TRY(cudaMemset2DAsync(dw, lddw * dtype_size(dw_dtype), 0, (size_t)d * dtype_size(dw_dtype), V, st));
    return GPT_OK;
  }
  unsigned* err = nullptr;
  CUDA_TRY(cudaGetSymbolAddress((void**)&err, g_ngram_err));
  uint8_t* b = static_cast<uint8_t*>(workspace);
  const CeRowScale scale{targets, dloss, dtok, N, V, err};
  unsigned* counter = reinterpret_cast<unsigned*>(b + p.counter);
  // the mean's factor: applied by the products in bf16, to dz in fp32 (as per-token gradients are in both)
  float* base = dtok ? nullptr : reinterpret_cast<float*>(b + p.base);
  const bool count_aside = N > (lp ? CE_COUNT_ROWS_BF16 : CE_COUNT_ROWS_F32);
  if (base && count_aside) {
    ++g_launches; launch_pdl(ce_base_kernel, 1, 1024, 0, st, scale, base);
    LAUNCH_CHECK();
  }
  const GemmCtx g{true, reinterpret_cast<float*>(b + p.splitk), p.splitk_elems, err, st, nullptr};  // bf16
  const size_t es = dtype_size(dtype);
  void* dz = b + p.dz;
  const bool one = p.piece >= V;  // dx needs no sum over pieces
  float* acc = lp ? reinterpret_cast<float*>(b + p.dx) : static_cast<float*>(dx);
  for (int v0 = 0; v0 < V; v0 += p.piece) {
    const int width = std::min(p.piece, V - v0);
    const uint8_t* wp = static_cast<const uint8_t*>(w) + (size_t)v0 * ldw * es;
    long long ldz = width;
    if (lp) {
      ldz = 64 * cdiv(width, 64);
      GemmEpilogue e = epi(EPI_DLOGITS, dz, ldz);
      e.softcap = softcap; e.targets = targets; e.vocab = V; e.col0 = v0; e.lse = lse; e.dtok = dtok; e.dloss = dloss;
      if (v0 == 0 && !count_aside) e.base_out = base;
      TRY(gemm_planned(g, tile_plan(N, width, d, 0, sms), N, width, d, op_k(x, ldx), op_k(wp, ldw), e));
    } else {
      float* z = static_cast<float*>(dz);
      const float* xf = static_cast<const float*>(x);
      const float* wf = reinterpret_cast<const float*>(wp);
      TRY(ce_products(ce_product(xf, ldx, 1, wf, ldw, 1, z, width, N, width, d, 0), CeProduct{},
                      CeGrad{lse, scale, count_aside ? base : nullptr, v0, softcap, counter}, st));
      CeProduct px = ce_no_product, pw = ce_no_product;
      if (dx) px = ce_product(z, width, 1, wf, ldw, 0, acc, lddx, N, d, width, v0 > 0);
      if (dw) pw = ce_product(z, width, 0, xf, ldx, 0, static_cast<float*>(dw) + v0 * lddw, lddw, width, d, N, dw_beta);
      ce_split(px, pw, reinterpret_cast<float*>(b + p.splitk), counter);
      TRY(ce_products(px, pw, CeGrad{}, st));
      continue;
    }
    if (dx) {
      GemmEpilogue e = one ? epi(EPI_STORE, dx, lddx) : epi(EPI_ACCUM_F32, acc, d, v0 > 0);
      if (one) e.scale_a = base;
      TRY(gemm_planned(g, tile_plan(N, d, width, p.splitk_elems, sms), N, d, width, op_k(dz, ldz), op_mn(wp, ldw), e));
    }
    if (dw) {
      uint8_t* out = static_cast<uint8_t*>(dw) + (size_t)v0 * lddw * dtype_size(dw_dtype);
      GemmEpilogue e = dw_dtype == GPT_DTYPE_BF16 ? epi(EPI_STORE, out, lddw) : epi(EPI_ACCUM_F32, out, lddw, dw_beta);
      e.scale_a = base;
      TRY(gemm_planned(g, tile_plan(width, d, N, p.splitk_elems, sms), width, d, N, op_mn(dz, ldz), op_mn(x, ldx), e));
    }
  }
  if (dx && lp && !one) {
    const int blocks = (int)std::min<long long>(((long long)N * d / 4 + 255) / 256, 8LL * device_sms());
    ++g_launches; launch_pdl(ce_dx_kernel, blocks, 256, 0, st, (const float*)acc, N, d, (const float*)base, (bf16*)dx, lddx);
    LAUNCH_CHECK();
  }
  return GPT_OK;
}

// ======================================================================== gradient clipping
extern "C" int grad_clip_workspace_bytes(int n, size_t* bytes) {
  if (!bytes || n < 0) return fail(GPT_ERR_ARG, "grad_clip_workspace_bytes: bad argument");
  *bytes = (size_t)std::max(1, cdiv(n, CLIP_MAX_TENSORS)) * CLIP_BLOCKS * sizeof(double);
  return GPT_OK;
}

template <int CAP>
static int clip_fill(ClipTable<CAP>& t, int n, const void* const* grads, void* const* outs, const long long* sizes,
                     const int* dtypes) {
  long long pieces = 0;
  t.n = n;
  for (int i = 0; i < n; ++i) {
    const bool lp = dtypes[i] == GPT_DTYPE_BF16;
    t.g[i] = grads[i];
    t.out[i] = outs ? outs[i] : const_cast<void*>(grads[i]);
    t.size_bf16[i] = (unsigned long long)sizes[i] << 1 | (lp ? 1 : 0);
    t.piece0[i] = (int)pieces;
    pieces += cdiv_ll(sizes[i], lp ? CLIP_PIECE / 2 : CLIP_PIECE / 4);
    if (pieces > 0x3fffffffLL) return fail(GPT_ERR_ARG, "grad_clip: too many elements");
  }
  t.piece0[n] = (int)pieces;
  return GPT_OK;
}

// both passes over all tensors, CAP of them a launch
template <int CAP>
static int clip_run(int n, const void* const* grads, void* const* outs, const long long* sizes, const int* dtypes,
                    float max_norm, float* norm_out, double* part, unsigned* err, cudaStream_t st) {
  ClipTable<CAP> t;
  const int launches = std::max(1, cdiv(n, CAP));
  int parts = 0;
  for (int pass = 0; pass < 2; ++pass)
    for (int l = 0; l < launches; ++l) {
      const int i0 = l * CAP, m = std::min(CAP, n - i0);
      if (pass == 0 || launches > 1)
        TRY(clip_fill(t, m, grads + i0, outs ? outs + i0 : nullptr, sizes + i0, dtypes + i0));
      const int grid = std::max(1, std::min(CLIP_BLOCKS, t.piece0[m]));
      ++g_launches;
      if (pass == 0) {
        launch_pdl(clip_sumsq_kernel<CAP>, grid, CLIP_THREADS, 0, st, t, part + parts);
        parts += grid;
      } else {
        // the norm alone needs no more than the first block
        const bool scale = outs || max_norm > 0.f;
        if (!scale && l > 0) break;
        launch_pdl(clip_scale_kernel<CAP>, scale ? grid : 1, CLIP_THREADS, 0, st, t, (const double*)part, parts, max_norm,
                   outs ? 0 : 1, l == 0 ? norm_out : nullptr, err);
      }
      LAUNCH_CHECK();
    }
  return GPT_OK;
}

// A tensor that overlaps what another one writes (two blocks would scale the
// same elements, or one would read what the other has scaled), or -1.  `order`:
// n ints of scratch.
static int clip_overlap(int n, const void* const* grads, void* const* outs, const long long* sizes, const int* dtypes,
                        int* order) {
  auto in0 = [&](int i) { return reinterpret_cast<uintptr_t>(grads[i]); };
  auto out0 = [&](int i) { return reinterpret_cast<uintptr_t>(outs ? outs[i] : grads[i]); };
  auto len = [&](int i) { return (uintptr_t)sizes[i] * dtype_size(dtypes[i]); };
  int m = 0;
  bool ascending = true;
  for (int i = 0; i < n; ++i) {
    if (sizes[i] == 0) continue;
    if (m > 0 && out0(order[m - 1]) > out0(i)) ascending = false;
    order[m++] = i;
  }
  if (!ascending) std::sort(order, order + m, [&](int a, int b) { return out0(a) < out0(b); });
  for (int k = 1; k < m; ++k)
    if (out0(order[k - 1]) + len(order[k - 1]) > out0(order[k])) return order[k];
  if (!outs) return -1;
  // the outputs are disjoint and sorted: those that an input meets are neighbours
  for (int i = 0; i < n; ++i) {
    if (sizes[i] == 0) continue;
    int lo = 0, hi = m;  // first output that ends behind the input's start
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (out0(order[mid]) + len(order[mid]) > in0(i)) hi = mid;
      else lo = mid + 1;
    }
    for (; lo < m && out0(order[lo]) < in0(i) + len(i); ++lo)
      if (order[lo] != i || out0(i) != in0(i)) return i;
  }
  return -1;
}

extern "C" int grad_clip(int n, const void* const* grads, void* const* outs, const long long* sizes, const int* dtypes,
                         float max_norm, float* norm_out, void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "grad_clip";
  if (n < 0 || (n > 0 && (!grads || !sizes || !dtypes)) || !(max_norm >= 0.f))
    return fail(GPT_ERR_ARG, "%s: bad argument (max_norm >= 0)", fn);
  size_t need = 0;
  TRY(grad_clip_workspace_bytes(n, &need));
  for (int i = 0; i < n; ++i) {
    if (dtypes[i] != GPT_DTYPE_F32 && dtypes[i] != GPT_DTYPE_BF16) return fail(GPT_ERR_ARG, "%s: tensor %d: bad dtype", fn, i);
    const size_t es = dtype_size(dtypes[i]);
    if (sizes[i] < 0 || sizes[i] > (1LL << 46) || (sizes[i] > 0 && (!grads[i] || (outs && !outs[i]))))
      return fail(GPT_ERR_ARG, "%s: tensor %d: null pointer or bad size", fn, i);
    if (sizes[i] > 0 && (misaligned(grads[i], es) || (outs && misaligned(outs[i], es))))
      return fail(GPT_ERR_ARG, "%s: tensor %d is not aligned to its elements", fn, i);
  }
  if (misaligned(norm_out, 4)) return fail(GPT_ERR_ARG, "%s: norm_out is not aligned to its elements", fn);
  if (!workspace || ws_bytes < need) return fail(GPT_ERR_WORKSPACE, "%s: needs %zu bytes of workspace", fn, need);
  if (misaligned(workspace, 256)) return fail(GPT_ERR_ARG, "workspace not 256-byte aligned");
  // blocks still read the partials while one writes the norm, and the tensors while
  // others write partials: both lie apart from everything else
  const Span own[] = {{"the workspace", workspace, 1, need, 0}, {"norm_out", norm_out, 1, 4, 0}};
  TRY(check_spans(fn, own, 1, 2));
  for (int i = 0; i < n; ++i)
    for (const void* p : {grads[i], outs ? static_cast<const void*>(outs[i]) : nullptr}) {
      const Span t{"a tensor", sizes[i] > 0 ? p : nullptr, 1, (unsigned long long)sizes[i] * dtype_size(dtypes[i]), 0};
      for (const Span& o : own)
        if (spans_overlap(o, t)) return fail(GPT_ERR_ARG, "%s: tensor %d overlaps %s", fn, i, o.name);
    }
  if (n > 0 && (outs || max_norm > 0.f)) {  // a norm alone writes no tensor
    int* order = static_cast<int*>(malloc((size_t)n * sizeof(int)));
    if (!order) return fail(GPT_ERR_ARG, "%s: out of host memory", fn);
    const int bad = clip_overlap(n, grads, outs, sizes, dtypes, order);
    free(order);
    if (bad >= 0) return fail(GPT_ERR_ARG, "%s: tensor %d overlaps another one that is written", fn, bad);
  }
  cudaStream_t st = (cudaStream_t)stream;
  ON_DEVICE_OF(fn, workspace);
  CHECK_PTR(fn, norm_out);
  for (int i = 0; i < n; ++i) {
    if (sizes[i] == 0) continue;
    CHECK_PTR(fn, grads[i]);
    if (outs) CHECK_PTR(fn, outs[i]);
  }
  unsigned* err = nullptr;
  CUDA_TRY(cudaGetSymbolAddress((void**)&err, g_ngram_err));
  double* part = static_cast<double*>(workspace);
  if (n <= CLIP_FEW_TENSORS)
    return clip_run<CLIP_FEW_TENSORS>(n, grads, outs, sizes, dtypes, max_norm, norm_out, part, err, st);
  return clip_run<CLIP_MAX_TENSORS>(n, grads, outs, sizes, dtypes, max_norm, norm_out, part, err, st);
}

// api_fp8.cu -- the C ABI of the 8-bit operators (sgemm_fp8.h): argument checks, workspace and launches.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdint>
#include <iterator>

#include "fp8_internal.h"
#include "sgemm_fp8.h"
#include "sgemm_internal.h"

using namespace sgemm_impl;

namespace {

constexpr int64_t kMaxDim = INT_MAX - 1024;  // column indices of the kernels' last chunks stay below 2^31

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int type_size(int type) { return type == SGEMM_BF16 ? 2 : 4; }
bool known_type(int type) { return type == SGEMM_F32 || type == SGEMM_BF16; }
bool known_format(int f) { return f == SGEMM_FP8_E4M3 || f == SGEMM_FP8_E5M2; }

// Rows of 16-byte vectors: the base and the row stride in bytes are multiples of 16 (a NULL matrix is not read).
bool rows16(const void* p, int64_t ld, int size) { return !p || (aligned(p, 16) && ld * size % 16 == 0); }

// Whether an output in an input's place has rows of its own: it would overwrite rows that are still to be read.
bool other_stride(const void* out, int64_t ld_out, const void* in, int64_t ld_in, int64_t rows) {
  return out == in && rows > 1 && ld_out != ld_in;
}

// ---------------------------------------------------------------- product

std::atomic<int> g_force_variant{SGEMM_VARIANT_AUTO}, g_force_tile{0}, g_force_split{0};

int op_code(char t) {
  if (t == 'N' || t == 'n') return 0;
  if (t == 'T' || t == 't' || t == 'C' || t == 'c') return 1;
  return -1;
}

// One operand of a product: `mn` output rows (or columns) x K, and how it is stored.
struct Operand {
  const sgemm_fp8_matrix_t* m = nullptr;
  int64_t rows = 0, cols = 0;  // stored
  int mn_major = 0;            // the stored rows run along the output, not along k
  Fp8Scales scales;
};

// Fills *o; false when a field of *m cannot be used (`read`: the operand is read at all).
bool check_operand(const sgemm_fp8_matrix_t* m, int64_t mn, int64_t K, bool mn_major, bool read, Operand* o) {
  if (!m) return !read;
  o->m = m;
  o->mn_major = mn_major ? 1 : 0;
  o->rows = mn_major ? K : mn;
  o->cols = mn_major ? mn : K;
  if (!known_format(m->format)) return false;
  const int along_k = mn_major ? m->block_rows : m->block_cols, along_mn = mn_major ? m->block_cols : m->block_rows;
  if (along_k != 128 || (along_mn != 1 && along_mn != 128)) return false;
  if (m->ld < std::max<int64_t>(1, o->cols) || m->lds < std::max<int64_t>(1, ceil_div(o->cols, m->block_cols)))
    return false;
  if (read && (!m->data || !m->scale || !aligned(m->scale, 4))) return false;
  o->scales.p = m->scale;
  o->scales.shift = along_mn == 128 ? 7 : 0;
  o->scales.si = mn_major ? 1 : m->lds;
  o->scales.sk = mn_major ? m->lds : 1;
  return true;
}

struct Product {
  int64_t M, N, K;
  float alpha;
  Operand a, b;
  Fp8Out out;
};

int check_product(char transA, char transB, int64_t M, int64_t N, int64_t K, float alpha, const sgemm_fp8_matrix_t* A,
                  const sgemm_fp8_matrix_t* B, float beta, const void* C, int64_t ldc, const void* D, int64_t ldd,
                  int type, Product* pr) {
  const int ta = op_code(transA), tb = op_code(transB);
  if (ta < 0) return -1;
  if (tb < 0) return -2;
  if (M < 0) return -3;
  if (N < 0) return -4;
  if (K < 0) return -5;
  const bool work = M > 0 && N > 0, read = work && K > 0 && alpha != 0.0f;
  *pr = Product{M, N, K, alpha, {}, {}, {}};
  if (!check_operand(A, M, K, ta != 0, read, &pr->a)) return -7;
  if (!check_operand(B, N, K, tb == 0, read, &pr->b)) return -8;
  if (!known_type(type)) return -14;
  const int size = type_size(type);
  if (work && beta != 0.0f && (!C || !aligned(C, size))) return -10;
  if (beta != 0.0f && ldc < std::max<int64_t>(1, N)) return -11;
  if (work && (!D || !aligned(D, size))) return -12;
  if (ldd < std::max<int64_t>(1, N) || (C == D && C && beta != 0.0f && ldc != ldd)) return -13;
  Fp8Out& o = pr->out;
  o.M = (int)std::min<int64_t>(M, INT_MAX);
  o.N = (int)std::min<int64_t>(N, INT_MAX);
  o.alpha = alpha;
  o.beta = beta;
  o.C = beta != 0.0f ? C : nullptr;
  o.D = const_cast<void*>(D);
  o.ldc = ldc;
  o.ldd = ldd;
  o.bf16 = type == SGEMM_BF16;
  o.vec = rows16(o.C, ldc, size) && rows16(D, ldd, size);
  return SGEMM_OK;
}

// TMA reads codes whose base and row stride (of more than one row) are multiples of 16 bytes; others are
// copied first.
int64_t repack_ld(const Operand& o) { return ceil_div(o.cols, 16) * 16; }
int64_t repack_bytes(const Operand& o) {
  return aligned(o.m->data, 16) && (o.m->ld % 16 == 0 || o.rows == 1) ? 0 : round256(o.rows * repack_ld(o));
}

// Times in ns that the choice of kernel goes by, fitted to 700 launches of 44 products (M, N, K from 1
// to 16384) forced to each kernel, tile and split on a GB300: they give those launches' times to about
// 15%, and for 34 further products the launch they choose took 4% longer than the fastest on average, 33%
// at most.  In the pair kernel, by tile width: a group of 128 k, and the rest of a tile.  On the short
// side: a group in a CTA that has its SM to itself, the rest of a tile, and what joining a tile's shares
// adds to it.
struct PairCost {
  int tile, group_ns, tile_ns;
};
constexpr PairCost kPairCost[] = {{256, 390, 3200}, {128, 325, 1850}, {64, 295, 950}};
constexpr PairCost kPairColsCost[] = {{256, 605, 3450}, {128, 490, 1650}, {64, 430, 1000}};  // B scaled by column
struct ShortCost {
  int tile, group_ns, tile_ns, join_ns;
};
constexpr ShortCost kShortCost[] = {{16, 310, 1500, 800}, {32, 330, 2400, 500}, {64, 445, 4100, 650}, {128, 545, 7300, 1550}};
constexpr double kPairLaunchNs = 4950, kShortLaunchNs = 2750;
constexpr double kSharedSm = 0.3;        // a group takes this much longer with a second CTA on the SM
constexpr double kSmBytesPerNs = 44.7;   // an SM's share of the memory bandwidth

// SMs that clusters of `split` CTAs can use at a time: groups of 4 or 8 do not fill every part of the chip.
int64_t cluster_sms(int sm_count, int split) {
  return split <= 2 ? sm_count : std::max(1, split == 4 ? sm_count * 18 / 19 : sm_count * 16 / 19);
}

int64_t short_ring(int tile) { return (tile == 128 ? 2 : 1) * 98 * 1024; }  // stages of two CTAs (one) per SM
int short_ctas_per_sm(int tile) { return tile == 128 ? 1 : 2; }

struct Choice {
  int variant = 0, tile = 0, split = 1;
  double ns = 1e30;
};

// The cheapest launch of a product, among the variant, tile and split that are forced (0: any); clusters:
// CTA pairs that run at a time, 0 on a device without clusters, where only unshared tiles can run.
Choice choose(const Product& pr, int64_t clusters, int sm_count, int variant, int tile, int split) {
  const int64_t groups = ceil_div(pr.K, 128), S = std::min(pr.M, pr.N), L = std::max(pr.M, pr.N);
  Choice best;
  const auto offer = [&](int v, int n, int k, double ns) {
    if (ns < best.ns) best = Choice{v, n, k, ns};
  };
  if (variant != SGEMM_VARIANT_FP8_SHORT && clusters > 0)
    for (const PairCost& c : pr.b.scales.shift == 0 ? kPairColsCost : kPairCost) {
      if (tile != 0 && tile != c.tile) continue;
      const int64_t rounds = ceil_div(ceil_div(pr.M, 256) * ceil_div(pr.N, c.tile), clusters);
      offer(SGEMM_VARIANT_FP8_PAIR, c.tile, 1, kPairLaunchNs + (double)rounds * (groups * c.group_ns + c.tile_ns));
    }
  if (variant != SGEMM_VARIANT_FP8_PAIR)
    for (const ShortCost& c : kShortCost) {
      if (tile != 0 ? tile != c.tile : c.tile > 16 && c.tile >= 2 * S) continue;
      const int64_t tiles = ceil_div(L, 128) * ceil_div(S, c.tile);
      for (int k = 1; k <= 8; k *= 2) {
        if (clusters == 0 && k > 1) break;
        if (split != 0 ? split != k : k > 1 && groups < 2 * k) continue;  // two groups per CTA at least
        const int per_sm = short_ctas_per_sm(c.tile);
        const double on_sm = std::min((double)per_sm, std::max(1.0, (double)tiles * k / sm_count));
        const double group = std::max(c.group_ns * (1.0 + kSharedSm * (on_sm - 1.0)), on_sm * (16384 + 64 * c.tile) / kSmBytesPerNs);
        const double rounds = (double)ceil_div(tiles * k, cluster_sms(sm_count, k) * per_sm);
        offer(SGEMM_VARIANT_FP8_SHORT, c.tile, k,
              kShortLaunchNs + rounds * (ceil_div(groups, k) * group + c.tile_ns + (k > 1 ? c.join_ns : 0)));
      }
    }
  return best;
}

int plan_product(const Product& pr, int sm_count, int pair_clusters, sgemm_plan_t* plan) {
  *plan = sgemm_plan_t{};
  plan->split_k = 1;
  if (pr.M == 0 || pr.N == 0) {
    plan->variant = SGEMM_VARIANT_NONE;
    return SGEMM_OK;
  }
  if (pr.M > kMaxDim || pr.N > kMaxDim || pr.K > kMaxDim) return SGEMM_ERR_UNSUPPORTED;
  if (pr.K == 0 || pr.alpha == 0.0f) {
    plan->variant = SGEMM_VARIANT_SCALE;
    plan->kernel_launches = 1;
    plan->threads = 256;
    return SGEMM_OK;
  }
  if (pr.a.m->ld > INT_MAX || pr.b.m->ld > INT_MAX) return SGEMM_ERR_UNSUPPORTED;
  const int64_t clusters = pair_clusters >= 0 ? pair_clusters : std::max(1, sm_count / 2);
  const int64_t groups = ceil_div(pr.K, 128);
  const int64_t S = std::min(pr.M, pr.N), L = std::max(pr.M, pr.N);
  const Choice choice = choose(pr, clusters, sm_count, g_force_variant.load(), g_force_tile.load(), g_force_split.load());
  const int variant = choice.variant;
  if (variant == 0) return SGEMM_ERR_UNSUPPORTED;  // forced to what needs clusters
  plan->variant = variant;
  plan->tile_k = 128;
  plan->kernel_launches = 1;
  plan->workspace_bytes = repack_bytes(pr.a) + repack_bytes(pr.b);
  plan->kernel_launches += (repack_bytes(pr.a) > 0) + (repack_bytes(pr.b) > 0);
  int64_t tiles;
  if (variant == SGEMM_VARIANT_FP8_PAIR) {
    plan->tile_m = 256;
    plan->tile_n = choice.tile;
    plan->stages = kFp8PairStages;
    plan->threads = kFp8PairThreads;
    plan->smem_bytes = fp8_pair_smem(pr.b.scales.shift == 0);
    tiles = ceil_div(pr.M, 256) * ceil_div(pr.N, plan->tile_n);
    plan->grid_x = 2 * std::min<int64_t>(tiles, clusters);
  } else {
    const Operand& s_op = pr.M <= pr.N ? pr.a : pr.b;
    plan->tile_m = 128;
    plan->tile_n = choice.tile;
    tiles = ceil_div(L, 128) * ceil_div(S, plan->tile_n);
    plan->split_k = choice.split;
    const int64_t stage = 16384 + (s_op.mn_major ? 16384 : plan->tile_n * 128);
    plan->stages = (int)std::min<int64_t>(kFp8ShortMaxStages, short_ring(plan->tile_n) / stage);
    plan->threads = kFp8ShortThreads;
    plan->smem_bytes = (int64_t)fp8_short_smem(plan->tile_n, plan->stages, (int)stage);
    plan->grid_x = tiles * choice.split;
  }
  plan->dp_tiles = tiles;
  plan->grid_y = 1;
  return plan->grid_x > INT_MAX || tiles * groups > INT_MAX ? SGEMM_ERR_UNSUPPORTED : SGEMM_OK;
}

// Tensor-core instruction descriptor, kind::f8f6f4: FP32 accumulator, operand formats, the
// operands' orders (1: MN-major), N and M of the instruction.
uint32_t instruction(const Operand& a, const Operand& b, int m, int n) {
  return (1u << 4) | ((uint32_t)a.m->format << 7) | ((uint32_t)b.m->format << 10) | ((uint32_t)a.mn_major << 15) |
         ((uint32_t)b.mn_major << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Tensor map of an operand's tiles (`mn` output rows each), after copying its codes to aligned rows
// at *ws where it needs that.
cudaError_t operand_map(const Operand& o, int mn, uint8_t** ws, CUtensorMap* map, const Guard& guard, cudaStream_t stream) {
  const void* data = o.m->data;
  int64_t ld = o.rows == 1 ? repack_ld(o) : o.m->ld;  // (a map wants a stride even where it steps over nothing)
  const int64_t copy = repack_bytes(o);
  if (copy > 0) {
    const cudaError_t e = launch_fp8_repack(data, o.m->ld, o.rows, o.cols, *ws, repack_ld(o), guard, stream);
    if (e != cudaSuccess) return e;
    data = *ws;
    ld = repack_ld(o);
    *ws += copy;
  }
  return encode_fp8_map(data, o.cols, o.rows, ld, o.mn_major ? 128 : mn, map);
}

cudaError_t launch_product(const Product& pr, const sgemm_plan_t& plan, const CallDevice& dev, uint8_t* ws,
                           cudaStream_t stream) {
  CUtensorMap ma, mb;
  if (plan.variant == SGEMM_VARIANT_FP8_PAIR) {
    cudaError_t e = operand_map(pr.a, 128, &ws, &ma, pr.out.guard, stream);
    if (e == cudaSuccess) e = operand_map(pr.b, plan.tile_n / 2, &ws, &mb, pr.out.guard, stream);
    if (e != cudaSuccess) return e;
    Fp8PairParams p;
    p.out = pr.out;
    p.K = (int)pr.K;
    p.sa = pr.a.scales;
    p.sb = pr.b.scales;
    p.a_mn = pr.a.mn_major;
    p.b_mn = pr.b.mn_major;
    p.idesc = instruction(pr.a, pr.b, 256, plan.tile_n);
    p.tiles_m = (int)ceil_div(pr.M, 256);
    p.tiles_n = (int)ceil_div(pr.N, plan.tile_n);
    p.clusters = (int)(plan.grid_x / 2);
    p.timeout_ns = wait_timeout_ns();
    p.fault = dev.fault;
    // TMA writes whole units of 16 bytes: where a row of D ends inside one, it would write what lies behind the row.
    // Such rows take 75 us in BF16 at 4096 x 4090 x 4096, whole ones 62 at 4096^3; with their ends written by the
    // lanes beside TMA in one kernel, calls of whole rows took 3 to 4% longer.
    const bool ends_inside = pr.N * (p.out.bf16 ? 2 : 4) % 16 != 0;
    if (!p.out.vec || (p.out.beta == 0.0f && ends_inside))
      return launch_fp8_pair_any(plan.tile_n, ma, mb, ma, p, stream);  // (D's map is not read)
    if (p.out.beta != 0.0f) return launch_fp8_pair_add(plan.tile_n, ma, mb, ma, p, stream);
    CUtensorMap md;
    e = encode_out_map(p.out.D, pr.N, pr.M, p.out.ldd, p.out.bf16 != 0, &md);
    return e == cudaSuccess ? launch_fp8_pair_plain(plan.tile_n, ma, mb, md, p, stream) : e;
  }
  const bool trans = pr.M <= pr.N;
  const Operand &l = trans ? pr.b : pr.a, &s = trans ? pr.a : pr.b;
  cudaError_t e = operand_map(l, 128, &ws, &ma, pr.out.guard, stream);
  if (e == cudaSuccess) e = operand_map(s, plan.tile_n, &ws, &mb, pr.out.guard, stream);
  if (e != cudaSuccess) return e;
  Fp8ShortParams p;
  p.out = pr.out;
  p.K = (int)pr.K;
  p.L = (int)(trans ? pr.N : pr.M);
  p.S = (int)(trans ? pr.M : pr.N);
  p.trans = trans;
  p.sl = l.scales;
  p.ss = s.scales;
  p.l_mn = l.mn_major;
  p.s_mn = s.mn_major;
  p.idesc = instruction(l, s, 128, plan.tile_n);
  p.tile_s = plan.tile_n;
  p.tiles_l = (int)ceil_div(p.L, 128);
  p.tiles_s = (int)ceil_div(p.S, plan.tile_n);
  p.split = plan.split_k;
  p.stages = plan.stages;
  p.stage_bytes = 16384 + (s.mn_major ? 16384 : plan.tile_n * 128);
  p.timeout_ns = wait_timeout_ns();
  p.fault = dev.fault;
  return launch_fp8_short(ma, mb, p, stream);
}

// ---------------------------------------------------------------- mixture of experts

// Whether the stored rows x cols matrices of `experts` experts can be read.
bool check_experts(const sgemm_fp8_experts_t* m, int64_t rows, int64_t cols, int64_t experts, bool read) {
  if (!m) return !read;
  if (m->ld < std::max<int64_t>(1, cols) || m->ld % 16 != 0 || m->ld > INT_MAX) return false;
  if (m->lds < std::max<int64_t>(1, ceil_div(cols, 128))) return false;
  if (experts > 1 && (m->stride < (rows - 1) * m->ld + cols || m->stride % 16 != 0 || m->stride >= (int64_t)1 << 39 ||
                      m->stride_scale < (ceil_div(rows, 128) - 1) * m->lds + ceil_div(cols, 128)))
    return false;
  return !read || (m->data && aligned(m->data, 16) && m->scale && aligned(m->scale, 4));
}

cudaError_t experts_map(const sgemm_fp8_experts_t& m, int64_t rows, int64_t cols, int64_t experts, int box,
                        CUtensorMap* map) {
  return encode_fp8_maps(m.data, cols, rows, m.ld, experts, experts > 1 ? m.stride : m.ld, box, map);
}

// Pieces of one workspace, 256 bytes apart (counted first, then placed).
struct Pieces {
  uint8_t* base = nullptr;
  int64_t at = 0;
  template <typename T>
  T* take(int64_t n) {
    T* r = base ? reinterpret_cast<T*>(base + at) : nullptr;
    at += round256(n * (int64_t)sizeof(T));
    return r;
  }
};

int launch_status(cudaError_t e) { return e == cudaSuccess ? SGEMM_OK : record_cuda_failure(e); }

}  // namespace

extern "C" {

int sgemm_fp8(char transA, char transB, int64_t M, int64_t N, int64_t K, float alpha, const sgemm_fp8_matrix_t* A,
              const sgemm_fp8_matrix_t* B, float beta, const void* C, int64_t ldc, void* D, int64_t ldd, int type,
              struct CUstream_st* stream_) {
  Product pr;
  int s = check_product(transA, transB, M, N, K, alpha, A, B, beta, C, ldc, D, ldd, type, &pr);
  if (s != SGEMM_OK || M == 0 || N == 0) return s;
  CallDevice dev;
  s = call_device(&dev);
  if (s != SGEMM_OK) return s;
  sgemm_plan_t plan;
  s = plan_product(pr, dev.sm_count, dev.pair_clusters, &plan);
  if (s != SGEMM_OK) return s;
  pr.out.guard = {dev.fault, dev.bounds};
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (plan.variant == SGEMM_VARIANT_SCALE) return launch_status(launch_fp8_scale(pr.out, stream));
  void* ws = nullptr;
  if (plan.workspace_bytes > 0) {
    const cudaError_t e = cudaMallocFromPoolAsync(&ws, (size_t)plan.workspace_bytes, dev.pool, stream);
    if (e != cudaSuccess) {
      record_cuda_failure(e);
      return e == cudaErrorMemoryAllocation ? SGEMM_ERR_NOMEM : SGEMM_ERR_CUDA;
    }
  }
  cudaError_t e = launch_product(pr, plan, dev, static_cast<uint8_t*>(ws), stream);
  if (ws) {
    const cudaError_t ef = cudaFreeAsync(ws, stream);
    if (e == cudaSuccess) e = ef;
  }
  return launch_status(e);
}

int sgemm_fp8_plan(char transA, char transB, int64_t M, int64_t N, int64_t K, float alpha, const sgemm_fp8_matrix_t* A,
                   const sgemm_fp8_matrix_t* B, float beta, const void* C, int64_t ldc, const void* D, int64_t ldd,
                   int type, int sm_count, sgemm_plan_t* plan) {
  if (!plan) return -16;
  Product pr;
  int s = check_product(transA, transB, M, N, K, alpha, A, B, beta, C, ldc, D, ldd, type, &pr);
  if (s != SGEMM_OK) return s;
  CallDevice dev;
  dev.sm_count = sm_count;
  dev.pair_clusters = -1;
  if (sm_count <= 0) {
    s = call_device(&dev);
    if (s != SGEMM_OK) return s;
  }
  return plan_product(pr, dev.sm_count, dev.pair_clusters, plan);
}

int sgemm_fp8_set_override(int variant, int tile_n, int split) {
  if (variant != SGEMM_VARIANT_AUTO && variant != SGEMM_VARIANT_FP8_PAIR && variant != SGEMM_VARIANT_FP8_SHORT)
    return -1;
  const bool is_short = variant == SGEMM_VARIANT_FP8_SHORT;
  const auto is_in = [&](const auto& tiles) { return std::find(std::begin(tiles), std::end(tiles), tile_n) != std::end(tiles); };
  const bool known = is_short ? is_in(kFp8ShortTiles) : variant == SGEMM_VARIANT_FP8_PAIR && is_in(kFp8PairTiles);
  if (tile_n != 0 && !known) return -2;
  if ((split != 0 && !is_short) || (split != 0 && split != 1 && split != 2 && split != 4 && split != 8)) return -3;
  g_force_variant.store(variant);
  g_force_tile.store(tile_n);
  g_force_split.store(split);
  return SGEMM_OK;
}

int sgemm_fp8_quantize(int64_t rows, int64_t cols, const void* X, int type, int64_t ldx, int format, int block_rows,
                       int block_cols, void* codes, int64_t ldq, float* scale, int64_t lds,
                       struct CUstream_st* stream) {
  if (rows < 0) return -1;
  if (cols < 0) return -2;
  const bool work = rows > 0 && cols > 0;
  if (!known_type(type)) return -4;
  if (work && (!X || !aligned(X, type_size(type)))) return -3;
  if (ldx < std::max<int64_t>(1, cols)) return -5;
  if (!known_format(format)) return -6;
  if (block_rows != 1 && block_rows != 128) return -7;
  if ((block_cols != 1 && block_cols != 128) || (block_rows == 1 && block_cols == 1)) return -8;
  if (work && !codes) return -9;
  if (ldq < std::max<int64_t>(1, cols)) return -10;
  if (work && (!scale || !aligned(scale, 4))) return -11;
  if (lds < std::max<int64_t>(1, ceil_div(cols, block_cols))) return -12;
  if (!work) return SGEMM_OK;
  if (rows > kMaxDim || cols > kMaxDim || ceil_div(rows, 128) * ceil_div(cols, 128) > INT_MAX)
    return SGEMM_ERR_UNSUPPORTED;
  CallDevice dev;
  const int s = call_device(&dev);
  if (s != SGEMM_OK) return s;
  QuantParams p;
  p.x = X;
  p.rows = rows;
  p.cols = cols;
  p.ldx = ldx;
  p.q = static_cast<uint8_t*>(codes);
  p.ldq = ldq;
  p.s = scale;
  p.lds = lds;
  p.format = format;
  p.guard = {dev.fault, dev.bounds};
  p.x_vec = rows16(X, ldx, type_size(type));
  return launch_status(launch_fp8_quantize(type, block_rows, block_cols, p, reinterpret_cast<cudaStream_t>(stream)));
}

int sgemm_fp8_rmsnorm(int64_t rows, int64_t cols, int type, const void* X, int64_t ldx, const void* R, int64_t ldr,
                      const void* W, float eps, void* H, int64_t ldh, void* Y, int64_t ldy, void* codes, int64_t ldq,
                      float* scale, int64_t lds, float* rstd, struct CUstream_st* stream) {
  if (rows < 0) return -1;
  if (cols < 0) return -2;
  if (!known_type(type)) return -3;
  const int size = type_size(type);
  const bool work = rows > 0 && cols > 0;
  const int64_t min_ld = std::max<int64_t>(1, cols);
  if (work && (!X || !aligned(X, size))) return -4;
  if (ldx < min_ld) return -5;
  if (R && !aligned(R, size)) return -6;
  if (R && ldr < min_ld) return -7;
  if (work && (!W || !aligned(W, size))) return -8;
  if (!(eps >= 0.0f)) return -9;
  if (H && !aligned(H, size)) return -10;
  if (H && (ldh < min_ld || other_stride(H, ldh, X, ldx, rows) || other_stride(H, ldh, R, ldr, rows))) return -11;
  if (Y && !aligned(Y, size)) return -12;
  if (Y && ldy < min_ld) return -13;
  if (codes && ldq < min_ld) return -15;
  if (work && codes && (!scale || !aligned(scale, 4))) return -16;
  if (codes && lds < std::max<int64_t>(1, ceil_div(cols, 128))) return -17;
  if (rstd && !aligned(rstd, 4)) return -18;
  if (rows == 0 || (cols == 0 && !rstd)) return SGEMM_OK;
  if (rows > kMaxDim || cols > kMaxDim) return SGEMM_ERR_UNSUPPORTED;
  CallDevice dev;
  const int s = call_device(&dev);
  if (s != SGEMM_OK) return s;
  if (cols == 0)  // the mean of nothing: NaNs
    return launch_status(cudaMemsetAsync(rstd, 0xFF, (size_t)rows * 4, reinterpret_cast<cudaStream_t>(stream)));
  NormParams p;
  p.rows = rows;
  p.cols = (int)cols;
  p.x = X;
  p.ldx = ldx;
  p.r = R;
  p.ldr = ldr;
  p.w = W;
  p.eps = eps;
  p.h = H;
  p.ldh = ldh;
  p.y = Y;
  p.ldy = ldy;
  p.q = static_cast<uint8_t*>(codes);
  p.ldq = ldq;
  p.s = scale;
  p.lds = lds;
  p.rstd = rstd;
  p.guard = {dev.fault, dev.bounds};
  p.vec = rows16(X, ldx, size) && rows16(R, ldr, size) && rows16(W, 0, size) && rows16(H, ldh, size) &&
          rows16(Y, ldy, size) && cols % 8 == 0;
  return launch_status(launch_fp8_rmsnorm(type, p, reinterpret_cast<cudaStream_t>(stream)));
}

int sgemm_fp8_rmsnorm_backward(int64_t rows, int64_t cols, int type, const void* dY, int64_t lddy, const void* H,
                               int64_t ldh, const void* W, const float* rstd, const void* dH, int64_t lddh, void* dX,
                               int64_t lddx, float* dW, struct CUstream_st* stream_) {
  if (rows < 0) return -1;
  if (cols < 0) return -2;
  if (!known_type(type)) return -3;
  const int size = type_size(type);
  const bool work = rows > 0 && cols > 0;
  const int64_t min_ld = std::max<int64_t>(1, cols);
  if (work && (!dY || !aligned(dY, size))) return -4;
  if (lddy < min_ld) return -5;
  if (work && (!H || !aligned(H, size))) return -6;
  if (ldh < min_ld) return -7;
  if (work && (!W || !aligned(W, size))) return -8;
  if (work && (!rstd || !aligned(rstd, 4))) return -9;
  if (dH && !aligned(dH, size)) return -10;
  if (dH && lddh < min_ld) return -11;
  if (work && (!dX || !aligned(dX, size))) return -12;
  if (lddx < min_ld) return -13;
  if (work && (other_stride(dX, lddx, dY, lddy, rows) || other_stride(dX, lddx, dH, lddh, rows))) return -13;
  if (dW && !aligned(dW, 4)) return -14;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (cols == 0 || (rows == 0 && !dW)) return SGEMM_OK;
  if (rows > kMaxDim || cols > kNormGradMaxCols) return SGEMM_ERR_UNSUPPORTED;
  CallDevice dev;
  const int s = call_device(&dev);
  if (s != SGEMM_OK) return s;
  if (rows == 0) return launch_status(cudaMemsetAsync(dW, 0, (size_t)cols * 4, stream));  // a sum of nothing
  NormGradParams p;
  p.rows = rows;
  p.cols = (int)cols;
  p.dy = dY;
  p.lddy = lddy;
  p.h = H;
  p.ldh = ldh;
  p.w = W;
  p.rstd = rstd;
  p.dh = dH;
  p.lddh = lddh;
  p.dx = dX;
  p.lddx = lddx;
  p.dw = dW;
  p.vec = rows16(dY, lddy, size) && rows16(H, ldh, size) && rows16(W, 0, size) && rows16(dH, lddh, size) &&
          rows16(dX, lddx, size) && cols % 8 == 0;
  p.timeout_ns = wait_timeout_ns();
  p.fault = dev.fault;
  p.guard = {dev.fault, dev.bounds};
  const int grid = fp8_rmsnorm_backward_grid(type, rows, (int)cols, p.vec != 0, dev.sm_count);
  if (dW) {
    void* ws = nullptr;
    cudaError_t e = cudaMallocFromPoolAsync(&ws, (size_t)grid * cols * 4, dev.pool, stream);
    if (e != cudaSuccess) {
      record_cuda_failure(e);
      return e == cudaErrorMemoryAllocation ? SGEMM_ERR_NOMEM : SGEMM_ERR_CUDA;
    }
    p.partial = static_cast<float*>(ws);
  }
  cudaError_t e = launch_fp8_rmsnorm_backward(type, p, grid, stream);
  if (p.partial) {
    const cudaError_t ef = cudaFreeAsync(p.partial, stream);
    if (e == cudaSuccess) e = ef;
  }
  return launch_status(e);
}

int sgemm_fp8_moe(int64_t tokens, int64_t hidden, int64_t inner, int64_t experts, int top_k,
                  const sgemm_fp8_matrix_t* X, const float* logits, int64_t ldl, int renormalize,
                  const sgemm_fp8_experts_t* gate, const sgemm_fp8_experts_t* up, const sgemm_fp8_experts_t* down,
                  void* Y, int64_t ldy, int type, struct CUstream_st* stream_) {
  if (tokens < 0) return -1;
  if (hidden < 0) return -2;
  if (inner < 0) return -3;
  if (experts < 0) return -4;
  if (top_k < 0 || top_k > experts) return -5;
  const bool work = tokens > 0 && hidden > 0, read = work && inner > 0 && top_k > 0;
  Operand x;
  if (!check_operand(X, tokens, hidden, false, read, &x)) return -6;
  if (X && (X->format != SGEMM_FP8_E4M3 || X->block_rows != 1)) return -6;
  if (read && (!logits || !aligned(logits, 4))) return -7;
  if (ldl < std::max<int64_t>(1, experts)) return -8;
  if (!check_experts(gate, inner, hidden, experts, read)) return -10;
  if (!check_experts(up, inner, hidden, experts, read)) return -11;
  if (!check_experts(down, hidden, inner, experts, read)) return -12;
  if (!known_type(type)) return -15;
  if (work && (!Y || !aligned(Y, type_size(type)))) return -13;
  if (ldy < std::max<int64_t>(1, hidden)) return -14;
  if (!work) return SGEMM_OK;
  if (tokens > kMoeMaxTokens || experts > kMoeMaxExperts || top_k > kMoeMaxTopK || hidden % 16 != 0 ||
      inner % 16 != 0 || hidden > kMaxDim || inner > kMaxDim || ldy > INT_MAX || (X && X->ld > INT_MAX))
    return SGEMM_ERR_UNSUPPORTED;
  CallDevice dev;
  const int s = call_device(&dev);
  if (s != SGEMM_OK) return s;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (!read) {  // a sum of nothing
    return launch_status(cudaMemset2DAsync(Y, (size_t)ldy * type_size(type), 0, (size_t)hidden * type_size(type),
                                           (size_t)tokens, stream));
  }
  MoeParams p;
  p.tokens = (int)tokens;
  p.hidden = (int)hidden;
  p.inner = (int)inner;
  p.experts = (int)experts;
  p.top_k = top_k;
  p.renormalize = renormalize != 0;
  p.logits = logits;
  p.ldl = ldl;
  p.sx = X->scale;
  p.ldsx = X->lds;
  p.sg = gate->scale;
  p.su = up->scale;
  p.sd = down->scale;
  p.ldsg = gate->lds;
  p.ldsu = up->lds;
  p.ldsd = down->lds;
  p.stride_sg = gate->stride_scale;
  p.stride_su = up->stride_scale;
  p.stride_sd = down->stride_scale;
  p.h_groups = (int)ceil_div(inner, 64);
  p.y = Y;
  p.ldy = ldy;
  p.bf16 = type == SGEMM_BF16;
  p.slots_max = (int)tokens * top_k;
  p.active_max = (int)std::min<int64_t>(experts, p.slots_max);
  p.timeout_ns = wait_timeout_ns();
  p.fault = dev.fault;
  p.guard = {dev.fault, dev.bounds};
  shape_fp8_moe(&p, dev.sm_count);
  uint8_t* x_copy = nullptr;
  const auto place = [&](Pieces* w) {
    p.h = w->take<uint8_t>(2 * (int64_t)p.slots_max * inner);
    p.sh = w->take<float>((int64_t)p.slots_max * p.h_groups);
    p.arrived = w->take<int>(ceil_div(hidden, 128));
    p.route = w->take<int>(2 + 2 * (int64_t)p.active_max + 2 * (int64_t)p.slots_max + tokens);
    p.part = w->take<float>(2 * (int64_t)p.down_grid * tokens * 128);
    x_copy = w->take<uint8_t>(repack_bytes(x));
  };
  Pieces count;
  place(&count);
  void* ws = nullptr;
  cudaError_t e = cudaMallocFromPoolAsync(&ws, (size_t)count.at, dev.pool, stream);
  if (e != cudaSuccess) {
    record_cuda_failure(e);
    return e == cudaErrorMemoryAllocation ? SGEMM_ERR_NOMEM : SGEMM_ERR_CUDA;
  }
  Pieces w;
  w.base = static_cast<uint8_t*>(ws);
  place(&w);
  MoeMaps maps;
  e = operand_map(x, tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64, &x_copy, &maps.x, p.guard, stream);
  if (e == cudaSuccess) e = experts_map(*gate, inner, hidden, experts, 64, &maps.gate);
  if (e == cudaSuccess) e = experts_map(*up, inner, hidden, experts, 64, &maps.up);
  if (e == cudaSuccess) e = experts_map(*down, hidden, inner, experts, 128, &maps.down);
  if (e == cudaSuccess) e = encode_fp8_map(p.h, inner, 2 * (int64_t)p.slots_max, inner, 32, &maps.h);
  if (e == cudaSuccess) e = launch_fp8_moe(maps, p, dev.sm_count, stream);
  const cudaError_t ef = cudaFreeAsync(ws, stream);
  return launch_status(e == cudaSuccess ? ef : e);
}

}  // extern "C"

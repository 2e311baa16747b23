// api_linear.cu -- the C ABI of the operators on BF16 layers (sgemm_linear.h): argument checks, workspace and launches.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdint>
#include <iterator>

#include "linear_internal.h"
#include "sgemm_internal.h"
#include "sgemm_linear.h"

using namespace sgemm_impl;

namespace {

constexpr int64_t kMaxDim = INT_MAX - 1024;  // indices of the kernels' last tiles stay below 2^31

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round8(int64_t n) { return ceil_div(n, 8) * 8; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int type_size(int type) { return type == SGEMM_BF16 ? 2 : 4; }
bool known_type(int type) { return type == SGEMM_F32 || type == SGEMM_BF16; }
bool known_act(int act) { return act >= SGEMM_ACT_NONE && act <= SGEMM_ACT_GELU_TANH; }

// Whether rows of elements of `size` bytes start at multiples of `n` bytes.
bool rows_at(const void* p, int64_t ld, int size, int n) { return aligned(p, n) && ld * size % n == 0; }

// A matrix argument: its memory is there (where it is used), aligned to its type, and its rows do not overlap.
bool usable(const void* p, int size, bool used) { return !used || (p && aligned(p, size)); }
bool wide_enough(int64_t ld, int64_t cols) { return ld >= std::max<int64_t>(1, cols); }
// A kept matrix (checked as a whole: one argument).
bool usable_kept(const sgemm_kept_t* k, int64_t cols, bool work) {
  if (!k) return true;
  if (!wide_enough(k->ld, cols) || k->ld > kMaxDim || !usable(k->data, k->scale ? 1 : 2, work)) return false;
  return !k->scale || (aligned(k->scale, 4) && wide_enough(k->lds, ceil_div(cols, 128)));
}

// ---------------------------------------------------------------- the choice of kernel

std::atomic<int> g_force_variant{SGEMM_VARIANT_AUTO}, g_force_tile{0}, g_force_split{0};

// A product: M x N over `segments` times K.
struct Shape {
  int64_t M = 0, N = 0, K = 0;
  int segments = 1, products = 1;
  bool gated = false, kept8 = false;
};

// Times in ns that the choice of kernel goes by.  In the pair kernel, by tile width: a K tile of 64, and the rest of a tile.
// On the short side: a K tile in a CTA that has its SM to itself, the rest of a tile, and what joining a tile's shares adds.
struct PairCost {
  int tile, k_ns, tile_ns;
};
constexpr PairCost kPairCost[] = {{256, 290, 1500}, {128, 190, 1200}, {64, 150, 1000}};
struct ShortCost {
  int tile, k_ns, tile_ns, join_ns;
};
constexpr ShortCost kShortCost[] = {{16, 160, 1200, 800}, {32, 170, 1600, 600}, {64, 220, 2400, 650}, {128, 300, 4000, 1200}};
constexpr double kPairLaunchNs = 4500, kShortLaunchNs = 2750;
constexpr double kSharedSm = 0.3;        // a K tile takes this much longer with a second CTA on the SM
constexpr double kSmBytesPerNs = 44.7;   // an SM's share of the memory bandwidth

// SMs that clusters of `split` CTAs can use at a time: groups of 4 or 8 do not fill every part of the chip.
int64_t cluster_sms(int sm_count, int split) {
  return split <= 2 ? sm_count : std::max(1, split == 4 ? sm_count * 18 / 19 : sm_count * 16 / 19);
}

bool short_alone(int tile, bool gated) { return gated || tile == 128; }  // one CTA per SM
int64_t short_ring(int tile, bool gated) { return (short_alone(tile, gated) ? 2 : 1) * 98 * 1024; }

bool pair_tile_fits(int tile, const Shape& s) {
  return s.gated ? tile >= (s.kept8 ? 256 : 128) : tile >= (s.kept8 ? 128 : 64);
}

struct Choice {
  int variant = 0, tile = 0, split = 1;
  double ns = 1e30;
};

// The cheapest launch, among the variant, tile and split that are forced (0: any); clusters: CTA pairs that run at a time, 0
// on a device without clusters, where only unshared tiles can run.
Choice choose(const Shape& s, int64_t clusters, int sm_count, int variant, int tile, int split) {
  const int64_t kt = ceil_div(s.K, 64) * s.segments;
  Choice best;
  const auto offer = [&](int v, int n, int k, double ns) {
    if (ns < best.ns) best = Choice{v, n, k, ns};
  };
  const auto forced_here = [&](const auto& tiles, const auto& fits) {
    return std::any_of(std::begin(tiles), std::end(tiles), [&](int t) { return t == tile && fits(t); });
  };
  if (variant != SGEMM_VARIANT_LINEAR_SHORT && clusters > 0) {
    const bool only = forced_here(kLinearPairTiles, [&](int t) { return pair_tile_fits(t, s); });
    for (const PairCost& c : kPairCost) {
      if (!pair_tile_fits(c.tile, s) || (only && c.tile != tile)) continue;
      const int64_t tiles = ceil_div(s.M, 256) * ceil_div(s.N, s.gated ? c.tile / 2 : c.tile) * s.products;
      offer(SGEMM_VARIANT_LINEAR_PAIR, c.tile, 1, kPairLaunchNs + (double)ceil_div(tiles, clusters) * (kt * c.k_ns + c.tile_ns));
    }
  }
  if (variant != SGEMM_VARIANT_LINEAR_PAIR) {
    const auto fits = [&](int t) { return !s.gated || t < 128; };
    const bool only = forced_here(kLinearShortTiles, fits);
    for (const ShortCost& c : kShortCost) {
      if (!fits(c.tile) || (only ? c.tile != tile : c.tile > 16 && c.tile >= 2 * s.M)) continue;
      const int64_t tiles = ceil_div(s.N, 128) * ceil_div(s.M, c.tile);
      if (tiles * 8 > INT_MAX) continue;
      const int wide = s.gated ? 2 : 1;
      for (int k = 1; k <= 8; k *= 2) {
        if (clusters == 0 && k > 1) break;
        if (split != 0 ? split != k : k > 1 && kt < 2 * k) continue;  // two K tiles per CTA at least
        const int per_sm = short_alone(c.tile, s.gated) ? 1 : 2;
        const double on_sm = std::min((double)per_sm, std::max(1.0, (double)tiles * k / sm_count));
        const double one = std::max(c.k_ns * wide * (1.0 + kSharedSm * (on_sm - 1.0)), on_sm * (16384 * wide + 64 * c.tile) / kSmBytesPerNs);
        const double rounds = (double)ceil_div(tiles * k, cluster_sms(sm_count, k) * per_sm);
        offer(SGEMM_VARIANT_LINEAR_SHORT, c.tile, k,
              s.products * (kShortLaunchNs + rounds * (ceil_div(kt, k) * one + c.tile_ns + (k > 1 ? c.join_ns : 0))));
      }
    }
  }
  return best;
}

int plan_shape(const Shape& s, bool s_mn, int sm_count, int pair_clusters, sgemm_plan_t* plan) {
  *plan = sgemm_plan_t{};
  plan->split_k = 1;
  const int64_t clusters = pair_clusters >= 0 ? pair_clusters : std::max(1, sm_count / 2);
  const Choice c = choose(s, clusters, sm_count, g_force_variant.load(), g_force_tile.load(), g_force_split.load());
  if (c.variant == 0) return SGEMM_ERR_UNSUPPORTED;  // forced to what needs clusters
  plan->variant = c.variant;
  plan->tile_k = 64;
  plan->kernel_launches = 1;
  plan->grid_y = 1;
  int64_t tiles;
  if (c.variant == SGEMM_VARIANT_LINEAR_PAIR) {
    plan->tile_m = 256;
    plan->tile_n = c.tile;
    plan->stages = kLinearPairStages;
    plan->threads = kLinearPairThreads;
    plan->smem_bytes = linear_pair_smem();
    tiles = ceil_div(s.M, 256) * ceil_div(s.N, s.gated ? c.tile / 2 : c.tile) * s.products;
    plan->grid_x = 2 * std::min<int64_t>(tiles, clusters);
    if (ceil_div(tiles, clusters) * ceil_div(s.K, 64) * s.segments > INT_MAX) return SGEMM_ERR_UNSUPPORTED;
  } else {
    plan->tile_m = 128;
    plan->tile_n = c.tile;
    plan->split_k = c.split;
    plan->kernel_launches = s.products;
    tiles = ceil_div(s.N, 128) * ceil_div(s.M, c.tile);
    const int64_t stage = (s.gated ? 2 : 1) * 16384 + (s_mn ? std::max(1, c.tile / 64) * 8192 : c.tile * 128);
    plan->stages = (int)std::min<int64_t>(kLinearShortMaxStages, short_ring(c.tile, s.gated) / stage);
    plan->threads = kLinearShortThreads;
    plan->smem_bytes = linear_short_smem(c.tile, s.gated, plan->stages, (int)stage);
    plan->grid_x = tiles * c.split;
  }
  plan->dp_tiles = tiles;
  return tiles > INT_MAX || plan->grid_x > INT_MAX ? SGEMM_ERR_UNSUPPORTED : SGEMM_OK;
}

// ---------------------------------------------------------------- operands and workspace

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

// A stored matrix of a product.  TMA reads BF16 rows that start at multiples of 16 bytes; others are copied first.
struct Operand {
  LinearKeptIn m;
  int64_t rows = 0, cols = 0;  // stored
  int mn = 0;                  // the stored rows run along the output, not along k
  void* copy = nullptr;
  bool copied = false;

  Operand() = default;
  Operand(const void* p, int64_t ld, const float* scale, int64_t lds, int64_t rows_, int64_t cols_, int mn_) : rows(rows_), cols(cols_), mn(mn_) {
    m.data = p;
    m.ld = ld;
    m.scale = scale;
    m.lds = lds;
    m.vec = scale ? rows_at(p, ld, 1, 8) : rows_at(p, ld, 2, 16);
    copied = scale || !aligned(p, 16) || (ld % 8 != 0 && rows > 1);
  }
  void place(Pieces* w) {
    if (copied) copy = w->take<uint16_t>(rows * round8(cols));
  }
  // Copies it where it needs that; an operand that several products read is copied once.
  cudaError_t make(const Guard& g, cudaStream_t stream) {
    if (!copied) return cudaSuccess;
    return launch_linear_expand(m, rows, cols, copy, round8(cols), g, stream);
  }
  cudaError_t map(int box_rows, CUtensorMap* out) const {
    const int64_t ld = copied || rows == 1 ? round8(cols) : m.ld;  // (a map wants a stride even where it steps over nothing)
    return encode_linear_map(copied ? copy : m.data, cols, rows, ld, mn ? 64 : box_rows, out);
  }
};

// Tensor-core instruction descriptor, kind::f16: FP32 accumulator, BF16 operands, their orders (1: MN-major), N and M.
uint32_t instruction(int a_mn, int b_mn, int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}

struct Product {
  Shape shape;
  Operand *a[2] = {nullptr, nullptr}, *b[2] = {nullptr, nullptr};  // the second of each: as the kernel's maps
  LinearOut out;
};

bool tma_writes(const void* p, int64_t ld, int64_t cols, int size) { return rows_at(p, ld, size, 16) && cols * size % 16 == 0; }

cudaError_t launch_product(Product& pr, const sgemm_plan_t& plan, const CallDevice& dev, cudaStream_t stream) {
  LinearOut& o = pr.out;
  const Shape& s = pr.shape;
  o.M = (int)s.M;
  o.N = (int)s.N;
  o.guard = {dev.fault, dev.bounds};
  o.bias_vec = aligned(o.bias, 16);
  const int size = o.f32 ? 4 : 2;
  const bool pair = plan.variant == SGEMM_VARIANT_LINEAR_PAIR;
  o.r_vec = rows_at(o.residual, o.ldr, 2, 16);
  LinearMaps maps = {};
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 2; ++i) {
    if (o.d[i]) {
      o.d_tma[i] = tma_writes(o.d[i], o.ldd[i], s.N, size);
      o.d_vec[i] = rows_at(o.d[i], o.ldd[i], size, 4 * size);
      if (pair && o.d_tma[i] && e == cudaSuccess) e = encode_out_map(o.d[i], s.N, s.M, o.ldd[i], !o.f32, &maps.d[i]);
    }
    LinearKept& k = o.kept[i];
    if (k.data) {
      k.vec = o.keep == 2 ? rows_at(k.data, k.ld, 1, 16) : tma_writes(k.data, k.ld, s.N, 2);
      o.kept_vec8[i] = rows_at(k.data, k.ld, 2, 8);
      if (pair && o.keep == 1 && k.vec && e == cudaSuccess) e = encode_out_map(k.data, s.N, s.M, k.ld, true, &maps.kept[i]);
    }
    const int tile = plan.tile_n;
    if (pr.a[i] && e == cudaSuccess) e = pr.a[i]->map(pair ? 128 : tile, &maps.a[i]);
    if (pr.b[i] && e == cudaSuccess) e = pr.b[i]->map(pair ? tile / 2 : 128, &maps.b[i]);
  }
  if (e != cudaSuccess) return e;
  if (pair) {
    LinearPairParams p;
    p.out = o;
    p.k_tiles = (int)ceil_div(s.K, 64);
    p.segments = s.segments;
    p.products = s.products;
    p.a_mn = pr.a[0]->mn;
    p.b_mn = pr.b[0]->mn;
    p.idesc = instruction(p.a_mn, p.b_mn, 256, plan.tile_n);
    p.tiles_m = (int)ceil_div(s.M, 256);
    p.tiles_n = (int)ceil_div(s.N, s.gated ? plan.tile_n / 2 : plan.tile_n);
    p.clusters = (int)(plan.grid_x / 2);
    p.timeout_ns = wait_timeout_ns();
    p.fault = dev.fault;
    return launch_linear_pair(plan.tile_n, s.gated, maps, p, stream);
  }
  LinearShortParams p;
  p.out = o;
  p.k_tiles = (int)ceil_div(s.K, 64);
  p.segments = s.segments;
  p.l_mn = pr.b[0]->mn;
  p.s_mn = pr.a[0]->mn;
  p.idesc = instruction(p.l_mn, p.s_mn, 128, plan.tile_n);
  p.tile_s = plan.tile_n;
  p.tiles_l = (int)ceil_div(s.N, 128);
  p.tiles_s = (int)ceil_div(s.M, plan.tile_n);
  p.split = plan.split_k;
  p.stages = plan.stages;
  p.stage_bytes = (s.gated ? 2 : 1) * 16384 + (p.s_mn ? std::max(1, plan.tile_n / 64) * 8192 : plan.tile_n * 128);
  p.timeout_ns = wait_timeout_ns();
  p.fault = dev.fault;
  for (int i = 0; i < s.products && e == cudaSuccess; ++i) {
    if (i == 1) {  // its own A and output, the same B
      maps.a[0] = maps.a[1];
      p.out.d[0] = o.d[1];
      p.out.ldd[0] = o.ldd[1];
      p.out.d_vec[0] = o.d_vec[1];
    }
    e = launch_linear_short(s.gated, maps, p, stream);
  }
  return e;
}

// Plans a product, and launches it.
int run_product(Product& pr, const CallDevice& dev, cudaStream_t stream, cudaError_t* e) {
  sgemm_plan_t plan;
  const int s = plan_shape(pr.shape, pr.a[0]->mn != 0, dev.sm_count, dev.pair_clusters, &plan);
  if (s != SGEMM_OK) return s;
  *e = launch_product(pr, plan, dev, stream);
  return SGEMM_OK;
}

// What is kept, as the kernels take it: 0 nothing, 1 BF16, 2 8-bit.
int keep_of(const sgemm_kept_t* k, LinearKept* out) {
  if (!k) return 0;
  out->data = k->data;
  out->ld = k->ld;
  out->scale = k->scale;
  out->lds = k->lds;
  return k->scale ? 2 : 1;
}
LinearKeptIn kept_in(const sgemm_kept_t* k) {
  LinearKeptIn m;
  if (!k) return m;
  m.data = k->data;
  m.ld = k->ld;
  m.scale = k->scale;
  m.lds = k->lds;
  m.vec = k->scale ? rows_at(k->data, k->ld, 1, 8) : rows_at(k->data, k->ld, 2, 16);
  return m;
}

int no_memory(cudaError_t e) {
  record_cuda_failure(e);
  return e == cudaErrorMemoryAllocation ? SGEMM_ERR_NOMEM : SGEMM_ERR_CUDA;
}
int launch_status(cudaError_t e) { return e == cudaSuccess ? SGEMM_OK : record_cuda_failure(e); }

// Allocates the workspace that `place` lays out, runs `work` (a status; CUDA's error in its argument) and frees it.
template <typename Place, typename Work>
int with_workspace(const CallDevice& dev, cudaStream_t stream, const Place& place, const Work& work) {
  Pieces w;
  place(&w);
  void* ws = nullptr;
  if (w.at > 0) {
    const cudaError_t e = cudaMallocFromPoolAsync(&ws, (size_t)w.at, dev.pool, stream);
    if (e != cudaSuccess) return no_memory(e);
    w = Pieces{static_cast<uint8_t*>(ws), 0};
    place(&w);
  }
  cudaError_t e = cudaSuccess;
  const int s = work(&e);
  if (ws) {
    const cudaError_t ef = cudaFreeAsync(ws, stream);
    if (e == cudaSuccess) e = ef;
  }
  return s != SGEMM_OK ? s : launch_status(e);
}

cudaError_t zero_rows(void* p, int64_t ld, int64_t rows, int64_t cols, int size, cudaStream_t stream) {
  return cudaMemset2DAsync(p, (size_t)ld * size, 0, (size_t)cols * size, (size_t)rows, stream);
}

bool too_large(std::initializer_list<int64_t> v) {
  return std::any_of(v.begin(), v.end(), [](int64_t x) { return x > kMaxDim; });
}

// The forward products: X (W0, gated: W1)^T with their epilogue.
int forward(int64_t tokens, int64_t inputs, int64_t outputs, const void* X, int64_t ldx, const void* W0, int64_t ldw0, const void* W1,
            int64_t ldw1, Product& pr, cudaStream_t stream) {
  CallDevice dev;
  const int s = linear_device(&dev);
  if (s != SGEMM_OK) return s;
  const bool gated = W1 != nullptr || pr.shape.gated;
  const bool empty = inputs == 0;  // a sum of nothing: 8 zeros per row instead
  const int64_t K = empty ? 8 : inputs;
  void* zeros = nullptr;
  Operand x(X, ldx, nullptr, 0, tokens, K, 0), w0(W0, ldw0, nullptr, 0, outputs, K, 0), w1(W1, ldw1, nullptr, 0, outputs, K, 0);
  if (empty) x.copied = w0.copied = w1.copied = false;
  pr.shape.M = tokens;
  pr.shape.N = outputs;
  pr.shape.K = K;
  pr.shape.gated = gated;
  pr.shape.kept8 = pr.out.keep == 2;
  pr.a[0] = &x;
  pr.b[0] = &w0;
  if (gated) pr.b[1] = &w1;
  return with_workspace(
      dev, stream,
      [&](Pieces* w) {
        if (empty) zeros = w->take<uint16_t>(8 * std::max(tokens, outputs));
        x.place(w);
        w0.place(w);
        if (gated) w1.place(w);
      },
      [&](cudaError_t* e) {
        const Guard g{dev.fault, dev.bounds};
        if (empty) {
          for (Operand* o : {&x, &w0, &w1}) o->m.data = zeros, o->m.ld = 8;
          *e = cudaMemsetAsync(zeros, 0, (size_t)std::max(tokens, outputs) * 16, stream);
        }
        if (*e == cudaSuccess) *e = x.make(g, stream);
        if (*e == cudaSuccess) *e = w0.make(g, stream);
        if (*e == cudaSuccess && gated) *e = w1.make(g, stream);
        return *e == cudaSuccess ? run_product(pr, dev, stream, e) : SGEMM_OK;
      });
}

}  // namespace

extern "C" {

int sgemm_linear(int64_t tokens, int64_t inputs, int64_t outputs, const void* X, int64_t ldx, const void* W, int64_t ldw, const void* bias,
                 int activation, const void* R, int64_t ldr, const sgemm_kept_t* kept, void* Y, int64_t ldy, int type,
                 struct CUstream_st* stream) {
  if (tokens < 0) return -1;
  if (inputs < 0) return -2;
  if (outputs < 0) return -3;
  const bool work = tokens > 0 && outputs > 0, read = work && inputs > 0;
  if (!usable(X, 2, read)) return -4;
  if (!wide_enough(ldx, inputs)) return -5;
  if (!usable(W, 2, read)) return -6;
  if (!wide_enough(ldw, inputs)) return -7;
  if (!usable(bias, 2, work && bias)) return -8;
  if (!known_act(activation)) return -9;
  if (!usable(R, 2, work && R)) return -10;
  if (R && !wide_enough(ldr, outputs)) return -11;
  if (!usable_kept(kept, outputs, work)) return -12;
  if (!known_type(type)) return -15;
  if (!usable(Y, type_size(type), work) || (work && Y == R && type != SGEMM_BF16)) return -13;
  if (!wide_enough(ldy, outputs) || (work && Y == R && tokens > 1 && ldy != ldr)) return -14;
  if (!work) return SGEMM_OK;
  if (too_large({tokens, inputs, outputs, ldx, ldw, ldy, R ? ldr : 0})) return SGEMM_ERR_UNSUPPORTED;
  Product pr;
  pr.out.d[0] = Y;
  pr.out.ldd[0] = ldy;
  pr.out.f32 = type == SGEMM_F32;
  pr.out.bias = bias;
  pr.out.residual = R;
  pr.out.ldr = ldr;
  pr.out.act = activation;
  pr.out.keep = keep_of(kept, &pr.out.kept[0]);
  return forward(tokens, inputs, outputs, X, ldx, W, ldw, nullptr, 0, pr, reinterpret_cast<cudaStream_t>(stream));
}

int sgemm_gated(int64_t tokens, int64_t inputs, int64_t outputs, const void* X, int64_t ldx, const void* gate, int64_t ldg, const void* up,
                int64_t ldu, int activation, const sgemm_kept_t* kept_gate, const sgemm_kept_t* kept_up, void* H, int64_t ldh,
                struct CUstream_st* stream) {
  if (tokens < 0) return -1;
  if (inputs < 0) return -2;
  if (outputs < 0) return -3;
  const bool work = tokens > 0 && outputs > 0, read = work && inputs > 0;
  if (!usable(X, 2, read)) return -4;
  if (!wide_enough(ldx, inputs)) return -5;
  if (!usable(gate, 2, read)) return -6;
  if (!wide_enough(ldg, inputs)) return -7;
  if (!usable(up, 2, read)) return -8;
  if (!wide_enough(ldu, inputs)) return -9;
  if (!known_act(activation)) return -10;
  if (!usable_kept(kept_gate, outputs, work)) return -11;
  if (!usable_kept(kept_up, outputs, work) || !kept_gate != !kept_up || (kept_up && !kept_gate->scale != !kept_up->scale)) return -12;
  if (!usable(H, 2, work)) return -13;
  if (!wide_enough(ldh, outputs)) return -14;
  if (!work) return SGEMM_OK;
  if (too_large({tokens, inputs, outputs, ldx, ldg, ldu, ldh})) return SGEMM_ERR_UNSUPPORTED;
  Product pr;
  pr.shape.gated = true;
  pr.out.d[0] = H;
  pr.out.ldd[0] = ldh;
  pr.out.act = activation;
  pr.out.keep = keep_of(kept_gate, &pr.out.kept[0]);
  keep_of(kept_up, &pr.out.kept[1]);
  return forward(tokens, inputs, outputs, X, ldx, gate, ldg, up, ldu, pr, reinterpret_cast<cudaStream_t>(stream));
}

int sgemm_linear_backward(int64_t tokens, int64_t inputs, int64_t outputs, const void* dY, int64_t lddy, const sgemm_kept_t* X,
                          const void* W, int64_t ldw, int activation, const sgemm_kept_t* kept, void* dX, int64_t lddx, void* dW,
                          int64_t lddw, int dw_type, float* dbias, struct CUstream_st* stream_) {
  if (tokens < 0) return -1;
  if (inputs < 0) return -2;
  if (outputs < 0) return -3;
  const bool read = tokens > 0 && outputs > 0, work = read && inputs > 0;
  if (!known_type(dw_type)) return -15;
  if (!known_act(activation)) return -9;
  if (!usable(dY, 2, read && (dX || dW || dbias))) return -4;
  if (!wide_enough(lddy, outputs)) return -5;
  if (dW && (!X || !usable_kept(X, inputs, work))) return -6;
  if (dX && !usable(W, 2, work)) return -7;
  if (dX && !wide_enough(ldw, inputs)) return -8;
  if (activation != SGEMM_ACT_NONE && (!kept || !usable_kept(kept, outputs, read))) return -10;
  if (!usable(dX, 2, dX != nullptr)) return -11;
  if (dX && !wide_enough(lddx, inputs)) return -12;
  if (!usable(dW, type_size(dw_type), dW != nullptr)) return -13;
  if (dW && !wide_enough(lddw, inputs)) return -14;
  if (!usable(dbias, 4, dbias != nullptr)) return -16;
  if (too_large({tokens, inputs, outputs, lddy, dX ? ldw : 0, dX ? lddx : 0, dW ? lddw : 0})) return SGEMM_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (tokens == 0 || inputs == 0 || outputs == 0) {  // nothing, or sums of nothing
    if (tokens == 0) {
      cudaError_t e = cudaSuccess;
      if (dW && inputs > 0 && outputs > 0) e = zero_rows(dW, lddw, outputs, inputs, type_size(dw_type), stream);
      if (e == cudaSuccess && dbias && outputs > 0) e = cudaMemsetAsync(dbias, 0, (size_t)outputs * 4, stream);
      return launch_status(e);
    }
    if (outputs == 0) return dX && inputs > 0 ? launch_status(zero_rows(dX, lddx, tokens, inputs, 2, stream)) : SGEMM_OK;
    dX = dW = nullptr;  // (no inputs: dbias alone)
  }
  if (!dX && !dW && !dbias) return SGEMM_OK;
  CallDevice dev;
  const int s = linear_device(&dev);
  if (s != SGEMM_OK) return s;
  const bool act = activation != SGEMM_ACT_NONE, products = dX || dW;
  LinearGradParams g;
  g.rows = tokens;
  g.cols = (int)outputs;
  g.dy = dY;
  g.lddy = lddy;
  g.dy_vec = rows_at(dY, lddy, 2, 16);
  if (act) g.a = kept_in(kept);
  g.act = activation;
  g.dbias = dbias;
  g.guard = {dev.fault, dev.bounds};
  g.row_blocks = linear_grad_row_blocks(tokens, (int)outputs, dev.sm_count);
  // dA: dY itself where it can be read as it is and there is no activation
  Operand d_n(dY, lddy, nullptr, 0, tokens, outputs, 0);
  const bool write = products && (act || d_n.copied);
  Operand w(W, ldw, nullptr, 0, outputs, inputs, 1);
  Operand x(X ? X->data : nullptr, X ? X->ld : 1, X ? X->scale : nullptr, X ? X->lds : 1, tokens, inputs, 1);
  const int64_t ldd = round8(outputs);
  return with_workspace(
      dev, stream,
      [&](Pieces* p) {
        g.da = write ? p->take<uint16_t>(tokens * ldd) : nullptr;
        g.partial = dbias && g.row_blocks > 1 ? p->take<float>((int64_t)g.row_blocks * outputs) : nullptr;
        if (dX) w.place(p);
        if (dW) x.place(p);
      },
      [&](cudaError_t* e) {
        g.ldd = ldd;
        if (write || dbias) *e = launch_linear_grad(g, stream);
        if (*e == cudaSuccess && dX) *e = w.make(g.guard, stream);
        if (*e == cudaSuccess && dW) *e = x.make(g.guard, stream);
        if (write) d_n = Operand(g.da, ldd, nullptr, 0, tokens, outputs, 0);
        int st = SGEMM_OK;
        if (*e == cudaSuccess && dX) {  // tokens x inputs over outputs
          Product pr;
          pr.shape.M = tokens;
          pr.shape.N = inputs;
          pr.shape.K = outputs;
          pr.a[0] = &d_n;
          pr.b[0] = &w;
          pr.out.d[0] = dX;
          pr.out.ldd[0] = lddx;
          st = run_product(pr, dev, stream, e);
        }
        if (*e == cudaSuccess && st == SGEMM_OK && dW) {  // outputs x inputs over tokens
          Operand d_t = d_n;
          d_t.mn = 1;
          Product pr;
          pr.shape.M = outputs;
          pr.shape.N = inputs;
          pr.shape.K = tokens;
          pr.a[0] = &d_t;
          pr.b[0] = &x;
          pr.out.d[0] = dW;
          pr.out.ldd[0] = lddw;
          pr.out.f32 = dw_type == SGEMM_F32;
          st = run_product(pr, dev, stream, e);
        }
        return st;
      });
}

int sgemm_gated_backward(int64_t tokens, int64_t inputs, int64_t outputs, const void* dH, int64_t lddh, const sgemm_kept_t* X,
                         const void* gate, int64_t ldg, const void* up, int64_t ldu, int activation, const sgemm_kept_t* kept_gate,
                         const sgemm_kept_t* kept_up, void* dX, int64_t lddx, void* dG, int64_t lddg, void* dU, int64_t lddu, int dw_type,
                         void* H, int64_t ldh, struct CUstream_st* stream_) {
  if (tokens < 0) return -1;
  if (inputs < 0) return -2;
  if (outputs < 0) return -3;
  const bool read = tokens > 0 && outputs > 0, work = read && inputs > 0;
  if (!usable(dH, 2, read && (dX || dG || dU || H))) return -4;
  if (!wide_enough(lddh, outputs)) return -5;
  if (dG && (!X || !usable_kept(X, inputs, work))) return -6;
  if (dX && !usable(gate, 2, work)) return -7;
  if (dX && !wide_enough(ldg, inputs)) return -8;
  if (dX && !usable(up, 2, work)) return -9;
  if (dX && !wide_enough(ldu, inputs)) return -10;
  if (!known_act(activation)) return -11;
  if (!kept_gate || !usable_kept(kept_gate, outputs, read)) return -12;
  if (!kept_up || !usable_kept(kept_up, outputs, read) || !kept_gate->scale != !kept_up->scale) return -13;
  if (!usable(dX, 2, dX != nullptr)) return -14;
  if (dX && !wide_enough(lddx, inputs)) return -15;
  if (!known_type(dw_type)) return -20;
  if (!usable(dG, type_size(dw_type), dG != nullptr)) return -16;
  if (dG && !wide_enough(lddg, inputs)) return -17;
  if (!usable(dU, type_size(dw_type), dU != nullptr) || !dG != !dU) return -18;
  if (dU && !wide_enough(lddu, inputs)) return -19;
  if (!usable(H, 2, H != nullptr)) return -21;
  if (H && !wide_enough(ldh, outputs)) return -22;
  if (too_large({tokens, inputs, outputs, lddh, dX ? ldg : 0, dX ? ldu : 0, dX ? lddx : 0, dG ? lddg : 0, dU ? lddu : 0, H ? ldh : 0}))
    return SGEMM_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (tokens == 0 || inputs == 0 || outputs == 0) {  // nothing, or sums of nothing
    if (tokens == 0) {
      cudaError_t e = cudaSuccess;
      if (dG && inputs > 0 && outputs > 0) e = zero_rows(dG, lddg, outputs, inputs, type_size(dw_type), stream);
      if (dG && inputs > 0 && outputs > 0 && e == cudaSuccess) e = zero_rows(dU, lddu, outputs, inputs, type_size(dw_type), stream);
      return launch_status(e);
    }
    if (outputs == 0) return dX && inputs > 0 ? launch_status(zero_rows(dX, lddx, tokens, inputs, 2, stream)) : SGEMM_OK;
    dX = dG = dU = nullptr;  // (no inputs: H alone)
  }
  if (!dX && !dG && !H) return SGEMM_OK;
  CallDevice dev;
  const int s = linear_device(&dev);
  if (s != SGEMM_OK) return s;
  LinearGradParams g;
  g.rows = tokens;
  g.cols = (int)outputs;
  g.dy = dH;
  g.lddy = lddh;
  g.dy_vec = rows_at(dH, lddh, 2, 16);
  g.a = kept_in(kept_gate);
  g.b = kept_in(kept_up);
  g.act = activation;
  g.h = H;
  g.ldh = ldh;
  g.h_vec = rows_at(H, ldh, 2, 16);
  g.guard = {dev.fault, dev.bounds};
  g.row_blocks = linear_grad_row_blocks(tokens, (int)outputs, dev.sm_count);
  Operand wg(gate, ldg, nullptr, 0, outputs, inputs, 1), wu(up, ldu, nullptr, 0, outputs, inputs, 1);
  Operand x(X ? X->data : nullptr, X ? X->ld : 1, X ? X->scale : nullptr, X ? X->lds : 1, tokens, inputs, 1);
  const int64_t ldd = round8(outputs);
  return with_workspace(
      dev, stream,
      [&](Pieces* p) {
        g.da = dX || dG ? p->take<uint16_t>(tokens * ldd) : nullptr;
        g.db = dX || dG ? p->take<uint16_t>(tokens * ldd) : nullptr;
        if (dX) {
          wg.place(p);
          wu.place(p);
        }
        if (dG) x.place(p);
      },
      [&](cudaError_t* e) {
        g.ldd = ldd;
        *e = launch_linear_grad(g, stream);
        if (*e == cudaSuccess && dX) *e = wg.make(g.guard, stream);
        if (*e == cudaSuccess && dX) *e = wu.make(g.guard, stream);
        if (*e == cudaSuccess && dG) *e = x.make(g.guard, stream);
        Operand da(g.da, ldd, nullptr, 0, tokens, outputs, 0), db(g.db, ldd, nullptr, 0, tokens, outputs, 0);
        int st = SGEMM_OK;
        if (*e == cudaSuccess && dX) {  // tokens x inputs, two sums over outputs
          Product pr;
          pr.shape.M = tokens;
          pr.shape.N = inputs;
          pr.shape.K = outputs;
          pr.shape.segments = 2;
          pr.a[0] = &da;
          pr.a[1] = &db;
          pr.b[0] = &wg;
          pr.b[1] = &wu;
          pr.out.d[0] = dX;
          pr.out.ldd[0] = lddx;
          st = run_product(pr, dev, stream, e);
        }
        if (*e == cudaSuccess && st == SGEMM_OK && dG) {  // twice outputs x inputs over tokens
          da.mn = db.mn = 1;
          Product pr;
          pr.shape.M = outputs;
          pr.shape.N = inputs;
          pr.shape.K = tokens;
          pr.shape.products = 2;
          pr.a[0] = &da;
          pr.a[1] = &db;
          pr.b[0] = &x;
          pr.out.d[0] = dG;
          pr.out.ldd[0] = lddg;
          pr.out.d[1] = dU;
          pr.out.ldd[1] = lddu;
          pr.out.f32 = dw_type == SGEMM_F32;
          st = run_product(pr, dev, stream, e);
        }
        return st;
      });
}

int sgemm_linear_plan(int64_t rows, int64_t cols, int64_t K, int gated, int kept8, int sm_count, sgemm_plan_t* plan) {
  if (rows < 1) return -1;
  if (cols < 1) return -2;
  if (K < 1) return -3;
  if (!plan) return -7;
  if (too_large({rows, cols, K})) return SGEMM_ERR_UNSUPPORTED;
  CallDevice dev;
  dev.sm_count = sm_count;
  dev.pair_clusters = -1;
  if (sm_count <= 0) {
    const int s = linear_device(&dev);
    if (s != SGEMM_OK) return s;
  }
  Shape s;
  s.M = rows;
  s.N = cols;
  s.K = K;
  s.gated = gated != 0;
  s.kept8 = kept8 != 0;
  return plan_shape(s, false, dev.sm_count, dev.pair_clusters, plan);
}

int sgemm_linear_set_override(int variant, int tile_n, int split) {
  if (variant != SGEMM_VARIANT_AUTO && variant != SGEMM_VARIANT_LINEAR_PAIR && variant != SGEMM_VARIANT_LINEAR_SHORT) return -1;
  const bool is_short = variant == SGEMM_VARIANT_LINEAR_SHORT;
  const auto is_in = [&](const auto& tiles) { return std::find(std::begin(tiles), std::end(tiles), tile_n) != std::end(tiles); };
  const bool known = is_short ? is_in(kLinearShortTiles) : variant == SGEMM_VARIANT_LINEAR_PAIR && is_in(kLinearPairTiles);
  if (tile_n != 0 && !known) return -2;
  if ((split != 0 && !is_short) || (split != 0 && split != 1 && split != 2 && split != 4 && split != 8)) return -3;
  g_force_variant.store(variant);
  g_force_tile.store(tile_n);
  g_force_split.store(split);
  return SGEMM_OK;
}

}  // extern "C"

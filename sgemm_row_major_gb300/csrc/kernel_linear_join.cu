// kernel_linear_join.cu -- the sums of products whose K tiles were shared by several units (kernel_linear_pair.cu), for sm_103a:
// added in the units' order, so that the result is the same every time, then what a layer does to them.
//
// A thread has up to 4 sums of 4 columns of a row on their way at once; 2, 4 or 8 threads share more than that (up to 32), whose
// parts are added through shared memory by the first of them, which does the rest.  (The sums lie in L2 as a rule, written just
// before.)  Two sums of 1024 x 1024 take 6.7 us with a cold L2; with them the weight gradient of 16384 tokens takes 39.4 us, and 43.5 with whole sums.
#include "linear_common.cuh"

namespace sgemm_impl {
namespace lin {
namespace {

constexpr int kThreads = 256, kEach = 4;
static_assert(kLinearMostShares <= 8 * kEach, "threads that share the sums");
int parts_of(int split) { return split <= kEach ? 1 : split <= 2 * kEach ? 2 : split <= 4 * kEach ? 4 : 8; }

__global__ void __launch_bounds__(kThreads) linear_join_kernel(const __grid_constant__ LinearJoinParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int which = 0;
  int64_t block = blockIdx.x;
  while (block >= p.part[which].blocks) block -= p.part[which++].blocks;
  const LinearJoin& t = p.part[which];
  const LinearJob& j = t.job;
  const LinearOut& o = p.out;
  const int chunks = (j.N + 3) / 4;
  const int parts = t.parts, per_block = kThreads / parts;
  const int part = (int)threadIdx.x / per_block, mine = (int)threadIdx.x % per_block;
  const int64_t i = block * per_block + mine, all = (int64_t)j.M * chunks;
  const bool there = i < all;
  const int row = !there ? 0 : all <= 0x7fffffff ? (int)((uint32_t)i / (uint32_t)chunks) : (int)(i / chunks);
  const int col = there ? (int)(i - (int64_t)row * chunks) * 4 : 0, n = min(4, j.N - col);
  const int64_t apart = (int64_t)t.rows_apart * t.ld, size = apart * t.split;
  const int64_t first = (int64_t)row * t.ld + col;  // (rows of the sums hold whole chunks)
  // this thread's sums: part, part + parts, ...
  float4 x[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int unit = part + parts * k;
    x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (there && unit < t.split && in_range(o.guard.fault, o.guard.word, f8::kSitePart, first + unit * apart, 4, size))
      x[k] = *reinterpret_cast<const float4*>(t.sums + first + unit * apart);
  }
  const auto plus = [](float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); };
  float4 s = x[0];
#pragma unroll
  for (int k = 1; k < kEach; ++k) s = plus(s, x[k]);
  if (parts > 1) {
    __shared__ float4 sums[kThreads];
    sums[threadIdx.x] = s;
    __syncthreads();
    if (part == 0)
      for (int k = 1; k < parts; ++k) s = plus(s, sums[k * per_block + mine]);
  }
  if (part != 0 || !there) return;
  float v[4] = {s.x, s.y, s.z, s.w};
  if (o.bias && in_range(o.guard.fault, o.guard.word, f8::kSiteIn, col, n, j.N)) {
    float x[4];
    get4(static_cast<const __nv_bfloat16*>(o.bias) + col, n, o.bias_vec, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += x[e];
  }
  if (o.keep && kept_ok(o, j, 0, row, col, n)) put4(static_cast<__nv_bfloat16*>(o.kept[0].data) + (int64_t)row * o.kept[0].ld + col, n, o.kept_vec8[0], v);
  with_act(o.act, [&](auto act) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) *reinterpret_cast<float2*>(&v[e]) = act_of<decltype(act)::value>(make_float2(v[e], v[e + 1]));
  });
  if (o.residual && r_ok(o, j, row, col, n)) {
    float x[4];
    get4(static_cast<const __nv_bfloat16*>(o.residual) + (int64_t)row * o.ldr + col, n, o.r_vec, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += x[e];
  }
  put_row(o, j, row, col, n, v);
}

}  // namespace
}  // namespace lin

cudaError_t launch_linear_join(LinearJoinParams& p, cudaStream_t stream) {
  int64_t blocks = 0;
  for (LinearJoin& t : p.part) {
    t.parts = lin::parts_of(t.split);
    const int64_t per_block = lin::kThreads / t.parts;
    t.blocks = t.sums ? ((int64_t)t.job.M * ((t.job.N + 3) / 4) + per_block - 1) / per_block : 0;
    blocks += t.blocks;
  }
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(lin::kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lin::linear_join_kernel, p);
}

}  // namespace sgemm_impl

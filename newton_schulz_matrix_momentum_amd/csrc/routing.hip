// Routing of tokens to experts: choice, weights and dispatch lists, the
// gradient of the weights, and the bias step that balances the experts.
//
// Forward: a wave takes a token; its lanes hold the token's scores.  Choices
// are decided in 64 bits, so near-equal ones fall as the definition says.
// The lists are a counting sort by expert that keeps the slots' order: each
// block counts its own slots, one block an expert turns the counts into the
// number of slots before, and every slot is then written to its place.
// Integer counts make every list reproducible.
#include "ckpt_code.h"

namespace muon {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * 64;

__device__ __forceinline__ double wave_max(double v) {
  for (int o = 32; o > 0; o >>= 1) v = fmax(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
// the larger value, the lower index among equals; values are never NaN here
__device__ __forceinline__ void wave_best(double &v, int &at) {
  for (int o = 32; o > 0; o >>= 1) {
    const double w = __shfl_xor(v, o, 64);
    const int i = __shfl_xor(at, o, 64);
    if (w > v || (w == v && i < at)) v = w, at = i;
  }
}

// LDS written by this wave's other lanes is visible
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

constexpr double kNone = -__builtin_huge_val();

// Scores of a token: s[r] of expert lane + 64 r
template <int R>
__device__ __forceinline__ void scores(const double (&l)[R], bool sigmoid, double (&s)[R]) {
  if (sigmoid) {
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = 1.0 / (1.0 + exp(-l[r]));
    return;
  }
  double top = kNone;
  bool nan = false;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    top = fmax(top, l[r]);
    nan |= l[r] != l[r];
  }
  top = wave_max(top);
  const bool bad = __any(nan);
  double z = 0.0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    s[r] = l[r] == kNone ? 0.0 : exp(l[r] - top);
    z += s[r];
  }
  z = wave_sum(z);
#pragma unroll
  for (int r = 0; r < R; ++r) s[r] = bad ? __builtin_nan("") : (z == 0.0 ? 0.0 : s[r] / z);
}

template <int DT, int R>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs args) {
  typedef typename Val<DT>::type T;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int E = args.experts, K = args.top_k;
  int *hist = (int *)smem;                                       // [E]
  int *slot = hist + E;                                          // [kRouteRows * K] ids
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double *choice = (double *)(smem + (((E + kRouteRows * K) * 4 + 15) & ~15)) + wave * E;   // grouped choice only
  const int64_t t0 = (int64_t)blockIdx.x * kRouteRows;
  const int rows = (int)min(args.tokens - t0, (int64_t)kRouteRows);
  for (int i = threadIdx.x; i < E; i += kThreads) hist[i] = 0;

  for (int q = wave; q < rows; q += kWaves) {
    const int64_t t = t0 + q;
    int id = -1;
    float w = 0.0f;
    if (!args.token_mask || args.token_mask[t]) {
      double l[R], s[R], by[R];
      const T *src = (const T *)args.logits + t * args.ld;
#pragma unroll
      for (int r = 0; r < R; ++r) l[r] = lane + 64 * r < E ? (double)Val<DT>::to(src[lane + 64 * r]) : kNone;
      scores<R>(l, args.sigmoid, s);
      bool nan = false;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int i = lane + 64 * r;
        nan |= i < E && s[r] != s[r];
        double c = s[r] + (args.bias && i < E ? (double)args.bias[i] : 0.0);
        if (l[r] == kNone || c != c) c = kNone;
        by[r] = args.bias ? c : l[r];
        if (args.top_groups < args.groups && i < E) choice[i] = c;
      }
      if (__any(nan)) {
        w = __builtin_nanf("");
      } else {
        if (args.top_groups < args.groups) {
          // lane g holds group g's score; the best top_groups stay
          const int size = E / args.groups;
          double best = kNone;
          int at = lane;
          wave_sync();
          if (lane < args.groups) {
            double a = kNone, b = kNone;
            for (int i = 0; i < size; ++i) {
              const double c = choice[lane * size + i];
              if (c > a) b = a, a = c;
              else if (c > b) b = c;
            }
            best = (args.group_top == 2 && size > 1) ? a + b : a;
            if (best != best) best = kNone;      // inf - inf
          }
          uint64_t kept = 0;
          bool open = lane < args.groups;
          for (int n = 0; n < args.top_groups; ++n) {
            double v = best;
            int g = open ? at : 1 << 20;
            if (!open) v = kNone;
            wave_best(v, g);
            kept |= 1ull << g;
            if (g == lane) open = false;
          }
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const int i = lane + 64 * r;
            if (i < E && !((kept >> (i / size)) & 1)) by[r] = kNone;
          }
        }
        double total = 0.0, mine = 0.0;
        for (int n = 0; n < K; ++n) {
          double v = kNone;
          int i = 1 << 20;
#pragma unroll
          for (int r = 0; r < R; ++r)
            if (by[r] > v) v = by[r], i = lane + 64 * r;
          wave_best(v, i);
          if (v == kNone) break;
          double p = 0.0;
#pragma unroll
          for (int r = 0; r < R; ++r)
            if (i == lane + 64 * r) p = s[r], by[r] = kNone;
          p = __shfl(p, i & 63, 64);
          total += p;
          if (lane == n) id = i, mine = p;
        }
        if (id >= 0) w = (float)(args.scale * (args.renormalize ? (total > 0.0 ? mine / total : 0.0) : mine));
      }
    }
    if (lane < K) {
      args.ids[t * K + lane] = id;
      args.weights[t * K + lane] = w;
      slot[q * K + lane] = id;
    }
  }
  if (!args.lists) return;
  __syncthreads();
  // place of each slot among the block's slots of its expert, 64 slots at a
  // time: the lanes with an equal id are found from one ballot a bit
  if (wave == 0) {
    const int n = rows * K;
    int bits = 0;
    while ((1 << bits) < E) ++bits;
    for (int base = 0; base < n; base += 64) {
      const int i = base + lane;
      const int id = i < n ? slot[i] : -1;
      uint64_t same = __ballot(id >= 0);
      for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((id >> b) & 1);
        same &= ((id >> b) & 1) ? set : ~set;
      }
      if (id >= 0) {
        const int before = __popcll(same & ((1ull << lane) - 1));
        const int had = hist[id];
        args.rank[t0 * K + i] = had + before;
        wave_sync();
        if (same >> lane == 1) hist[id] = had + before + 1;    // the last of them
      }
      wave_sync();
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < E; i += kThreads) args.hist[(int64_t)i * args.blocks + blockIdx.x] = hist[i];
}

// hist[e][.] -> slots of expert e in the blocks before; counts[e]
__global__ __launch_bounds__(kThreads) void route_scan_kernel(RouteArgs args) {
  __shared__ int part[kWaves];
  const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int *h = args.hist + (int64_t)e * args.blocks;
  int before = 0;
  for (int base = 0; base < args.blocks; base += kThreads) {
    const int i = base + (int)threadIdx.x;
    const int v = i < args.blocks ? h[i] : 0;
    int sum = v;
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(sum, o, 64);
      if (lane >= o) sum += u;
    }
    if (lane == 63) part[wave] = sum;
    __syncthreads();
    int add = before, all = 0;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) add += part[w];
      all += part[w];
    }
    if (i < args.blocks) h[i] = add + sum - v;
    before += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    args.counts[e] = before;
    if (args.load) args.load[e] += before;
  }
}

// every slot to its place; places past the last slot hold -1
__global__ __launch_bounds__(kThreads) void route_place_kernel(RouteArgs args) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  int *offset = (int *)smem;     // [E + 1]
  const int E = args.experts, K = args.top_k;
  if (threadIdx.x < 64) {
    int before = 0;
    for (int base = 0; base < E; base += 64) {
      const int i = base + (int)threadIdx.x;
      const int v = i < E ? args.counts[i] : 0;
      int sum = v;
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(sum, o, 64);
        if ((int)threadIdx.x >= o) sum += u;
      }
      if (i < E) offset[i] = before + sum - v;
      before += __shfl(sum, 63, 64);
    }
    if (threadIdx.x == 0) offset[E] = before;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= E; i += kThreads) args.offsets[i] = offset[i];
  const int64_t t0 = (int64_t)blockIdx.x * kRouteRows;
  const int n = (int)min(args.tokens - t0, (int64_t)kRouteRows) * K;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int64_t flat = t0 * K + i;
    const int id = args.ids[flat];
    if (id >= 0) {
      const int place = offset[id] + args.hist[(int64_t)id * args.blocks + blockIdx.x] + args.rank[flat];
      args.order[place] = (int)flat;
      args.rows[place] = (int)(flat / K);
    }
    if (flat >= offset[E]) args.order[flat] = args.rows[flat] = -1;
  }
}

// One wave a token: lanes hold the scores and their gradients.  With weights
// renormalised over the taken experts, a softmax's gradient outside them is
// zero (their weights are a softmax of the taken logits alone).
template <int DT, int R>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(RouteArgs args) {
  typedef typename Val<DT>::type T;
  const int E = args.experts, K = args.top_k;
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= args.tokens) return;
  const T *src = (const T *)args.logits + t * args.ld;
  float l[R], s[R], ds[R];
  float top = -INFINITY;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    l[r] = lane + 64 * r < E ? Val<DT>::to(src[lane + 64 * r]) : -INFINITY;
    top = fmaxf(top, l[r]);
    ds[r] = 0.0f;
  }
  if (args.sigmoid) {
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = 1.0f / (1.0f + expf(-l[r]));
  } else {
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    float z = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] = l[r] == -INFINITY ? 0.0f : expf(l[r] - top);
      z += s[r];
    }
    for (int o = 32; o > 0; o >>= 1) z += __shfl_xor(z, o, 64);
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = z > 0.0f ? s[r] / z : s[r];
  }
  // lane j < K: pick j
  int id = lane < K ? args.ids[t * K + lane] : -1;
  if (id >= E) id = -1;
  float p = 0.0f;
  const float dw = id >= 0 ? args.grad_weights[t * K + lane] : 0.0f;
  for (int j = 0; j < K; ++j) {
    const int i = __shfl(id, j, 64);
    float v = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (i == lane + 64 * r) v = s[r];
    v = __shfl(v, i & 63, 64);
    if (lane == j && i >= 0) p = v;
  }
  float d = dw;
  if (args.renormalize) {
    float total = p, dot = dw * p;
    for (int o = 32; o > 0; o >>= 1) {
      total += __shfl_xor(total, o, 64);
      dot += __shfl_xor(dot, o, 64);
    }
    d = (id >= 0 && total > 0.0f) ? (dw - dot / total) / total : 0.0f;
  }
  d *= args.scale;
  float dot = id >= 0 ? d * p : 0.0f;
  for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, 64);
  for (int j = 0; j < K; ++j) {
    const int i = __shfl(id, j, 64);
    const float v = __shfl(d, j, 64);
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (i == lane + 64 * r) ds[r] += v;
  }
  T *dst = (T *)args.grad_logits + t * args.ld_grad;
  const bool none = __ballot(id >= 0) == 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = lane + 64 * r;
    float g;
    if (args.sigmoid) g = ds[r] == 0.0f ? 0.0f : s[r] * (1.0f - s[r]) * ds[r];
    else if (args.renormalize) g = ds[r] == 0.0f ? 0.0f : s[r] * ds[r];
    else g = none ? 0.0f : s[r] * (ds[r] - dot);
    if (i < E) dst[i] = Val<DT>::from(g);
  }
}

template <typename C>
__global__ __launch_bounds__(kThreads) void balance_kernel(float *bias, const C *counts, int experts, float rate) {
  __shared__ int64_t part[kWaves];
  const int64_t first = (int64_t)blockIdx.x * experts;
  int64_t sum = 0;
  for (int i = threadIdx.x; i < experts; i += kThreads) sum += (int64_t)counts[first + i];
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = 0;
  for (int w = 0; w < kWaves; ++w) sum += part[w];
  for (int i = threadIdx.x; i < experts; i += kThreads) {
    const int64_t d = sum - (int64_t)experts * (int64_t)counts[first + i];
    bias[first + i] += d > 0 ? rate : (d < 0 ? -rate : 0.0f);
  }
}

template <int DT>
hipError_t route_for(const RouteArgs &args, hipStream_t s) {
  const size_t lists = ((size_t)(args.experts + kRouteRows * args.top_k) * 4 + 15) & ~(size_t)15;
  const size_t lds = lists + (args.top_groups < args.groups ? (size_t)kWaves * args.experts * 8 : 0);
  const dim3 g(args.blocks), b(kThreads);
  const int r = (args.experts + 63) / 64;
  if (r <= 1) hipLaunchKernelGGL((route_kernel<DT, 1>), g, b, lds, s, args);
  else if (r <= 2) hipLaunchKernelGGL((route_kernel<DT, 2>), g, b, lds, s, args);
  else if (r <= 4) hipLaunchKernelGGL((route_kernel<DT, 4>), g, b, lds, s, args);
  else if (r <= 8) hipLaunchKernelGGL((route_kernel<DT, 8>), g, b, lds, s, args);
  else hipLaunchKernelGGL((route_kernel<DT, 16>), g, b, lds, s, args);
  return hipGetLastError();
}

template <int DT>
hipError_t backward_for(const RouteArgs &args, hipStream_t s) {
  const dim3 g((unsigned)((args.tokens + kWaves - 1) / kWaves)), b(kThreads);
  const int r = (args.experts + 63) / 64;
  if (r <= 1) hipLaunchKernelGGL((route_backward_kernel<DT, 1>), g, b, 0, s, args);
  else if (r <= 2) hipLaunchKernelGGL((route_backward_kernel<DT, 2>), g, b, 0, s, args);
  else if (r <= 4) hipLaunchKernelGGL((route_backward_kernel<DT, 4>), g, b, 0, s, args);
  else if (r <= 8) hipLaunchKernelGGL((route_backward_kernel<DT, 8>), g, b, 0, s, args);
  else hipLaunchKernelGGL((route_backward_kernel<DT, 16>), g, b, 0, s, args);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs &args, int dtype, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (args.blocks > 0) {
    e = dtype == kF32 ? route_for<kF32>(args, s) : dtype == kBF16 ? route_for<kBF16>(args, s) : route_for<kF16>(args, s);
    if (e != hipSuccess) return e;
  }
  if (!args.lists) return e;
  hipLaunchKernelGGL(route_scan_kernel, dim3(args.experts), dim3(kThreads), 0, s, args);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(route_place_kernel, dim3(args.blocks > 0 ? args.blocks : 1), dim3(kThreads), (size_t)(args.experts + 1) * 4, s, args);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteArgs &args, int dtype, hipStream_t s) {
  return dtype == kF32 ? backward_for<kF32>(args, s) : dtype == kBF16 ? backward_for<kBF16>(args, s) : backward_for<kF16>(args, s);
}

hipError_t launch_balance(float *bias, const void *counts, int count_bytes, int64_t layers, int experts, float rate, hipStream_t s) {
  const dim3 g((unsigned)layers), b(kThreads);
  if (count_bytes == 4) hipLaunchKernelGGL(balance_kernel<int32_t>, g, b, 0, s, bias, (const int32_t *)counts, experts, rate);
  else hipLaunchKernelGGL(balance_kernel<int64_t>, g, b, 0, s, bias, (const int64_t *)counts, experts, rate);
  return hipGetLastError();
}

}  // namespace muon

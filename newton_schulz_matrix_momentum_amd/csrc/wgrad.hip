// Weight gradients out of an 8-bit checkpoint:
//   dW_e[n][d] = sum_i dy[i][n] x^[rows_of[i]][d]   over the expert's slots i.
//
// Both operands lie with the summed axis (tokens) slowest, while an MFMA lane
// wants 8 consecutive tokens of one column.  The tiles go to LDS as they lie,
// 16-bit rows of tokens (x^ decoded on the way: exact in bf16), and the
// fragments come back through gfx950's transposing LDS reads
// (ds_read_b64_tr_b16: within each 16-lane group, lane l receives element
// l % 4 of the 8 bytes that lane 4 e + l / 4 addressed, as its element e).
#include "ckpt_code.h"

namespace muon {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ void mma(const u32x4 &a, const u32x4 &b, f32x4 &c) {
  if constexpr (DT == kBF16)
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <int DT>
__device__ __forceinline__ uint32_t pair(float a, float b) {
  if constexpr (DT == kF16) a = saturate_f16(a), b = saturate_f16(b);
  return (uint32_t)__builtin_bit_cast(uint16_t, Val<DT>::from(a)) | ((uint32_t)__builtin_bit_cast(uint16_t, Val<DT>::from(b)) << 16);
}

// 16 codes with one scale as 16-bit operands
template <int DT, int FMT>
__device__ __forceinline__ void decode16(const u32x4 &w, uint32_t b, u32x4 &lo, u32x4 &hi) {
  const float s = scale_of(b);
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    decode4<FMT>(w[i], s, v);
    const uint32_t p = pair<DT>(v[0], v[1]), q = pair<DT>(v[2], v[3]);
    if (i < 2) lo[2 * i] = p, lo[2 * i + 1] = q;
    else hi[2 * (i - 2)] = p, hi[2 * (i - 2) + 1] = q;
  }
}

// One expert's slots [lo, hi), read clamped to the list's length
__device__ __forceinline__ void slot_range(const WgradArgs &args, int e, int64_t &lo, int64_t &hi) {
  if (args.offsets) {
    lo = min(max((int64_t)args.offsets[e], (int64_t)0), args.slots);
    hi = min(max((int64_t)args.offsets[e + 1], lo), args.slots);
  } else {
    lo = 0;
    hi = args.slots;
  }
}

// Checkpoint row of a slot, -1: left out
__device__ __forceinline__ int64_t row_of(const WgradArgs &args, int64_t slot, int64_t hi) {
  if (slot >= hi) return -1;
  if (!args.rows_of) return slot;
  const int r = args.rows_of[slot];
  return (r >= 0 && r < args.ckpt_rows) ? (int64_t)r : (int64_t)-1;
}

template <int OT>
__device__ __forceinline__ void put4(void *out, int64_t at, int n, bool vec, bool accumulate, f32x4 v) {
  typedef typename Val<OT>::type T;
  T *p = (T *)out + at;
  if (accumulate) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) v[i] += Val<OT>::to(p[i]);
  }
  if (vec && n >= 4) {
    if constexpr (OT == kF32) *(f32x4 *)p = v;
    else *(uint2 *)p = make_uint2((uint32_t)__builtin_bit_cast(uint16_t, Val<OT>::from(v[0])) | ((uint32_t)__builtin_bit_cast(uint16_t, Val<OT>::from(v[1])) << 16),
                                  (uint32_t)__builtin_bit_cast(uint16_t, Val<OT>::from(v[2])) | ((uint32_t)__builtin_bit_cast(uint16_t, Val<OT>::from(v[3])) << 16));
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) p[i] = Val<OT>::from(v[i]);
}

__device__ __forceinline__ void put4_any(void *out, int dtype, int64_t at, int n, bool vec, bool acc, f32x4 v) {
  if (dtype == kF32) put4<kF32>(out, at, n, vec, acc, v);
  else if (dtype == kBF16) put4<kBF16>(out, at, n, vec, acc, v);
  else put4<kF16>(out, at, n, vec, acc, v);
}

// 128 outs x 128 columns per block of four waves (64 x 64 each), 32 tokens a
// step, double-buffered through registers.
//
// LDS rows hold one token's 128 values, 256 bytes; the 32-byte chunk c of row
// r is kept at c ^ key(r): the 8 rows that half a wave reads at once (a
// 16-lane group takes 4 rows) have distinct keys, so their equal chunks fall
// into distinct banks.
constexpr int kThreads = 256;
constexpr int kRowBytes = kWgradTile * 2;
__device__ __forceinline__ int key(int r) { return (r & 3) | ((r >> 1) & 4); }

template <int DT, int FMT, bool TRANS>
__global__ __launch_bounds__(kThreads, 2) void wgrad_kernel(WgradArgs args) {
  typedef typename Val<DT>::type T;
  __shared__ __attribute__((aligned(16))) char lds[2][2][kWgradK * kRowBytes];   // [buffer][dy, x^]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn = wave >> 1, wd = wave & 1;
  const int tn = blockIdx.x / args.tiles_d, td = blockIdx.x % args.tiles_d;
  const int e = blockIdx.y;
  int64_t lo, hi;
  slot_range(args, e, lo, hi);
  if (args.splits > 1) {
    lo += blockIdx.z * args.split_len;
    hi = min(hi, lo + args.split_len);
  }
  const int n0 = tn * kWgradTile, d0 = td * kWgradTile;

  // dy: thread covers tokens tid / 16 and 16 + tid / 16, 8 columns from 8 (tid % 16)
  const int y_row = tid >> 4, y_col = (tid & 15) * 8;
  const int y_n = min(args.outs - (n0 + y_col), 8);
  // x^: thread covers token tid / 8, 16 columns from 16 (tid % 8)
  const int x_row = tid >> 3, x_col = (tid & 7) * 16;
  const bool x_in = d0 + x_col < args.cols;
  const T *dy = (const T *)args.dy + n0 + y_col;
  const uint8_t *codes = args.codes + d0 + x_col;
  const uint8_t *scales = args.scales + (d0 + x_col) / kCkptBlock;

  u32x4 ry[2], rx = {};
  uint32_t rb = 0;
  auto fetch = [&](int64_t base) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t slot = base + y_row + 16 * i;
      ry[i] = u32x4{};
      if (row_of(args, slot, hi) >= 0 && y_n > 0) {
        const T *p = dy + slot * args.ld_dy;
        if (y_n == 8) {
          ry[i] = *(const u32x4u *)p;
        } else {
          uint16_t t[8] = {};
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < y_n) t[k] = __builtin_bit_cast(uint16_t, p[k]);
#pragma unroll
          for (int k = 0; k < 4; ++k) ry[i][k] = (uint32_t)t[2 * k] | ((uint32_t)t[2 * k + 1] << 16);
        }
      }
    }
    const int64_t r = row_of(args, base + x_row, hi);
    rx = u32x4{};
    rb = 127;
    if (r >= 0 && x_in) {
      rx = *(const u32x4 *)(codes + r * args.codes_ld);
      rb = scales[r * args.scales_ld];
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = y_row + 16 * i, c = (tid & 15) >> 1;
      *(u32x4 *)(&lds[buf][0][r * kRowBytes + ((c ^ key(r)) * 32) + (tid & 1) * 16]) = ry[i];
    }
    u32x4 a, b;
    decode16<DT, FMT>(rx, rb, a, b);
    char *p = &lds[buf][1][x_row * kRowBytes + (((tid & 7) ^ key(x_row)) * 32)];
    *(u32x4 *)p = a;
    *(u32x4 *)(p + 16) = b;
  };
  // fragment of 16 columns from 16 c: tokens 8 g .. 8 g + 7 of the lane's column
  const int g = lane >> 4, j = lane & 15;
  auto frag = [&](const char *t, int c) {
    const int r0 = 8 * g + (j >> 2), r1 = r0 + 4;
    const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) i16x4 *)(t + r0 * kRowBytes + ((c ^ key(r0)) * 32) + (j & 3) * 8));
    const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) i16x4 *)(t + r1 * kRowBytes + ((c ^ key(r1)) * 32) + (j & 3) * 8));
    const uint2 a = __builtin_bit_cast(uint2, x), b = __builtin_bit_cast(uint2, y);
    return u32x4{a.x, a.y, b.x, b.y};
  };

  // acc[i][k]: the MFMA's rows are the index that is contiguous in the output
  f32x4 acc[4][4] = {};
  if (lo < hi) {
    fetch(lo);
    stage(0);
    __syncthreads();
    int buf = 0;
    for (int64_t base = lo; base < hi; base += kWgradK) {
      const bool more = base + kWgradK < hi;
      if (more) fetch(base + kWgradK);
      u32x4 fy[4], fx[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        fy[i] = frag(lds[buf][0], wn * 4 + i);
        fx[i] = frag(lds[buf][1], wd * 4 + i);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (TRANS) mma<DT>(fy[i], fx[k], acc[i][k]);
          else mma<DT>(fx[i], fy[k], acc[i][k]);
        }
      if (more) stage(buf ^ 1);
      __syncthreads();
      buf ^= 1;
    }
  }

  const int rows = TRANS ? args.cols : args.outs, width = TRANS ? args.outs : args.cols;
  const int row_base = TRANS ? d0 + wd * 64 : n0 + wn * 64, col_base = TRANS ? n0 + wn * 64 : d0 + wd * 64;
  const int64_t size = (int64_t)args.outs * args.cols;
  const bool split = args.splits > 1;
  const int ot = split ? (int)kF32 : args.out_dtype;
  const bool vec = (width & 3) == 0 && (((uintptr_t)(split ? (void *)args.part : args.out)) & 15) == 0;
  const int64_t first = (split ? (int64_t)blockIdx.z : (int64_t)e) * size;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = row_base + 16 * k + (lane & 15), col = col_base + 16 * i + 4 * (lane >> 4);
      if (row < rows && col < width)
        put4_any(split ? (void *)args.part : args.out, ot, first + (int64_t)row * width + col, min(width - col, 4), vec,
                 !split && args.accumulate, acc[i][k]);
    }
}

// out = (out +) the sum of the parts, in their order
__global__ __launch_bounds__(256) void wgrad_join_kernel(WgradArgs args) {
  const int64_t size = (int64_t)args.outs * args.cols;
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= size) return;
  const int n = (int)min(size - at, (int64_t)4);
  f32x4 v = {};
  const bool vec = (size & 3) == 0;
  for (int p = 0; p < args.splits; ++p) {
    const float *src = args.part + p * size + at;
    if (vec) {
      v += *(const f32x4 *)src;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) v[i] += src[i];
    }
  }
  put4_any(args.out, args.out_dtype, at, n, (((uintptr_t)args.out) & 15) == 0, args.accumulate, v);
}

}  // namespace

hipError_t launch_wgrad(const WgradArgs &args, int dtype, int format, hipStream_t s) {
  const dim3 g(args.tiles_n * args.tiles_d, args.experts, args.splits), b(kThreads);
#define MUON_WGRAD(DT, FMT)                                                                             \
  if (args.transposed) hipLaunchKernelGGL((wgrad_kernel<DT, FMT, true>), g, b, 0, s, args);             \
  else hipLaunchKernelGGL((wgrad_kernel<DT, FMT, false>), g, b, 0, s, args);                            \
  break;
  switch (dtype * 2 + format) {
    case kF16 * 2 + MUON_E4M3: MUON_WGRAD(kF16, MUON_E4M3)
    case kF16 * 2 + MUON_INT8: MUON_WGRAD(kF16, MUON_INT8)
    case kBF16 * 2 + MUON_E4M3: MUON_WGRAD(kBF16, MUON_E4M3)
    case kBF16 * 2 + MUON_INT8: MUON_WGRAD(kBF16, MUON_INT8)
    default: return hipErrorInvalidValue;
  }
#undef MUON_WGRAD
  return hipGetLastError();
}

hipError_t launch_wgrad_join(const WgradArgs &args, hipStream_t s) {
  const int64_t size = (int64_t)args.outs * args.cols;
  hipLaunchKernelGGL(wgrad_join_kernel, dim3((unsigned)((size + 1023) / 1024)), dim3(256), 0, s, args);
  return hipGetLastError();
}

}  // namespace muon

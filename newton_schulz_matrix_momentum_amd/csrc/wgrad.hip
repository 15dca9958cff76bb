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

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
template <int DT>
__device__ __forceinline__ uint32_t pair(float a, float b) {
  const f32x2v v = {a, b};      // one packed conversion
  if constexpr (DT == kF16) {
    const f32x2v c = {saturate_f16(a), saturate_f16(b)};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(c, f16x2));
  } else {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  }
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

// ---------------------------------------------------------------------------
// Large products: BN outs x BD columns per block (256 x 128 or 128 x 256), four
// waves of half the sides, two blocks a CU, so that one block's prologue and
// stores run beside the other's products.
//
// A step is 32 tokens.  dy goes global -> LDS by DMA into a ring of kRing
// stages, issued kRing steps ahead; x^ passes through registers (codes loaded
// four steps ahead, decoded and written two ahead) into a ring of two.  Every
// step issues the same memory operations (rows outside the expert come from a
// page of zeros, or are zeroed while they are decoded), so the wait for a
// stage's DMA is a constant count.
//
// A wave holds the short operand's four fragments and half of the long
// operand's eight.  Step i: products of the first half while the second half
// is read; then one barrier, behind which stage i + 1 is complete and stage
// i's buffers are free; then products of the second half while stage i + 1's
// first fragments are read and the buffers are refilled.
constexpr int kRing = 4;
constexpr uint64_t kRowBits = 0x0101010101010101ull;

#define MUON_WGRAD_VMCNT(n) (0x0F70 | ((n) & 15) | (((n) >> 4) << 14))   // s_waitcnt vmcnt(n) alone

template <int I> struct IntC { static constexpr int value = I; };

template <int DT, int FMT, bool TRANS, bool GATHER, int BN, int BD>
__global__ __launch_bounds__(kThreads, 2) void wgrad_wide_kernel(WgradArgs args) {
  static_assert(BN * BD == 256 * 128, "two fragment shapes");
  constexpr int YROW = BN * 2, XROW = BD * 2;                // bytes of a token's row in LDS
  constexpr int YSTAGE = kWgradK * YROW, XSTAGE = kWgradK * XROW;
  constexpr int ND = YSTAGE / 4096;                          // DMA instructions of a wave and step
  constexpr int LPR = YROW / 16;                             // lanes of a DMA instruction on one row
  constexpr int NX = BD / 128;                               // 16-code chunks of a thread and step
  constexpr int CPR = BD / 16;                               // chunks of a row
  constexpr bool LONG_Y = BN == 256;
  // One array a stage: the compiler then sees which stage a read and a DMA in
  // flight belong to, and does not wait for the others' DMA before a read.
  __shared__ __attribute__((aligned(1024))) char y0[YSTAGE], y1[YSTAGE], y2[YSTAGE], y3[YSTAGE];
  __shared__ __attribute__((aligned(1024))) char x0[XSTAGE], x1[XSTAGE];
  static_assert(kRing == 4, "one array a stage");
  auto ybuf = [&](auto sc) -> char * {
    constexpr int S = decltype(sc)::value & 3;
    if constexpr (S == 0) return y0;
    else if constexpr (S == 1) return y1;
    else if constexpr (S == 2) return y2;
    else return y3;
  };
  auto xbuf = [&](auto sc) -> char * {
    if constexpr ((decltype(sc)::value & 1) == 0) return x0;
    else return x1;
  };

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave >> 1, wd = wave & 1;
  // consecutive blocks go to the XCDs in turn: each XCD walks one contiguous
  // run of tiles, whose operand panels its L2 then holds
  const int total = (int)gridDim.x, per = total / 8, rem = total % 8, xcd = blockIdx.x % 8;
  int tile = (xcd < rem ? xcd * (per + 1) : rem * (per + 1) + (xcd - rem) * per) + blockIdx.x / 8;
  const int tiles = args.tiles_n * args.tiles_d;
  const int part = tile / tiles;                             // expert, or part of the token range
  tile -= part * tiles;
  const int e = args.splits > 1 ? 0 : part;
  int64_t lo, hi;
  slot_range(args, e, lo, hi);
  if (args.splits > 1) {
    lo += part * args.split_len;
    hi = min(hi, lo + args.split_len);
  }
  const int n0 = (tile / args.tiles_d) * BN, d0 = (tile % args.tiles_d) * BD;
  const int steps = (int)((max(hi - lo, (int64_t)0) + kWgradK - 1) / kWgradK);

  f32x4 acc[8][4] = {};
  if (steps > 0) {
    const int64_t last = hi - 1;
    // dy: wave w moves rows 8 w .. 8 w + 7 of a stage.  A step's rows are a
    // buffer that ends with the expert's last row, so rows behind it read as
    // zeros, as do slots that are left out (an offset past any end).  Columns
    // past outs (whole chunks: outs is a multiple of 8) read the last ones.
    constexpr int RPI = 64 / LPR;                            // rows of a DMA instruction
    constexpr int NO = RPI == 2 ? 2 : 1;                     // lane offsets that differ between instructions
    const uint32_t y_pitch = (uint32_t)args.ld_dy * 2;
    uint32_t y_off[NO];
#pragma unroll
    for (int o = 0; o < NO; ++o) {
      const int r = wave * 8 + o * RPI + lane / LPR, q = lane % LPR, c = (((q >> 1) ^ key(r)) << 1) | (q & 1);
      y_off[o] = (uint32_t)(wave * 8 + lane / LPR) * y_pitch + (uint32_t)min(n0 + c * 8, args.outs - 8) * 2;
    }
    auto dma = [&](int step, auto sc, uint64_t valid) {
      const int64_t row = lo + (int64_t)step * kWgradK;
      const int64_t left = min(max(hi - row, (int64_t)0), (int64_t)kWgradK);
      const __amdgpu_buffer_rsrc_t rows = __builtin_amdgcn_make_buffer_rsrc(
          (void *)((const char *)args.dy + row * args.ld_dy * 2), 0, left > 0 ? (int)((uint32_t)(left - 1) * y_pitch + (uint32_t)args.outs * 2) : 0, 0x00020000);
#pragma unroll
      for (int j = 0; j < ND; ++j) {
        uint32_t off = y_off[j % NO];
        if constexpr (GATHER) {
          if (valid != kRowBits && !((valid >> (8 * (j * RPI + lane / LPR))) & 1)) off = 0x80000000u;
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rows, (__attribute__((address_space(3))) void *)(ybuf(sc) + (wave * 8 * YROW + j * 1024)), 16,
                                                 (int)off, (int)((uint32_t)(j * RPI) * y_pitch), 0, 0);
      }
    };
    // x^: rows 8 w + lane / 8 (one chunk), or 8 w + lane / 16 and 4 further (two)
    const int x_sub = lane / CPR, x_row = wave * 8 + x_sub, x_chunk = lane % CPR;
    const uint32_t x_col = (uint32_t)min(d0 + x_chunk * 16, (args.cols - 1) & ~15);
    struct Saved {
      u32x4 w[NX];
      uint32_t b[NX];
      uint64_t in;           // bit 8 k: row 8 w + k is in (of kRowBits)
    } saved[2];
    // GATHER: a stage's checkpoint rows are loaded two steps before they are
    // checked (check: -1 where the slot is left out) and used
    int row[2][NX];
    auto find = [&](int step, int (&out)[NX]) {
#pragma unroll
      for (int x = 0; x < NX; ++x) out[x] = args.rows_of[min(lo + (int64_t)step * kWgradK + x_row + 4 * x, last)];
    };
    auto check = [&](int step, int (&r)[NX]) -> uint64_t {
      uint64_t m[NX];
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        const bool in = lo + (int64_t)step * kWgradK + x_row + 4 * x < hi && r[x] >= 0 && r[x] < args.ckpt_rows;
        r[x] = in ? r[x] : -1;
        m[x] = __ballot(in);
      }
      // a row's lanes start at 8 k (one chunk a thread) or at 16 k (two)
      if constexpr (NX == 1) return m[0] & kRowBits;
      uint64_t v = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) v |= ((m[0] >> (16 * k)) & 1) << (8 * k) | ((m[NX - 1] >> (16 * k)) & 1) << (8 * (k + 4));
      return v;
    };
    auto fetch = [&](int step, Saved &s, const int (&from)[NX], uint64_t valid) {
      const int64_t base = lo + (int64_t)step * kWgradK + wave * 8;
      const int64_t first = min(base, last);                 // wave-uniform
      s.in = valid;
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        if constexpr (GATHER) {
          const int64_t r = max(from[x], 0);
          s.w[x] = *(const u32x4 *)(args.codes + r * args.codes_ld + x_col);
          s.b[x] = args.scales[r * args.scales_ld + x_col / kCkptBlock];
        } else {
          const uint32_t k = min((uint32_t)(x_sub + 4 * x), (uint32_t)min(last - first, (int64_t)7));
          s.w[x] = *(const u32x4 *)(args.codes + first * args.codes_ld + (k * (uint32_t)args.codes_ld + x_col));
          s.b[x] = *(args.scales + first * args.scales_ld + (k * (uint32_t)args.scales_ld + x_col / kCkptBlock));
        }
      }
    };
    // validity of a stage's 8 rows of this wave without a list
    auto tail = [&](int step) -> uint64_t {
      const int64_t left = hi - (lo + (int64_t)step * kWgradK + wave * 8);
      return left >= 8 ? kRowBits : left <= 0 ? 0ull : ((1ull << (8 * left)) - 1) & kRowBits;
    };
    auto stage = [&](auto sc, const Saved &s) {
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        u32x4 a, b, w = s.w[x];
        uint32_t sb = s.b[x];
        if (s.in != kRowBits && !((s.in >> (8 * (x_sub + 4 * x))) & 1)) w = u32x4{}, sb = 127;
        decode16<DT, FMT>(w, sb, a, b);
        const int r = x_row + 4 * x;
        const int o = r * XROW + ((x_chunk ^ key(r)) * 32);
        *(u32x4 *)(xbuf(sc) + o) = a;
        *(u32x4 *)(xbuf(sc) + (o + 16)) = b;
      }
    };
    // Fragment c of a stage (16 columns): tokens 8 g .. 8 g + 7 of the lane's
    // column, from rows r0 and r0 + 4 (their keys are equal).  Its chunk's
    // place differs from fragment 0's by c in the three bits of the key, so
    // the offset is one exclusive or.  The base passes through an empty asm
    // each step: kept apart for each fragment, the offsets would cost 12
    // registers, and as a chain of sums they lose the stage they point into.
    constexpr int LROW = LONG_Y ? YROW : XROW, SROW = LONG_Y ? XROW : YROW;
    const int r0 = 8 * (lane >> 4) + ((lane & 15) >> 2), lc = (LONG_Y ? wn : wd) * 8, sc0 = (LONG_Y ? wd : wn) * 4;
    int at_long = r0 * LROW + ((lc ^ key(r0)) * 32) + (lane & 3) * 8;
    int at_short = r0 * SROW + ((sc0 ^ key(r0)) * 32) + (lane & 3) * 8;
    auto fresh = [](int &o) { asm volatile("" : "+v"(o)); };
    auto frag = [&](const char *t, int o, int half) {
      const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4 *)(t + o));
      const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4 *)(t + o + half));
      const uint2 a = __builtin_bit_cast(uint2, x), b = __builtin_bit_cast(uint2, y);
      return u32x4{a.x, a.y, b.x, b.y};
    };
    auto frag_long = [&](auto sc, int i) {
      if constexpr (LONG_Y) return frag(ybuf(sc), at_long ^ (i * 32), 4 * YROW);
      else return frag(xbuf(sc), at_long ^ (i * 32), 4 * XROW);
    };
    auto frag_short = [&](auto sc, int i) {
      if constexpr (LONG_Y) return frag(xbuf(sc), at_short ^ (i * 32), 4 * XROW);
      else return frag(ybuf(sc), at_short ^ (i * 32), 4 * YROW);
    };
    u32x4 fs[4], fl[4], fh[4];
    auto column = [&](int base, const u32x4 (&f)[4], int k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (TRANS == LONG_Y) mma<DT>(f[i], fs[k], acc[base + i][k]);    // rows: the long operand's index
        else mma<DT>(fs[k], f[i], acc[base + i][k]);
      }
    };

    // fill: steps 0 .. 3 in the steady order (dma, codes), steps 0 and 1 decoded
    if constexpr (GATHER) {
      find(0, row[0]);
      find(1, row[1]);
    }
    auto fill = [&](auto sc) {
      constexpr int i = decltype(sc)::value;
      const uint64_t v = GATHER ? check(i, row[i & 1]) : tail(i);
      dma(i, sc, v);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (i >= 2) stage(sc, saved[i & 1]);
      __builtin_amdgcn_sched_barrier(0);
      fetch(i, saved[i & 1], row[i & 1], v);
      if constexpr (GATHER) find(i + 2, row[i & 1]);
      __builtin_amdgcn_sched_barrier(0);
    };
    fill(IntC<0>{});
    fill(IntC<1>{});
    fill(IntC<2>{});
    fill(IntC<3>{});
    // row[] now holds steps 4 and 5
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < 4; ++k) fs[k] = frag_short(IntC<0>{}, k), fl[k] = frag_long(IntC<0>{}, k);

    auto step = [&](auto sc, int i) {
      constexpr int S = decltype(sc)::value;                 // i % 4
      const IntC<S + 1> next;
      Saved &s = saved[S & 1];
      int (&r)[NX] = row[S & 1];
      fresh(at_long);
      fresh(at_short);
#pragma unroll
      for (int k = 0; k < 4; ++k) fh[k] = frag_long(sc, 4 + k);
#pragma unroll
      for (int k = 0; k < 4; ++k) column(0, fl, k);
      // stage i + 1: its dma has landed (behind it: three steps of codes and
      // indices, two of dma; the newest of those may stay on their way), its
      // codes are written; stage i is in registers
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(MUON_WGRAD_VMCNT(2 * ND + 2 * NX * (GATHER ? 3 : 2)));
      __builtin_amdgcn_s_waitcnt(0xC07F);     // lgkmcnt(0)
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      const uint64_t v = GATHER ? check(i + 4, r) : tail(i + 4);
      dma(i + 4, sc, v);
      __builtin_amdgcn_sched_barrier(0);
      stage(sc, s);
      __builtin_amdgcn_sched_barrier(0);
      fetch(i + 4, s, r, v);
      if constexpr (GATHER) find(i + 6, r);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < 4; ++k) fl[k] = frag_long(next, k);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        column(4, fh, k);
        fs[k] = frag_short(next, k);
      }
    };
#pragma unroll 1
    for (int i = 0;;) {
      step(IntC<0>{}, i);
      if (++i >= steps) break;
      step(IntC<1>{}, i);
      if (++i >= steps) break;
      step(IntC<2>{}, i);
      if (++i >= steps) break;
      step(IntC<3>{}, i);
      if (++i >= steps) break;
    }
    // nothing may still be on its way to LDS when the block's LDS is given on
    __builtin_amdgcn_s_waitcnt(0);
  }

  const int rows = TRANS ? args.cols : args.outs, width = TRANS ? args.outs : args.cols;
  const int64_t size = (int64_t)args.outs * args.cols;
  const bool split = args.splits > 1;
  const int ot = split ? (int)kF32 : args.out_dtype;
  void *const out = split ? (void *)args.part : args.out;
  const bool vec = (width & 3) == 0 && (((uintptr_t)out) & 15) == 0;
  const int64_t first = (int64_t)part * size;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // the MFMA's rows (4 consecutive a lane) are contiguous in the output
      const int il = 16 * i + (TRANS == LONG_Y ? 4 * (lane >> 4) : (lane & 15));
      const int is = 16 * k + (TRANS == LONG_Y ? (lane & 15) : 4 * (lane >> 4));
      const int n = n0 + wn * (BN / 2) + (LONG_Y ? il : is), d = d0 + wd * (BD / 2) + (LONG_Y ? is : il);
      const int r = TRANS ? d : n, c = TRANS ? n : d;
      if (r < rows && c < width) put4_any(out, ot, first + (int64_t)r * width + c, min(width - c, 4), vec, !split && args.accumulate, acc[i][k]);
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

template <int DT, int FMT>
hipError_t launch_wide(const WgradArgs &args, hipStream_t s) {
  const dim3 g((unsigned)(args.tiles_n * args.tiles_d * (args.splits > 1 ? args.splits : args.experts))), b(kThreads);
#define MUON_WIDE(TRANS, GATHER)                                                                                             \
  if (args.wide == 1) hipLaunchKernelGGL((wgrad_wide_kernel<DT, FMT, TRANS, GATHER, 256, 128>), g, b, 0, s, args);           \
  else hipLaunchKernelGGL((wgrad_wide_kernel<DT, FMT, TRANS, GATHER, 128, 256>), g, b, 0, s, args)
  if (args.transposed && args.rows_of) MUON_WIDE(true, true);
  else if (args.transposed) MUON_WIDE(true, false);
  else if (args.rows_of) MUON_WIDE(false, true);
  else MUON_WIDE(false, false);
#undef MUON_WIDE
  return hipGetLastError();
}

hipError_t launch_wgrad(const WgradArgs &args, int dtype, int format, hipStream_t s) {
  if (args.wide) {
    if (dtype == kF16) return format == MUON_E4M3 ? launch_wide<kF16, MUON_E4M3>(args, s) : launch_wide<kF16, MUON_INT8>(args, s);
    return format == MUON_E4M3 ? launch_wide<kBF16, MUON_E4M3>(args, s) : launch_wide<kBF16, MUON_INT8>(args, s);
  }
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

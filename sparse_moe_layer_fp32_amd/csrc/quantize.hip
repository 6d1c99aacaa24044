// Quantisation to e4m3 codes with an fp32 scale for each block: of 1 x 128 (the
// rows of a product's left operand) or 128 x 128 (its weights).
//
//   a = max(largest |v| of the block, 2^-90);  scale = a / 448;
//   code = e4m3(v * (448 / a)), to nearest even
//
// (448 is e4m3's largest value; the least a keeps 448 / a and the scale
// ordinary fp32 numbers, also for a block of zeros.)  The product v * (448 / a)
// is at most 448 (1 + 2^-22), which rounds to 448, so no code overflows.  A block
// that holds a NaN or an infinity has that for its scale, so that no product of
// it is finite.
//
// Bound: HBM, 3 bytes a value.  A lane takes 16 values of a row: two loads and
// one store of 16 bytes; eight lanes share a block of 128.  65536 rows of 1280: 44
// us, 5.8 TB/s; 8192 tokens of 4096 to 8 rows each: 55 us, 6.3 TB/s; weights of 288 x
// 1280 x 4096 797, 5.7 TB/s.

#include "activation.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kQuantThreads = 256;
constexpr int kLaneValues = 16;
constexpr int kBlockLanes = 128 / kLaneValues;
constexpr float kLargest = 448.0f;
constexpr uint32_t kLeast = 0x12800000u;  // 2^-90

struct F16 {
  F8 lo, hi;
};

__device__ __forceinline__ F16 load16(const uint16_t* p) { return {load8(p), load8(p + 8)}; }

// Largest magnitude as bits: of non-negative floats these order as the values
// do, with infinity and NaN above all others.
__device__ __forceinline__ uint32_t largest(const F16& v) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    m = max(m, __float_as_uint(v.lo.v[q]) & 0x7FFFFFFFu);
    m = max(m, __float_as_uint(v.hi.v[q]) & 0x7FFFFFFFu);
  }
  return m;
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return static_cast<uint32_t>(w);
}

__device__ __forceinline__ u32x4 encode(const F16& v, float inv) {
  const float* l = v.lo.v;
  const float* h = v.hi.v;
  return u32x4{codes4(l[0] * inv, l[1] * inv, l[2] * inv, l[3] * inv),
               codes4(l[4] * inv, l[5] * inv, l[6] * inv, l[7] * inv),
               codes4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv),
               codes4(h[4] * inv, h[5] * inv, h[6] * inv, h[7] * inv)};
}

// Eight lanes take a block of a row, of all rows one after the other.  STREAM:
// codes are stored with the non-temporal hint.
template <bool STREAM>
__global__ __launch_bounds__(kQuantThreads) void quantize_rows_kernel(
    const uint16_t* __restrict__ x, const int32_t* __restrict__ pos, int64_t tokens, int64_t rows,
    int top_k, int cols, uint32_t blocks, uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const uint32_t id = blockIdx.x * kQuantThreads + threadIdx.x;
  const uint32_t block = id / kBlockLanes, lane = id % kBlockLanes;
  const uint32_t row = block / blocks, b = block - row * blocks;
  const int64_t t = row;
  const int c = static_cast<int>(b) * 128 + static_cast<int>(lane) * kLaneValues;
  const bool live = t < tokens && c < cols;
  F16 v{};
  if (live) v = load16(x + t * cols + c);
  uint32_t m = max(largest(v), kLeast);
#pragma unroll
  for (int off = 1; off < kBlockLanes; off <<= 1)
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), off)));
  if (!live) return;
  const float a = __uint_as_float(m);
  const u32x4 w = encode(v, kLargest / a);
  const float scale = a / kLargest;
  auto put = [&](int64_t r) {
    u32x4* const to = reinterpret_cast<u32x4*>(codes + r * cols + c);
    if (STREAM)
      __builtin_nontemporal_store(w, to);
    else
      *to = w;
    if (lane == 0) scales[r * blocks + b] = scale;
  };
  if (!pos) {
    put(t);
    return;
  }
  for (int j = 0; j < top_k; ++j) {
    const int r = pos[t * top_k + j];
    if (r >= 0 && r < rows) put(r);
  }
}

// A workgroup takes a block: four rows of 16 values a thread, in registers.
__global__ __launch_bounds__(kQuantThreads) void quantize_weight_kernel(
    const uint16_t* __restrict__ w, int F, int K, int fblocks, int kblocks,
    uint8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ uint32_t most[kQuantThreads / 64];
  const int kb = blockIdx.x % kblocks;
  const int rest = blockIdx.x / kblocks;
  const int fb = rest % fblocks;
  const int64_t g = rest / fblocks;
  const int c = kb * 128 + threadIdx.x % kBlockLanes * kLaneValues;
  const int row0 = fb * 128 + threadIdx.x / kBlockLanes;
  F16 v[4];
  uint32_t m = kLeast;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + 32 * i;
    v[i] = F16{};
    if (row < F && c < K) v[i] = load16(w + (g * F + row) * K + c);
    m = max(m, largest(v[i]));
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1)
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), off)));
  if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(most[0], most[1]), max(most[2], most[3]));
  const float a = __uint_as_float(m);
  const float inv = kLargest / a;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + 32 * i;
    if (row < F && c < K)
      *reinterpret_cast<u32x4*>(codes + (g * F + row) * K + c) = encode(v[i], inv);
  }
  if (threadIdx.x == 0) scales[(g * fblocks + fb) * kblocks + kb] = a / kLargest;
}

}  // namespace

hipError_t launch_quantize_rows(const uint16_t* x, const int32_t* pos, int64_t tokens,
                                int64_t rows, int top_k, int cols, uint8_t* codes, float* scales,
                                hipStream_t stream) {
  if (tokens == 0 || rows == 0) return hipSuccess;
  const int blocks = (cols + 127) / 128;
  const int64_t threads = tokens * blocks * kBlockLanes;
  const unsigned grid = static_cast<unsigned>((threads + kQuantThreads - 1) / kQuantThreads);
  // Codes that do not stay in the 256 MB last-level cache until they are read go
  // past it (8192 tokens of 4096 to 8 rows each: 55 us, from 70).
  const bool past = rows_past_cache(tokens, rows, top_k, cols + 4 * blocks);
  if (past)
    quantize_rows_kernel<true><<<grid, kQuantThreads, 0, stream>>>(x, pos, tokens, rows, top_k, cols,
                                                                   blocks, codes, scales);
  else
    quantize_rows_kernel<false><<<grid, kQuantThreads, 0, stream>>>(x, pos, tokens, rows, top_k,
                                                                    cols, blocks, codes, scales);
  return hipGetLastError();
}

hipError_t launch_quantize_weight(const uint16_t* w, int groups, int F, int K, uint8_t* codes,
                                  float* scales, hipStream_t stream) {
  const int fb = (F + 127) / 128, kb = (K + 127) / 128;
  const int64_t blocks = static_cast<int64_t>(groups) * fb * kb;
  if (blocks == 0) return hipSuccess;
  quantize_weight_kernel<<<static_cast<unsigned>(blocks), kQuantThreads, 0, stream>>>(
      w, F, K, fb, kb, codes, scales);
  return hipGetLastError();
}

}  // namespace moe

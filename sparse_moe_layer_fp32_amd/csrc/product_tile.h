// One output tile of a linear or grouped product on gfx950 matrix cores: the
// forward product y = x W^T, the input gradient dx = dy W and the weight
// gradient dW = dy^T x share this mainloop.
//
//  * bf16 x bf16 -> fp32 on v_mfma_f32_32x32x16_bf16, contraction steps of 64.
//  * An operand whose contraction runs along its rows in memory (x and W of
//    the forward product, dy of the input gradient) is laid down in LDS as
//    [tile row][64], 128-byte rows, and a fragment is one 16-byte read.  An
//    operand whose contraction runs across rows (W of the input gradient,
//    both of the weight gradient) is laid down as it lies in memory, [64][tile
//    column], and a fragment is two transposing reads (ds_read_b64_tr_b16: the
//    16 lanes of a group read four rows of 16 columns and each gets one
//    column's four values), so no operand is transposed in memory.
//  * 16-byte chunks are XOR-swizzled: contiguous rows by (row >> 1) & 7,
//    strided rows by 4 (row & 3) (the four rows a lane group reads land in
//    different 64-byte quarters of the banks).
//  * Panels go memory -> LDS with buffer_load ... lds.  A lane whose row or
//    column lies outside the operand gets an offset past the buffer's end,
//    which reads as zero without touching memory, so ragged edges of every
//    dimension cost no branches and no operand needs padding.
//  * A and B have rings of SA and SB stages; s_waitcnt vmcnt plus a bare
//    barrier order them, so later stages stay in flight.
//  * The fp32 tile leaves through LDS in whole rows (finish8): bias,
//    activation and residual act on eight consecutive columns per thread, and
//    stores are whole lines.
#pragma once

#include <type_traits>

#include "activation.h"
#include "products.h"

namespace moe {

namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef const __attribute__((address_space(4))) int const_int;

constexpr int kStep = 64;                     // contraction values per stage
// Buffers are described with kRecords bytes whatever they hold: what keeps a
// lane inside its operand is its offset, kOutside where it has nothing to read.
constexpr uint32_t kRecords = 0xF0000000u;
constexpr uint32_t kOutside = 0xFFFFFFF0u;

template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// The work of one block: a tile of one group's output and a contraction range.
struct Unit {
  int g;      // group
  int row0;   // first output row (forward, input gradient: a row of all P;
              // weight gradient: an out feature)
  int rows;   // output rows in the tile, >= 1
  int col0;   // first output column
  int begin;  // the group's first row and row count
  int len;
  int split;
};

// Bias, z, activation, residual and the store of eight consecutive columns.
// Rounded once per output, from the fp32 sum.
__device__ __forceinline__ void finish8(const ProductArgs& p, F8 v, const float* bias, int64_t row,
                                        int col, int N) {
  const int64_t at = row * N + col;
  if (bias) {
    const F8 b = load8(bias + col);
#pragma unroll
    for (int q = 0; q < 8; ++q) v.v[q] += b.v[q];
  }
  if (p.z) store8(p.z + at, v);
  if (p.act != MOE_ACT_NONE)
#pragma unroll
    for (int q = 0; q < 8; ++q) v.v[q] = activate(v.v[q], p.act);
  if (p.residual) {
    const F8 r = load8(p.residual + at);
#pragma unroll
    for (int q = 0; q < 8; ++q) v.v[q] += r.v[q];
  }
  if (p.y_f32) {
    float* y = static_cast<float*>(p.y) + at;
    if (p.accumulate) {
      const F8 o = load8(y);
#pragma unroll
      for (int q = 0; q < 8; ++q) v.v[q] += o.v[q];
    }
    store8(y, v);
  } else {
    uint16_t* y = static_cast<uint16_t*>(p.y) + at;
    if (p.accumulate) {
      const F8 o = load8(y);
#pragma unroll
      for (int q = 0; q < 8; ++q) v.v[q] += o.v[q];
    }
    store8(y, v);
  }
}

// x's row of row r, or -1.
__device__ __forceinline__ int64_t source_row(const ProductArgs& p, int r) {
  if (!p.src) return r;
  const int id = p.src[r];
  if (id < 0) return -1;
  const int s = id / p.row_div;
  return s < p.x_rows ? s : -1;
}

// One transposing read.  The restrict parameter gives the call alias
// information; without any, the compiler takes it for a possible reader of
// every LDS DMA in flight and waits for all of them (vmcnt(0)) first.  The
// rings' own waits and barriers order the two.
__device__ __forceinline__ s16x4 read_transposed(lds_s16x4* __restrict__ at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(at);
}

// A panel of D tile rows (or columns) by kStep contraction values in LDS,
// filled by pieces of 1 KiB (one wave instruction each).
template <int D, bool STRIDED>
struct Panel {
  static constexpr int BYTES = D * kStep * 2;
  static constexpr int PIECES = BYTES / 1024;
  static constexpr int CPR = STRIDED ? D / 8 : 8;  // 16-byte chunks per LDS row
  static constexpr int RPP = 64 / CPR;             // LDS rows per piece
  static __device__ __forceinline__ int swz(int row) {
    return !STRIDED ? (row >> 1) & 7 : D >= 128 ? 4 * (row & 3) : 4 * ((row >> 1) & 1);
  }
  // Fragment base address of this lane for the 32 rows (columns) from `first`.
  static __device__ __forceinline__ int frag_base(int first, int lane) {
    if (!STRIDED) return (first + (lane & 31)) * 128;
    // row 8 (lane / 32) + (lane % 16) / 4, columns first + 16 ((lane / 16) % 2) + 4 (lane % 4)
    const int row = 8 * (lane >> 5) + ((lane & 15) >> 2);
    const int chunk = first / 8 + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    return row * D * 2 + (chunk ^ swz(row)) * 16 + (lane & 1) * 8;
  }
  // The 8 contraction values 16 ks + 8 (lane / 32) .. of the lane's row.
  static __device__ __forceinline__ bf16x8 frag(uint8_t* panel, int base, int ks, int lane) {
    if constexpr (!STRIDED) {
      const int sw = ((2 * ks + (lane >> 5)) ^ (((lane & 31) >> 1) & 7)) * 16;
      return *reinterpret_cast<const bf16x8*>(panel + base + sw);
    } else {
      // rows 4 apart share row & 3 (and, D = 64, differ in (row >> 1) & 1 by none)
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      const s16x4 lo = read_transposed((lds_s16x4*)(panel + base + 16 * ks * D * 2));
      const s16x4 hi = read_transposed((lds_s16x4*)(panel + base + (16 * ks + 4) * D * 2));
      return __builtin_bit_cast(bf16x8,
                                s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    }
  }
};

template <int OP, int BM_, int BN_, int WM_, int WN_, int SA_, int SB_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, SA = SA_, SB = SB_;
  static constexpr int NW = WM * WN, THREADS = 64 * NW;
  static constexpr int MB = BM / WM / 32, NB = BN / WN / 32;  // 32 x 32 blocks per wave
  using PA = Panel<BM, OP == kWeightGrad>;
  using PB = Panel<BN, OP != kForward>;
  static constexpr int JA = PA::PIECES / NW, JB = PB::PIECES / NW;  // pieces per wave and stage
  static constexpr int KS = kStep / 16;
  static constexpr int RING = SA * PA::BYTES + SB * PB::BYTES;
  // the fp32 tile leaves in passes that fit the ring
  static constexpr int PASSES = (BM * BN * 4 + RING - 1) / RING;
  static_assert(MB >= 1 && NB >= 1 && JA >= 1 && JB >= 1 && MB % PASSES == 0, "tile shape");
  static_assert(SA == SB || (SA == 2 && SB > 2), "ring depths");
  static_assert((SB - 1) * (JA + JB) < 64, "vmcnt budget");
};

// DB (weight gradient): the tile also sums dy over the rows, by one product
// more per 16 rows with a matrix of ones; the waves side by side take a block
// of 32 out features each.
template <int OP, class T, bool GATHER, bool DB>
__device__ __forceinline__ void product_tile(const ProductArgs& p, uint8_t* smem, const Unit& un) {
  using PA = typename T::PA;
  using PB = typename T::PB;
  const int N = OP == kForward ? p.F : p.K;
  const int L = OP == kForward ? p.K : OP == kInputGrad ? p.F : un.len;
  const int KT = (L + kStep - 1) / kStep;
  const int per = (KT + p.splits - 1) / p.splits;
  const int k_first = min(KT, un.split * per), k_last = min(KT, k_first + per);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid / T::WN, wn = wid % T::WN;
  const int cols = min(T::BN, N - un.col0);

  // ---- sources: per lane a byte offset from a base that moves with the step
  const char *abase, *bbase;
  int64_t astep, bstep;
  if (OP == kWeightGrad) {
    abase = reinterpret_cast<const char*>(p.a + static_cast<int64_t>(un.begin) * p.F + un.row0);
    astep = static_cast<int64_t>(kStep) * p.F * 2;
    if (GATHER) {
      bbase = reinterpret_cast<const char*>(p.b + un.col0);
      bstep = 0;
    } else {
      bbase = reinterpret_cast<const char*>(p.b + static_cast<int64_t>(un.begin) * p.K + un.col0);
      bstep = static_cast<int64_t>(kStep) * p.K * 2;
    }
  } else {
    const int64_t wsize = static_cast<int64_t>(p.F) * p.K;
    const uint16_t* w = p.b + un.g * wsize;
    astep = kStep * 2;
    if (OP == kForward && p.src) {
      abase = reinterpret_cast<const char*>(p.a);
      } else {
      abase = reinterpret_cast<const char*>(p.a + static_cast<int64_t>(un.row0) * L);
      }
    if (OP == kForward) {
      bbase = reinterpret_cast<const char*>(w + static_cast<int64_t>(un.col0) * L);
      bstep = kStep * 2;
    } else {
      bbase = reinterpret_cast<const char*>(w + un.col0);
      bstep = static_cast<int64_t>(kStep) * N * 2;
    }
  }
  uint32_t aoff[T::JA], boff[T::JB];
  bool atail[T::JA], btail[T::JB];  // the lane's values lie behind L in the last step
  const int lim = L - (KT - 1) * kStep;
#pragma unroll
  for (int j = 0; j < T::JA; ++j) {
    const int row = PA::RPP * (wid * T::JA + j) + lane / PA::CPR;
    const int chunk = (lane % PA::CPR) ^ PA::swz(row);
    atail[j] = (OP == kWeightGrad ? row : chunk * 8) >= lim;
    if (OP == kWeightGrad) {
      aoff[j] = chunk * 8 < p.F - un.row0 ? static_cast<uint32_t>(row) * p.F * 2 + chunk * 16
                                          : kOutside;
    } else {
      int64_t s = row;
      if (row >= un.rows)
        s = -1;
      else if (OP == kForward && p.src)
        s = source_row(p, un.row0 + row);
      aoff[j] = s >= 0 ? static_cast<uint32_t>(s * L * 2 + chunk * 16) : kOutside;
    }
  }
#pragma unroll
  for (int j = 0; j < T::JB; ++j) {
    const int row = PB::RPP * (wid * T::JB + j) + lane / PB::CPR;
    const int chunk = (lane % PB::CPR) ^ PB::swz(row);
    btail[j] = (OP == kForward ? chunk * 8 : row) >= lim;
    if (OP == kForward) {
      boff[j] = row < cols ? static_cast<uint32_t>(row) * L * 2 + chunk * 16 : kOutside;
    } else {
      const uint32_t r = GATHER ? 0 : static_cast<uint32_t>(row) * N * 2;
      // db alone (no y): x is not read
      boff[j] = chunk * 8 < cols && (OP != kWeightGrad || p.y) ? r + chunk * 16 : kOutside;
    }
  }
  uint8_t* const aring = smem;
  uint8_t* const bring = smem + T::SA * PA::BYTES;
  auto load = [&](const char* base, int64_t step, int kt, uint32_t off, uint8_t* lds) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(base + kt * step), 0, static_cast<int>(kRecords), 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, off, 0, 0, 0);
  };
  auto issue_a = [&](int kt, int j) {
    const uint32_t off = (kt == KT - 1 && atail[j]) ? kOutside : aoff[j];
    load(abase, astep, kt, off,
         aring + ((kt - k_first) % T::SA) * PA::BYTES + (wid * T::JA + j) * 1024);
  };
  // Gathered rows of the weight gradient: the wave's rows of a stage are
  // consecutive, so their sources come by scalar loads, a stage ahead.
  constexpr int IDS = GATHER ? PB::RPP * T::JB : 1;
  int ids[IDS];
  auto fetch_ids = [&](int kt) {
    if constexpr (GATHER) {
      if (kt < k_last) {
        const const_int* s = (const const_int*)(p.src + un.begin + kt * kStep + wid * IDS);
#pragma unroll
        for (int i = 0; i < IDS; ++i) {
          const int id = s[i];  // in the padding behind the last row at most
          ids[i] = kt * kStep + wid * IDS + i < L ? id : -1;
        }
      }
    }
  };
  auto issue_b = [&](int kt, int j) {
    uint32_t off = boff[j];
    if constexpr (GATHER) {
      int s = ids[PB::RPP * j];
#pragma unroll
      for (int i = 1; i < PB::RPP; ++i) s = lane / PB::CPR == i ? ids[PB::RPP * j + i] : s;
      off = s < 0 || off == kOutside ? kOutside : off + static_cast<uint32_t>(s) * p.K * 2;
    } else {
      off = (kt == KT - 1 && btail[j]) ? kOutside : off;
    }
    load(bbase, bstep, kt, off,
         bring + ((kt - k_first) % T::SB) * PB::BYTES + (wid * T::JB + j) * 1024);
  };

  // ---- fragments and products
  int abase_l[T::MB], bbase_l[T::NB];
#pragma unroll
  for (int mb = 0; mb < T::MB; ++mb)
    abase_l[mb] = PA::frag_base(wm * (T::BM / T::WM) + 32 * mb, lane);
#pragma unroll
  for (int nb = 0; nb < T::NB; ++nb)
    bbase_l[nb] = PB::frag_base(wn * (T::BN / T::WN) + 32 * nb, lane);
  f32x16 acc[T::MB][T::NB];
#pragma unroll
  for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) acc[mb][nb] = f32x16{};
  f32x16 dbacc{};
  const __bf16 one = static_cast<__bf16>(1.0f);
  const bf16x8 ones{one, one, one, one, one, one, one, one};

  bf16x8 af[2][T::MB], bf[2][T::NB];
  auto load_frags = [&](int kt, int ks, int set) {
    uint8_t* sa = aring + ((kt - k_first) % T::SA) * PA::BYTES;
    uint8_t* sb = bring + ((kt - k_first) % T::SB) * PB::BYTES;
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) bf[set][nb] = PB::frag(sb, bbase_l[nb], ks, lane);
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb) af[set][mb] = PA::frag(sa, abase_l[mb], ks, lane);
  };
  auto barrier = [] { asm volatile("s_barrier" ::: "memory"); };
  // Split rings (SA == 2 < SB): A is requested one step ahead, as a step
  // starts, B SB - 1 steps ahead between the products.  Loads return in
  // order, so when a step ends only the B stage requested in it may be in
  // flight.  Equal rings: both are requested S - 1 steps ahead.
  constexpr bool SPLIT = T::SA != T::SB;
  constexpr int REFILLS = SPLIT ? T::JB : T::JA + T::JB;
  auto refill = [&](int kt, int d) {
    if (SPLIT)
      issue_b(kt + T::SB - 1, d);
    else if (d < T::JA)
      issue_a(kt + T::SB - 1, d);
    else
      issue_b(kt + T::SB - 1, d - T::JA);
  };
  auto step_end = [&](int kt) {
    if (kt + T::SB - 1 < k_last)
      wait_loads<(SPLIT ? T::JB : (T::SB - 2) * (T::JA + T::JB))>();
    else
      wait_loads<0>();
    barrier();
  };
  if (k_first < k_last) {
#pragma unroll
    for (int s = 0; s < T::SB - 1; ++s)
      if (k_first + s < k_last) {
        fetch_ids(k_first + s);
        if (s < T::SA - 1)
#pragma unroll
          for (int j = 0; j < T::JA; ++j) issue_a(k_first + s, j);
#pragma unroll
        for (int j = 0; j < T::JB; ++j) issue_b(k_first + s, j);
      }
    fetch_ids(k_first + T::SB - 1);
    if (k_first + T::SB - 2 < k_last)
      wait_loads<(T::SB - 2) * (SPLIT ? T::JB : T::JA + T::JB)>();
    else
      wait_loads<0>();
    barrier();
    constexpr int MFMAS = T::KS * T::MB * T::NB;
    constexpr int EVERY = MFMAS / REFILLS > 0 ? MFMAS / REFILLS : 1;
    const bool has_work = wm * (T::BM / T::WM) < un.rows && wn * (T::BN / T::WN) < cols;
    if (!has_work && !DB) {
      for (int kt = k_first; kt < k_last; ++kt) {
        if (SPLIT && kt + 1 < k_last)
#pragma unroll
          for (int j = 0; j < T::JA; ++j) issue_a(kt + 1, j);
        if (kt + T::SB - 1 < k_last)
#pragma unroll
          for (int d = 0; d < REFILLS; ++d) refill(kt, d);
        fetch_ids(kt + T::SB);
        if (kt + 1 < k_last) step_end(kt);
      }
    } else {
      auto step = [&](int kt, auto REFILL) {
        constexpr bool more = decltype(REFILL)::value;
        if (SPLIT && kt + 1 < k_last)
#pragma unroll
          for (int j = 0; j < T::JA; ++j) issue_a(kt + 1, j);
        load_frags(kt, 0, 0);
#pragma unroll
        for (int ks = 0; ks < T::KS; ++ks) {
          if (ks + 1 < T::KS) load_frags(kt, ks + 1, (ks + 1) & 1);
          if constexpr (DB) {
            bf16x8 mine = af[ks & 1][0];
#pragma unroll
            for (int mb = 1; mb < T::MB; ++mb) mine = wn == mb ? af[ks & 1][mb] : mine;
            dbacc = mfma32(ones, mine, dbacc);
          }
#pragma unroll
          for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
            for (int nb = 0; nb < T::NB; ++nb) {
              acc[mb][nb] = mfma32(bf[ks & 1][nb], af[ks & 1][mb], acc[mb][nb]);
              const int i = (ks * T::MB + mb) * T::NB + nb;
              if (more && i % EVERY == EVERY - 1 && i / EVERY < REFILLS) refill(kt, i / EVERY);
            }
          __builtin_amdgcn_sched_barrier(0);
        }
        if (more && MFMAS / EVERY < REFILLS)
#pragma unroll
          for (int d = MFMAS / EVERY; d < REFILLS; ++d) refill(kt, d);
        if (more) fetch_ids(kt + T::SB);
        if (kt + 1 < k_last) step_end(kt);
      };
      int kt = k_first;
      for (; kt + T::SB - 1 < k_last; ++kt) step(kt, std::true_type{});
      for (; kt < k_last; ++kt) step(kt, std::false_type{});
    }
  }

  // ---- the tile leaves.  acc[mb][nb]: lane l holds row 32 mb + l % 32 and,
  // for r = 4 g .. 4 g + 3, columns 8 g + 4 (l / 32) + 0..3 of block nb.
  const int64_t out_row0 = (OP == kWeightGrad ? static_cast<int64_t>(un.g) * p.F : 0) + un.row0;
  const int64_t out_rows = OP == kWeightGrad ? static_cast<int64_t>(p.G) * p.F : p.P;
  if constexpr (DB) {
    const int r = wm * (T::BM / T::WM) + 32 * wn + (lane & 31);
    if (wn < T::MB && lane < 32 && r < un.rows) {
      const int64_t i = out_row0 + r;
      if (p.splits > 1)
        p.part_db[un.split * out_rows + i] = dbacc[0];
      else
        p.db[i] = p.accumulate ? p.db[i] + dbacc[0] : dbacc[0];
    }
  }
  if (OP == kWeightGrad && !p.y) return;
  const float* bias =
      OP == kForward && p.bias ? p.bias + static_cast<int64_t>(un.g) * p.F : nullptr;
  constexpr int Q = T::BN / 4;                        // 16-byte chunks per staged row
  constexpr int WROWS = T::BM / T::WM / T::PASSES;    // staged rows per wave row and pass
  constexpr int SROWS = T::BM / T::PASSES;
  float* const stage = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int pass = 0; pass < T::PASSES; ++pass) {
    __syncthreads();
#pragma unroll
    for (int m = 0; m < T::MB / T::PASSES; ++m) {
      const int mb = pass * (T::MB / T::PASSES) + m;
      const int sr = wm * WROWS + 32 * m + (lane & 31);
#pragma unroll
      for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x16& v = acc[mb][nb];
          const int q = (wn * (T::BN / T::WN) + 32 * nb + 8 * g) / 4 + (lane >> 5);
          *reinterpret_cast<f32x4*>(stage + (sr * Q + (q ^ (sr & 15))) * 4) =
              f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
        }
    }
    __syncthreads();
    for (int i = tid; i < SROWS * (T::BN / 8); i += T::THREADS) {
      const int sr = i / (T::BN / 8), c = i % (T::BN / 8);
      const int row = sr / WROWS * (T::BM / T::WM) + pass * WROWS + sr % WROWS;
      if (row >= un.rows || c * 8 >= cols) continue;
      const f32x4 lo = *reinterpret_cast<const f32x4*>(stage + (sr * Q + ((2 * c) ^ (sr & 15))) * 4);
      const f32x4 hi =
          *reinterpret_cast<const f32x4*>(stage + (sr * Q + ((2 * c + 1) ^ (sr & 15))) * 4);
      const F8 v{{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}};
      if (p.splits > 1)
        store8(p.part + (un.split * out_rows + out_row0 + row) * N + un.col0 + c * 8, v);
      else
        finish8(p, v, bias, out_row0 + row, un.col0 + c * 8, N);
    }
  }
}

}  // namespace

}  // namespace moe

// One output tile of a linear or grouped product on gfx950 matrix cores: the
// forward product y = x W^T, the input gradient dx = dy W and the weight
// gradient dW = dy^T x share this mainloop.
//
//  * bf16 x bf16 -> fp32 on v_mfma_f32_32x32x16_bf16, contraction steps of 64 (or 32).
//  * An operand whose contraction runs along its rows in memory (x and W of
//    the forward product, dy of the input gradient) is laid down in LDS as
//    [tile row][step], and a fragment is one 16-byte read.  An
//    operand whose contraction runs across rows (W of the input gradient,
//    both of the weight gradient) is laid down as it lies in memory, [step][tile
//    column], and a fragment is two transposing reads (ds_read_b64_tr_b16: the
//    16 lanes of a group read four rows of 16 columns and each gets one
//    column's four values), so no operand is transposed in memory.
//  * 16-byte chunks are XOR-swizzled: 128-byte rows by (row >> 1) & 7,
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

// The tile's lambdas hold its accumulators by reference: one that is called
// rather than inlined would put them in memory.
#define MOE_INLINE __attribute__((always_inline))

typedef __attribute__((address_space(3))) void lds_void;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

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

// Bias, z, activation, residual and the store of eight consecutive columns at
// element `at` of the output, rounded once per output from the fp32 sum.
// bias and res are zeros where there is none; ACT: the activation, or -1 for
// p.act.
template <int ACT>
__device__ __forceinline__ void finish8(const ProductArgs& p, F8 v, const F8& bias, const F8& res,
                                        int64_t at) {
#pragma unroll
  for (int q = 0; q < 8; ++q) v.v[q] += bias.v[q];
  if (p.z) store8(p.z + at, v);
  const int act = ACT < 0 ? p.act : ACT;
  if (act != MOE_ACT_NONE)
#pragma unroll
    for (int q = 0; q < 8; ++q) v.v[q] = activate(v.v[q], act);
#pragma unroll
  for (int q = 0; q < 8; ++q) v.v[q] += res.v[q];
  if (p.y_f32)
    store8(static_cast<float*>(p.y) + at, v);
  else
    store8(static_cast<uint16_t*>(p.y) + at, v);
}

// The same for one piece on its own.
__device__ __forceinline__ void finish_one(const ProductArgs& p, const F8& v, const float* bias,
                                           int64_t row, int col, int N) {
  const int64_t at = row * N + col;
  const F8 b = bias ? load8(bias + col) : F8{};
  const F8 r = p.residual ? load8(p.residual + at) : F8{};
  finish8<-1>(p, v, b, r, at);
}

// A gradient's eight consecutive columns: stored, or added to what is there.
// STREAM: with the non-temporal hint (a constant, as stores that differ in the
// hint alone are merged without it).
template <bool STREAM, class E>
__device__ __forceinline__ void put_grad8(E* y, F8 v, bool accumulate) {
  if (accumulate) {
    const F8 o = load8(y);
#pragma unroll
    for (int q = 0; q < 8; ++q) v.v[q] += o.v[q];
  }
  if (STREAM)
    stream8(y, v);
  else
    store8(y, v);
}
template <bool STREAM>
__device__ __forceinline__ void put_grad8(const ProductArgs& p, const F8& v, int64_t at) {
  if (p.y_f32)
    put_grad8<STREAM>(static_cast<float*>(p.y) + at, v, p.accumulate);
  else
    put_grad8<STREAM>(static_cast<uint16_t*>(p.y) + at, v, p.accumulate);
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

// A panel of D tile rows (or columns) by BK contraction values in LDS, filled
// by pieces of 1 KiB (one wave instruction each).
template <int D, int BK, bool STRIDED>
struct Panel {
  static constexpr int BYTES = D * BK * 2;
  static constexpr int PIECES = BYTES / 1024;
  static constexpr int CPR = STRIDED ? D / 8 : BK / 8;  // 16-byte chunks per LDS row
  static constexpr int RPP = 64 / CPR;                  // LDS rows per piece
  static_assert(BK == 64 || BK == 32, "contraction step");
  static __device__ __forceinline__ int swz(int row) {
    if (!STRIDED) return BK == 64 ? (row >> 1) & 7 : (row >> 2) & 3;
    return D >= 128 ? 4 * (row & 3) : 4 * ((row >> 1) & 1);
  }
  // Fragment base address of this lane for the 32 rows (columns) from `first`.
  static __device__ __forceinline__ int frag_base(int first, int lane) {
    if (!STRIDED) return (first + (lane & 31)) * BK * 2;
    // row 8 (lane / 32) + (lane % 16) / 4, columns first + 16 ((lane / 16) % 2) + 4 (lane % 4)
    const int row = 8 * (lane >> 5) + ((lane & 15) >> 2);
    const int chunk = first / 8 + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    return row * D * 2 + (chunk ^ swz(row)) * 16 + (lane & 1) * 8;
  }
  // The 8 contraction values 16 ks + 8 (lane / 32) .. of the lane's row.
  static __device__ __forceinline__ bf16x8 frag(uint8_t* panel, int base, int ks, int lane) {
    if constexpr (!STRIDED) {
      const int sw = ((2 * ks + (lane >> 5)) ^ swz(lane & 31)) * 16;
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

template <int OP, int BM_, int BN_, int WM_, int WN_, int SA_, int SB_, int BK_ = 64>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, SA = SA_, SB = SB_, BK = BK_;
  static constexpr int NW = WM * WN, THREADS = 64 * NW;
  static constexpr int MB = BM / WM / 32, NB = BN / WN / 32;  // 32 x 32 blocks per wave
  using PA = Panel<BM, BK, OP == kWeightGrad>;
  using PB = Panel<BN, BK, OP != kForward>;
  static constexpr int JA = PA::PIECES / NW, JB = PB::PIECES / NW;  // pieces per wave and stage
  static constexpr int KS = BK / 16;
  static constexpr int RING = SA * PA::BYTES + SB * PB::BYTES;
  // the fp32 tile leaves in passes that fit the ring
  static constexpr int NEED = (BM * BN * 4 + RING - 1) / RING;
  static constexpr int PASSES = MB % NEED == 0 ? NEED : MB;
  static_assert(MB >= 1 && NB >= 1 && JA >= 1 && JB >= 1 && MB % PASSES == 0 &&
                    BM * BN * 4 / PASSES <= RING,
                "tile shape");
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
  constexpr int kStep = T::BK;
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
  auto load = [&](const char* base, int64_t step, int kt, uint32_t off, uint8_t* lds) MOE_INLINE {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(base + kt * step), 0, static_cast<int>(kRecords), 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, off, 0, 0, 0);
  };
  auto issue_a = [&](int kt, int j) MOE_INLINE {
    const uint32_t off = (kt == KT - 1 && atail[j]) ? kOutside : aoff[j];
    load(abase, astep, kt, off,
         aring + ((kt - k_first) % T::SA) * PA::BYTES + (wid * T::JA + j) * 1024);
  };
  // Gathered rows of the weight gradient: each lane loads the sources of its
  // rows of a stage one step before the stage is requested and ahead of that
  // step's other loads, so that the ring's own wait covers them.
  int ids[T::JB], ids_now[T::JB];
  auto use_ids = [&]() MOE_INLINE {
    if constexpr (GATHER)
#pragma unroll
      for (int j = 0; j < T::JB; ++j) ids_now[j] = ids[j];
  };
  auto fetch_ids = [&](int kt) MOE_INLINE {
    if constexpr (GATHER) {
      if (kt < k_last) {
        const int32_t* s = p.src + un.begin + kt * kStep;  // into the padding at most
#pragma unroll
        for (int j = 0; j < T::JB; ++j)
          ids[j] = s[PB::RPP * (wid * T::JB + j) + lane / PB::CPR];
      }
    }
  };
  auto issue_b = [&](int kt, int j) MOE_INLINE {
    uint32_t off = boff[j];
    if constexpr (GATHER) {
      const int s = ids_now[j];
      off = s < 0 || off == kOutside || (kt == KT - 1 && btail[j])
                ? kOutside
                : off + static_cast<uint32_t>(s) * p.K * 2;
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
  // db: the wave's blocks of out features are wn, wn + WN, ..
  constexpr int DBN = (T::MB + T::WN - 1) / T::WN;
  f32x16 dbacc[DBN];
  // (read on its own: chosen among the wave's fragments, the compiler would
  // index them in scratch memory)
  int dbbase[DBN];
#pragma unroll
  for (int i = 0; i < DBN; ++i) {
    dbacc[i] = f32x16{};
    dbbase[i] = PA::frag_base(wm * (T::BM / T::WM) + 32 * ((wn + i * T::WN) % T::MB), lane);
  }
  const __bf16 one = static_cast<__bf16>(1.0f);
  const bf16x8 ones{one, one, one, one, one, one, one, one};

  bf16x8 af[2][T::MB], bf[2][T::NB];
  bf16x8 dbf[2][DBN];
  auto load_frags = [&](int kt, int ks, int set) MOE_INLINE {
    uint8_t* sa = aring + ((kt - k_first) % T::SA) * PA::BYTES;
    uint8_t* sb = bring + ((kt - k_first) % T::SB) * PB::BYTES;
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) bf[set][nb] = PB::frag(sb, bbase_l[nb], ks, lane);
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb) af[set][mb] = PA::frag(sa, abase_l[mb], ks, lane);
    if constexpr (DB)
#pragma unroll
      for (int i = 0; i < DBN; ++i) dbf[set][i] = PA::frag(sa, dbbase[i], ks, lane);
  };
  // The rings.  Step kt multiplies stage kt.  Before its last products, with
  // all of the stage's fragments in registers, the waves wait for stage kt + 1
  // and meet at a barrier, so that the first fragments of the next step load
  // under these products and no step begins with empty registers.  After the
  // barrier the slots of stage kt are free.  Split rings (SA == 2 < SB): A(kt +
  // 2) is requested right there, B(kt + SB - 1) between the products before;
  // loads return in order, so at the barrier only that B stage may be in
  // flight.  Equal rings: both are requested S - 1 steps ahead between the
  // products.
  constexpr bool SPLIT = T::SA != T::SB;
  constexpr int REFILLS = SPLIT ? T::JB : T::JA + T::JB;
  auto refill = [&](int kt, int d) MOE_INLINE {
    if (SPLIT)
      issue_b(kt + T::SB - 1, d);
    else if (d < T::JA)
      issue_a(kt + T::SB - 1, d);
    else
      issue_b(kt + T::SB - 1, d - T::JA);
  };
  auto meet = [&](int kt) MOE_INLINE {
    if (kt + T::SB - 1 < k_last)
      wait_loads<(SPLIT ? T::JB : (T::SB - 2) * (T::JA + T::JB))>();
    else
      wait_loads<0>();
    // the wave's reads of stage kt have returned before another wave refills
    // its slots
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (SPLIT && kt + 2 < k_last)
#pragma unroll
      for (int j = 0; j < T::JA; ++j) issue_a(kt + 2, j);
  };
  if (k_first < k_last) {
#pragma unroll
    for (int s = 0; s < T::SB - 1; ++s)
      if (k_first + s < k_last) {
        fetch_ids(k_first + s);
        use_ids();
        if (s < T::SA - 1)
#pragma unroll
          for (int j = 0; j < T::JA; ++j) issue_a(k_first + s, j);
#pragma unroll
        for (int j = 0; j < T::JB; ++j) issue_b(k_first + s, j);
      }
    fetch_ids(k_first + T::SB - 1);  // for the first step's refill
    if (k_first + T::SB - 2 < k_last)
      wait_loads<(T::SB - 2) * (SPLIT ? T::JB : T::JA + T::JB)>();
    else
      wait_loads<0>();
    asm volatile("s_barrier" ::: "memory");
    if (SPLIT && k_first + 1 < k_last)
#pragma unroll
      for (int j = 0; j < T::JA; ++j) issue_a(k_first + 1, j);
    constexpr int EARLY = (T::KS - 1) * T::MB * T::NB;  // products before the barrier
    constexpr int EVERY = EARLY / REFILLS > 0 ? EARLY / REFILLS : 1;
    const bool has_work = wm * (T::BM / T::WM) < un.rows && wn * (T::BN / T::WN) < cols;
    if (!has_work && !DB) {
      for (int kt = k_first; kt < k_last; ++kt) {
        use_ids();
        fetch_ids(kt + T::SB);
        if (kt + T::SB - 1 < k_last)
#pragma unroll
          for (int d = 0; d < REFILLS; ++d) refill(kt, d);
        if (kt + 1 < k_last) meet(kt);
      }
    } else {
      load_frags(k_first, 0, 0);
      auto step = [&](int kt, auto REFILL) MOE_INLINE {
        constexpr bool more = decltype(REFILL)::value;
        if (more) {
          use_ids();
          fetch_ids(kt + T::SB);
        }
#pragma unroll
        for (int ks = 0; ks < T::KS; ++ks) {
          if (ks + 1 < T::KS) {
            load_frags(kt, ks + 1, (ks + 1) & 1);
          } else {
            if (more && EARLY / EVERY < REFILLS)
#pragma unroll
              for (int d = EARLY / EVERY; d < REFILLS; ++d) refill(kt, d);
            if (kt + 1 < k_last) {
              meet(kt);
              load_frags(kt + 1, 0, 0);
            }
          }
          if constexpr (DB)
#pragma unroll
            for (int i = 0; i < DBN; ++i) dbacc[i] = mfma32(ones, dbf[ks & 1][i], dbacc[i]);
#pragma unroll
          for (int mb = 0; mb < T::MB; ++mb)
#pragma unroll
            for (int nb = 0; nb < T::NB; ++nb) {
              acc[mb][nb] = mfma32(bf[ks & 1][nb], af[ks & 1][mb], acc[mb][nb]);
              const int i = (ks * T::MB + mb) * T::NB + nb;
              if (more && i < EARLY && i % EVERY == EVERY - 1 && i / EVERY < REFILLS)
                refill(kt, i / EVERY);
            }
          if constexpr (T::MB * T::NB == 8 && T::NW == 8) {
            // Big: three fragment reads, then one after every two products
            // (+1 to 1.5% on 8192 cubed; one after each product, or half of
            // them first: +-0; the smaller tiles lose 2% to any such order).
            __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
#pragma unroll
            for (int q = 0; q < 3; ++q) {
              __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);
              __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      static_assert(T::KS % 2 == 0, "the next step's first fragments take set 0");
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
#pragma unroll
    for (int i = 0; i < DBN; ++i) {
      const int b = wn + i * T::WN, r = wm * (T::BM / T::WM) + 32 * b + (lane & 31);
      if (b < T::MB && lane < 32 && r < un.rows) {
        const int64_t at = out_row0 + r;
        if (p.splits > 1)
          p.part_db[un.split * out_rows + at] = dbacc[i][0];
        else
          p.db[at] = p.accumulate ? p.db[at] + dbacc[i][0] : dbacc[i][0];
      }
    }
  }
  if (OP == kWeightGrad && !p.y) return;
  // In passes through LDS: the fp32 blocks laid down by rows (16-byte chunks
  // XOR-rotated by the row), then each thread takes eight columns, the same in
  // every row it takes, of rows RSTEP apart: its bias is loaded once, and
  // UNROLL rows' residuals and LDS reads are under way together.
  constexpr int Q = T::BN / 4;                      // 16-byte chunks per staged row
  constexpr int WROWS = T::BM / T::WM / T::PASSES;  // staged rows per wave row and pass
  constexpr int SROWS = T::BM / T::PASSES;
  constexpr int CH = T::BN / 8;
  constexpr int RSTEP = T::THREADS / CH, ITERS = SROWS / RSTEP;
  constexpr int UNROLL = ITERS % 4 == 0 ? 4 : 2;
  static_assert(T::THREADS % CH == 0 && SROWS % RSTEP == 0 && ITERS % UNROLL == 0, "copy-out");
  float* const stage = reinterpret_cast<float*>(smem);
  const int c = tid % CH, r0 = tid / CH;
  const bool live = c * 8 < cols;
  F8 bias{};
  if (OP == kForward && p.bias && live && p.splits == 1)
    bias = load8(p.bias + static_cast<int64_t>(un.g) * p.F + un.col0 + c * 8);
  auto run_pass = [&](auto PASS) MOE_INLINE {  // a constant: the blocks stay in registers
    constexpr int pass = decltype(PASS)::value;
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
    auto take = [&](int sr) MOE_INLINE {
      const f32x4 lo = *reinterpret_cast<const f32x4*>(stage + (sr * Q + ((2 * c) ^ (sr & 15))) * 4);
      const f32x4 hi =
          *reinterpret_cast<const f32x4*>(stage + (sr * Q + ((2 * c + 1) ^ (sr & 15))) * 4);
      return F8{{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}};
    };
    auto tile_row = [&](int sr) MOE_INLINE {
      return sr / WROWS * (T::BM / T::WM) + pass * WROWS + sr % WROWS;
    };
    auto copy_out = [&](auto each) MOE_INLINE {
      for (int it = 0; it < ITERS; it += UNROLL) each(r0 + it * RSTEP);
    };
    const int64_t at0 = out_row0 * N + un.col0 + c * 8;
    if (p.splits > 1) {
      float* part = p.part + un.split * out_rows * N + at0;
      copy_out([&](int sr0) MOE_INLINE {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
          const int row = tile_row(sr0 + u * RSTEP);
          if (row < un.rows && live) store8(part + static_cast<int64_t>(row) * N, take(sr0 + u * RSTEP));
        }
      });
    } else if constexpr (OP == kForward) {
      auto with_act = [&](auto ACT) MOE_INLINE {
        copy_out([&](int sr0) MOE_INLINE {
          F8 res[UNROLL], v[UNROLL];
#pragma unroll
          for (int u = 0; u < UNROLL; ++u) {
            const int row = tile_row(sr0 + u * RSTEP);
            res[u] = F8{};
            if (p.residual && row < un.rows && live)
              res[u] = load8(p.residual + at0 + static_cast<int64_t>(row) * N);
            v[u] = take(sr0 + u * RSTEP);
          }
#pragma unroll
          for (int u = 0; u < UNROLL; ++u) {
            const int row = tile_row(sr0 + u * RSTEP);
            if (row < un.rows && live)
              finish8<decltype(ACT)::value>(p, v[u], bias, res[u],
                                            at0 + static_cast<int64_t>(row) * N);
          }
        });
      };
      // one loop per activation: a switch per element costs more than relu
      switch (p.act) {
        case MOE_ACT_RELU: with_act(std::integral_constant<int, MOE_ACT_RELU>{}); break;
        case MOE_ACT_GELU: with_act(std::integral_constant<int, MOE_ACT_GELU>{}); break;
        case MOE_ACT_GELU_TANH: with_act(std::integral_constant<int, MOE_ACT_GELU_TANH>{}); break;
        case MOE_ACT_SILU: with_act(std::integral_constant<int, MOE_ACT_SILU>{}); break;
        default: with_act(std::integral_constant<int, MOE_ACT_NONE>{}); break;
      }
    } else {
      auto put = [&](auto STREAM) MOE_INLINE {
        copy_out([&](int sr0) MOE_INLINE {
#pragma unroll
          for (int u = 0; u < UNROLL; ++u) {
            const int row = tile_row(sr0 + u * RSTEP);
            if (row < un.rows && live)
              put_grad8<decltype(STREAM)::value>(p, take(sr0 + u * RSTEP),
                                                 at0 + static_cast<int64_t>(row) * N);
          }
        });
      };
      if (OP == kWeightGrad && p.stream)
        put(std::true_type{});
      else
        put(std::false_type{});
    }
  };
  static_assert(T::PASSES <= 3, "passes");
  run_pass(std::integral_constant<int, 0>{});
  if constexpr (T::PASSES > 1) run_pass(std::integral_constant<int, 1>{});
  if constexpr (T::PASSES > 2) run_pass(std::integral_constant<int, 2>{});
}

}  // namespace

}  // namespace moe

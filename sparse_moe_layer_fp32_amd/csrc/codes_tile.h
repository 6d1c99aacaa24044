// One output tile of a product of e4m3 codes on gfx950 matrix cores: y = x W^T
// with a scale for each row and block of 128 codes of x, and for each block of
// 128 x 128 of W.  Panels, swizzles, DMA with lanes outside the operand reading
// zero, and the way out are those of product_tile.h, and so are the addresses: a
// row of K codes travels as one of K / 2 16-bit values, and a step is 128 bytes
// of a row, which is one block of scales.
//
//  * A step's products are summed on their own, and the sums added to the
//    accumulators times the scales of their row and column block, in fp32: 16
//    FMAs for every two products of 64 codes.  They run under the next products.
//  * Widened codes are bound by the widening: each wave converts its 32 + 32 rows
//    of a step for eight products of 32 x 32 x 16 (777 x 1296 -> 2056, 429 tiles of
//    64 x 64: 12.9 us, MFMA busy 17%, waiting 36%).  Native 64 x 64 and 128 x 256
//    tiles serve few rows, where W's stream bounds them (512 rows in 288 groups,
//    4096 -> 1280: 130 us, 5.4 TB/s).
//  * 64 x 64 tiles have three stages, so that three blocks share a CU (there 141 us
//    with four stages and two blocks, 140 with two and four; 2048 rows: 261, 283 and
//    284; 8 rows in 8 groups, where a CU has one block: 14.4, 14.0 and 22.5).
//  * One loop serves all steps: loads of stages behind the last see an empty
//    buffer and bring zeros without touching memory.
#pragma once

#include <algorithm>

#include "product_tile.h"

namespace moe {

namespace {

// How a tile multiplies codes.
//
// kNative: v_mfma_f32_32x32x64_f8f6f4, twice the bf16 rate.  It sums the eight
// products of consecutive codes in fixed point, cut 2^-13 below the largest of
// them (measured: a product 2^-14 of its neighbour is lost, one of another eight
// is not), and everything else in fp32: of normal values a block of 128 is off
// by 1.4e-5 of itself in the 2-norm, little beside the 1.7e-3 of a bf16 result,
// for which alone it is used.
// kExact: codes widened to bf16, which holds them, on the bf16 matrix cores:
// exact products, fp32 sums, for fp32 results.
enum CodesKind : int { kNative = 1, kExact = 2 };

// Rings of S stages: both panels S - 1 steps ahead, and with them the scales of
// the tile's rows, one piece of a wave more per 64 rows (the waves without rows
// load nothing into a place of their own, so that all count the same loads).
template <int KIND_, int BM_, int BN_, int WM_, int WN_, int S_>
struct CodesTile {
  static constexpr int KIND = KIND_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_;
  static constexpr int BK = 64;  // in pairs of codes
  static constexpr int NW = WM * WN, THREADS = 64 * NW;
  static constexpr int MB = BM / WM / 32, NB = BN / WN / 32;  // 32 x 32 blocks per wave
  using PA = Panel<BM, BK, false>;
  using PB = Panel<BN, BK, false>;
  static constexpr int JA = PA::PIECES / NW, JB = PB::PIECES / NW;  // pieces per wave and stage
  static constexpr int AHEAD = S - 1;
  static constexpr int RING = S * (PA::BYTES + PB::BYTES);
  static constexpr int SWAVES = BM / 64;
  static constexpr int SBYTES = BM * 4;
  static constexpr int LDS = RING + S * SBYTES + 256;
  static constexpr int J = JA + JB + 1;  // pieces per wave and stage, all told
  // the fp32 tile leaves in passes that fit the ring
  static constexpr int NEED = (BM * BN * 4 + RING - 1) / RING;
  static constexpr int PASSES = MB % NEED == 0 ? NEED : MB;
  static_assert(MB >= 1 && NB >= 1 && JA >= 1 && JB >= 1 && MB % PASSES == 0 &&
                    BM * BN * 4 / PASSES <= RING && LDS <= 160 * 1024,
                "tile shape");
  static_assert(AHEAD * J < 64, "vmcnt budget");
  static_assert(BM % 64 == 0 && SWAVES <= NW, "row scales");
  static_assert(128 % (BN / WN) == 0, "a wave's columns share their scale");
};

template <class T>
__device__ __forceinline__ void codes_tile(const CodesArgs& p, uint8_t* smem, const Unit& un) {
  using PA = typename T::PA;
  using PB = typename T::PB;
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  struct U32x8 {
    u32x4 lo, hi;
  };
  const int N = p.F, L = p.K;
  constexpr int kStep = T::BK;
  const int KT = (L + kStep - 1) / kStep;
  const int per = (KT + p.splits - 1) / p.splits;
  const int k_first = min(KT, un.split * per), k_last = min(KT, k_first + per);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid / T::WN, wn = wid % T::WN;
  const int cols = min(T::BN, N - un.col0);

  // ---- sources: per lane a byte offset from a base that moves with the step
  const char* const abase = reinterpret_cast<const char*>(
      p.a + (p.src ? 0 : static_cast<int64_t>(un.row0) * L));
  const char* const bbase = reinterpret_cast<const char*>(
      p.b + (static_cast<int64_t>(un.g) * N + un.col0) * L);
  uint32_t aoff[T::JA], boff[T::JB];
  bool atail[T::JA], btail[T::JB];  // the lane's codes lie behind L in the last step
  const int lim = L - (KT - 1) * kStep;
#pragma unroll
  for (int j = 0; j < T::JA; ++j) {
    const int row = PA::RPP * (wid * T::JA + j) + lane / PA::CPR;
    const int chunk = (lane % PA::CPR) ^ PA::swz(row);
    atail[j] = chunk * 8 >= lim;
    int64_t s = row;
    if (row >= un.rows)
      s = -1;
    else if (p.src)
      s = source_row(p, un.row0 + row);
    aoff[j] = s >= 0 ? static_cast<uint32_t>(s * L * 2 + chunk * 16) : kOutside;
  }
#pragma unroll
  for (int j = 0; j < T::JB; ++j) {
    const int row = PB::RPP * (wid * T::JB + j) + lane / PB::CPR;
    const int chunk = (lane % PB::CPR) ^ PB::swz(row);
    btail[j] = chunk * 8 >= lim;
    boff[j] = row < cols ? static_cast<uint32_t>(row) * L * 2 + chunk * 16 : kOutside;
  }
  uint8_t* const aring = smem;
  uint8_t* const bring = smem + T::S * PA::BYTES;
  uint8_t* const sring = smem + T::RING;
  auto records = [&](int kt) MOE_INLINE { return static_cast<int>(kt < k_last ? kRecords : 0u); };
  auto load = [&](const char* base, int kt, uint32_t off, uint8_t* to) MOE_INLINE {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(base + static_cast<int64_t>(kt) * kStep * 2), 0, records(kt), 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 16, off, 0, 0, 0);
  };
  auto issue_a = [&](int kt, int j) MOE_INLINE {
    const uint32_t off = (kt == KT - 1 && atail[j]) ? kOutside : aoff[j];
    load(abase, kt, off,
         aring + ((kt - k_first) % T::S) * PA::BYTES + (wid * T::JA + j) * 1024);
  };
  auto issue_b = [&](int kt, int j) MOE_INLINE {
    const uint32_t off = (kt == KT - 1 && btail[j]) ? kOutside : boff[j];
    load(bbase, kt, off,
         bring + ((kt - k_first) % T::S) * PB::BYTES + (wid * T::JB + j) * 1024);
  };

  // ---- scales: of this lane's rows, and of the wave's columns
  const char* const sbase = reinterpret_cast<const char*>(
      p.a_scale + (p.src ? 0 : static_cast<int64_t>(un.row0) * KT));
  auto scale_offset = [&](int row) MOE_INLINE {
    if (row >= un.rows) return kOutside;
    const int64_t s = p.src ? source_row(p, un.row0 + row) : row;
    return s >= 0 ? static_cast<uint32_t>(s * KT * 4) : kOutside;
  };
  // of the row whose scale this lane fetches
  const uint32_t soff = wid < T::SWAVES ? scale_offset(64 * wid + lane) : kOutside;
  const int fblocks = (N + 127) / 128;
  const int fb = min((un.col0 + wn * (T::BN / T::WN)) / 128, fblocks - 1);
  const float* const wscale = p.b_scale + (static_cast<int64_t>(un.g) * fblocks + fb) * KT;
  float ws_held = 0.0f;  // lane i: the column block's scale of step i of 64
  auto hold_scales = [&](int kt) MOE_INLINE { ws_held = wscale[min(kt + lane, KT - 1)]; };
  auto issue_s = [&](int kt) MOE_INLINE {
    uint8_t* const to = wid < T::SWAVES
                            ? sring + ((kt - k_first) % T::S) * T::SBYTES + wid * 256
                            : sring + T::S * T::SBYTES;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(sbase + static_cast<int64_t>(kt) * 4), 0, records(kt), 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 4, soff, 0, 0, 0);
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

  // A half of a step: two chunks of a row, 32 codes of each half of the wave.
  // Which codes meet in which product is the same for both operands, and that is
  // all that a sum over them asks.
  u32x4 bq[T::NB][4], aq[4];
  auto load_b = [&](int kt, int half) MOE_INLINE {
    uint8_t* sb = bring + ((kt - k_first) % T::S) * PB::BYTES;
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
      for (int c = 2 * half; c < 2 * half + 2; ++c)
        bq[nb][c] = __builtin_bit_cast(u32x4, PB::frag(sb, bbase_l[nb], c, lane));
  };
  auto load_a = [&](int kt, int mb, int half) MOE_INLINE {
    uint8_t* sa = aring + ((kt - k_first) % T::S) * PA::BYTES;
#pragma unroll
    for (int c = 2 * half; c < 2 * half + 2; ++c)
      aq[c] = __builtin_bit_cast(u32x4, PA::frag(sa, abase_l[mb], c, lane));
  };
  // Block nb's sums of the step in the wave's present row block.
  f32x16 t[T::NB];
  auto multiply = [&](int nb, int half) MOE_INLINE {
    const u32x4 b0 = bq[nb][2 * half], b1 = bq[nb][2 * half + 1];
    const u32x4 a0 = aq[2 * half], a1 = aq[2 * half + 1];
    f32x16 v = half ? t[nb] : f32x16{};
    if constexpr (T::KIND == kNative) {
      const i32x8 b = __builtin_bit_cast(i32x8, U32x8{b0, b1});
      const i32x8 a = __builtin_bit_cast(i32x8, U32x8{a0, a1});
      v = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, v, 0, 0, 0, 0, 0, 0);
    } else {
      v = mfma32(e4m3x8_to_bf16(b0[0], b0[1]), e4m3x8_to_bf16(a0[0], a0[1]), v);
      v = mfma32(e4m3x8_to_bf16(b0[2], b0[3]), e4m3x8_to_bf16(a0[2], a0[3]), v);
      v = mfma32(e4m3x8_to_bf16(b1[0], b1[1]), e4m3x8_to_bf16(a1[0], a1[1]), v);
      v = mfma32(e4m3x8_to_bf16(b1[2], b1[3]), e4m3x8_to_bf16(a1[2], a1[3]), v);
    }
    t[nb] = v;
  };
  auto add = [&](int mb, int nb, float scale) MOE_INLINE {
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[mb][nb][i] = fmaf(scale, t[nb][i], acc[mb][nb][i]);
  };
  // At the end of step kt: the wave's reads of stage kt have returned before
  // another wave refills its slots, and stage kt + 1 is there.
  auto meet = [&]() MOE_INLINE {
    wait_loads<(T::AHEAD - 1) * T::J>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  // Piece d of stage kt + AHEAD.
  auto refill = [&](int kt, int d) MOE_INLINE {
    if (d < T::JA)
      issue_a(kt + T::AHEAD, d);
    else if (d < T::JA + T::JB)
      issue_b(kt + T::AHEAD, d - T::JA);
    else
      issue_s(kt + T::AHEAD);
  };

  if (k_first < k_last) {
    hold_scales(k_first);  // (first: the rings' first wait covers it)
#pragma unroll
    for (int s = 0; s < T::AHEAD; ++s)
#pragma unroll
      for (int d = 0; d < T::J; ++d) refill(k_first + s - T::AHEAD, d);
    wait_loads<(T::AHEAD - 1) * T::J>();
    asm volatile("s_barrier" ::: "memory");
    const bool has_work = wm * (T::BM / T::WM) < un.rows && wn * (T::BN / T::WN) < cols;
    if (!has_work) {
      for (int kt = k_first; kt < k_last; ++kt) {
#pragma unroll
        for (int d = 0; d < T::J; ++d) refill(kt, d);
        meet();
      }
    } else {
      // A row block's sums are added when the next one's products replace them
      // one by one, so that the additions run under products; the last block's
      // in the next step, with the scale of its own (`last`; at first 0, times
      // sums of 0).  Fragments are replaced as soon as their products are issued.
      float rs[T::MB], last = 0.0f;
#pragma unroll
      for (int nb = 0; nb < T::NB; ++nb) t[nb] = f32x16{};
      auto step = [&](int kt) MOE_INLINE {
        // Pieces of the refill by row block, and what is left in the last one.
        constexpr int FIRST = T::MB - 1;
        constexpr int PER = FIRST > 0 ? (T::J + FIRST - 1) / std::max(FIRST, 1) : 0;
        const float w = __builtin_bit_cast(
            float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ws_held), (kt - k_first) & 63));
#pragma unroll
        for (int mb = 0; mb < T::MB; ++mb) {
          rs[mb] = w * *reinterpret_cast<const float*>(
                           sring + ((kt - k_first) % T::S) * T::SBYTES +
                           (wm * (T::BM / T::WM) + 32 * mb + (lane & 31)) * 4);
        }
        if (((kt + 1 - k_first) & 63) == 0) hold_scales(kt + 1);
#pragma unroll
        for (int mb = 0; mb < T::MB; ++mb) {
          const bool final = mb + 1 == T::MB;
          if (final) {
#pragma unroll
            for (int d = FIRST * PER; d < T::J; ++d) refill(kt, d);
            meet();
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int nb = 0; nb < T::NB; ++nb) {
              if (half == 0) add(mb ? mb - 1 : T::MB - 1, nb, mb ? rs[mb - 1] : last);
              __builtin_amdgcn_sched_barrier(0);  // (the products take the sums' registers)
              multiply(nb, half);
              __builtin_amdgcn_sched_barrier(0);
            }
            if (!final) {
              load_a(kt, mb + 1, half);
            } else {
              load_a(kt + 1, 0, half);
              load_b(kt + 1, half);
            }
          }
          if (!final)
#pragma unroll
            for (int d = mb * PER; d < (mb + 1) * PER && d < T::J; ++d) refill(kt, d);
          __builtin_amdgcn_sched_barrier(0);
        }
        last = rs[T::MB - 1];
      };
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        load_b(k_first, half);
        load_a(k_first, 0, half);
      }
      // (a first step of its own, which the compiler would make, spills registers)
#pragma clang loop unroll(disable)
      for (int kt = k_first; kt < k_last; ++kt) step(kt);
#pragma unroll
      for (int nb = 0; nb < T::NB; ++nb) add(T::MB - 1, nb, last);
    }
    wait_loads<0>();  // (of stages behind the last, whose zeros go to LDS)
  }
  tile_leaves<kForward, T>(p, smem, un, acc, wm, wn);
}

template <int Q> using CodesHalf = CodesTile<Q, 128, 256, 2, 4, 3>;
template <int Q> using CodesSmall = CodesTile<Q, 64, 64, 2, 2, 3>;

}  // namespace

}  // namespace moe

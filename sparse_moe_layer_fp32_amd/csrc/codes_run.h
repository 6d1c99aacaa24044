// Large products of codes: blocks that stay on their CU and take one 256 x 256
// tile after the other, for bf16 results.
//
// A tile by itself starts with loads that have nothing to hide behind, and ends
// with stores that have not either.  Here the rings run on across tiles: the last
// two steps of a tile load the first two stages of the next, which arrive while the
// tile leaves (8192 x 512 -> 8192, four steps a tile: 74 us, from 88; at 32 steps a
// tile 1%).
//
// Bound: power and the matrix pipe.  8192 x 4096 -> 11264 takes 323 us here, 2.3
// PFLOP/s, at 1.97 GHz (2.4 with operands of zeros); MFMA busy 57%, the additions
// of blocks under their scales 12% of the cycles, tiles' ends 9%, loads 8%, LDS
// reads 6%, the barrier in mid-step 3%.  Gathered rows of few a group take longer:
// 65536 rows of 288 groups, 4096 -> 1280, 466 us, MFMA busy 45%.  Their L2s fetch 2.5
// GB, of which memory has to give W's 1.5 (x's 34 MB stay in the last-level cache),
// and the compiler holds x's buffer in vector registers: each of its loads runs in a
// loop that makes it scalar, four a step, and 13 vector registers are spilled.
//
//  * Rings: three stages of x, two of W, all 160 KB.  A wave holds a step's
//    fragments of W from the step's start, so W's slot is free after a barrier in
//    mid-step, and both panels are loaded two steps ahead.
//  * A tile leaves wave by wave, without barriers, through the slot of x's last
//    stage, which the next tile's third stage fills: wave w stages 16 rows of its
//    64 columns at a time in the 4 KB that its own loads of that stage will
//    overwrite, so that its own order is all the order there is to keep.
//  * Waves take the 32-row blocks of a tile in turn (block b: wave row b % 2), so
//    that a tile of fewer rows, a group's remainder or a cut tile, costs both
//    waves of a SIMD as much less; rows outside the tile are not loaded.
//  * The rows' scales come from a copy ordered by steps (codes_prepare_kernel), 128
//    bytes to a load: read as they lie, 32 rows 128 bytes apart, they took as long
//    to fetch as the panels (13% of 8192 x 4096 -> 11264; the copy takes 5 us).
#pragma once

#include "codes_tile.h"

namespace moe {

namespace {

// (constant while a kernel of this file runs, and so loaded by scalar loads, which
// do not queue behind the rings')
typedef const __attribute__((address_space(4))) RowTile ConstTile;
typedef const __attribute__((address_space(4))) int32_t ConstInt;

// An offset past every x (kMaxGatherBytes in the C entries), with room for a
// row's length to be added.
constexpr uint32_t kFar = 0xF0000000u;

struct CodesRun {
  static constexpr int BM = 256, BN = 256, THREADS = 512;
  static constexpr int MB = 4;           // 32-row blocks of a wave
  static constexpr int IB = 8, NB = 4;   // its products of 16 x 16: rows, columns
  static constexpr int SA = 3, SB = 2, AHEAD = 2;
  using Pan = Panel<256, 64, false>;
  static constexpr int JP = Pan::PIECES / 8;  // pieces of a panel per wave
  static constexpr int J = 2 * JP;
  static constexpr int LDS = (SA + SB) * Pan::BYTES;
  static_assert(LDS == 160 * 1024, "all of LDS");
};

// A block's next tile: its place in the walk of the virtual grid of one block per
// tile (find_unit's, with the same mapping of blocks to XCDs).  The rings' look
// ahead needs tiles of two steps at least.
struct Walk {
  int bid, limit;       // next virtual block, and their number
  int NT, units, cut;   // column tiles; tiles; dense: the first that is cut, or -1
};

__device__ __forceinline__ Walk start_walk(const CodesArgs& p) {
  Walk w;
  w.bid = blockIdx.x;
  w.NT = (p.F + CodesRun::BN - 1) / CodesRun::BN;
  const int rows = p.tiles ? *(ConstInt*)p.num_tiles : static_cast<int>((p.P + CodesRun::BM - 1) / CodesRun::BM);
  w.units = rows * w.NT;
  w.cut = p.whole >= 0 ? p.whole / kNumXcd * kNumXcd : -1;
  w.limit = w.cut >= 0 ? w.cut + (w.units - w.cut) * p.slices : w.units;
  w.limit = (w.limit + kNumXcd - 1) / kNumXcd * kNumXcd;
  return w;
}

__device__ __forceinline__ bool next_tile(const CodesArgs& p, Walk* w, Unit* un) {
  for (; w->bid < w->limit; w->bid += gridDim.x) {
    int part = 0, parts = 1;
    const int v = w->cut >= 0 ? cut_unit(w->bid, w->cut, w->units, p.slices, &part)
                              : xcd_remap(w->bid, w->units);
    if (v < 0) continue;
    if (w->cut >= 0 && v >= w->cut) parts = p.slices;
    // runs of kGroupM row tiles of a group, the row tile fastest
    int first = 0, tiles = w->units / w->NT;
    if (p.tiles) {
      ConstTile* t = (ConstTile*)p.tiles + v / w->NT;
      first = t->first;
      tiles = t->tiles;
    }
    const int i = v - first * w->NT;
    const int run = i / (kGroupM * w->NT) * kGroupM;
    const int gm = min(kGroupM, tiles - run);
    const int x = i - run * w->NT;
    const int rt = run + x % gm;
    // (readfirstlane: all of it is the block's, and stays in scalar registers)
    un->col0 = __builtin_amdgcn_readfirstlane(x / gm * CodesRun::BN);
    if (p.tiles) {
      ConstTile* t = (ConstTile*)p.tiles + first + rt;
      un->row0 = __builtin_amdgcn_readfirstlane(t->row0);
      un->rows = __builtin_amdgcn_readfirstlane(t->rows);
      un->g = __builtin_amdgcn_readfirstlane(t->g);
    } else {
      un->row0 = __builtin_amdgcn_readfirstlane(rt * CodesRun::BM + part * (CodesRun::BM / parts));
      un->rows = __builtin_amdgcn_readfirstlane(
          min(CodesRun::BM / parts, static_cast<int>(p.P) - un->row0));
      un->g = 0;
    }
    if (un->rows <= 0) continue;
    w->bid += gridDim.x;
    return true;
  }
  return false;
}

// 32 rows' values in both halves of a wave -> 16 rows' each in all four quarters.
__device__ __forceinline__ void split_rows(float v, float* lo, float* hi) {
  const uint32_t u = __float_as_uint(v);
  const auto both = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  *lo = __uint_as_float(both[0]);
  *hi = __uint_as_float(both[1]);
}

// GATHER: x's rows are named by p.src.  ACT: there is an activation.
template <bool GATHER, bool ACT>
__global__ __launch_bounds__(CodesRun::THREADS, 2) void codes_run_kernel(CodesArgs p) {
  using R = CodesRun;
  using Pan = R::Pan;
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  struct U32x8 {
    u32x4 lo, hi;
  };
  __shared__ __attribute__((aligned(1024))) uint8_t smem[R::LDS];
  Walk walk = start_walk(p);
  Unit un, nx;
  if (!next_tile(p, &walk, &un)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid / 4, wn = wid % 4;
  const int N = p.F, L = p.K, KT = (L + 63) / 64;
  const int lim = L - (KT - 1) * 64;  // of a row, in the last step
  uint8_t* const aring = smem;
  uint8_t* const bring = smem + R::SA * Pan::BYTES;

  // ---- loads: stage `lk` of the tile that is being loaded, in buffers that move
  // with the step.  W's rows, and x's without a gather, are kept inside by the
  // buffer's length, gathered ones by their offset.  A lane's offsets are the same
  // in both panels (row 8 (4 wid + j) + lane / 8 of piece j) without a gather.
  const char *aload, *bload;
  int alen, blen;  // bytes of the buffers: 0 when there is no further tile
  int lk = 0;
  uint32_t off[R::JP], aoff[GATHER ? R::JP : 1];
  auto chunk_of = [&](int j) MOE_INLINE {  // lane % 8, swizzled by the row
    return (lane & 7) ^ Pan::swz(8 * (R::JP * wid + j) + (lane >> 3));
  };
  const uint32_t pitch = static_cast<uint32_t>(L) * 2;
  // Gathered: the offsets of the next tile's rows in x (codes_prepare), kFar where
  // there is none.
  uint32_t far[GATHER ? R::JP : 1];
  auto fetch_sources = [&](const Unit& u) MOE_INLINE {
#pragma unroll
    for (int j = 0; j < R::JP; ++j)
      far[GATHER ? j : 0] = p.sources[u.row0 + 8 * (R::JP * wid + j) + (lane >> 3)];
  };
  auto scalar = [](const void* q) MOE_INLINE {
    const uint64_t v = reinterpret_cast<uint64_t>(q);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return reinterpret_cast<const char*>(static_cast<uint64_t>(hi) << 32 | lo);
  };
  auto load_from = [&](const Unit& u) MOE_INLINE {
    lk = 0;
    bload = scalar(p.b + (static_cast<int64_t>(u.g) * N + u.col0) * L);
    blen = min(R::BN, N - u.col0) * static_cast<int>(pitch);
    aload = scalar(p.a + (GATHER ? 0 : static_cast<int64_t>(u.row0) * L));
    alen = GATHER ? static_cast<int>(kFar) : u.rows * static_cast<int>(pitch);
#pragma unroll
    for (int j = 0; j < R::JP; ++j) {
      const int row = 8 * (R::JP * wid + j) + (lane >> 3);
      off[j] = row * pitch + chunk_of(j) * 16;
      if (GATHER)
        aoff[GATHER ? j : 0] = (row < u.rows ? far[GATHER ? j : 0] : kFar) + chunk_of(j) * 16;
    }
  };
  auto load_nothing = [&]() MOE_INLINE {
    alen = blen = 0;
  };
  int aslot = 0, bslot = 0;  // of the stage that is loaded next
  auto load = [&](const char* base, int bytes, uint32_t at, uint8_t* to) MOE_INLINE {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, bytes, 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 16, at, 0, 0, 0);
  };
  auto issue_a = [&](int j) MOE_INLINE {
    load(aload, alen, GATHER ? aoff[GATHER ? j : 0] : off[j],
         aring + aslot * Pan::BYTES + (wid * R::JP + j) * 1024);
  };
  auto issue_b = [&](int j) MOE_INLINE {
    load(bload, blen, off[j], bring + bslot * Pan::BYTES + (wid * R::JP + j) * 1024);
  };
  // The stage is complete: on to the next one.
  auto advance = [&]() MOE_INLINE {
    ++lk;
    aload += 128;
    bload += 128;
    if (!GATHER) alen = max(alen - 128, 0);
    blen = max(blen - 128, 0);
    aslot = aslot == R::SA - 1 ? 0 : aslot + 1;
    bslot ^= 1;
  };
  // Before a tile's last stage: lanes whose codes lie behind the row's end read
  // nothing.
  auto cut_tail = [&]() MOE_INLINE {
    if (lk == KT - 1 && lim < 64)
#pragma unroll
      for (int j = 0; j < R::JP; ++j)
        if (chunk_of(j) * 8 >= lim) {
          off[j] = kOutside;
          if (GATHER) aoff[GATHER ? j : 0] = kOutside;
        }
  };

  // ---- scales: of the wave's rows, a step ahead, and of its columns, 64 steps a
  // lane each
  const char* sload;
  int slen = 0;  // bytes of the tile's rows
  const uint32_t srow = (32 * wm + (lane & 31)) * 4;
  float rs_next[R::MB], ws_held;
  const float* wscale;
  const int fblocks = (N + 127) / 128;
  const int64_t sstep = p.a_scale_step * 4;
  auto scales_from = [&](const Unit& u) MOE_INLINE {
    sload = scalar(p.a_scale + u.row0);
    slen = u.rows * 4;
    const int fb = min((u.col0 + wn * 64) / 128, fblocks - 1);
    wscale = p.b_scale + (static_cast<int64_t>(u.g) * fblocks + fb) * KT;
  };
  auto fetch_scales = [&]() MOE_INLINE {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(sload), 0, slen, 0x00027000);
#pragma unroll
    for (int mb = 0; mb < R::MB; ++mb)
      rs_next[mb] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(r, srow + 256 * mb, 0, 0));
    sload += sstep;
  };
  auto hold_scales = [&](int kt) MOE_INLINE { ws_held = wscale[min(kt + lane, KT - 1)]; };

  // ---- fragments and products: v_mfma_f32_16x16x128_f8f6f4, a step at once, W's
  // rows first, so that a lane's four sums belong to one row of x and four columns.
  // Lane l holds row l % 16 and two chunks of 16 codes, l / 16 and l / 16 + 4 (of
  // both operands, which is all that a sum over them asks; with 2 (l / 16) and the
  // next, the 64 lanes' reads conflict and a step takes 5% more cycles).
  f32x4 acc[R::IB][R::NB], t[4];
  u32x4 bq[R::NB][2], aq[2][2];
  int ause = 0, buse = 0;  // slots of the stage whose fragments are read next
  const int frag = (lane & 15) * 128 + ((lane >> 4) ^ ((lane & 15) >> 1)) * 16;
  const int abase = frag + 32 * 128 * wm, bbase = frag + 64 * 128 * wn;
  auto load_b = [&](int nb) MOE_INLINE {
    const uint8_t* sb = bring + buse * Pan::BYTES + 16 * 128 * nb;
    bq[nb][0] = *reinterpret_cast<const u32x4*>(sb + bbase);
    bq[nb][1] = *reinterpret_cast<const u32x4*>(sb + (bbase ^ 64));
  };
  auto load_a = [&](int i) MOE_INLINE {
    const uint8_t* sa = aring + ause * Pan::BYTES + 64 * 128 * (i / 2) + 16 * 128 * (i % 2);
    aq[i & 1][0] = *reinterpret_cast<const u32x4*>(sa + abase);
    aq[i & 1][1] = *reinterpret_cast<const u32x4*>(sa + (abase ^ 64));
  };
  auto multiply = [&](int i, int nb) MOE_INLINE {
    const i32x8 b = __builtin_bit_cast(i32x8, U32x8{bq[nb][0], bq[nb][1]});
    const i32x8 a = __builtin_bit_cast(i32x8, U32x8{aq[i & 1][0], aq[i & 1][1]});
    t[nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, f32x4{}, 0, 0, 0, 0, 0, 0);
  };
  auto meet = [&]() MOE_INLINE {
    wait_loads<R::J>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  auto meet_b = [&]() MOE_INLINE { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
  bool more;  // there is a next tile
  // What is loaded from step kt on: the next tile's stages from the last step but
  // one, its first scales in the last step.
  auto turn = [&](int kt) MOE_INLINE {
    if (kt == KT - R::AHEAD) {
      if (more)
        load_from(nx);
      else
        load_nothing();
    }
    cut_tail();
  };

  if (GATHER) fetch_sources(un);
  scales_from(un);
  hold_scales(0);
  fetch_scales();
  load_from(un);
#pragma unroll
  for (int s = 0; s < R::AHEAD; ++s) {
    cut_tail();
#pragma unroll
    for (int j = 0; j < R::JP; ++j) issue_a(j);
#pragma unroll
    for (int j = 0; j < R::JP; ++j) issue_b(j);
    advance();
  }
  wait_loads<R::J>();
  asm volatile("s_barrier" ::: "memory");

  // The steps of a tile of whose 32-row blocks the wave has B.
  auto steps = [&](auto BLOCKS) MOE_INLINE {
    constexpr int B = decltype(BLOCKS)::value;
    if constexpr (B == 0) {
      for (int kt = 0; kt < KT; ++kt) {
        if (kt == KT - 1 && more) {
          scales_from(nx);
          hold_scales(0);
          fetch_scales();
        }
        turn(kt);
#pragma unroll
        for (int j = 0; j < R::JP; ++j) issue_a(j);
        meet_b();
#pragma unroll
        for (int j = 0; j < R::JP; ++j) issue_b(j);
        advance();
        ause = ause == R::SA - 1 ? 0 : ause + 1;
        buse ^= 1;
        meet();
      }
      return;
    } else {
      // A product's four sums are added, times the scale of their row and columns,
      // three products later: one product and four additions in turn keep both
      // pipes busy.  The last three of a step are added in the next (`last`: the
      // scale; at first 0, times sums of 0).
      constexpr int I = 2 * B;
      float rs[I], last = 0.0f;
#pragma unroll
      for (int i = 0; i < R::IB; ++i)
#pragma unroll
        for (int nb = 0; nb < R::NB; ++nb) acc[i][nb] = f32x4{};
#pragma unroll
      for (int nb = 0; nb < R::NB; ++nb) {
        t[nb] = f32x4{};
        load_b(nb);
      }
      load_a(0);
      auto add = [&](int m) MOE_INLINE {  // the step's product m, or the last step's
        const int i = m < 0 ? I - 1 : m / R::NB, nb = (m + R::NB) % R::NB;
        const float w = m < 0 ? last : rs[i];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][nb][q] = fmaf(w, t[nb][q], acc[i][nb][q]);
      };
#pragma clang loop unroll(disable)
      for (int kt = 0; kt < KT; ++kt) {
        const float w = __builtin_bit_cast(
            float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ws_held), kt & 63));
#pragma unroll
        for (int mb = 0; mb < B; ++mb) {
          split_rows(rs_next[mb] * w, &rs[2 * mb], &rs[2 * mb + 1]);
        }
        const bool end = kt == KT - 1;
        if (end ? more : ((kt + 1) & 63) == 0) {
          if (end) scales_from(nx);
          hold_scales(end ? 0 : kt + 1);
        }
        if (end && !more) slen = 0;
        fetch_scales();
        turn(kt);
#pragma unroll
        for (int i = 0; i < I; ++i) {
          // the products so far have taken all of W's panel
          if (i == 1) {
            meet_b();
            if (I == 2) {
#pragma unroll
              for (int j = 0; j < R::JP; ++j) issue_b(j);
              advance();
            }
          }
          if (i == I - 1) {
            ause = ause == R::SA - 1 ? 0 : ause + 1;
            buse ^= 1;
            meet();
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int nb = 0; nb < R::NB; ++nb) {
            multiply(i, nb);
            add(4 * i + nb - 3);
            if (nb == 0) load_a(i + 1 < I ? i + 1 : 0);
            if (i == I - 1) load_b(nb);
            // the refill: x's pieces among the first rows' products, W's among the
            // following ones
            constexpr int ROWS = I > 2 ? I - 2 : 1;
            constexpr int PER = (R::JP + ROWS - 1) / ROWS;
            if (i == 0) issue_a(nb);
            if (I > 2 && i > 0 && nb < PER && (i - 1) * PER + nb < R::JP) {
              issue_b((i - 1) * PER + nb);
              if ((i - 1) * PER + nb == R::JP - 1) advance();
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        last = rs[I - 1];
      }
#pragma unroll
      for (int m = -3; m < 0; ++m) add(m);
    }
  };

  // The tile leaves: 16 rows of the wave's 64 columns at a time through the wave's
  // own part of the slot behind the last stage's.
  auto leaves = [&](auto BLOCKS) MOE_INLINE {
    constexpr int B = decltype(BLOCKS)::value;
    // (hidden from the compiler, which would compute all addresses before the first
    // tile and keep them in memory)
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    float* const stage = reinterpret_cast<float*>(aring + aslot * Pan::BYTES + wid * 4096);
    const int c = lane & 7;  // eight columns of the wave's
    const int col = un.col0 + wn * 64 + c * 8;
    const bool live = col < N;
    F8 bias{};
    if (p.bias && live) bias = load8(p.bias + static_cast<int64_t>(un.g) * N + col);
#pragma unroll
    for (int i = 0; i < 2 * B; ++i) {
      const int wr = lane & 15;
#pragma unroll
      for (int nb = 0; nb < R::NB; ++nb)
        *reinterpret_cast<f32x4*>(stage + (wr * 16 + ((4 * nb + (lane >> 4)) ^ wr)) * 4) =
            acc[i][nb];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int sr = lane / 8 + 8 * h;
        const int row = 32 * (2 * (i / 2) + wm) + 16 * (i % 2) + sr;
        const f32x4 lo = *reinterpret_cast<const f32x4*>(stage + (sr * 16 + ((2 * c) ^ sr)) * 4);
        const f32x4 hi = *reinterpret_cast<const f32x4*>(stage + (sr * 16 + ((2 * c + 1) ^ sr)) * 4);
        if (row < un.rows && live) {
          const int64_t at = static_cast<int64_t>(un.row0 + row) * N + col;
          const F8 res = p.residual ? load8(p.residual + at) : F8{};
          const F8 v{{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}};
          if (!ACT)
            finish8<MOE_ACT_NONE>(p, v, bias, res, at);
          else
            switch (p.act) {
              case MOE_ACT_RELU: finish8<MOE_ACT_RELU>(p, v, bias, res, at); break;
              case MOE_ACT_GELU: finish8<MOE_ACT_GELU>(p, v, bias, res, at); break;
              case MOE_ACT_GELU_TANH: finish8<MOE_ACT_GELU_TANH>(p, v, bias, res, at); break;
              default: finish8<MOE_ACT_SILU>(p, v, bias, res, at); break;
            }
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // before the loads that follow here
  };

  do {
    more = next_tile(p, &walk, &nx);
    if (GATHER && more) fetch_sources(nx);
    const int blocks = (un.rows + 31) / 32;
    const int mine = wn * 64 < N - un.col0 ? (blocks - wm + 1) / 2 : 0;
    switch (mine) {
      case 4: steps(std::integral_constant<int, 4>{}); leaves(std::integral_constant<int, 4>{}); break;
      case 3: steps(std::integral_constant<int, 3>{}); leaves(std::integral_constant<int, 3>{}); break;
      case 2: steps(std::integral_constant<int, 2>{}); leaves(std::integral_constant<int, 2>{}); break;
      case 1: steps(std::integral_constant<int, 1>{}); leaves(std::integral_constant<int, 1>{}); break;
      default: steps(std::integral_constant<int, 0>{}); break;
    }
    un = nx;
  } while (more);
  wait_loads<0>();  // nothing comes into LDS behind the block's end
}

}  // namespace

}  // namespace moe

// The experts' products on 256 x 256 tiles, 16-bit types with whole 16-byte chunks everywhere.
//
// Eight waves a workgroup, one workgroup a CU, two waves a SIMD. Waves 0-3 compute the tile's
// rows 0-127, waves 4-7 rows 128-255, 128 x 64 each (4 x 2 blocks of the 32x32x16 MFMA). The
// contraction moves through LDS 64 values (128 bytes) at a time, DMA'd into a ring of two 64 KB
// stages. Every stage is two steps of 16 MFMAs, and a step is two phases: a wave reads all the
// step's fragments into registers (and, under the latency of the reads, issues its share of the
// DMA), then computes from registers alone. The two waves of a SIMD run half a step apart, so one
// always reads while the other computes; a barrier ends every phase.
//
// Because a step's reads come in one burst, its part of the stage is free for the stage after
// next as soon as both halves have read it: the DMA runs one and a quarter to one and a half
// stages ahead of its use in a ring of two. The steps split a stage so that each has its own 1 KB
// pieces: by rows of A where A is contraction-contiguous (step 1: all of B and rows 0-63 of either
// half; step 2: the other rows), by the contraction where both operands are contraction-major.
//
// The tiles of a workgroup form one stream of stages: the DMA goes on into the next tile while
// this one's last stages and its stores run. Results leave the registers as 16-byte stores: the
// MFMAs run with the operands swapped, so a lane holds runs of four columns of one row, one swap of
// lane halves makes them eight, and one of rows of 16 lanes puts 64 bytes of a row into four lanes
// (weight gradient of 64 x 1408 x 2048, 384 rows each: 191 us with 32 bytes a row, 182 so).
//
// An XCD takes a part of the tile list. A weight gradient's tiles cost as many stages as their expert has rows, so
// its parts have equal cost (cost_list): 27 x 2048 x 7168 of a router's 32768 rows 1044 us with equal numbers of tiles,
// 867 so. SPLIT: the last round of a dense product (last_round), 509 rows of 18432 x 7168 forward 336 to 265 us,
// input gradient 551 to 298. The gated block's activation is chosen once a tile: chosen value by value, its code came three
// times for each and the instructions were fetched again and again (384 rows each over 64 x 1408 x 2048, silu, 383 us, 326 so).
//
// Bound by the board's power and LDS. 4 x 2048 rows against 2048 x 7168, bf16, held for a second:
// 177 us (1357 TFLOP/s) at 1.59 GHz and 1330 W, 2500 cycles a stage of 2048 MFMA cycles; on zeros
// 129 us (1867 TFLOP/s) at 2.35 GHz. Without the DMA's waits 5 % less, without the LDS reads 30 %
// less. What was slower on the same products (27 to 32 experts, 32768 rows): sixteen waves of 64 x
// 64 at four a SIMD, a stage behind (840 against 745 us); eight or four waves that read the next
// group under the current one's MFMAs with one barrier a stage (830, 920); the DMA issued before
// the phase's reads (775).
#pragma once

#include "expert_gemm.hpp"

namespace mns {

struct TilePP {
  static constexpr int BM = 256, BN = 256, NT = 512, OCC = 2;
  static constexpr int OPB = 256 * 128;   // bytes of an operand's stage
  static constexpr int LDS = 4 * OPB;
};

// A value the compiler cannot see through: what is computed from it is computed where it stands
// and not kept in registers across the loops.
__device__ inline int opaque(int v) {
  __asm__ __volatile__("" : "+v"(v));
  return v;
}

// A pointer that is equal in every lane, in scalar registers: a buffer resource made from values
// that the compiler keeps in vector registers costs a loop at every use.
__device__ inline const char* uniform(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = (uint32_t)wave_uniform((int)(uint32_t)v), hi = (uint32_t)wave_uniform((int)(uint32_t)(v >> 32));
  return reinterpret_cast<const char*>((uint64_t)hi << 32 | lo);
}

template <typename T> using FragOf = typename Frag<T>::type;

template <typename T>
__device__ inline f32x16 mma32(const FragOf<T>& a, const FragOf<T>& b, const f32x16& c) {
  if constexpr (__is_same(T, __bf16)) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// dma16 from inline assembly: the compiler does not see that it writes LDS and does not wait for
// the queue before reads of other pieces. The kernel's own waits and barriers order it. Nor does the
// compiler count the wait states between a vector instruction's write of a scalar (readfirstlane)
// and this load's read of it: rs comes through settled(). Nothing else in the kernel uses m0.
__device__ inline void dma16_unseen(u32x4 rs, uint32_t lds_at, uint32_t voff) {
  __asm__ __volatile__("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds_at), "v"(voff), "s"(rs) : "memory");
}

// Five wait states, after which a load may read these scalars, whoever wrote them. Once a stage (in
// every dma16_unseen, input gradient of 64 x 1408 x 2048, 384 rows each, fp16: 172 to 178 us).
__device__ inline void settled(const char*& a, const char*& b, uint32_t& c, uint32_t& d) {
  __asm__ __volatile__("s_nop 4" : "+s"(a), "+s"(b), "+s"(c), "+s"(d));
}

// A fragment of 32 columns from a contraction-major stage (rows of 512 bytes): two transposing
// reads (see kmajor_frag_off for their lanes); `at`: the lane's place for the group.
template <typename T>
__device__ inline FragOf<T> read_major(const char* at) {
  typedef __attribute__((address_space(3))) s16x4* lds4;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(char*)at);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(char*)(at + 4 * 512));
  return __builtin_bit_cast(FragOf<T>, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// A block's 32 columns of 32 rows to the result at (r0, c0) of the tile. A lane holds runs of four columns of one row;
// a swap of lane halves makes them eight, and a swap of rows of 16 lanes then puts the 32 columns of one row
// into four lanes, so that a store writes 64 bytes of each of 16 rows. value(e): column run e / 4 (8 apart, and 4
// for the upper half), e % 4 of it.
template <typename T, class V>
__device__ inline void store_block(int ln, const __amdgpu_buffer_rsrc_t& rs, int r0, int c0, int ld, const ExpertTile& x, int n, V&& value) {
  uint32_t w[2][4];                  // [half of the columns][16 bytes]
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const auto s = __builtin_amdgcn_permlane32_swap(pack2<T>(value(q * 8 + 2 * e), value(q * 8 + 2 * e + 1)),
                                                      pack2<T>(value(q * 8 + 4 + 2 * e), value(q * 8 + 4 + 2 * e + 1)), false, false);
      w[q][e] = s[0];
      w[q][2 + e] = s[1];
    }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const auto s = __builtin_amdgcn_permlane16_swap(w[0][e], w[1][e], false, false);
    w[0][e] = s[0];
    w[1][e] = s[1];
  }
  const int c = c0 + ((ln >> 4) & 1) * 16 + (ln >> 5) * 8;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = r0 + k * 16 + (ln & 15);
    const uint32_t off = x.row0 + r < x.m && x.col0 + c < n ? (uint32_t)(r * ld + c) * 2 : OOB;
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[k][0], w[k][1], w[k][2], w[k][3]}, rs, off, 0, 0);
  }
}

// The last round of an XCD's list where it leaves at least half of the workgroups idle (SPLIT): each of its
// `over` tiles is cut along the contraction into `parts` that as many workgroups take, and expert_split_sum adds
// them up. full: tiles of the rounds before.
struct LastRound {
  int full, over, parts;
};
__host__ __device__ inline LastRound last_round(int tiles, int wgs) {
  const int over = tiles % wgs, parts = over ? wgs / over : 1;
  return parts < 2 ? LastRound{tiles, 0, 1} : LastRound{tiles - over, over, parts};
}

template <int MODE, typename T, bool SPLIT = false>
__global__ void __launch_bounds__(TilePP::NT, TilePP::OCC) expert_gemm_pp(const typename ArgsOf<MODE>::type p) {
  constexpr int BK = 64, OPB = TilePP::OPB, NT = TilePP::NT;
  constexpr bool AKM = ex_dw(MODE), BKM = !ex_fwd(MODE);
  // A's two stages, then B's
  __shared__ __align__(1024) char lds[4 * OPB];
  __shared__ int first[EXPERT_MAX + 2];
  __shared__ int2 rows[EXPERT_MAX + 1];
  __shared__ int wsum[NT / 64];
  typedef FragOf<T> F;
  const int wave = wave_uniform(threadIdx.x >> 6), wm = wave >> 2, wn = wave & 3;
  const int lane = threadIdx.x & 63;
  expert_tiles<NT, TilePP::BM, true, ex_dw(MODE)>(p, first, wsum, rows);
  ExpertList l;
  if constexpr (ex_dw(MODE)) l = cost_list(p, first, (int64_t)((p.m + 255) / 256) * p.tiles_n * (MODE == EX_DW2 ? 2 : 1));
  else l = expert_list<MODE, TilePP>(p, first);
  const int step = gridDim.x >> 3;
  int t = blockIdx.x >> 3;
  const int own = t;
  LastRound last{l.n, 0, 1};
  if constexpr (SPLIT) {
    last = last_round(l.n, step);
    if (own >= last.over * last.parts && own >= last.full) return;
  } else if (t >= l.n) {
    return;
  }
  // the workgroup's tile in the round that begins with tile at - own: its place in the list, or -1
  auto tile_of = [&](int at) {
    if (!SPLIT || at < last.full) return at < l.n ? at : -1;
    return at == last.full + own && own < last.over * last.parts ? last.full + own / last.parts : -1;
  };
  // the stages of it that the workgroup takes
  auto stages_of = [&](int at, int nk, int* begin, int* end) {
    const bool cut = SPLIT && at >= last.full;
    *begin = cut ? nk * (own % last.parts) / last.parts : 0;
    *end = cut ? nk * (own % last.parts + 1) / last.parts : nk;
  };

  // ------------------------------------------------------------------ the stages on their way
  // A piece is 1 KB of an operand's stage: rows 8 i .. 8 i + 7 of a contiguous operand, contraction
  // rows 2 i, 2 i + 1 of a major one. A wave brings eight of each stage, four in each step where A
  // is major, six and two where it is contiguous. What lies outside the operand falls to the
  // buffer's range check and becomes zero; a stage of no tile is all outside.
  auto a_piece = [&](int j) {        // A's pieces of this wave: j = 0, 1 in step 1, 2, 3 in step 2
    if constexpr (AKM) return (j >> 1) * 16 + wave * 2 + (j & 1);
    else return (j >> 1) * 8 + wave * 2 + (j & 1) + (wave >= 4 ? 8 : 0);   // rows 0-63 and 128-191, then the others
  };
  auto b_piece = [&](int j) {
    if constexpr (AKM) return (j >> 1) * 16 + wave * 2 + (j & 1);
    else return wave * 4 + j;
  };
  uint32_t offa[4], offb[4];         // lane's byte offset in each piece
  const char* srca = p.A; const char* srcb = p.B;   // where the stage begins
  uint32_t lena = 0, lenb = 0;       // bytes from there to the operand's end
  int exta = 0, extb = 0;            // rows or columns of the tile that exist
  const int rba = (int)p.lda * 2;    // bytes per row of memory
  int rbb = (int)p.ldb * 2;
  if constexpr (MODE == EX_GATE)     // a wave brings rows of one of the two matrices
    if (wave & 1) rbb = (int)p.ldb2 * 2;
  const char* later_a = nullptr; const char* later_b = nullptr;   // EX_DX2: the contraction that follows
  bool follows = false;
  int ti = t - step;                 // tile being issued
  int klen = 0, k0 = 0;              // its contraction length, the stage being issued
  int efrom = 0, islot = 1;
  bool live = true;
  int left = 0;                      // SPLIT: stages of the tile that are not issued yet
  const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) char*)lds;
  auto offset = [&](int l0, bool km, int rb, int ext, int i) {
    if (km) {
      const int k = i * 2 + (l0 >> 5), c = ((l0 & 31) ^ kmajor_swizzle(k & 3)) * 8;
      return c < ext ? (uint32_t)(k * rb + c * 2) : OOB;
    }
    const int r = i * 8 + (l0 >> 3);
    return (uint32_t)(r * rb + ((l0 & 7) ^ chunk_swizzle<8>(r)) * 16);
  };
  // EX_GATE: rows 64 b .. 64 b + 31 of the stage are rows 32 b .. of W, the next 32 those of W2
  auto offset_b = [&](int l0, int ext, int j) {
    if constexpr (MODE == EX_GATE) {
      const int r = b_piece(j) * 8 + (l0 >> 3), row = (wave >> 1) * 32 + j * 8 + (l0 >> 3);
      return (uint32_t)(row * rbb + ((l0 & 7) ^ chunk_swizzle<8>(r)) * 16);
    } else {
      return offset(l0, BKM, rbb, ext, b_piece(j));
    }
  };
  // the next stage of the stream: of this tile, of the next tile that has any, or none
  auto advance = [&]() {
    islot ^= 1;
    k0 += BK;
    srca += AKM ? (int64_t)BK * rba : BK * 2;
    srcb += BKM ? (int64_t)BK * rbb : BK * 2;
    auto follow = [&]() {              // EX_DX2: to the second contraction
      follows = false;
      k0 = 0;
      srca = later_a;
      srcb = later_b;
      if constexpr (MODE == EX_DX2) rbb = (int)p.ldb2 * 2;
      const int l0 = opaque(lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) offb[j] = offset_b(l0, extb, j);
    };
    bool done = k0 >= klen;
    if constexpr (SPLIT) done = --left <= 0;
    if (MODE == EX_DX2 && k0 >= klen && follows && !(SPLIT && done)) {
      follow();
    } else if (done) {
      k0 = klen = 0;
      while (live && klen == 0) {
        ti += step;
        const int place = tile_of(ti);
        live = place >= 0;
        if (!live) break;
        const ExpertTile x = expert_tile<MODE, T, TilePP, true>(p, first, l, place, &efrom, rows);
        klen = x.k;
        if (klen > 0) {
          srca = x.a + (AKM ? (int64_t)x.row0 * 2 : (int64_t)x.row0 * rba);
          if constexpr (MODE == EX_GATE) {
            srcb = (wave & 1 ? x.b2 : x.b) + (int64_t)x.col0 * rbb;
          } else {
            if constexpr (MODE == EX_DX2) {
              rbb = (int)p.ldb * 2;
              later_a = x.a2 + (int64_t)x.row0 * rba;
              later_b = x.b2 + (int64_t)x.col0 * 2;
              follows = true;
            }
            srcb = x.b + (BKM ? (int64_t)x.col0 * 2 : (int64_t)x.col0 * rbb);
          }
          exta = min(x.m - x.row0, 256);
          if constexpr (MODE == EX_DW2) exta = (exta + 7) & ~7;   // whole chunks, zeros behind the end
          extb = min(p.n - x.col0, tile_cols<MODE, TilePP>());
          const int l0 = opaque(lane);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            offa[j] = offset(l0, AKM, rba, exta, a_piece(j));
            offb[j] = offset_b(l0, extb, j);
          }
          if constexpr (SPLIT) {
            const int nh = (klen + BK - 1) / BK;
            int begin, end;
            stages_of(ti, MODE == EX_DX2 ? 2 * nh : nh, &begin, &end);
            left = end - begin;
            if (MODE == EX_DX2 && begin >= nh) {
              follow();
              begin -= nh;
            }
            k0 = begin * BK;
            srca += AKM ? (int64_t)k0 * rba : (int64_t)k0 * 2;
            srcb += BKM ? (int64_t)k0 * rbb : (int64_t)k0 * 2;
          }
        }
      }
    }
    const int rest = klen - k0;
    srca = uniform(srca);
    srcb = uniform(srcb);
    const int resta = MODE == EX_DX2 ? (rest + 7) & ~7 : rest;   // whole chunks as well
    lena = !live ? 0 : AKM ? (min(rest, BK) - 1) * rba + exta * 2 : (exta - 1) * rba + resta * 2;
    lenb = !live ? 0 : BKM ? (min(rest, BK) - 1) * rbb + extb * 2 : (extb - 1) * rbb + rest * 2;
    lena = wave_uniform(lena);
    lenb = wave_uniform(lenb);
    settled(srca, srcb, lena, lenb);
  };
  const int kin0 = ((lane & 7) ^ chunk_swizzle<8>(lane >> 3)) * 8, kin1 = ((lane & 7) ^ chunk_swizzle<8>(8 + (lane >> 3))) * 8;
  auto bring = [&](bool isa, int j) {
    const bool km = isa ? AKM : BKM;
    const int i = isa ? a_piece(j) : b_piece(j);
    uint32_t off = isa ? offa[j] : offb[j];
    // a chunk behind the end of its row would be the next row's
    if (!km) off = (i & 1 ? kin1 : kin0) < klen - k0 ? off : OOB;
    const uint64_t v = reinterpret_cast<uint64_t>(isa ? srca : srcb);
    const u32x4 rs = {(uint32_t)v, (uint32_t)(v >> 32) & 0xffffu, isa ? lena : lenb, 0x00020000u};
    dma16_unseen(rs, lds0 + (isa ? 0 : 2 * OPB) + islot * OPB + i * 1024, off);
  };
  // the pieces of step `st` of the stage
  auto issue = [&](auto st_c) {
    constexpr int st = decltype(st_c)::value;
#pragma unroll
    for (int j = 0; j < 2; ++j) bring(true, st * 2 + j);
    if constexpr (AKM) {
#pragma unroll
      for (int j = 0; j < 2; ++j) bring(false, st * 2 + j);
    } else if constexpr (st == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) bring(false, j);
    }
  };

  // ------------------------------------------------------------------------------ the tiles
  f32x16 acc[4][2];
  F fa[2][4], fb[2][4];              // [block][group]; AKM: block i, group g of A at [i >> 1][(i & 1) * 2 + g]
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  };
  // the lane's places in the stage's slot: of the groups (contiguous) or blocks (major)
  int ata[4], atb[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int ck = ((2 * g + (lane >> 5)) ^ chunk_swizzle<8>(lane & 31)) << 4;
    ata[g] = AKM ? kmajor_frag_off<512>(lane, wm * 128 + g * 32) : (wm * 128 + (lane & 31)) * 128 + ck;
    atb[g] = 2 * OPB + (BKM ? kmajor_frag_off<512>(lane, wn * 64 + (g & 1) * 32) : (wn * 64 + (lane & 31)) * 128 + ck);
  }
  auto rowfrag = [&](int at) { return *reinterpret_cast<const F*>(lds + at); };
  auto read = [&](auto st_c) {
    constexpr int st = decltype(st_c)::value;
    if constexpr (AKM) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int j = 0; j < 2; ++j) fb[j][g] = read_major<T>(lds + atb[j] + st * 16384 + g * 8192);
#pragma unroll
        for (int i = 0; i < 4; ++i) fa[i >> 1][(i & 1) * 2 + g] = read_major<T>(lds + ata[i] + st * 16384 + g * 8192);
      }
    } else {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if constexpr (st == 0) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if constexpr (BKM) fb[j][g] = read_major<T>(lds + atb[j] + g * 8192);
            else fb[j][g] = rowfrag(atb[g] + j * 4096);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) fa[i][g] = rowfrag(ata[g] + st * 8192 + i * 4096);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto compute = [&](auto st_c) {
    constexpr int st = decltype(st_c)::value;
    __builtin_amdgcn_s_setprio(1);
    if constexpr (AKM) {
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = mma32<T>(fb[j][g], fa[i >> 1][(i & 1) * 2 + g], acc[i][j]);
    } else {
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[st * 2 + i][j] = mma32<T>(fb[j][g], fa[i][g], acc[st * 2 + i][j]);
    }
    __builtin_amdgcn_s_setprio(0);
  };
  // at most eight pieces still on their way, and the stores of the tile before if `stored`
  auto landed = [&](bool stored) {
    if constexpr (MODE == EX_GATE) {
      if (p.C2) wait_vmcnt<8 + 24>();
      else wait_vmcnt<8 + 8>();
    } else {
      wait_vmcnt<8 + 16>();
    }
    if (!stored) wait_vmcnt<8>();
  };
  auto phase_end = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    barrier_nofence();
    __builtin_amdgcn_sched_barrier(0);
  };
  // Stores: 16 a wave whatever the tile (rows and columns outside fall to the range check); EX_GATE: 8, or 24
  // with both products.
  auto put_block = [&](int ln, const __amdgpu_buffer_rsrc_t& rs, int r0, int c0, int ld, const ExpertTile& x, auto&& value) {
    store_block<T>(ln, rs, r0, c0, ld, x, p.n, value);
  };
  auto result = [&](const char* to, int64_t ld, const ExpertTile& x) {
    return make_rsrc(uniform(to + ((int64_t)x.row0 * ld + x.col0) * 2), 0x7ffffff0u);
  };
  auto store = [&](const ExpertTile& x) {
    const int ln = opaque(lane);
    if constexpr (MODE == EX_GATE) {
      auto each = [&](const char* to, int64_t ld, auto&& value) {
        const __amdgpu_buffer_rsrc_t rs = result(to, ld, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) put_block(ln, rs, wm * 128 + i * 32, wn * 32, (int)ld, x, [&](int e) { return value(i, e); });
      };
      if (x.c2) {
        each(x.c2, p.ldc2, [&](int i, int e) { return acc[i][0][e]; });
        each(x.c3, p.ldc3, [&](int i, int e) { return acc[i][1][e]; });
      }
      with_activation(p.act, [&](auto act) {
        each(x.c, p.ldc, [&](int i, int e) { return activated<T, act.value>(acc[i][0][e]) * acc[i][1][e]; });
      });
    } else {
      const int64_t ldc = row_step<MODE>(p, x);
      const __amdgpu_buffer_rsrc_t rs = result(x.c, ldc, x);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          put_block(ln, rs, wm * 128 + i * 32, wn * 64 + j * 32, (int)ldc, x, [&](int e) { return acc[i][j][e]; });
    }
  };
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;

  // stage 0 whole and the first step of stage 1 on their way; the first step of stage 0 has landed
  advance();
  issue(S0{});
  issue(S1{});
  advance();
  issue(S0{});
  wait_vmcnt<8>();
  barrier_nofence();
  if (wm) barrier_nofence();         // waves 4-7 run half a step behind

  int cfrom = 0;
  int toggle = OPB;
  bool begin = true;                 // no stores yet
  clear();
  for (;; t += step) {
    const int place = tile_of(t);
    if (place < 0) break;
    const ExpertTile x = expert_tile<MODE, T, TilePP, true>(p, first, l, place, &cfrom, rows);
    int nk = (x.k + BK - 1) / BK * (MODE == EX_DX2 ? 2 : 1);
    if constexpr (SPLIT) {
      int begin, end;
      stages_of(t, nk, &begin, &end);
      nk = end - begin;
    }
    // blocks whose rows all lie outside are not computed (the barriers stay)
    const bool busy0 = x.row0 + wm * 128 < x.m, busy1 = x.row0 + wm * 128 + (AKM ? 0 : 64) < x.m;
    for (int kt = 0; kt < nk; ++kt) {
      // In the queue at the end of either reading phase: eight pieces, and before the oldest of
      // them, in a tile's first stage, the stores of the tile before it.
      const bool stored = kt == 0 && !begin;
      if (busy0) read(S0{});
      issue(S1{});                   // step 2 of the next stage
      wait_lgkmcnt0();
      landed(stored);   // step 2 of this stage has landed
      phase_end();
      if (busy0) compute(S0{});
      phase_end();
      if (busy1) read(S1{});
      advance();
      issue(S0{});                   // step 1 of the stage after next
      wait_lgkmcnt0();
      landed(stored);   // step 1 of the next stage has landed
      phase_end();
      if (busy1) compute(S1{});
      phase_end();
#pragma unroll
      for (int g = 0; g < 4; ++g) {  // the other slot
        ata[g] += toggle;
        atb[g] += toggle;
      }
      toggle = -toggle;
    }
    if constexpr (SPLIT) {
      if (t >= last.full) {            // the last: its sums as they lie in the registers
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(uniform(reinterpret_cast<const char*>(p.parts) + (int64_t)blockIdx.x * (256 * 256 * 4)), 256 * 256 * 4);
        const uint32_t at = opaque((wave * 64 + lane) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, at, ((i * 2 + j) * 4 + q) * NT * 16, 0);
            }
        break;
      }
    }
    store(x);
    __builtin_amdgcn_sched_barrier(0);
    clear();
    begin = false;
  }
  if (!wm) barrier_nofence();
  wait_vmcnt<0>();                   // the last pieces land before the LDS is given back
}

// The parts of a cut tile added up in order, and the tile's epilogue: a wave takes 32 rows of one wave's share of
// a tile.
template <int MODE, typename T>
__global__ void __launch_bounds__(64) expert_split_sum(const typename ArgsOf<MODE>::type p) {
  __shared__ int first[EXPERT_MAX + 2];
  __shared__ int2 rows[EXPERT_MAX + 1];
  __shared__ int wsum[1];
  expert_tiles<64, TilePP::BM, true>(p, first, wsum, rows);
  const ExpertList l = expert_list<MODE, TilePP>(p, first);
  const LastRound last = last_round(l.n, p.wgs);
  const int i = (blockIdx.x >> 3) & 3, wave = (blockIdx.x >> 5) & 7, q = blockIdx.x >> 8, lane = threadIdx.x;
  if (q >= last.over) return;
  int from = 0;
  const ExpertTile x = expert_tile<MODE, T, TilePP, true>(p, first, l, last.full + q, &from, rows);
  f32x4 acc[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[j][r] = f32x4{0.f, 0.f, 0.f, 0.f};
  const f32x4* parts = reinterpret_cast<const f32x4*>(p.parts) + wave * 64 + lane;
  for (int s = 0; s < last.parts; ++s) {
    const f32x4* part = parts + (int64_t)((q * last.parts + s) * 8 + (blockIdx.x & 7)) * (256 * 64);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[j][r] += part[((i * 2 + j) * 4 + r) * TilePP::NT];
  }
  const int r0 = (wave >> 2) * 128 + i * 32, wn = wave & 3;
  auto result = [&](const char* to, int64_t ld) { return make_rsrc(uniform(to + ((int64_t)x.row0 * ld + x.col0) * 2), 0x7ffffff0u); };
  if constexpr (MODE == EX_GATE) {
    if (x.c2) {
      store_block<T>(lane, result(x.c2, p.ldc2), r0, wn * 32, (int)p.ldc2, x, p.n, [&](int e) { return acc[0][e >> 2][e & 3]; });
      store_block<T>(lane, result(x.c3, p.ldc3), r0, wn * 32, (int)p.ldc3, x, p.n, [&](int e) { return acc[1][e >> 2][e & 3]; });
    }
    with_activation(p.act, [&](auto act) {
      store_block<T>(lane, result(x.c, p.ldc), r0, wn * 32, (int)p.ldc, x, p.n,
                     [&](int e) { return activated<T, act.value>(acc[0][e >> 2][e & 3]) * acc[1][e >> 2][e & 3]; });
    });
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      store_block<T>(lane, result(x.c, p.ldc), r0, wn * 64 + j * 32, (int)p.ldc, x, p.n, [&](int e) { return acc[j][e >> 2][e & 3]; });
  }
}

}  // namespace mns

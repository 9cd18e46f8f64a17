// Matrix products on MXFP4 / FP8 operands for many rows: LDS-tiled, operands fetched
// by direct loads into LDS several stages ahead of the matrix instructions.
#include "mxq_mm.h"

namespace mxq {

namespace {

// A workgroup of 2 x WN waves owns 64 MI x 32 NI WN results, a wave 32 MI x 32 NI. The
// contraction runs in steps of 64 elements, two to a unit of 128. Each operand has a ring
// of four slots in LDS, 64 bytes of a row in each: a unit of an MXFP4 row or a step of
// an FP8 row. Direct loads fill the slots three ahead, evenly over the steps: a burst
// would stall the waves at the memory pipe's door. Fragments of the next step are read
// from LDS while the matrix cores work on the current one; one barrier a slot (every unit,
// with FP8 every step) is all that the waves wait for.
template <bool A8, bool B8, int MI, int NI, int WN>
struct Tile {
  static constexpr int Waves = 2 * WN, Threads = 64 * Waves;
  static constexpr int BM = 64 * MI, BN = 32 * NI * WN;
  static constexpr int Ring = 4, ASlot = BM * 64, BSlot = BN * 64;
  static constexpr int BRing = Ring * ASlot, SRing = BRing + Ring * BSlot;  // offsets in LDS
  static constexpr int DA = ASlot / 1024 / Waves, DB = BSlot / 1024 / Waves;  // 1 KiB loads of a wave for a slot
  // loads of a step, and those younger than the slot a barrier waits for
  static constexpr int Issued = (A8 ? DA : DA / 2) + (B8 ? DB : DB / 2);
  static constexpr int Younger = A8 ? Issued : 3 * Issued;
  // scales: 16 bytes of a row cover a chunk of four units; two such chunks
  static constexpr int SRows = BM + BN, SChunk = SRows * 16;
  static constexpr int SLoads = SRows / 16 / Waves;  // 256-byte loads of a wave in a chunk (16 rows each)
  static constexpr int Lds = SRing + 2 * SChunk;
  static constexpr int PadN = 32 * NI + 4;  // floats of a row parked for the epilogue
  static_assert(DA % 2 == 0 && DB % 2 == 0, "half a slot is whole loads");
  static_assert(Waves * (MI > 2 ? 2 : MI) * 32 * PadN * 4 <= Lds, "the epilogue's rows fit");
};

__device__ __forceinline__ v4i buffer_of(const void* base, int64_t bytes) {
  const uint64_t a = (uint64_t)base;
  const uint32_t n = bytes > 0xFFFFFFFFll ? 0xFFFFFFFFu : (uint32_t)bytes;
  return v4i{(int)(uint32_t)a, (int)((a >> 32) & 0xFFFFu), (int)n, 0x00020000};
}

// Direct loads into LDS: lane l's 16 (or 4) bytes land at lds + 16 l (4 l). They have no
// destination register; the kernel waits for them by count before the barrier that
// precedes their first reader. (Written in assembly because the compiler would wait
// for all of them ahead of every LDS read.)
__device__ __forceinline__ void load_lds16(v4i buf, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
               "s"(buf), "s"(soff)
               : "memory");
}
__device__ __forceinline__ void load_lds4(v4i buf, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
               "s"(buf), "s"(soff)
               : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void barrier() {
  asm volatile("s_barrier" ::: "memory");
}

// Which 16-byte piece of a row's slot holds logical piece c: rows are spread over the
// banks so that the reads of a fragment collide in none.
__device__ __forceinline__ int piece(int row, int c) { return c ^ ((row >> 2) & 3); }

template <bool FP8>
struct Frag {
  v4i w[FP8 ? 2 : 1];
};

// This lane's row of a fragment for step s of a unit, from the slot that holds it.
template <bool FP8, bool EXACT>
__device__ __forceinline__ Frag<FP8> read_frag(const uint8_t* slot, int row, int s, int h) {
  Frag<FP8> f;
  if constexpr (FP8) {
    f.w[0] = *reinterpret_cast<const v4i*>(slot + row * 64 + 16 * piece(row, EXACT ? 2 * h : h));
    f.w[1] = *reinterpret_cast<const v4i*>(slot + row * 64 + 16 * piece(row, EXACT ? 2 * h + 1 : 2 + h));
  } else {
    f.w[0] = *reinterpret_cast<const v4i*>(slot + row * 64 + 16 * piece(row, 2 * s + h));
  }
  return f;
}

template <bool FP8>
__device__ __forceinline__ v8i operand_of(const Frag<FP8>& f) {
  if constexpr (FP8)
    return __builtin_shufflevector(f.w[0], f.w[1], 0, 1, 2, 3, 4, 5, 6, 7);
  else
    return widen(f.w[0]);
}

template <bool FP8>
__device__ __forceinline__ bf16x8 bf16_of(const Frag<FP8>& f, int j, float scale) {
  if constexpr (FP8)
    return bf16_from_e4m3((uint32_t)f.w[j / 2][2 * (j % 2)], (uint32_t)f.w[j / 2][2 * (j % 2) + 1], scale);
  else
    return bf16_from_e2m1((uint32_t)f.w[0][j], scale);
}

// The scale register of a unit: MXFP4 byte 0 (2) is the block of this lane half in the
// first (second) step; FP8 byte 0 is the group's exponent.
template <bool FP8>
__device__ __forceinline__ uint32_t scale_reg(uint32_t raw, int h) {
  return FP8 ? raw >> 23 : raw >> (8 * h);
}

// One step on the matrix cores, the first (S = 0) or second of a unit. `between` is called MI times in the course of it
// (with 0 .. MI - 1) to issue loads while the matrix cores are busy.
template <bool A8, bool B8, bool EXACT, int MI, int NI, int S, typename F>
__device__ __forceinline__ void multiply(f32x16 (&c)[MI][NI], const Frag<A8> (&a)[MI], const Frag<B8> (&b)[NI],
                                         const uint32_t (&sa)[MI], const uint32_t (&sb)[NI], F&& between) {
  if constexpr (!EXACT) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
      for (int j = 0; j < NI; ++j)
        c[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            operand_of<B8>(b[j]), operand_of<A8>(a[i]), c[i][j], B8 ? kE4M3 : kE2M1, A8 ? kE4M3 : kE2M1,
            B8 ? 0 : 2 * S, (int)sb[j], A8 ? 0 : 2 * S, (int)sa[i]);
      __builtin_amdgcn_sched_barrier(0);
      between(i);
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
    float fa[MI], fb[NI];
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[i] = e8m0_operand((A8 ? sa[i] : sa[i] >> (16 * S)) & 255u);
#pragma unroll
    for (int j = 0; j < NI; ++j) fb[j] = e8m0_operand((B8 ? sb[j] : sb[j] >> (16 * S)) & 255u);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      bf16x8 wa[MI];
#pragma unroll
      for (int i = 0; i < MI; ++i) wa[i] = bf16_of<A8>(a[i], t, fa[i]);
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const bf16x8 wb = bf16_of<B8>(b[j], t, fb[j]);
#pragma unroll
        for (int i = 0; i < MI; ++i) c[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb, wa[i], c[i][j], 0, 0, 0);
      }
      if (t * MI % 4 == 0) between(t * MI / 4);
    }
  }
}

// Workgroup `b` of `total` as the b-th of a list in which every XCD (workgroups are dealt
// to the eight in turn) walks consecutive entries, so that tiles which share operand
// rows share an L2.
__device__ __forceinline__ int xcd_order(int b, int total) {
  const int x = b & 7, q = total >> 3, r = total & 7;
  return x * q + (x < r ? x : r) + (b >> 3);
}

template <bool A8, bool B8, bool EXACT, int MI, int NI, int WN, bool ODDK, typename T>
__global__ __launch_bounds__(128 * WN, MI *NI > 8 ? 1 : 2) void mm_tile_kernel(MmLaunch p, int col_tiles) {
  using G = Tile<A8, B8, MI, NI, WN>;
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;

  // the tile
  const int row_tiles = p.offsets ? segment_tiles(p.offsets, p.groups, p.rows, G::BM)
                                  : (int)((p.rows + G::BM - 1) / G::BM);
  const int64_t total = (int64_t)row_tiles * col_tiles;
  if ((int64_t)blockIdx.x >= total) return;
  const int at = xcd_order(blockIdx.x, (int)total);
  constexpr int Group = 8;  // row tiles walked together over the columns
  const int band = at / (Group * col_tiles), in_band = at - band * (Group * col_tiles);
  const int tall = row_tiles - band * Group < Group ? row_tiles - band * Group : Group;
  const int row_tile = band * Group + in_band % tall, col_tile = in_band / tall;
  Segment s{0, 0, p.rows, row_tile};
  if (p.offsets && !find_segment(p.offsets, p.groups, p.rows, G::BM, row_tile, s)) return;

  const int64_t abytes = A8 ? p.k : p.k / 2, bbytes = B8 ? p.k : p.k / 2;
  const int64_t asbytes = A8 ? p.k / 128 * 4 : p.k / 32, bsbytes = B8 ? p.k / 128 * 4 : p.k / 32;
  const int64_t arow0 = s.begin + (int64_t)s.tile * G::BM;
  const int64_t brow0 = (int64_t)s.expert * p.n + (int64_t)col_tile * G::BN;
  const int arows = (int)(s.count - (int64_t)s.tile * G::BM < G::BM ? s.count - (int64_t)s.tile * G::BM : G::BM);
  const int brows = (int)(p.n - (int64_t)col_tile * G::BN < G::BN ? p.n - (int64_t)col_tile * G::BN : G::BN);
  const v4i abuf = buffer_of(p.a + arow0 * abytes, arows * abytes);
  const v4i bbuf = buffer_of(p.b + brow0 * bbytes, brows * bbytes);
  const uint8_t* ascale = static_cast<const uint8_t*>(p.a_scales) + arow0 * asbytes;
  const uint8_t* bscale = static_cast<const uint8_t*>(p.b_scales) + brow0 * bsbytes;
  const v4i asbuf = buffer_of(ascale, arows * asbytes);
  const v4i bsbuf = buffer_of(bscale, brows * bsbytes);

  // byte offsets of this lane's pieces in the slots' loads; rows past the end repeat the last
  uint32_t va[G::DA], vb[G::DB];
#pragma unroll
  for (int j = 0; j < G::DA; ++j) {
    const int row = (wave * G::DA + j) * 16 + lane / 4;
    va[j] = (uint32_t)((row < arows ? row : arows - 1) * abytes) + 16 * piece(row, lane % 4);
  }
#pragma unroll
  for (int j = 0; j < G::DB; ++j) {
    const int row = (wave * G::DB + j) * 16 + lane / 4;
    vb[j] = (uint32_t)((row < brows ? row : brows - 1) * bbytes) + 16 * piece(row, lane % 4);
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const int units = (int)((p.k + 127) / 128);
  const int tail = (int)(p.k % 128) / 32;  // blocks of the last unit, 0: all four (MXFP4 only: ODDK)

  // Before the last unit is loaded: pieces past the rows' end repeat the row's first one.
  auto trim = [&](int t) {
    if (ODDK && tail && t == units - 1) {
#pragma unroll
      for (int j = 0; j < G::DA; ++j) {
        const int c = piece((wave * G::DA + j) * 16 + lane / 4, lane % 4);
        va[j] -= c >= tail ? 16 * c : 0;
      }
#pragma unroll
      for (int j = 0; j < G::DB; ++j) {
        const int c = piece((wave * G::DB + j) * 16 + lane / 4, lane % 4);
        vb[j] -= c >= tail ? 16 * c : 0;
      }
    }
  };
  // Loads j0 <= j < j1 of slot number q of A (of B): unit q of an MXFP4 operand, step q of an
  // FP8 one. Past the last slot they load nothing, so that every step has the same number
  // outstanding.
  auto load_a = [&](int q, int j0, int j1) {
    v4i buf = abuf;
    buf[2] = q < (A8 ? 2 * units : units) ? buf[2] : 0;
#pragma unroll
    for (int j = j0; j < j1; ++j)
      load_lds16(buf, va[j], (uint32_t)q * 64, lds0 + (q & 3) * G::ASlot + (wave * G::DA + j) * 1024);
  };
  auto load_b = [&](int q, int j0, int j1) {
    v4i buf = bbuf;
    buf[2] = q < (B8 ? 2 * units : units) ? buf[2] : 0;
#pragma unroll
    for (int j = j0; j < j1; ++j)
      load_lds16(buf, vb[j], (uint32_t)q * 64, lds0 + G::BRing + (q & 3) * G::BSlot + (wave * G::DB + j) * 1024);
  };
  // Part u of MI of the loads issued in step s of unit t.
  auto load_part = [&](int t, int s, int u) {
    constexpr int NA = A8 ? G::DA : G::DA / 2, NB = B8 ? G::DB : G::DB / 2;
    const int a0 = A8 ? 0 : s * NA, b0 = B8 ? 0 : s * NB;
    load_a(A8 ? 2 * t + s + 3 : t + 3, a0 + u * NA / MI, a0 + (u + 1) * NA / MI);
    load_b(B8 ? 2 * t + s + 3 : t + 3, b0 + (u * NB + MI - 1) / MI, b0 + ((u + 1) * NB + MI - 1) / MI);
  };

  uint8_t* const sring = lds + G::SRing;
  // Chunk c of the scales: four dwords of every row, by direct loads. A dword past the
  // row's end repeats its last one.
  auto load_scales = [&](int c) {
    const uint32_t slot = lds0 + G::SRing + (uint32_t)(c & 1) * G::SChunk;
    const int want = 4 * c + (lane & 3), most = (int)(p.k / 128) - 1, dword = want < most ? want : most;
#pragma unroll
    for (int j = 0; j < G::SLoads; ++j) {
      const int first = (wave * G::SLoads + j) * 16;  // uniform: 16 rows of A or of B
      const int row = first + (lane >> 2);
      if (first < G::BM)
        load_lds4(asbuf, (uint32_t)((row < arows ? row : arows - 1) * asbytes) + 4 * dword, 0, slot + first * 16);
      else
        load_lds4(bsbuf, (uint32_t)((row - G::BM < brows ? row - G::BM : brows - 1) * bsbytes) + 4 * dword, 0,
                  slot + first * 16);
    }
  };
  // The same through registers where rows of block bytes do not start on dwords.
  constexpr int SR = (G::SRows + G::Threads - 1) / G::Threads;
  v4i held[SR];
  auto fetch_scales = [&](int c) {
#pragma unroll
    for (int j = 0; j < SR; ++j) {
      const int row = threadIdx.x + G::Threads * j;
      if (row < G::SRows) {
        const bool is_a = row < G::BM;
        const int rr = is_a ? (row < arows ? row : arows - 1) : (row - G::BM < brows ? row - G::BM : brows - 1);
        const uint8_t* q = (is_a ? ascale + rr * asbytes : bscale + rr * bsbytes) + 16 * c;
        const int left = (int)(p.k / 32) - 16 * c;
        uint32_t w[4];
        if (left >= 16) {
          __builtin_memcpy(w, q, 16);
        } else {
          // blocks past the row's end: 2^0, their codes are cleared
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = 0x7F7F7F7Fu;
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (4 * i + u < left) w[i] = (w[i] & ~(255u << (8 * u))) | (uint32_t)q[4 * i + u] << (8 * u);
          }
        }
        held[j] = v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
      }
    }
  };
  auto park_scales = [&](int c) {
#pragma unroll
    for (int j = 0; j < SR; ++j) {
      const int row = threadIdx.x + G::Threads * j;
      if (row < G::SRows) *reinterpret_cast<v4i*>(sring + (c & 1) * G::SChunk + row * 16) = held[j];
    }
  };
  // The last unit's last step has one block where `tail` is odd: clears the other one.
  auto clear_tail = [&]() {
    uint8_t* a = lds + ((units - 1) & 3) * G::ASlot;
    uint8_t* b = lds + G::BRing + ((units - 1) & 3) * G::BSlot;
    for (int row = threadIdx.x; row < G::SRows; row += G::Threads) {
      const int x = row < G::BM ? row : row - G::BM;
      *reinterpret_cast<v4i*>((row < G::BM ? a : b) + x * 64 + 16 * piece(x, tail)) = v4i{0, 0, 0, 0};
    }
    wait_loads<0>();
    barrier();
  };

  const int wm = wave / WN, wn = wave % WN;
  const int arow = wm * 32 * MI + r, brow = wn * 32 * NI + r;
  Frag<A8> fa[2][MI];
  Frag<B8> fb[2][NI];
  uint32_t sa[MI], sb[NI], ra[MI], rb[NI];
  f32x16 c[MI][NI] = {};

  auto read_step = [&](int t, int s, Frag<A8>(&xa)[MI], Frag<B8>(&xb)[NI]) {
    const uint8_t* a = lds + ((A8 ? 2 * t + s : t) & 3) * G::ASlot;
    const uint8_t* b = lds + G::BRing + ((B8 ? 2 * t + s : t) & 3) * G::BSlot;
#pragma unroll
    for (int i = 0; i < MI; ++i) xa[i] = read_frag<A8, EXACT>(a, arow + 32 * i, s, h);
#pragma unroll
    for (int j = 0; j < NI; ++j) xb[j] = read_frag<B8, EXACT>(b, brow + 32 * j, s, h);
  };
  // The scales of unit t as they lie in LDS; select_scales makes them the instructions'.
  auto read_scales = [&](int t) {
    const uint8_t* q = sring + ((t >> 2) & 1) * G::SChunk + 4 * (t & 3);
#pragma unroll
    for (int i = 0; i < MI; ++i) ra[i] = *reinterpret_cast<const uint32_t*>(q + 16 * (arow + 32 * i));
#pragma unroll
    for (int j = 0; j < NI; ++j) rb[j] = *reinterpret_cast<const uint32_t*>(q + 16 * (G::BM + brow + 32 * j));
  };
  auto select_scales = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = scale_reg<A8>(ra[i], h);
#pragma unroll
    for (int j = 0; j < NI; ++j) sb[j] = scale_reg<B8>(rb[j], h);
  };
  auto idle = [](int) {};

  if constexpr (ODDK) {
    fetch_scales(0);
    park_scales(0);
  } else {
    load_scales(0);
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    trim(q);
    load_a(q, 0, G::DA);
    load_b(q, 0, G::DB);
  }
  wait_loads<2 * (G::DA + G::DB)>();
  barrier();
  if (ODDK && (tail & 1) && units == 1) clear_tail();
  read_step(0, 0, fa[0], fb[0]);
  read_scales(0);
  select_scales();

  for (int t = 0; t + 1 < units; ++t) {
    // first step
    if constexpr (A8) {
      wait_loads<G::Younger>();
      barrier();
    }
    trim(t + 3);
    if constexpr (ODDK) {
      // chunk c + 1 is fetched in the first unit of chunk c and parked in the third
      if ((t & 3) == 0 && t + 4 < units) fetch_scales((t >> 2) + 1);
      if ((t & 3) == 2 && t + 2 < units) park_scales((t >> 2) + 1);
    } else {
      if ((t & 3) == 0 && t + 4 < units) load_scales((t >> 2) + 1);
    }
    read_step(t, 1, fa[1], fb[1]);
    __builtin_amdgcn_sched_barrier(0);
    multiply<A8, B8, EXACT, MI, NI, 0>(c, fa[0], fb[0], sa, sb, [&](int u) { load_part(t, 0, u); });
    __builtin_amdgcn_sched_barrier(0);
    // second step: the next slots have landed once at most the younger loads are outstanding,
    // and every wave has read its last fragments of the slots that are filled next
    wait_loads<G::Younger>();
    barrier();
    if (ODDK && (tail & 1) && t + 2 == units) clear_tail();
    read_step(t + 1, 0, fa[0], fb[0]);
    read_scales(t + 1);
    __builtin_amdgcn_sched_barrier(0);
    multiply<A8, B8, EXACT, MI, NI, 1>(c, fa[1], fb[1], sa, sb, [&](int u) { load_part(t, 1, u); });
    __builtin_amdgcn_sched_barrier(0);
    select_scales();
  }
  if constexpr (A8) {
    wait_loads<G::Younger>();
    barrier();
  }
  const bool both = !ODDK || tail == 0 || tail > 2;
  if (both) read_step(units - 1, 1, fa[1], fb[1]);
  multiply<A8, B8, EXACT, MI, NI, 0>(c, fa[0], fb[0], sa, sb, idle);
  if (both) multiply<A8, B8, EXACT, MI, NI, 1>(c, fa[1], fb[1], sa, sb, idle);

  // Epilogue: a block of rows at a time through LDS, so that rows leave as whole runs.
  wait_loads<0>();
  barrier();
  constexpr int V = sizeof(T) == 2 ? 8 : 4, PerRow = 32 * NI / V, RowsAtOnce = 64 / PerRow;
  constexpr int Park = MI > 2 ? 2 : MI;  // 32-row blocks parked at a time
  float* park = reinterpret_cast<float*>(lds) + wave * Park * 32 * G::PadN;
  const int prow = lane / PerRow, pcol = (lane % PerRow) * V;
  RunEpilogue<T, V> out(p.ep, s.expert, (int64_t)col_tile * G::BN + wn * 32 * NI + pcol);
#pragma unroll 1
  for (int block = 0; block < MI / Park; ++block) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i / Park == block) {
        float* to = park + (i % Park * 32 + r) * G::PadN + 4 * h;
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4*>(to + 32 * j + 8 * q) =
                make_float4(c[i][j][4 * q], c[i][j][4 * q + 1], c[i][j][4 * q + 2], c[i][j][4 * q + 3]);
      }
    }
    __builtin_amdgcn_wave_barrier();
    const int first = wm * 32 * MI + block * Park * 32 + prow;
    out.rows(p.ep, park + prow * G::PadN + pcol, RowsAtOnce * G::PadN, arow0 + first, arows - first, RowsAtOnce,
             Park * 32 / RowsAtOnce);
    __builtin_amdgcn_wave_barrier();
  }
}

template <bool A8, bool B8, bool EXACT, int MI, int NI, int WN, bool ODDK, typename T>
hipError_t launch_tile(const MmLaunch& a, hipStream_t st) {
  using G = Tile<A8, B8, MI, NI, WN>;
  const int64_t col_tiles = (a.n + G::BN - 1) / G::BN;
  const int64_t row_tiles = a.offsets ? a.rows / G::BM + (a.rows < a.groups ? a.rows : a.groups)
                                      : (a.rows + G::BM - 1) / G::BM;
  auto k = mm_tile_kernel<A8, B8, EXACT, MI, NI, WN, ODDK, T>;
  static const hipError_t set =
      hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, G::Lds);
  if (set != hipSuccess) return set;
  k<<<dim3((uint32_t)(row_tiles * col_tiles)), G::Threads, G::Lds, st>>>(a, (int)col_tiles);
  return hipGetLastError();
}

template <int MI, int NI, int WN, int ENI, int EWN>
hipError_t launch_sized(const MmLaunch& a, hipStream_t st) {
  const bool f32 = a.ep.out_f32;
  if (a.a_fmt && a.b_fmt)
    return f32 ? launch_tile<true, true, true, MI, ENI, EWN, false, float>(a, st)
               : launch_tile<true, true, false, MI, NI, WN, false, __bf16>(a, st);
  if (a.a_fmt)
    return f32 ? launch_tile<true, false, true, MI, ENI, EWN, false, float>(a, st)
               : launch_tile<true, false, false, MI, NI, WN, false, __bf16>(a, st);
  if (a.k % 128)
    return f32 ? launch_tile<false, false, false, MI, NI, WN, true, float>(a, st)
               : launch_tile<false, false, false, MI, NI, WN, true, __bf16>(a, st);
  return f32 ? launch_tile<false, false, false, MI, NI, WN, false, float>(a, st)
             : launch_tile<false, false, false, MI, NI, WN, false, __bf16>(a, st);
}

}  // namespace

hipError_t launch_gemm_tiles(const MmLaunch& a, bool large, hipStream_t st) {
  return large ? launch_sized<4, 4, 2, 4, 2>(a, st) : launch_sized<2, 2, 2, 2, 2>(a, st);
}

}  // namespace mxq

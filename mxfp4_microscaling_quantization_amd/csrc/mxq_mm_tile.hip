// Matrix products on MXFP4 / FP8 operands for many rows: LDS-tiled, operands fetched
// by direct loads into LDS several stages ahead of the matrix instructions.
#include <atomic>

#include "mxq_mm.h"

namespace mxq {

namespace {

constexpr int kCUs = 256;  // of an MI355X; the tiles' LDS leaves room for one workgroup of each

// A workgroup of 2 x WN waves owns 64 MI x 32 NI WN results, a wave 32 MI x 32 NI. The
// contraction runs in steps of 64 elements, four to a turn of 256. Each operand has R
// slots in LDS with 128 bytes of every row in each, a whole cache line: a turn of an
// MXFP4 row or half a turn of an FP8 row. (A CU's direct loads of 1 KiB take 18 cycles each as
// 8 rows of 128 bytes, 36 as 16 rows of 64, with all CUs at work on data in the L2s; 16 of
// either alone.) A slot is filled again from the moment when every
// wave has read its last fragments, the loads spread over the steps. Fragments of the next
// step are read from LDS while the matrix cores work on the current one; one barrier a
// slot is all that the waves wait for.
// Tiles of 128 leave few products between a fragment's read and its use: there, except for
// FP8 instructions (512 x 14336 x 4096: 50 us with two groups, 44 with one), KS = 2 groups of
// waves hold the same results and take two steps of every turn each; their sums are added
// at the end, each group finishing half of the rows. Tiles of 64 leave room for a second
// workgroup on the CU instead (and gained nothing from a ring of eight slots, and up to a
// tenth from two groups at FP4).
// What bounds it: large tiles, the matrix cores under the chip's power limit while they run
// (8192 x 8192 x 16384: MXFP4 4.2 PFLOP/s, where a loop of its products alone reaches 6.2 to 6.9
// on such data; FP8 2.4 of 4.2), and the results' bytes between (8192 x 14336 x 4096 MXFP4
// to bf16 275 us, with GELU 291, with bias, GELU and z 335; to fp32 on a residual 389). The
// exact products of FP8 operands to fp32, on bf16 instructions, take 882 us there (MXFP4 weights 850).
// Tiles of 128 and 64: the 1 KiB loads of a CU, at 18 cycles each, and one turn's latency
// (256 x 4096 x 14336: MXFP4 26 us, FP8 33); with LOOSE scales the wait ahead of park_scales is for
// all loads, so every second turn empties the ring (777 x 1336 x 4128 to fp32: 19 us).
// Weight gradient of 16 uneven experts, 16384 tokens, 2048 x 7168: 509 us, of which the
// results are 470 MB (accumulated in fp32: 990); 13 us of every tile are its start and its results, 4.0 us a turn.
template <bool A8, bool B8, int MI, int NI, int WN, int KS, int R, bool WG>
struct Tile {
  static constexpr int Waves = 2 * WN * KS, Threads = 64 * Waves;
  static constexpr int BM = 64 * MI, BN = 32 * NI * WN;
  static constexpr int ASlot = BM * 128, BSlot = BN * 128;
  static constexpr int Slot = ASlot + BSlot, SRing = R * Slot;                // offsets in LDS
  static constexpr int DA = ASlot / 1024 / Waves, DB = BSlot / 1024 / Waves;  // 1 KiB loads of a wave for a slot
  // loads of the slots after the one that a barrier waits for (the fewest that are certain)
  static constexpr int Younger = KS == 2 && A8 ? 0 : (R - 2) * (A8 == B8 ? DA + DB : DA);
  // scales: 16 bytes of a row cover a chunk of two turns; R chunks, loaded R / 2 ahead
  static constexpr int SRows = BM + BN, SChunk = SRows * 16, Ahead = R / 2;
  static constexpr int SLoads = SRows / 16 / Waves;  // 256-byte loads of a wave in a chunk (16 rows each)
  // weight gradient: a ninth piece of every row, beside each slot
  static constexpr int XRing = SRing + R * SChunk, XSlot = SRows * 16;
  static constexpr int Lds = XRing + (WG ? R * XSlot : 0);
  // 32 rows of every wave, parked for the epilogue from the second slot on
  static constexpr int ParkBytes = Waves * 32 * 32 * NI * 4;
  static_assert(KS == 1 || (MI == 2 && DA == MI && DB == MI), "two groups: half of the rows and a load a part");
  static_assert(Slot + ParkBytes <= SRing, "the parked rows fit beside the first slot");
  static_assert(DA % 2 == 0 && DB % 2 == 0, "a wave's loads of a slot come in pairs");
};

__device__ __forceinline__ v4i buffer_of(const void* base, int64_t bytes) {
  const uint64_t a = (uint64_t)base;
  const uint32_t n = bytes > 0xFFFFFFFFll ? 0xFFFFFFFFu : (uint32_t)bytes;
  return v4i{(int)(uint32_t)a, (int)((a >> 32) & 0xFFFFu), (int)n, 0x00020000};
}

// Direct loads into LDS: lane l's 16 (or 4) bytes land at lds + 16 l (4 l), lds in m0, an operand
// like the others, so that the compiler knows what the register holds. They have no
// destination register; the kernel waits for them by count before the barrier that
// precedes their first reader. (Written in assembly because the compiler would wait
// for all of them ahead of every LDS read.) A vector memory instruction may read a scalar
// register five wait states after a vector instruction wrote it: the compiler, which does
// not look into the statement, may just have fetched a spilled descriptor with v_readlane.
__device__ __forceinline__ void load_lds16(v4i buf, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"{m0}"(__builtin_amdgcn_readfirstlane(lds)),
               "v"(voff), "s"(buf), "s"(__builtin_amdgcn_readfirstlane(soff))
               : "memory");
}
__device__ __forceinline__ void load_lds4(v4i buf, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_nop 4\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"{m0}"(__builtin_amdgcn_readfirstlane(lds)),
               "v"(voff), "s"(buf), "s"(__builtin_amdgcn_readfirstlane(soff))
               : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void barrier() {
  asm volatile("s_barrier" ::: "memory");
}

// Which 16-byte piece of a row's slot holds logical piece c: rows are spread over the
// banks so that the reads of a fragment collide in none.
__device__ __forceinline__ int piece(int row, int c) { return c ^ ((row >> 1) & 7); }

template <bool FP8>
struct Frag {
  v4i w[FP8 ? 2 : 1];
};

// Byte offset in a slot of this lane's first piece of the fragment whose first row is 0, and
// the fragment of step s of a turn: a step's pieces differ from the first step's in whole
// bits, so one register serves all. (FP8: pieces h and 2 + h, or the lane's 32 elements
// in order, 2h and 2h + 1, for the exact product.)
template <bool FP8, bool EXACT>
__device__ __forceinline__ int frag_base(int row, int h) {
  return row * 128 + 16 * piece(row, FP8 && EXACT ? 2 * h : h);
}
__device__ __forceinline__ int row16(int base) { return (base >> 7) * 16; }  // 16 times its row
template <bool FP8, bool EXACT>
__device__ __forceinline__ Frag<FP8> read_frag(const uint8_t* slot, int base, int i, int s) {
  Frag<FP8> f;
  const int at = base ^ (FP8 ? 64 * (s & 1) : 32 * s);
  f.w[0] = *reinterpret_cast<const v4i*>(slot + at + 4096 * i);
  if constexpr (FP8) f.w[1] = *reinterpret_cast<const v4i*>(slot + (at ^ (EXACT ? 16 : 32)) + 4096 * i);
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

// The scale register of two steps: MXFP4 byte 0 (2) is the block of this lane half in the
// first (second) one; FP8 byte 0 is the group's exponent.
template <bool FP8>
__device__ __forceinline__ uint32_t scale_reg(uint32_t raw, int h) {
  return FP8 ? raw >> 23 : raw >> (8 * h);
}

// The byte select of the scale operands is part of the instruction.
template <bool A8, bool B8>
__device__ __forceinline__ f32x16 multiply_scaled(const Frag<A8>& a, const Frag<B8>& b, uint32_t sa, uint32_t sb,
                                                  int step, f32x16 c) {
  constexpr int FA = A8 ? kE4M3 : kE2M1, FB = B8 ? kE4M3 : kE2M1;
  if (step == 0)
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand_of<B8>(b), operand_of<A8>(a), c, FB, FA, 0, (int)sb,
                                                           0, (int)sa);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand_of<B8>(b), operand_of<A8>(a), c, FB, FA,
                                                         B8 ? 0 : 2, (int)sb, A8 ? 0 : 2, (int)sa);
}

// One step on the matrix cores, the first (step 0) or second of a scale register's two.
// `between` is called MI times in the course of it (with 0 .. MI - 1) to issue loads while
// the matrix cores are busy.
template <bool A8, bool B8, bool EXACT, int MI, int NI, typename F>
__device__ __forceinline__ void multiply(f32x16 (&c)[MI][NI], const Frag<A8> (&a)[MI], const Frag<B8> (&b)[NI],
                                         const uint32_t (&sa)[MI], const uint32_t (&sb)[NI], int step, F&& between) {
  if constexpr (!EXACT) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
      for (int j = 0; j < NI; ++j)
        c[i][j] = multiply_scaled<A8, B8>(a[i], b[j], sa[i], sb[j], step, c[i][j]);
      __builtin_amdgcn_sched_barrier(0);
      between(i);
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
    float fa[MI], fb[NI];
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[i] = e8m0_operand((A8 ? sa[i] : sa[i] >> (16 * step)) & 255u);
#pragma unroll
    for (int j = 0; j < NI; ++j) fb[j] = e8m0_operand((B8 ? sb[j] : sb[j] >> (16 * step)) & 255u);
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

// A workgroup takes entry `turn` of its share of the tiles. Workgroups are dealt to the eight
// XCDs in turn; entries are ordered so that the workgroups of an XCD hold consecutive
// ones, which share operand rows in its L2.
__device__ __forceinline__ int64_t list_entry(int64_t turn) {
  const int grid = gridDim.x, x = blockIdx.x & 7, q = grid >> 3, r = grid & 7;
  return turn * grid + x * q + (x < r ? x : r) + (blockIdx.x >> 3);
}

template <bool A8, bool B8, bool EXACT, int MI, int NI, int WN, int KS, int R, bool LOOSE, bool WG, typename T>
__global__ __launch_bounds__(128 * WN * KS, MI * NI > 8 ? 1 : 2) void mm_tile_kernel(MmLaunch p, int col_tiles) {
  using G = Tile<A8, B8, MI, NI, WN, KS, R, WG>;
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;

  const bool listed = p.offsets && !WG;  // its row tiles are known on the device only
  int row_tiles = (int)(((WG ? p.n : p.rows) + G::BM - 1) / G::BM);
  if (listed) {
    // (malformed offsets make no more work than well-formed ones can)
    const int most = (int)most_tiles(p.rows, p.groups, G::BM);
    row_tiles = segment_tiles(p.offsets, p.groups, p.rows, G::BM);
    row_tiles = row_tiles < most ? row_tiles : most;
  }
  const int64_t total = (int64_t)row_tiles * col_tiles * (WG ? p.groups : 1);
  const int64_t abytes = WG ? p.ld_a : A8 ? p.k : p.k / 2, bbytes = WG ? p.ld_b : B8 ? p.k : p.k / 2;
  const int64_t asbytes = WG ? 4 * p.ld_as : A8 ? p.k / 128 * 4 : p.k / 32;
  const int64_t bsbytes = WG ? 4 * p.ld_bs : B8 ? p.k / 128 * 4 : p.k / 32;
  // weight gradient: bytes and scales that a column has at most
  const int64_t col_bytes = (p.rows + 15) / 16 * 16;
  const int col_scales = (int)((p.rows + 127 * (int64_t)p.groups) / 128);
  const uint32_t apitch = (uint32_t)(16 * abytes), bpitch = (uint32_t)(16 * bbytes);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;

  // The tile in work: its expert, first row of d and first column, rows and columns there are,
  int expert = 0, arows = 0, brows = 0;
  int64_t orow0 = 0, col0 = 0;
  // its operands. Weight gradient: the contraction runs over the expert's tokens, whose first
  // byte of a column lies `shift` past a 16-byte boundary; first_slot: their first scale.
  int64_t depth = 0;
  int shift = 0, first_slot = 0;
  v4i abuf = {}, bbuf = {}, asbuf = {}, bsbuf = {};
  const uint8_t *ascale = nullptr, *bscale = nullptr;
  // Byte offsets of this lane's pieces in a wave's first two loads of a slot; the others lie
  // whole rows further on. Rows past the tile's last are past the buffer's end: zeros.
  uint32_t va[2], vb[2];
  int turns = 0, halves = 0;  // slots of an MXFP4 operand, of an FP8 operand
  int tail = 0;               // blocks of the last turn, 0: all eight
  int last_steps = 0;
  auto set_up = [&](int64_t entry) {
    if (entry >= total) return false;
    expert = WG ? (int)(entry / ((int64_t)row_tiles * col_tiles)) : 0;
    const int at = (int)(entry - (int64_t)expert * row_tiles * col_tiles);
    constexpr int Group = 8;  // row tiles walked together over the columns
    const int band = at / (Group * col_tiles), in_band = at - band * (Group * col_tiles);
    const int tall = row_tiles - band * Group < Group ? row_tiles - band * Group : Group;
    const int row_tile = band * Group + in_band % tall, col_tile = in_band / tall;
    Segment s{expert, 0, p.rows, row_tile};
    if (listed && !find_segment(p.offsets, p.groups, p.rows, G::BM, row_tile, s)) return false;
    depth = p.k;
    if constexpr (WG) {
      s.begin = clamp_row(p.offsets[expert], p.rows);
      depth = clamp_row(p.offsets[expert + 1], p.rows) - s.begin;
      depth = depth < 0 ? 0 : depth;
      shift = (int)(s.begin & 15);
      first_slot = segment_tiles(p.offsets, expert, p.rows, 128);
    }
    expert = s.expert;
    const int64_t arow0 = WG ? (int64_t)row_tile * G::BM : s.begin + (int64_t)s.tile * G::BM;
    col0 = (int64_t)col_tile * G::BN;
    const int64_t brow0 = (WG ? 0 : (int64_t)expert * p.n) + col0;
    orow0 = WG ? expert * p.n + arow0 : arow0;
    const int64_t aleft = WG ? p.n - arow0 : s.count - (int64_t)s.tile * G::BM;
    const int64_t bleft = (WG ? p.k : p.n) - col0;
    arows = (int)(aleft < G::BM ? aleft : G::BM);
    brows = (int)(bleft < G::BN ? bleft : G::BN);
    const int64_t from = WG ? s.begin - shift : 0;  // bytes of a row before the first piece
    // (of the last column no more than it has: it may end a wider tensor)
    abuf = buffer_of(p.a + arow0 * abytes + from, (arows - 1) * abytes + (WG ? col_bytes : abytes) - from);
    bbuf = buffer_of(p.b + brow0 * bbytes + from, (brows - 1) * bbytes + (WG ? col_bytes : bbytes) - from);
    ascale = static_cast<const uint8_t*>(p.a_scales) + arow0 * asbytes;
    bscale = static_cast<const uint8_t*>(p.b_scales) + brow0 * bsbytes;
    asbuf = buffer_of(ascale, (arows - 1) * asbytes + (WG ? 4 * col_scales : asbytes));
    bsbuf = buffer_of(bscale, (brows - 1) * bsbytes + (WG ? 4 * col_scales : bsbytes));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int arow = (wave * G::DA + j) * 8 + lane / 8, brow = (wave * G::DB + j) * 8 + lane / 8;
      va[j] = (uint32_t)(arow * abytes) + 16 * piece(arow, lane % 8);
      vb[j] = (uint32_t)(brow * bbytes) + 16 * piece(brow, lane % 8);
    }
    turns = (int)((depth + 255) / 256);
    halves = (int)(WG ? (depth + 127) / 128 : depth / 128);
    tail = WG ? 4 * (halves & 1) : (int)(depth % 256) / 32;
    last_steps = tail ? (tail + 1) / 2 : 4;
    return true;
  };

  // Before the last turn of an MXFP4 operand is loaded: pieces past the rows' end repeat the
  // row's first one.
  auto trim = [&](int t) {
    if (tail && t == turns - 1) {
      int l = lane;
      asm volatile("" : "+v"(l));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int ca = piece((wave * G::DA + j) * 8 + l / 8, l % 8);
        const int cb = piece((wave * G::DB + j) * 8 + l / 8, l % 8);
        if (!A8 && ca >= tail) va[j] -= 16 * ca;
        if (!B8 && cb >= tail) vb[j] -= 16 * cb;
      }
    }
  };
  // (Weight gradient: the last group's pieces may pass the end of the last column, so the
  // offset in the row is part of what the buffer's bounds are checked against.)
  // Load j of slot number q of A, and of B (q counts turns of an MXFP4 operand, half turns of
  // an FP8 one). Past the last slot it loads nothing.
  auto load_a = [&](int q, int j) {
    v4i buf = abuf;
    buf[2] = q < (A8 ? halves : turns) ? buf[2] : 0;
    const uint32_t at = (uint32_t)q * 128;
    load_lds16(buf, va[j & 1] + (j >> 1) * apitch + (WG ? at : 0), WG ? 0 : at,
               lds0 + (q & (R - 1)) * G::Slot + (wave * G::DA + j) * 1024);
  };
  auto load_b = [&](int q, int j) {
    v4i buf = bbuf;
    buf[2] = q < (B8 ? halves : turns) ? buf[2] : 0;
    const uint32_t at = (uint32_t)q * 128;
    load_lds16(buf, vb[j & 1] + (j >> 1) * bpitch + (WG ? at : 0), WG ? 0 : at,
               lds0 + G::ASlot + (q & (R - 1)) * G::Slot + (wave * G::DB + j) * 1024);
  };
  // Weight gradient. Tokens [0, 128) of a group lie at bytes [shift, 128 + shift) of nine
  // 16-byte pieces. The first piece's leading bytes, which belong to other tokens, are
  // replaced by the ninth's when a fragment is read: the sum does not depend on the order
  // of the tokens, and both operands have the same shift.
  auto load_ninth = [&](int q) {
    if (!WG || shift == 0) return;
    int l = lane;
    asm volatile("" : "+v"(l));  // (addresses formed here, not held over the turns)
#pragma unroll
    for (int j = wave; j < G::SRows / 64; j += G::Waves) {
      const bool is_a = j < G::BM / 64;
      v4i buf = is_a ? abuf : bbuf;
      buf[2] = q < halves ? buf[2] : 0;
      const uint32_t row = (is_a ? j : j - G::BM / 64) * 64 + l;
      load_lds16(buf, row * (uint32_t)(is_a ? abytes : bbytes) + (uint32_t)q * 128 + 128, 0,
                 lds0 + G::XRing + (q & (R - 1)) * G::XSlot + j * 1024);
    }
  };
  uint32_t keep_second = h ? ~0u : 0u;  // the second lane half holds other pieces
  auto merge_ninth = [&](v4i w, int q, int at) {
    const v4i x = *reinterpret_cast<const v4i*>(lds + G::XRing + (q & (R - 1)) * G::XSlot + at);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int lead = shift - 4 * d;  // leading bytes of this dword that are replaced
      const uint32_t own = lead <= 0 ? ~0u : lead >= 4 ? 0u : ~0u << (8 * lead);
      const uint32_t keep = own | keep_second;
      w[d] = (int)(((uint32_t)w[d] & keep) | ((uint32_t)x[d] & ~keep));
    }
    return w;
  };
  // The last group's bytes past its last token become zeros, in both operands.
  auto clear_group = [&](int q) {
    const int last = (int)(depth - (int64_t)q * 128);
    if (last >= 128) return;
    for (int i = threadIdx.x; i < G::SRows * 9; i += G::Threads) {
      const int row = i / 9, c = i % 9, keep = last + shift - 16 * c;  // leading bytes that stay
      if (keep >= 16 || (c == 8 && shift == 0)) continue;
      const int x = row < G::BM ? row : row - G::BM;
      uint8_t* slot = row < G::BM ? lds + (q & (R - 1)) * G::Slot : lds + G::ASlot + (q & (R - 1)) * G::Slot;
      v4i* at = c == 8 ? reinterpret_cast<v4i*>(lds + G::XRing + (q & (R - 1)) * G::XSlot + row * 16)
                       : reinterpret_cast<v4i*>(slot + x * 128 + 16 * piece(x, c));
      v4i w = *at;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int left = keep - 4 * d;
        w[d] = left >= 4 ? w[d] : left <= 0 ? 0 : (int)((uint32_t)w[d] & ~(~0u << (8 * left)));
      }
      *at = w;
    }
    wait_loads<0>();
    barrier();
  };
  // The loads issued in step s of turn t, part u of MI of them: those of an FP8 slot in the
  // odd step that frees it and the step after, those of an MXFP4 slot in the last step and
  // the first two of the next turn (A's earlier than B's).
  // Two groups: in the second step, which frees a turn's slots, and the first of the next.
  auto load_part = [&](int t, int s, int u) {
    if constexpr (KS == 2) {
      const int q8 = s ? 2 * t + R : 2 * t - 1 + R;
      if (WG && u == 0) load_ninth(q8);
      if (A8)
        load_a(q8, u);
      else if (s)
        load_a(t + R, u);
      if (B8)
        load_b(q8, u);
      else if (!s)
        load_b(t - 1 + R, u);
      return;
    }
    if (WG && (s & 1) && u == 0) load_ninth(2 * t + (s + 1) / 2 - 1 + R);
    if constexpr (A8) {
#pragma unroll
      for (int j = 0; j < G::DA; ++j)
        if ((s & 1) == (j >= G::DA / 2 ? 0 : 1) && j % (G::DA / 2) * MI / (G::DA / 2) == u)
          load_a(2 * t + (s + 1) / 2 - 1 + R, j);
    } else {
#pragma unroll
      for (int j = 0; j < G::DA; ++j)
        if (s == (j < 3 ? 3 : 0) && j % 3 % MI == u) load_a(s == 3 ? t + R : t + R - 1, j);
    }
    if constexpr (B8) {
#pragma unroll
      for (int j = 0; j < G::DB; ++j)
        if ((s & 1) == (j >= G::DB / 2 ? 0 : 1) && (j % (G::DB / 2) * MI + MI / 2) / (G::DB / 2) == u)
          load_b(2 * t + (s + 1) / 2 - 1 + R, j);
    } else {
#pragma unroll
      for (int j = 0; j < G::DB; ++j)
        if (s == (j < 2 ? 0 : 1) && (j + (j < 2)) % MI == u) load_b(t + R - 1, j);
    }
  };

  uint8_t* const sring = lds + G::SRing;
  // Chunk c of the scales: four dwords of every row, by direct loads. A dword past the
  // row's end repeats its last one.
  auto load_scales = [&](int c) {
    const uint32_t slot = lds0 + G::SRing + (uint32_t)(c & (R - 1)) * G::SChunk;
    int l = lane;
    asm volatile("" : "+v"(l));  // (addresses formed here, not held over the turns)
    const int want = 4 * c + (l & 3), most = halves - 1;
    int dword = first_slot + (want < most ? want : most);
    if (WG) dword = dword < col_scales ? dword : 0;  // malformed offsets stay inside
#pragma unroll
    for (int j = 0; j < G::SLoads; ++j) {
      const int first = (wave * G::SLoads + j) * 16;  // uniform: 16 rows of A or of B
      const int row = first + (l >> 2);
      if (first < G::BM)
        load_lds4(asbuf, (uint32_t)((row < arows ? row : arows - 1) * asbytes) + 4 * dword, 0, slot + first * 16);
      else
        load_lds4(bsbuf, (uint32_t)((row - G::BM < brows ? row - G::BM : brows - 1) * bsbytes) + 4 * dword, 0,
                  slot + first * 16);
    }
  };
  // The same through registers (LOOSE) where rows of block bytes do not start on dwords: k is not a
  // multiple of 128, or the caller's scales start at another byte.
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
      if (row < G::SRows) *reinterpret_cast<v4i*>(sring + (c & (R - 1)) * G::SChunk + row * 16) = held[j];
    }
  };
  // The last turn's last step has one block where `tail` is odd: clears the other one.
  auto clear_tail = [&]() {
    uint8_t* a = lds + ((turns - 1) & (R - 1)) * G::Slot;
    uint8_t* b = lds + G::ASlot + ((turns - 1) & (R - 1)) * G::Slot;
    for (int row = threadIdx.x; row < G::SRows; row += G::Threads) {
      const int x = row < G::BM ? row : row - G::BM;
      *reinterpret_cast<v4i*>((row < G::BM ? a : b) + x * 128 + 16 * piece(x, tail)) = v4i{0, 0, 0, 0};
    }
    wait_loads<0>();
    barrier();
  };

  // kg: the wave's group; its steps of a turn are 2 kg and 2 kg + 1 where there are two
  const int kg = KS == 2 ? wave / (2 * WN) : 0, wm = wave / WN % 2, wn = wave % WN;
  const int arow = wm * 32 * MI + r, brow = wn * 32 * NI + r;
  int abase = frag_base<A8, EXACT>(arow, h) ^ (A8 ? 0 : 64 * kg);
  int bbase = frag_base<B8, EXACT>(brow, h) ^ (B8 ? 0 : 64 * kg);
  // Two FP8 fragment sets of A do not fit the registers: a fragment is then replaced by the
  // next step's as soon as its last product is issued.
  constexpr bool Roll = A8 && B8 && !EXACT && KS == 1 && MI > 2;
  Frag<A8> fa[Roll ? 1 : 2][MI];
  Frag<B8> fb[2][NI];
  uint32_t sa[MI], sb[NI], ra[MI], rb[NI];
  f32x16 c[MI][NI];
  // The sums pass through an empty statement after every step: the products, which have
  // no side effects, would else sink below the barriers and keep every fragment alive.
  auto pin = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        if constexpr (MI * NI > 8)
          asm volatile("" : "+a"(c[i][j]));
        else
          asm volatile("" : "+v"(c[i][j]));
      }
  };
  auto read_a = [&](int t, int s, int i) {
    Frag<A8> f = read_frag<A8, EXACT>(lds + ((A8 ? 2 * t + (s >> 1) + kg : t) & (R - 1)) * G::Slot, abase, i, s);
    if (WG && (s & 1) == 0) f.w[0] = merge_ninth(f.w[0], 2 * t + (s >> 1) + kg, row16(abase) + 512 * i);
    return f;
  };
  // Fragments of step s of turn t: B's, and A's where they are not replaced one by one.
  auto read_step = [&](int t, int s) {
    const uint8_t* b = lds + G::ASlot + ((B8 ? 2 * t + (s >> 1) + kg : t) & (R - 1)) * G::Slot;
    if constexpr (!Roll) {
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[s & 1][i] = read_a(t, s, i);
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      fb[s & 1][j] = read_frag<B8, EXACT>(b, bbase, j, s);
      if (WG && (s & 1) == 0)
        fb[s & 1][j].w[0] = merge_ninth(fb[s & 1][j].w[0], 2 * t + (s >> 1) + kg, 16 * G::BM + row16(bbase) + 512 * j);
    }
  };
  // The scales of steps 2u and 2u + 1 as they lie in LDS; select_scales makes them the
  // instructions'.
  auto read_scales = [&](int u) {
    const uint8_t* q = sring + ((u >> 2) & (R - 1)) * G::SChunk + 4 * (u & 3);
#pragma unroll
    for (int i = 0; i < MI; ++i) ra[i] = *reinterpret_cast<const uint32_t*>(q + row16(abase) + 512 * i);
#pragma unroll
    for (int j = 0; j < NI; ++j) rb[j] = *reinterpret_cast<const uint32_t*>(q + 16 * G::BM + row16(bbase) + 512 * j);
  };
  auto select_scales = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = scale_reg<A8>(ra[i], h);
#pragma unroll
    for (int j = 0; j < NI; ++j) sb[j] = scale_reg<B8>(rb[j], h);
  };

  // The loads that start a tile: its first scales and slot 0, then the other slots, of the
  // last one only what the steps to come do not load.
  auto start_first = [&]() {
    if (WG && turns == 0) return;
    if constexpr (LOOSE) {
      fetch_scales(0);
      park_scales(0);
    } else {
#pragma unroll
      for (int c = 0; c < G::Ahead; ++c)
        if (c == 0 || 2 * c < turns) load_scales(c);
    }
    trim(0);
    load_ninth(0);
#pragma unroll
    for (int j = 0; j < G::DA; ++j) load_a(0, j);
#pragma unroll
    for (int j = 0; j < G::DB; ++j) load_b(0, j);
  };
  constexpr int PartA = A8 ? (KS == 2 ? 0 : G::DA / 2) : G::DA < 3 ? G::DA : 3;
  constexpr int PartB = B8 ? (KS == 2 ? 0 : G::DB / 2) : 0;
  auto start_rest = [&]() {
    if (WG && turns == 0) return;
#pragma unroll
    for (int q = 1; q < R; ++q) {
      trim(q);
      load_ninth(q);
#pragma unroll
      for (int j = 0; j < (q < R - 1 ? G::DA : PartA); ++j) load_a(q, j);
#pragma unroll
      for (int j = 0; j < (q < R - 1 ? G::DB : PartB); ++j) load_b(q, j);
    }
  };
  // the last turn: one to four steps (two or four where k is a multiple of 128)
  auto last_step = [&](int s) {
    if (s + 1 < last_steps) {
      read_step(turns - 1, s + 1);
      if (s == 1) read_scales(2 * turns - 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    multiply<A8, B8, EXACT, MI, NI>(c, fa[Roll ? 0 : s & 1], fb[s & 1], sa, sb, s & 1, [&](int u) {
      if constexpr (Roll)
        if (s + 1 < last_steps) fa[0][u] = read_a(turns - 1, s + 1, u);
      if (s == 0) load_part(turns - 1, 0, u);
    });
    pin();
    if (s == 1) select_scales();
  };

  if (!set_up(list_entry(0))) return;
  start_first();
  for (int64_t entry = 0;; ++entry) {
    start_rest();
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) c[i][j] = f32x16{};
    if (!WG || turns > 0) {
      wait_loads<KS == 2 && A8 ? G::DA + G::DB : PartA + PartB + (R - 2) * (G::DA + G::DB)>();
      barrier();
      if (LOOSE && (tail & 1) && turns == 1) clear_tail();
      if (WG && (KS == 2 ? turns == 1 : halves == 1)) clear_group(halves - 1);
      read_step(0, 0);
      if constexpr (Roll) {
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[0][i] = read_a(0, 0, i);
      }
      read_scales(kg);
      select_scales();

      if constexpr (KS == 2) {
        for (int t = 0; t + 1 < turns; ++t) {
          asm volatile("" : "+v"(abase), "+v"(bbase));
          if constexpr (WG) asm volatile("" : "+v"(keep_second));
          if constexpr (LOOSE) {
            if ((t & 1) == 0 && t + 2 < turns) fetch_scales((t >> 1) + 1);
            if ((t & 1) == 1) park_scales((t >> 1) + 1);
          }
          read_step(t, 1);
          __builtin_amdgcn_sched_barrier(0);
          multiply<A8, B8, EXACT, MI, NI>(c, fa[0], fb[0], sa, sb, 0, [&](int u) { load_part(t, 0, u); });
          pin();
          __builtin_amdgcn_sched_barrier(0);
          // the next turn's slots have landed, and every wave has its last fragments of this one's
          wait_loads<G::Younger>();
          barrier();
          if (WG && t + 2 == turns) clear_group(halves - 1);
          if (LOOSE && (tail & 1) && t + 2 == turns) clear_tail();
          trim(t + R);
          if constexpr (!LOOSE)
            if ((t & 1) == 0 && t + 2 * G::Ahead < turns) load_scales((t >> 1) + G::Ahead);
          read_step(t + 1, 0);
          read_scales(2 * t + 2 + kg);
          __builtin_amdgcn_sched_barrier(0);
          multiply<A8, B8, EXACT, MI, NI>(c, fa[1], fb[1], sa, sb, 1, [&](int u) { load_part(t, 1, u); });
          pin();
          __builtin_amdgcn_sched_barrier(0);
          select_scales();
        }
        auto none = [](int) {};
        if (last_steps > 2 * kg) {
          if (last_steps > 2 * kg + 1) read_step(turns - 1, 1);
          multiply<A8, B8, EXACT, MI, NI>(c, fa[0], fb[0], sa, sb, 0, none);
          pin();
          if (last_steps > 2 * kg + 1) {
            multiply<A8, B8, EXACT, MI, NI>(c, fa[1], fb[1], sa, sb, 1, none);
            pin();
          }
        }
      } else {
        for (int t = 0; t + 1 < turns; ++t) {
          // addresses and masks are formed where used, not held
          asm volatile("" : "+v"(abase), "+v"(bbase));
          if constexpr (WG) asm volatile("" : "+v"(keep_second));
          if constexpr (LOOSE) {
            // chunk c + 1 is fetched in the first turn of chunk c and parked in the second
            if ((t & 1) == 0 && t + 2 < turns) fetch_scales((t >> 1) + 1);
            if ((t & 1) == 1 && t + 1 < turns) park_scales((t >> 1) + 1);
          }
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const int tn = s == 3 ? t + 1 : t, sn = (s + 1) & 3;
            auto advance = [&]() {
              // the next slots have landed, and every wave has its last fragments of the current ones
              if (s == 3 || (s == 1 && (A8 || B8))) {
                wait_loads<G::Younger>();
                barrier();
                if (WG && s == 3 && t + 2 == turns && (halves & 1)) clear_group(halves - 1);
              }
              if (s == 3) {
                if (LOOSE && (tail & 1) && t + 2 == turns) clear_tail();
                trim(t + R);
                if constexpr (!LOOSE)
                  if ((t & 1) == 0 && t + 2 * G::Ahead < turns) load_scales((t >> 1) + G::Ahead);
              }
              read_step(tn, sn);
              if (s & 1) read_scales(2 * t + (s + 1) / 2);
            };
            // Where A's fragments are replaced one by one, the last of them has just been read: its
            // step's first products go ahead of the wait.
            const bool late = Roll && !WG && (s & 1);  // (the weight gradient's registers do not allow it)
            if (!late) advance();
            __builtin_amdgcn_sched_barrier(0);
            multiply<A8, B8, EXACT, MI, NI>(c, fa[Roll ? 0 : s & 1], fb[s & 1], sa, sb, s & 1, [&](int u) {
              if (late && u == 0) {
                pin();
                advance();
              }
              if constexpr (Roll) fa[0][u] = read_a(tn, sn, u);
              load_part(t, s, u);
            });
            pin();
            __builtin_amdgcn_sched_barrier(0);
            if (s & 1) select_scales();
          }
        }
        last_step(0);
        if (!LOOSE || last_steps > 1) {
          if constexpr (A8 || B8) {
            wait_loads<G::Younger>();
            barrier();
            if (WG && 2 * turns == halves) clear_group(halves - 1);
          }
          last_step(1);
          if (last_steps > 2) {
            last_step(2);
            if (!LOOSE || last_steps > 3) last_step(3);
          }
        }
      }
    }
    // Every wave is done with the slots: the next tile's first loads start before this one's
    // results are finished and stored, 32 rows at a time through LDS, so that rows leave as
    // whole runs.
    wait_loads<0>();
    barrier();
    constexpr int V = sizeof(T) == 2 ? 8 : 4, PerRow = 32 * NI / V, RowsAtOnce = 64 / PerRow;
    constexpr int Pieces = 8 * NI;  // 16-byte pieces of a parked row, exchanged so that no read or write collides
    float* park = reinterpret_cast<float*>(lds + G::Slot) + wave * 32 * 32 * NI;
    const int prow = lane / PerRow, pcol = lane % PerRow * V;
    const int64_t out_row = orow0 + 32 * MI * wm + 32 * MI / KS * kg + prow;
    // (two groups: each finishes half of the rows)
    constexpr int WaveRows = 32 * MI / KS;
    const int left = arows - 32 * MI * wm - WaveRows * kg, out_rows = (left < WaveRows ? left : WaveRows) - prow;
    constexpr int Runs = 32 / RowsAtOnce;
    RunEpilogue<T, V, (Runs < 4 ? Runs : 4)> out;
    const int64_t out_col = col0 + wn * 32 * NI + pcol;
    const int out_expert = expert;
    out.template start<RowsAtOnce>(p.ep, out_col, out_row, out_rows);
    const bool more = set_up(list_entry(entry + 1));
    if (more) start_first();
    out.fetch_bias(p.ep, out_expert, out_col);
    if constexpr (KS == 2) {
      // each group hands the other the rows that that one finishes, and adds what it gets
      float4* give = reinterpret_cast<float4*>(lds + G::Slot) + wave * 64 * 4 * NI + lane;
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& x = kg ? c[0][j] : c[1][j];
          give[64 * (4 * j + q)] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
        }
      wait_lds();
      barrier();
      const float4* take = reinterpret_cast<const float4*>(lds + G::Slot) + (wave ^ (2 * WN)) * 64 * 4 * NI + lane;
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 y = take[64 * (4 * j + q)];
          const f32x16& x = kg ? c[1][j] : c[0][j];
          const f32x16 keep = x;
          c[0][j][4 * q] = keep[4 * q] + y.x;
          c[0][j][4 * q + 1] = keep[4 * q + 1] + y.y;
          c[0][j][4 * q + 2] = keep[4 * q + 2] + y.z;
          c[0][j][4 * q + 3] = keep[4 * q + 3] + y.w;
        }
      wait_lds();
      barrier();
    }
#pragma unroll
    for (int i = 0; i < (KS == 2 ? 1 : MI); ++i) {
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<float4*>(park + r * 32 * NI + 4 * ((8 * j + 2 * q + h) ^ (r & (Pieces - 1)))) =
              make_float4(c[i][j][4 * q], c[i][j][4 * q + 1], c[i][j][4 * q + 2], c[i][j][4 * q + 3]);
      __builtin_amdgcn_wave_barrier();
      out.template finish<Runs, RowsAtOnce>(p.ep, [&](int k, float(&z)[V]) {
        const int row = prow + k * RowsAtOnce;
#pragma unroll
        for (int v = 0; v < V; v += 4) {
          const int at = row * 32 * NI + 4 * ((pcol / 4 + v / 4) ^ (row & (Pieces - 1)));
          const float4 x = *reinterpret_cast<const float4*>(park + at);
          z[v] = x.x, z[v + 1] = x.y, z[v + 2] = x.z, z[v + 3] = x.w;
        }
      });
      __builtin_amdgcn_wave_barrier();
    }
    if (!more) return;
    wait_lds();
    barrier();
  }
}

// The limit of a kernel's dynamic LDS belongs to the kernel on one device: raised at its first
// launch there (and again after a failure).
hipError_t allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& set) {
  int device = 0;
  if (const hipError_t e = hipGetDevice(&device); e != hipSuccess) return e;
  const uint64_t bit = device < 64 ? (uint64_t)1 << device : 0;
  if (set.load(std::memory_order_relaxed) & bit) return hipSuccess;
  const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess)
    set.fetch_or(bit, std::memory_order_relaxed);
  else
    (void)hipGetLastError();  // it is returned here
  return e;
}

template <bool A8, bool B8, bool EXACT, int MI, int NI, int WN, int KS, int R, bool LOOSE, bool WG, typename T>
hipError_t launch_tile(const MmLaunch& a, hipStream_t st) {
  using G = Tile<A8, B8, MI, NI, WN, KS, R, WG>;
  const int64_t col_tiles = ((WG ? a.k : a.n) + G::BN - 1) / G::BN;
  const int64_t row_tiles = WG          ? (a.n + G::BM - 1) / G::BM * a.groups
                            : a.offsets ? most_tiles(a.rows, a.groups, G::BM)
                                        : (a.rows + G::BM - 1) / G::BM;
  auto k = mm_tile_kernel<A8, B8, EXACT, MI, NI, WN, KS, R, LOOSE, WG, T>;
  static std::atomic<uint64_t> set{0};  // bit d: on device d
  if (const hipError_t e = allow_lds(reinterpret_cast<const void*>(k), G::Lds, set); e != hipSuccess) return e;
  const int64_t tiles = row_tiles * col_tiles, most = kCUs * (2 * G::Lds <= 160 * 1024 ? 2 : 1);
  k<<<dim3((uint32_t)(tiles < most ? tiles : most)), G::Threads, G::Lds, st>>>(a, (int)col_tiles);
  return hipGetLastError();
}

// Waves of 32 MI x 32 NI results, WN of them across, KS groups; the exact product's need the
// registers of a wave that has a SIMD for itself in the large tile (ENI, EWN), and those with
// FP8 rows of A that are not exact take KS8 groups.
template <int MI, int NI, int WN, int ENI, int EWN, int KS, int KS8, int R>
hipError_t launch_sized(const MmLaunch& a, hipStream_t st) {
  const bool f32 = a.ep.out_f32;
  if (a.a_fmt && a.b_fmt)
    return f32 ? launch_tile<true, true, true, MI, ENI, EWN, KS, R, false, false, float>(a, st)
               : launch_tile<true, true, false, MI, NI, WN, KS8, R, false, false, __bf16>(a, st);
  const bool loose = a.k % 128 || ((uintptr_t)a.a_scales | (uintptr_t)a.b_scales) % 4;
  if (a.a_fmt && loose)
    return f32 ? launch_tile<true, false, true, MI, ENI, EWN, KS, R, true, false, float>(a, st)
               : launch_tile<true, false, false, MI, NI, WN, KS8, R, true, false, __bf16>(a, st);
  if (a.a_fmt)
    return f32 ? launch_tile<true, false, true, MI, ENI, EWN, KS, R, false, false, float>(a, st)
               : launch_tile<true, false, false, MI, NI, WN, KS8, R, false, false, __bf16>(a, st);
  if (loose)
    return f32 ? launch_tile<false, false, false, MI, NI, WN, KS, R, true, false, float>(a, st)
               : launch_tile<false, false, false, MI, NI, WN, KS, R, true, false, __bf16>(a, st);
  return f32 ? launch_tile<false, false, false, MI, NI, WN, KS, R, false, false, float>(a, st)
             : launch_tile<false, false, false, MI, NI, WN, KS, R, false, false, __bf16>(a, st);
}

}  // namespace

hipError_t launch_gemm_tiles(const MmLaunch& a, int side, hipStream_t st) {
  if (side == 256) return launch_sized<4, 2, 4, 4, 2, 1, 1, 2>(a, st);
  return side == 128 ? launch_sized<2, 2, 2, 2, 2, 2, 1, 4>(a, st) : launch_sized<1, 1, 2, 1, 2, 1, 1, 4>(a, st);
}

int tile_side(int64_t rows, int64_t cols, int64_t experts, int64_t each) {
  const int64_t least = rows < experts ? rows : experts;
  auto rounds = [&](int64_t side, int64_t at_once) {
    const int64_t full = rows / side + experts / 2 + 1;
    const int64_t tiles = (full < least ? least : full) * ((cols + side - 1) / side) * each;
    return (tiles + at_once - 1) / at_once;
  };
  if (rounds(64, 2 * kCUs) == 1) return 64;
  return 22 * rounds(256, kCUs) <= 10 * rounds(128, kCUs) ? 256 : 128;
}

hipError_t launch_grouped_wgrad(const MmLaunch& a, hipStream_t st) {
  const bool f32 = a.ep.out_f32;
  switch (tile_side(a.n - 1, a.k, 0, a.groups)) {
    case 64:
      return f32 ? launch_tile<true, true, true, 1, 1, 2, 1, 4, false, true, float>(a, st)
                 : launch_tile<true, true, false, 1, 1, 2, 1, 4, false, true, __bf16>(a, st);
    case 128:
      return f32 ? launch_tile<true, true, true, 2, 2, 2, 2, 4, false, true, float>(a, st)
                 : launch_tile<true, true, false, 2, 2, 2, 1, 4, false, true, __bf16>(a, st);
    default:
      return f32 ? launch_tile<true, true, true, 4, 4, 2, 1, 2, false, true, float>(a, st)
                 : launch_tile<true, true, false, 4, 2, 4, 1, 2, false, true, __bf16>(a, st);
  }
}

}  // namespace mxq

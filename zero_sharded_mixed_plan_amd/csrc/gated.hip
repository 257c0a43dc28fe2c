// HIP kernels for gfx950 (CDNA4): the gated feed-forward block's two projections with
// the activation and the product in one kernel, and the products of its backward pass.
#include <algorithm>

#include "products.h"

namespace zk {
namespace {

// ---------------------------------------------------------------------------
// 16-bit types at multiples of 16 bytes
// ---------------------------------------------------------------------------

// Tiles of TILE x TILE results (of gate and up in the forward pass TILE x TILE / 2 each).
// A wave has XB x 2 blocks of 32 x 32 results.  The operands' tiles go from global memory
// straight into LDS (16 bytes a lane, no registers between), two to four steps of 32 of k
// before they are used: under load a copy takes a microsecond and more, a step of matrix
// instructions 0.6.
//
// Rows of k are copied 64 of k at a time, whole lines of the L2 (with half lines its
// requests doubled, and the 8192 x 4096 x 14336 forward pass took 1626 us in place of 1525).
// A deep tile can be refilled only when both of its steps have been read, two steps before it is
// needed; where both operands have them, the second has a third one, which fills the 160 KB of a CU:
// 1530 us with two and two, 1436 with three (1339 TFLOP/s).
// The DMA writes LDS in lane order, 1024 bytes a wave, so a lane fetches the unit that belongs
// at its place.
template <int TILE>
constexpr int kTileThreads = TILE == 256 ? 512 : 256;
template <int TILE, bool BY_K, bool DEEP>
constexpr int kTileBytes = TILE * kDeep<DEEP> * 2 + (TILE == 256 && !BY_K ? 512 : 0);
// This thread's place of round q in an operand's tile: byte offset from the tile's first element.
// i0, ni: the tile's first row (column) and the matrix's number of them, beyond which the last
// ones stand in (what they give is not stored).
template <int TILE, bool BY_K>
__device__ __forceinline__ u32 place_of(int q, int64_t ld, int64_t i0, int64_t ni) {
  constexpr u32 kN = kTileThreads<TILE>;
  const u32 t = threadIdx.x;
  if constexpr (BY_K) {
    const u32 row = q * (kN / 8) + t / 8;
    return (u32)min((int64_t)row, ni - 1 - i0) * (u32)ld + ((t % 8) ^ (t / 16 % 8)) * 16;
  } else {
    constexpr u32 kUnits = TILE / 8;
    const u32 k = q * (kN / kUnits) + t / kUnits;
    const u32 col = ((t % kUnits) ^ swizzle<TILE>(k)) * 8;
    return k * (u32)ld + (u32)min((int64_t)col, ni - 8 - i0) * 2;
  }
}
// Whether it lies within the last `left` of k.
template <int TILE, bool BY_K>
__device__ __forceinline__ bool inside(int q, int left) {
  constexpr u32 kN = kTileThreads<TILE>, kUnits = TILE / 8;
  u32 t = threadIdx.x;
  asm volatile("" : "+v"(t));  // what this needs is not held in registers through the loop
  return (int)(BY_K ? ((t % 8) ^ (t / 16 % 8)) * 8 : q * (kN / kUnits) + t / kUnits) < left;
}

// What copies read from: bytes from p on, by 32-bit offsets.  A buffer descriptor costs a copy no vector
// instruction and no register for its address.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const char* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, 0x7fffffff, 0x00020000);
}

// Starts the copy of round q.  PART: the last of k, beyond whose `left` there are zeros.
template <int TILE, bool BY_K, bool PART>
__device__ __forceinline__ void copy_place(char* lds, __amdgpu_buffer_rsrc_t from, u32 off, int q, int left) {
  constexpr u32 kN = kTileThreads<TILE>;
  char* const to = lds + chunk_at<TILE, BY_K>(q * (kN / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64));
  if (!PART || inside<TILE, BY_K>(q, left)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, off, 0, 0, 0);
  } else {
    u32 t = threadIdx.x, zero = 0;
    asm volatile("" : "+v"(t), "+v"(zero));
    *reinterpret_cast<vec4*>(to + t % 64 * 16) = vec4{zero, zero, zero, zero};
  }
}

// All but the newest LATER copies have arrived, for every wave, and every wave's reads are done.
template <int LATER>
__device__ __forceinline__ void turn() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x70 | (LATER & 15) | (LATER >> 4) << 14);  // vmcnt(LATER) lgkmcnt(0), known to the compiler, which adds no others
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Orders the scheduling region: one matrix instruction, one of the copies, EACH reads of LDS, and so on.
template <int MFMA, int COPIES, int READS, int EACH>
__device__ __forceinline__ void interleave() {
  if constexpr (MFMA > 0) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (COPIES > 0) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    if constexpr (READS > 0) __builtin_amdgcn_sched_group_barrier(0x100, READS < EACH ? READS : EACH, 0);
    interleave<MFMA - 1, (COPIES > 0 ? COPIES - 1 : 0), (READS > EACH ? READS - EACH : 0), EACH>();
  }
}

// f(0), f(1) .. f(N - 1), as constants
template <int N, int J = 0, class F>
__device__ __forceinline__ void each_step(F&& f) {
  f(std::integral_constant<int, J>{});
  if constexpr (J + 1 < N) each_step<N, J + 1>(f);
}

template <class T, Product KIND, int TILE, bool ALONE>
__global__ __launch_bounds__(kTileThreads<TILE>) void tiled_kernel(const ProductLaunch a, u32 down, u32 across, u32 splits) {
  constexpr bool kQByK = KIND != kWeight, kPByK = KIND == kForward;
  constexpr int WC = 2, WR = TILE == 256 ? 4 : 2;
  constexpr int XB = TILE / WC / 32, YB = TILE / WR / 32;
  constexpr u32 kCols = KIND == kForward ? TILE / 2 : TILE;  // columns of the results
  // Names of their own, so that the compiler sees that reads of one and copies to another do not
  // meet, and waits for none of them; it tells seven apart.  An operand has two deep tiles (of the forward
  // pass's two the second has three), or four; where a tile is alone on its CU four deep ones.
  static_assert(!ALONE || TILE == 128, "tiles of 256 have no room for more");
  constexpr bool kPDeep = kPByK || ALONE, kQDeep = kQByK || ALONE, kThree = kPByK && kQByK && !ALONE;
  constexpr int kPTiles = kPDeep && !ALONE ? 2 : 4, kQTiles = kThree ? 3 : kQDeep && !ALONE ? 2 : 4;
  constexpr int kP = kTileBytes<TILE, kPByK, kPDeep>, kQ = kTileBytes<TILE, kQByK, kQDeep>;
  constexpr bool kEight = kPTiles + kQTiles == 8;
  __shared__ __attribute__((aligned(128))) char p1[kP], p2[kPTiles > 2 ? kP : 16], p3[kPTiles > 3 ? kP : 16];
  __shared__ __attribute__((aligned(128))) char q1[kQ], q2[kQTiles > 2 ? kQ : 16], q3[kQTiles > 3 ? kQ : 16];
  __shared__ __attribute__((aligned(128))) char p0[kEight ? kP + kQ : kP], q0[kEight ? 16 : kQ];
  u32 tr, tc;
  const u32 halves = KIND == kWeight ? 2 : 1;
  const u32 split = KIND == kForward ? 0 : blockIdx.x / (down * halves * across);
  tile_of(KIND == kForward ? blockIdx.x : blockIdx.x % (down * halves * across), down * halves, across, tr, tc);
  const int which = KIND == kWeight && tr >= down;
  const int64_t r0 = (int64_t)(tr - which * down) * TILE, c0 = (int64_t)tc * kCols;
  const u32 wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const u32 wc = wave % WC, wr = wave / WC;

  constexpr int kRP = kRounds<kPDeep>, kRQ = kRounds<kQDeep>;
  u32 op[kRP], oq[kRQ];
#pragma unroll
  for (int i = 0; i < kRP; ++i)  // in the forward pass gate's columns, then up's
    op[i] = place_of<TILE, kPByK>(KIND == kForward ? i % (kRP / 2) : i, a.ld_p[0], c0, a.cols);
#pragma unroll
  for (int i = 0; i < kRQ; ++i) oq[i] = place_of<TILE, kQByK>(i, a.ld_q[0], r0, a.rows);
  u32 at_p[XB], at_q[YB];
  block_offsets<TILE, kQByK>(at_q, wr * YB * 32);
  if constexpr (KIND == kForward) {  // blocks of gate, then of up
    u32 gate[XB / 2];
    block_offsets<TILE, kPByK>(gate, wc * (XB / 2) * 32);
#pragma unroll
    for (int x = 0; x < XB; ++x) at_p[x] = gate[x % (XB / 2)] + x / (XB / 2) * (TILE / 2) * 128;
  } else {
    block_offsets<TILE, kPByK>(at_p, wc * XB * 32);
  }
  f32x16 acc[XB][YB] = {};
  struct Fragments {
    i16x8 p[kStep / 16][XB], q[kStep / 16][YB];
  };
  // a split has a run of the 64s of k, in the input gradient of gate's and then up's
  constexpr u32 kParts = KIND == kInput ? 2 : 1;
  const u32 units = (u32)((a.k + 63) / 64);
  const u32 from = (u32)((u64)units * kParts * split / splits), to = (u32)((u64)units * kParts * (split + 1) / splits);
  for (u32 part = 0; part < kParts; ++part) {
    const u32 lo = max(from, part * units) - part * units, hi = min(to, (part + 1) * units) - part * units;
    if (KIND != kForward && (from >= (part + 1) * units || to <= part * units)) continue;
    const int64_t k_lo = KIND == kForward ? 0 : (int64_t)lo * 64;
    const int k = (int)((KIND == kForward ? a.k : min(a.k, (int64_t)hi * 64)) - k_lo);
    const u32 steps = (u32)(k + kStep - 1) / kStep, whole = (u32)k / kStep;
    const u32 iq = KIND == kWeight ? which : part, ip = KIND == kInput ? part : 0;
    // where the next copies begin, how far a copy goes, and what is left of k there
    const char* next_q = a.q[iq] + (kQByK ? r0 * a.ld_q[0] + k_lo * 2 : k_lo * a.ld_q[0] + r0 * 2);
    const char* next_p[2] = {a.p[ip] + (kPByK ? c0 * a.ld_p[0] + k_lo * 2 : k_lo * a.ld_p[0] + c0 * 2),
                             KIND == kForward ? a.p[1] + c0 * a.ld_p[0] : nullptr};
    const int64_t far_q = kDeep<kQDeep> * (kQByK ? 2 : a.ld_q[0]), far_p = kDeep<kPDeep> * (kPByK ? 2 : a.ld_p[0]);
    int left_p = k, left_q = k;
    auto copy_p = [&](char* to, auto all_whole) {
      auto start = [&](auto is_part) {
#pragma unroll
        for (int i = 0; i < kRP; ++i)
          copy_place<TILE, kPByK, decltype(is_part)::value>(to, buffer_at(next_p[KIND == kForward ? i / (kRP / 2) : 0]), op[i], i,
                                                            left_p);
      };
      if (decltype(all_whole)::value || left_p >= kDeep<kPDeep>) start(std::false_type{});
      else start(std::true_type{});
      next_p[0] += far_p;
      if constexpr (KIND == kForward) next_p[1] += far_p;
      left_p -= kDeep<kPDeep>;
    };
    auto copy_q = [&](char* to, auto all_whole) {
      auto start = [&](auto is_part) {
#pragma unroll
        for (int i = 0; i < kRQ; ++i) copy_place<TILE, kQByK, decltype(is_part)::value>(to, buffer_at(next_q), oq[i], i, left_q);
      };
      if (decltype(all_whole)::value || left_q >= kDeep<kQDeep>) start(std::false_type{});
      else start(std::true_type{});
      next_q += far_q;
      left_q -= kDeep<kQDeep>;
    };
    // Steps go round J = 0 .. kRound - 1.  The tile of step J, or of two steps where it is deep:
    auto tile_p = [&](auto j) -> char* {
      constexpr int J = (kPDeep ? decltype(j)::value / 2 : decltype(j)::value) % kPTiles;
      return J == 0 ? p0 : J == 1 ? p1 : J == 2 ? p2 : p3;
    };
    auto tile_q = [&](auto j) -> char* {
      constexpr int J = (kQDeep ? decltype(j)::value / 2 : decltype(j)::value) % kQTiles;
      return J == 0 ? (kEight ? p0 + kP : q0) : J == 1 ? q1 : J == 2 ? q2 : q3;
    };
    auto read = [&](auto j, Fragments& f) {
      constexpr u32 J = decltype(j)::value;
#pragma unroll
      for (u32 s = 0; s < kStep / 16; ++s) {
#pragma unroll
        for (int y = 0; y < YB; ++y)
          f.q[s][y] = fragment<TILE, kQByK>(tile_q(j), at_q[y], s + (kQDeep ? J % 2 * 2 : 0));
#pragma unroll
        for (int x = 0; x < XB; ++x)
          f.p[s][x] = fragment<TILE, kPByK>(tile_p(j), at_p[x], s + (kPDeep ? J % 2 * 2 : 0));
      }
    };
    // A step multiplies fragments that are in registers, while those of the next one are read, and starts
    // the copies that fit into what has been read: a step's tile four steps ahead, or with its
    // second step a deep tile, kPFar (kQFar) steps ahead.  The second operand's third or fourth deep tile is
    // started by the step after that.
    constexpr bool kLater = kQTiles > 2 && kQDeep;
    constexpr u32 kPFar = kPDeep ? 2 * kPTiles - 1 : 4, kQFar = !kQDeep ? 4 : kLater ? 2 * kQTiles - 2 : 2 * kQTiles - 1;
    auto copies = [&](auto j, u32 s, auto all_whole) {
      constexpr int J = decltype(j)::value;
      if constexpr (!kPDeep || J % 2 == 1)
        if (decltype(all_whole)::value || s + kPFar < steps) copy_p(tile_p(std::integral_constant<int, J + kPFar>{}), all_whole);
      if constexpr (!kQDeep || J % 2 == (kLater ? 0 : 1))
        if (decltype(all_whole)::value || s + kQFar < steps) copy_q(tile_q(std::integral_constant<int, J + kQFar>{}), all_whole);
    };
    auto multiply_and_read = [&](auto j, const Fragments& f, Fragments& next) {
      constexpr int J = decltype(j)::value;
      read(std::integral_constant<int, J + 1>{}, next);
#pragma unroll
      for (u32 s = 0; s < kStep / 16; ++s)
#pragma unroll
        for (int x = 0; x < XB; ++x)
#pragma unroll
          for (int y = 0; y < YB; ++y) acc[x][y] = mfma32<T>(f.p[s][x], f.q[s][y], acc[x][y]);
      // a few reads behind each matrix instruction, so that neither waits for the other
      constexpr int kReads = kStep / 16 * ((kPByK ? 1 : 2) * XB + (kQByK ? 1 : 2) * YB);
      constexpr int kMfma = kStep / 16 * XB * YB;
      constexpr int kEach = (kReads + kMfma - 3) / (kMfma - 2);
      interleave<kMfma, (!kPDeep || J % 2 ? kRP : 0) + (!kQDeep || J % 2 == (kLater ? 0 : 1) ? kRQ : 0), kReads, kEach>();
    };
    // When step J is done, what the next one reads has arrived: deep tiles started by the step before an even
    // one; tiles of one step started two before; with four deep tiles what was started more than four steps before.
    constexpr int kEven = (kPDeep ? 0 : kRP) + (kQDeep && !kLater ? 0 : kRQ);  // copies started by an even step
    constexpr auto later = [](int J) { return ALONE ? 16 : (kPDeep || kQDeep) && J % 2 == 0 ? kEven : 8; };
    constexpr u32 kAhead = ALONE ? 9 : kThree ? 6 : 5;  // a step's copies lie within as many steps
    auto step = [&](auto j, const Fragments& f, Fragments& next) {
      constexpr int J = decltype(j)::value;
      copies(j, 0, std::true_type{});
      multiply_and_read(j, f, next);
      turn<later(J)>();
    };
    auto last_steps = [&](auto j, u32 s, const Fragments& f, Fragments& next) {
      if (s >= steps) return;
      copies(j, s, std::false_type{});
      multiply_and_read(j, f, next);
      if (s + kAhead <= whole) turn<later(decltype(j)::value)>();  // whole copies were started until now
      else turn<0>();
    };
    constexpr int kRound = ALONE ? 8 : kThree ? 12 : 4;
    Fragments f, g;
    // in the steps' order, but for what step 0 starts and later ones
    constexpr u32 kFirst = kPDeep || kQDeep ? (ALONE ? 8 : 4) : 4;
    each_step<kFirst>([&](auto j) {
      constexpr u32 J = decltype(j)::value;
      if (J > 0 && J >= steps) return;
      if constexpr (!kPDeep || J % 2 == 0) copy_p(tile_p(j), std::false_type{});
      if constexpr (!kQDeep || (J % 2 == 0 && (!kLater || J < kQFar))) copy_q(tile_q(j), std::false_type{});
    });
    constexpr int kBegun = ALONE ? 20 : 8;
    if (whole >= kFirst) turn<kBegun>();  // the later steps' copies may still be under way
    else turn<0>();
    read(std::integral_constant<int, 0>{}, f);
    turn<kBegun>();
    u32 s = 0;
    for (; s + kRound - 1 + kAhead <= whole; s += kRound)  // copies of whole steps only
      each_step<kRound>([&](auto j) {
        if constexpr (decltype(j)::value % 2 == 0) step(j, f, g);
        else step(j, g, f);
      });
#pragma unroll 1
    for (; s < steps; s += kRound)
      each_step<kRound>([&](auto j) {
        if constexpr (decltype(j)::value % 2 == 0) last_steps(j, s + decltype(j)::value, f, g);
        else last_steps(j, s + decltype(j)::value, g, f);
      });
  }

  // the results leave by way of LDS, where the copies no longer need it
  constexpr u32 kOf = kPByK ? 2 : 4, kEach = WC * WR / kOf;
  const u32 slot = wave / kEach;
  char* at_slot = slot == 0 ? p0 : p1;
  if constexpr (!kPByK) at_slot = slot == 2 ? p2 : slot == 3 ? p3 : at_slot;
  char* const mine = at_slot + wave % kEach * kStageBytes;
  finish_tile<T, KIND, XB, YB>(acc, mine, r0 + wr * YB * 32, c0 + wc * (KIND == kForward ? XB / 2 : XB) * 32, which, split, splits);
}

// ---------------------------------------------------------------------------
// a few tokens
// ---------------------------------------------------------------------------

// Every weight is read once, and what counts is the bytes in flight and that all CUs have a like share
// of them.  A workgroup has COLS columns of gate and of up, 16 or 32 (a block, where they are held in 8 bits); its waves take turns of 64 of k and work alone: each copies its
// turns' weights and tokens into LDS, whole lines, RING turns ahead, and waits for no other wave before its
// sums are added to theirs.  Weights loaded straight into the registers that the matrix
// instructions take them from, 16 bytes of every row a lane, reached half of the bandwidth: each
// lane of such a load is a line of its own to the L1.  TOKENS: a multiple of 16.
template <class T, int TOKENS, int COLS, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void few_kernel(const ProductLaunch a) {
  constexpr int N = TOKENS / 16, H = COLS / 16, kRing = N <= 2 ? 3 : 2;
  constexpr int kTurnBytes = (2 * COLS + TOKENS) * 128;  // rows of gate, of up, of tokens
  constexpr int kCopies = kTurnBytes / 1024;
  __shared__ __attribute__((aligned(128))) char s0[WAVES * kTurnBytes], s1[WAVES * kTurnBytes],
      s2[kRing > 2 ? WAVES * kTurnBytes : 16];
  const u32 lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t c0 = (int64_t)blockIdx.x * COLS;
  // Chunk i of 8 rows: lane l fetches the unit of row 8 i + l / 8 whose place is l % 8 (unit j of row r at
  // j ^ (r / 2 % 8)).  Rows beyond the last stand for it.
  u32 off[COLS / 8], off_x[2 * N];
#pragma unroll
  for (u32 i = 0; i < COLS / 8; ++i)
    off[i] = (u32)min((int64_t)(8 * i + lane / 8), a.cols - 1 - c0) * (u32)a.ld_p[0] + ((lane % 8) ^ ((4 * i + lane / 16) % 8)) * 16;
#pragma unroll
  for (u32 i = 0; i < 2 * N; ++i)
    off_x[i] = (u32)min((int64_t)(8 * i + lane / 8), a.rows - 1) * (u32)a.ld_q[0] + ((lane % 8) ^ ((4 * i + lane / 16) % 8)) * 16;
  u32 at = wave * kTurnBytes + lane % 16 * 128 + ((lane / 16) ^ (lane / 2 % 8)) * 16;  // 16 rows further: + 2048
  asm("" : "+v"(at));

  auto copy = [&](char* slot, int64_t u) {
    const int64_t left = a.k - u * 64;
    auto start = [&](auto is_part) {
      auto one = [&](__amdgpu_buffer_rsrc_t from, u32 from_off, u32 i, u32 chunk) {
        char* const to = slot + wave * kTurnBytes + chunk * 1024;
        if (!decltype(is_part)::value || (int64_t)(((lane % 8) ^ ((4 * i + lane / 16) % 8)) * 8) < left)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, from_off, 0, 0, 0);
        else
          *reinterpret_cast<vec4*>(to + lane * 16) = vec4{0, 0, 0, 0};  // beyond the end of k
      };
#pragma unroll
      for (u32 m = 0; m < 2; ++m)
#pragma unroll
        for (u32 i = 0; i < COLS / 8; ++i) one(buffer_at(a.p[m] + c0 * a.ld_p[0] + u * 128), off[i], i, COLS / 8 * m + i);
#pragma unroll
      for (u32 i = 0; i < 2 * N; ++i) one(buffer_at(a.q[0] + u * 128), off_x[i], i, COLS / 4 + i);
    };
    if (left >= 64) start(std::false_type{});
    else start(std::true_type{});
  };
  f32x4 acc[2][H][N] = {};
  // this wave's turns are 64 of k from 64 (wave + WAVES i) on
  const int64_t all = (a.k + 63) / 64, turns = (all - wave + WAVES - 1) / WAVES;
  const int64_t whole = (a.k / 64 - wave + WAVES - 1) / WAVES;  // of them without an end of k inside
  auto turn = [&](char* slot, int64_t i) {
    if (i >= turns) return;
    // the ring's other turns may be under way still; one with an end of k inside starts fewer copies
    if (i + kRing - 1 < whole) __builtin_amdgcn_s_waitcnt(0x70 | ((kRing - 1) * kCopies & 15) | ((kRing - 1) * kCopies >> 4) << 14);
    else __builtin_amdgcn_s_waitcnt(0x70);
    i16x8 w[2][H][2], x[N][2];
#pragma unroll
    for (u32 s = 0; s < 2; ++s) {
#pragma unroll
      for (u32 m = 0; m < 2; ++m)
#pragma unroll
        for (u32 h = 0; h < H; ++h) w[m][h][s] = *reinterpret_cast<const i16x8*>(slot + ((at ^ (s * 64)) + (H * m + h) * 2048));
#pragma unroll
      for (int t = 0; t < N; ++t) x[t][s] = *reinterpret_cast<const i16x8*>(slot + ((at ^ (s * 64)) + (2 * H + t) * 2048));
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): what was read may be written over
    asm volatile("" ::: "memory");
    if (i + kRing < turns) copy(slot, wave + WAVES * (i + kRing));
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < N; ++t)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < H; ++h) acc[m][h][t] = mfma16<T>(w[m][h][s], x[t][s], acc[m][h][t]);
  };
  if (0 < turns) copy(s0, wave);
  if (1 < turns) copy(s1, wave + WAVES);
  if (kRing > 2 && 2 < turns) copy(s2, wave + 2 * WAVES);
#pragma unroll 1
  for (int64_t i = 0; i < turns; i += kRing) {
    turn(s0, i);
    turn(s1, i + 1);
    if constexpr (kRing > 2) turn(s2, i + 2);
  }

  static_assert(2 * TOKENS * COLS * 4 <= kTurnBytes, "the sums fit where the copies were");
  finish_few<T, TOKENS, COLS, WAVES>(acc, reinterpret_cast<float*>(s0), a, c0);
}

template <class T, int TOKENS>
int few_as(const ProductLaunch& a, hipStream_t s) {
  auto go = [&](auto columns, auto waves) {
    constexpr int C = decltype(columns)::value, W = decltype(waves)::value;
    hipLaunchKernelGGL((few_kernel<T, TOKENS, C, W>), dim3((u32)((a.cols + C - 1) / C)), dim3(W * 64), 0, s, a);
  };
  using Two = std::integral_constant<int, 2>;
  using Four = std::integral_constant<int, 4>;
  const bool many = a.cols > 16 * 512;  // more than two workgroups a CU
  // With 64 tokens their rows are more than the weights' of 16 columns, and a workgroup of four waves has a CU
  // to itself.  Several sets of weights in turn, so that they come from HBM: 64 tokens, 4096 x 14336 53 us with 32
  // columns, 64 with 16, 4096 x 11008 48 and 50, 40 tokens, 4096 x 8000 30 and 33; but 2048 x 4000 15.5 and
  // 11.8, 512 x 1376 6.7 and 4.1: few columns need the workgroups.  Between them 4096 x 5504 takes 27.5 and 32.0, or
  // 27.4 and 24.9 from the last-level cache.  16 tokens, 4096 x 14336 45 and 45, 4096 x 11008 39.7 and 35.7.
  if ((TOKENS == 64 && a.cols > 16 * 384) || a.held[0].codes) {
    a.cols > 32 * 256 ? go(std::integral_constant<int, 32>{}, Two{}) : go(std::integral_constant<int, 32>{}, Four{});
  } else if constexpr (TOKENS == 64) {
    go(std::integral_constant<int, 16>{}, Four{});
  } else {
    many ? go(std::integral_constant<int, 16>{}, Two{}) : go(std::integral_constant<int, 16>{}, Four{});
  }
  return launched("gated projections");
}

// Whether the copies of 16 bytes find whole units: addresses, strides, and the lengths
// along which an operand's rows lie.  Offsets within a tile are 32 bits.
bool tiles_fit(Product kind, const ProductLaunch& a) {
  auto ok = [](const char* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 16 == 0 && ld < (1 << 22); };
  const int nq = kind == kForward ? 1 : 2, np = kind == kWeight ? 1 : 2;
  for (int i = 0; i < nq; ++i)
    if (!ok(a.q[i], a.ld_q[i])) return false;
  for (int i = 0; i < np; ++i)
    if (!ok(a.p[i], a.ld_p[i])) return false;
  const bool q_by_k = kind != kWeight, p_by_k = kind == kForward;
  if (a.k < 1 || a.ld_p[0] != a.ld_p[np - 1] || a.ld_q[0] != a.ld_q[nq - 1]) return false;
  return (q_by_k ? a.k : a.rows) % 8 == 0 && (p_by_k ? a.k : a.cols) % 8 == 0;
}

// The size of the tiles and the number of splits of k.  Few tiles leave CUs without work; splits of a long k
// give it to them, at the price of fp32 partial results that are written and read once more.  The
// estimate is of microseconds, from these measurements: 64 of k take a tile of 256 1.5, of
// 128 0.4 alone on a CU and 0.95 where two share it (the 8192 x 4096 x 14336 forward pass 1498 us with
// tiles of 256, 1873 with 128); a tile begins and ends in 8 and 5; partial results move at 5 TB/s,
// and another launch takes 3.
// Where no tile of 128 shares its CU, nothing covers its waits; four deep tiles an operand, in LDS that no other
// workgroup needs, have copies under way for seven steps: 128 tokens, 4096 x 11008, forward 57.7 -> 51.2 us with
// weights from HBM (35.5 -> 31.8 from the last-level cache); input gradient of 1024 tokens there 251 -> 203, of 4096
// tokens, 768 x 2048, 49.6 -> 38.5. The weight gradient gains nothing (173 and 173, 55.3 and 55.8), short sums lose (300
// tokens, 512 x 1376: 6.6 and 7.1, 12.0 and 12.8).
// The estimate is low where sums are short: 8192 x 512 x 1376 it gives 23 us for the input gradient and 31 for the
// weight gradient's products, which take 29 to 33 and 32 to 35.
struct TilePlan {
  int tile;
  u32 splits;
  bool alone;
};

TilePlan tile_plan(Product kind, const ProductLaunch& a) {
  const int64_t halves = kind == kWeight ? 2 : 1, units = (a.k + 63) / 64 * (kind == kInput ? 2 : 1);
  const int64_t bytes = halves * a.rows * a.cols * 4;
  TilePlan best{128, 1, false};
  double least = 1e300;
  for (int tile : {128, 256}) {
    const int64_t cols = kind == kForward ? tile / 2 : tile;
    const int64_t tiles = (a.rows + tile - 1) / tile * ((a.cols + cols - 1) / cols) * halves;
    for (u32 n = 1; n <= kMaxSplits / 2; ++n) {
      if (n > 1 && (kind == kForward || units / n < 4 || bytes > kMaxPartialBytes / n || a.cols % 8 != 0)) break;
      const int64_t groups = tiles * n;
      double each, begin, rounds;
      if (tile == 256) each = 1.5, begin = 8.0, rounds = (double)((groups + 255) / 256);
      else if (groups <= 256) each = 0.4, begin = 5.0, rounds = 1.0;
      else each = 0.95, begin = 5.0, rounds = (double)((groups + 511) / 512);
      double t = rounds * (each * (double)units / n + begin);
      if (n > 1) t += 3.0 + 2.0 * n * (double)bytes / 5e6;
      if (t < least) {
        least = t;
        best = TilePlan{tile, n, kind != kWeight && tile == 128 && groups <= 256 && units / n >= 32};
      }
    }
  }
  return best;
}

template <class T, Product KIND, int TILE, bool ALONE>
int tiled_as(const ProductLaunch& a, u32 splits, hipStream_t s) {
  constexpr int cols = KIND == kForward ? TILE / 2 : TILE;
  const u32 down = (u32)((a.rows + TILE - 1) / TILE), across = (u32)((a.cols + cols - 1) / cols);
  hipLaunchKernelGGL((tiled_kernel<T, KIND, TILE, ALONE>), dim3(down * across * (KIND == kWeight ? 2 : 1) * splits),
                     dim3(kTileThreads<TILE>), 0, s, a, down, across, splits);
  return launched(KIND == kForward ? "gated projections" : KIND == kInput ? "gated input gradient" : "gated weight gradient");
}

template <class T, Product KIND>
int tiled_of(const ProductLaunch& a, hipStream_t s) {
  if constexpr (KIND == kForward) {
    // With weights from HBM, tiles take longer but for the widest layers: one token, 4096 x 11008 35.7 us and 41.3; 64
    // tokens 512 x 1376 4.1 and 8.3, 2048 x 4000 11.7 and 19.8, 4096 x 5504 32 and 36, 4096 x 11008 48 and 44, 4096 x 14336
    // 53 and 50 (from the last-level cache 36 and 30, 42 and 37).
    if (a.rows <= 16) return few_as<T, 16>(a, s);
    if (a.rows <= 32) return few_as<T, 32>(a, s);
    if (a.rows <= 64) return few_as<T, 64>(a, s);
  }
  const TilePlan plan = tile_plan(KIND, a);
  if (int rc = plan.tile == 256 ? tiled_as<T, KIND, 256, false>(a, plan.splits, s)
               : plan.alone     ? tiled_as<T, KIND, 128, KIND != kWeight>(a, plan.splits, s)
                                : tiled_as<T, KIND, 128, false>(a, plan.splits, s))
    return rc;
  return plan.splits > 1 ? launch_join(KIND, a, std::is_same<T, BF16>::value ? ZERO_BF16 : ZERO_F16, plan.splits, s) : ZERO_OK;
}

template <Product KIND>
int product_of(const ProductLaunch& a, zero_dtype_t t, hipStream_t s) {
  if (t == ZERO_F32 || !tiles_fit(KIND, a)) return launch_product_any(KIND, a, t, s);
  return t == ZERO_BF16 ? tiled_of<BF16, KIND>(a, s) : tiled_of<F16, KIND>(a, s);
}

// A launch has fewer than 2^32 threads: larger results are taken in parts.
constexpr int64_t kMostSide = int64_t(1) << 18;

ProductLaunch part_of(Product kind, const ProductLaunch& a, zero_dtype_t t, int64_t r, int64_t c) {
  const int64_t eb = t == ZERO_F32 ? 4 : 2, ob = kind == kWeight && a.out_type == ZERO_F32 ? 4 : kind == kWeight ? 2 : eb;
  ProductLaunch b = a;
  for (int i = 0; i < 2; ++i) {
    if (b.q[i]) b.q[i] += r * (kind == kWeight ? eb : b.ld_q[i]);
    if (b.p[i]) b.p[i] += c * (kind == kForward ? b.ld_p[i] : eb);
    if (b.out[i]) b.out[i] += r * b.ld_out[i] + c * ob;
    if (b.kept[i]) b.kept[i] += r * b.ld_kept[i] + c * eb;
    if (b.held[i].codes) {
      b.held[i].codes += r * b.held[i].ld_codes + c;
      b.held[i].scales += r * b.held[i].ld_scales + c / kBlock;
    }
  }
  b.rows = std::min(kMostSide, a.rows - r);
  b.cols = std::min(kMostSide, a.cols - c);
  return b;
}

}  // namespace

int64_t product_ws_bytes(int64_t tokens, int64_t dim, int64_t hidden) {
  const double most = 4.0 * kMaxSplits * (double)partial_cols(dim) * (double)std::max(tokens, 2 * hidden);
  return most < (double)kMaxPartialBytes ? (int64_t)most : kMaxPartialBytes;
}

int launch_product(Product kind, const ProductLaunch& a, zero_dtype_t t, void* stream) {
  for (int64_t r = 0; r < a.rows; r += kMostSide)
    for (int64_t c = 0; c < a.cols; c += kMostSide) {
      const ProductLaunch b = part_of(kind, a, t, r, c);
      const hipStream_t s = (hipStream_t)stream;
      if (int rc = kind == kForward  ? product_of<kForward>(b, t, s)
                   : kind == kInput ? product_of<kInput>(b, t, s)
                                    : product_of<kWeight>(b, t, s))
        return rc;
    }
  return ZERO_OK;
}

}  // namespace zk

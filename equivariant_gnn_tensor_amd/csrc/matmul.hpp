// Matrix products on the gfx950 matrix cores with the dense layer's epilogue (templates;
// matmul_*.hip hold the instantiations of one element type each).
//
//   C(m, n) = epilogue(sum_k A(m, k) B(k, n)),  sums in fp32
//
// An operand is either contiguous along k ("rows": A[m lda + k], B[n ldb + k]) or along its
// other index ("columns": A[k lda + m], B[k ldb + n]).  The layer's three products need three
// of the four pairs (MatmulForm).
//
// A workgroup owns a BM x BN tile of C and walks k in slices of 128 bytes (64 elements of 16
// bits, 32 of 32) through a ring of slices in LDS.
//   LDS, rows: [row][8 chunks of 16 bytes], chunk c of row r at c ^ (r / 2 mod 8).  The 64 banks
//   hold two rows, and a fragment read takes one chunk of each of 16 rows at a time: the exclusive
//   or puts those of the eight even (odd) rows on different banks (with r mod 8 half of all LDS
//   cycles were conflicts).
//   LDS, columns: [k][columns].  16-bit fragments hold eight k of one column, so they are read
//   with the transposing LDS load, 32 bytes of each of four k and two neighbouring blocks at a
//   time, which an exclusive or of the block with k spreads over all banks.  fp32 fragments are
//   one number a lane.
// Slices come in by loads that write LDS directly, kGrain bytes a lane: 16 where both operands are
// aligned to it and hold whole chunks, 4 where they allow that (fp32 always, 16-bit rows of even
// length and stride).  They need no registers, and what lies past the end is cleared by their range
// check.  Anything else (kGrain 0) goes through registers, chunk by chunk, ends masked.
//
// v_mfma_f32_32x32x16 (16 bits) and v_mfma_f32_32x32x2 (fp32) take B's fragment first, so a
// lane ends up with four adjacent columns of one row at a time; the epilogue turns them over
// to whole row segments through LDS and is then plain row code: bias, pre-activation,
// activation, residual, one rounding, 16-byte accesses of any alignment.
//
// Tiles: 256 x 256 by eight waves of 128 x 64 (16 bits), 128 x 128 by four of 64 x 64, 64 x 64 by four of
// 32 x 32; matmul_shape chooses.  8192 x 8192 -> 8192 f16: 880 us, 1250 TFLOP/s with the first
// (LDS busy a quarter of the time, the matrix pipes 76 %, the clock held at about 1.6 GHz by power),
// 1057 with the second; 256 x 128 tiles of half slices, two workgroups a CU, 971.
// 65408 x 1024 -> 4096 bf16 501 us (1095), 65408 x 1024 -> 1024 fp32 989 us (139; the matrix
// instructions' peak is 157).  The large tile's results cost 50 us of the 501 (LDS) and 25 (stores).
#pragma once

#include <algorithm>
#include <type_traits>

#include "activation.hpp"
#include "fragments.hpp"
#include "linear.hpp"
#include "rows.hpp"

namespace etpc {
namespace mm {

// kGrain bytes a lane from base + off (zeros past the range) to LDS from `lds` on, lane after lane.  In
// assembly, so that the compiler's own counting of loads does not wait for more of them (and of the
// epilogue's stores among them) than barrier_after_loads; nothing but LDS and m0 is written (the
// compiler keeps nothing in m0: it sets it before each use); the wait states cover m0 and scalars that
// a vector instruction has just written.  What the compiler counts itself is only waited for earlier.
typedef int Range __attribute__((ext_vector_type(4)));
template <int kGrain>
__device__ inline void load_lds(uint32_t lds, const Range& range, int off) {
  if (kGrain == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(range));
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(range));
}
__device__ inline uint32_t lds_address(const char* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)p));
}

// One operand's slice: SIDE rows (columns) of the tile by one slice of k.
template <class T, int SIDE, bool kCols, int kThreads>
struct Side {
  static constexpr int E = 16 / sizeof(T), BK = slice<T>();
  static constexpr int kBytes = SIDE * kSliceBytes;
  static constexpr int kPer = kBytes / 16 / kThreads;      // chunks a thread
  static constexpr int kRow = kCols ? SIDE / E : 8;        // chunks of a row in LDS
  static_assert(kPer >= 1 && kBytes % (16 * kThreads) == 0, "whole chunks for every thread");
  static_assert((kThreads / kRow) % (kCols ? 4 : 16) == 0, "a thread's chunks share their swizzle");

  // Logical chunk at place p of LDS row r.
  static __device__ inline int unswizzle(int p, int r) {
    if (!kCols) return p ^ ((r >> 1) & 7);
    return sizeof(T) == 2 ? p ^ spread(r) : p;
  }
  // Chunks of columns move in pairs (32 bytes, what the transposing load takes of one k).
  static __device__ inline int spread(int k) { return SIDE >= 128 ? (k & 3) << 2 : (k & 2) << 1; }

  // Reads slices from k0 on (first: the tile's first row or column) into LDS.
  template <int kGrain>
  struct Direct {
    static constexpr int kLoads = kPer * 16 / kGrain;
    int off[kLoads];
    const char* p;
    uint64_t left;        // bytes from p to the operand's end
    int64_t step;         // bytes of a slice
    static constexpr int kFar = 0x7ffffff0, kMost = 0x7fffff00;   // an offset out of any range
    // Row r in LDS and first element in it of load i.
    static __device__ inline int place(int i, int& r) {
      const int g = threadIdx.x + i * kThreads, q = g / (16 / kGrain);
      r = q / kRow;
      return unswizzle(q % kRow, r) * E + g % (16 / kGrain) * (kGrain / static_cast<int>(sizeof(T)));
    }
    __device__ inline void start(const T* base, int64_t ld, int64_t first, int n, int K, int k0) {
      const int64_t at = kCols ? k0 * ld + first : first * ld + k0;
      const int64_t all = kCols ? (K - 1) * ld + n : (n - 1) * ld + K;
      p = reinterpret_cast<const char*>(base + at);
      left = static_cast<uint64_t>((all - at) * static_cast<int64_t>(sizeof(T)));
      step = (kCols ? BK * ld : BK) * static_cast<int64_t>(sizeof(T));
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        int r;
        const int c = place(i, r);
        off[i] = (static_cast<int>(r * ld) + c) * static_cast<int>(sizeof(T));
      }
    }
    // With `have` k values from here to the end, fewer than a slice: chunks past it are read as zero,
    // in this and every later slice.
    __device__ inline void end(int have) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        int r;
        const int c = place(i, r);
        if ((kCols ? r : c) >= have) off[i] = kFar;
      }
    }
    // Load i of the slice; the last one moves on to the next slice.
    __device__ inline void issue(char* lds, int wave, int i) {
      const uint64_t at = reinterpret_cast<uint64_t>(p);
      const Range range = {static_cast<int>(at), static_cast<int>(at >> 32 & 0xffff),
                           left >= kMost ? kMost : static_cast<int>(left), 0x00020000};
      load_lds<kGrain>(lds_address(lds) + wave * 64 * kGrain + i * kThreads * kGrain, range, off[i]);
      if (i == kLoads - 1) {
        p += step;
        left -= static_cast<uint64_t>(step);
      }
    }
    __device__ inline void commit(char*) {}
  };

  // Slices that lie inside the operand as a whole are plain 16-byte loads of any alignment; others go
  // chunk by chunk, ends masked.
  struct Staged {
    static constexpr int kLoads = 1;   // all at once
    Chunk t[kPer];
    int64_t off[kPer];
    const T* p;
    int64_t ld, first, k0;
    int n, K;
    __device__ inline void start(const T* base, int64_t ld_, int64_t first_, int n_, int K_, int k0_) {
      p = base, ld = ld_, first = first_, n = n_, K = K_, k0 = k0_;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int q = threadIdx.x + i * kThreads, r = q / kRow, c = unswizzle(q % kRow, r) * E;
        off[i] = kCols ? r * ld + first + c : (first + r) * ld + c;
      }
    }
    __device__ inline void end(int) {}
    __device__ inline void issue(char*, int, int) {
      const T* const at = p + (kCols ? k0 * ld : k0);
      if (k0 + BK <= K && first + SIDE <= n) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) __builtin_memcpy(&t[i], at + off[i], 16);
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int q = threadIdx.x + i * kThreads, r = q / kRow, c = unswizzle(q % kRow, r) * E;
          t[i] = Chunk{};
          if (kCols) {
            if (k0 + r < K) t[i] = fetch_chunk(p + (k0 + r) * ld, static_cast<int>(first) + c, n);
          } else {
            if (first + r < n) t[i] = fetch_chunk(p + (first + r) * ld, static_cast<int>(min<int64_t>(k0 + c, K)), K);
          }
        }
      }
      k0 += BK;
    }
    __device__ inline void commit(char* lds) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        *reinterpret_cast<Chunk*>(lds + (threadIdx.x + i * kThreads) * 16) = t[i];
    }
  };

  // Fragment: 16 bytes a lane, k = 2E s + E (lane / 32) .., index at + lane % 32.
  static __device__ inline Chunk fragment(const char* lds, int at, int s, int lane) {
    const int h = lane >> 5;
    if (!kCols) {
      const int r = at + (lane & 31);
      return *reinterpret_cast<const Chunk*>(lds + r * 128 + (((2 * s + h) ^ ((r >> 1) & 7)) << 4));
    }
    Chunk t;
    if (sizeof(T) == 2) {
      const int k = 16 * s + 8 * h + ((lane & 15) >> 2);
      const int col = at + (lane & 16) + (lane & 3) * 4;
      const int place = (((col >> 3) ^ spread(k)) << 4) + ((col & 7) << 1);
      const char* p = lds + k * (SIDE * 2) + place;
      const Tr4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsTr4*)p);
      const Tr4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsTr4*)(p + 4 * (SIDE * 2)));
      __builtin_memcpy(&t, &lo, 8);
      __builtin_memcpy(reinterpret_cast<char*>(&t) + 8, &hi, 8);
    } else {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(lds) + (8 * s + 4 * h) * SIDE + at + (lane & 31);
#pragma unroll
      for (int j = 0; j < 4; ++j) t[j] = p[j * SIDE];
    }
    return t;
  }
};

// Barrier after which every wave's loads into LDS, but for its kPending youngest loads and stores,
// have arrived, and its reads and writes of LDS are done.  (The library's barrier would wait for
// loads into LDS in some places and for all loads in others.)
template <int kPending>
__device__ inline void barrier_after_loads() {
  static_assert(kPending < 64, "six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (kPending & 15) | (kPending >> 4) << 14);   // vmcnt(kPending) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

__device__ inline void barrier_after_reads() { barrier_after_loads<63>(); }

// Where chunk c (four floats) of row r lies among a wave's 32 x TN results on their way out: writes
// take one chunk of 16 rows at a time, reads all of one or two rows, both from all banks.
template <int TN>
__device__ inline int turn_at(int r, int c) {
  return r * TN + ((c ^ (TN == 64 ? r & 15 : (r >> 1) & 7)) << 2);
}

// Tile of id (bands of eight tile rows, so that the tiles that run together share rows and columns).
__device__ inline void place_tile(int id, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int band = id / (8 * tiles_n), in = id - band * 8 * tiles_n, high = min(8, tiles_m - 8 * band);
  tn = in / high;
  tm = 8 * band + in - tn * high;
}

template <class T, int BM, int BN, int WM, int WN, int kStages, bool kACols, bool kBCols, int kGrain>
__global__ __launch_bounds__(64 * WM * WN) void matmul_kernel(const MatmulArgs a) {
#ifdef __HIP_DEVICE_COMPILE__   // the host's pass needs no body, and drops launch stubs over builtins it does not know
  constexpr bool kDirect = kGrain > 0;
  constexpr int kWaves = WM * WN, kThreads = 64 * kWaves, BK = slice<T>();
  constexpr int TM = BM / WM, TN = BN / WN, MI = TM / 32, NI = TN / 32;
  using A = Side<T, BM, kACols, kThreads>;
  using B = Side<T, BN, kBCols, kThreads>;
  constexpr int kStage = A::kBytes + B::kBytes;
  static_assert(32 * TN * 4 * kWaves <= kStage, "the epilogue turns its rows over in the second slice's space");
  constexpr int kVecs = TN / 8, kRows = 64 / kVecs;   // of the epilogue: vectors a row, rows a pass
  constexpr int kPasses = 32 / kRows, kStores = MI * kPasses;
  static_assert(kDirect || kStages == 2, "registers hold one slice");
  __shared__ __attribute__((aligned(16))) char ring[kStages * kStage];
  char* const one = ring;
  char* const two = ring + kStage;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int per = a.tiles_m * a.tiles_n, total = per * a.splits;
  const int h = lane >> 5;
  using LoadA = typename std::conditional<kDirect, typename A::template Direct<kDirect ? kGrain : 16>, typename A::Staged>::type;
  using LoadB = typename std::conditional<kDirect, typename B::template Direct<kDirect ? kGrain : 16>, typename B::Staged>::type;
  LoadA la;
  LoadB lb;
  int64_t m0, n0;
  int k0, k1;
  constexpr int kLoads = LoadA::kLoads + LoadB::kLoads;
  const auto issue_one = [&](char* lds, int i) __attribute__((always_inline)) {
    if (i < LoadA::kLoads) la.issue(lds, wave, i);
    else lb.issue(lds + A::kBytes, wave, i - LoadA::kLoads);
  };
  const auto issue = [&](char* lds) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) issue_one(lds, i);
  };
  // A tile's place, and its first slice's loads on their way to `one`.
  const auto open = [&](int id) __attribute__((always_inline)) {
    const int split = id / per;
    int tm, tn;
    place_tile(id - split * per, a.tiles_m, a.tiles_n, tm, tn);
    m0 = static_cast<int64_t>(tm) * BM, n0 = static_cast<int64_t>(tn) * BN;
    k0 = split * a.k_split, k1 = a.K - k0 < a.k_split ? a.K : k0 + a.k_split;
    la.start(static_cast<const T*>(a.a), a.lda, m0, a.M, a.K, k0);
    lb.start(static_cast<const T*>(a.b), a.ldb, n0, a.N, a.K, k0);
    if (kDirect && k1 - k0 < BK) la.end(k1 - k0), lb.end(k1 - k0);
    issue(one);
  };
  int id = node_block(blockIdx.x, gridDim.x);
  open(id);
  bool whole = false;   // the tile before lay inside C as a whole: each wave issued kStores stores at least for y (and z)
  for (;;) {
    const int slices = (k1 - k0 - 1) / BK + 1;
    Acc acc[MI][NI] = {};
    // Loads of slice t on their way (in order of t).
    const auto prepare = [&](int t) __attribute__((always_inline)) {
      const int64_t have = k1 - k0 - static_cast<int64_t>(t) * BK;
      if (kDirect && have < BK) la.end(static_cast<int>(have)), lb.end(static_cast<int>(have));
    };
    const auto commit = [&](char* lds) __attribute__((always_inline)) {
      la.commit(lds);
      lb.commit(lds + A::kBytes);
    };
    // Fragments are read one step of k ahead of their products.
    Chunk fa[2][MI], fb[2][NI];
    const auto read_one = [&](const char* lds, int s, int i) __attribute__((always_inline)) {
      if (i < NI) fb[s & 1][i] = B::fragment(lds + A::kBytes, wn * TN + 32 * i, s, lane);
      else fa[s & 1][i - NI] = A::fragment(lds, wm * TM + 32 * (i - NI), s, lane);
    };
    // The products of step s, with the reads of step `next` of `from` and, with kLoad, the loads to
    // `to` spread between them: the matrix pipe is never without work while those are issued.
    const auto step = [&](int s, const char* from, int next, auto load, char* to) __attribute__((always_inline)) {
      constexpr int kReads = MI + NI, kProducts = MI * NI;
#pragma unroll
      for (int i = 0; i < kProducts; ++i) {
        const int m = i / NI, n = m & 1 ? NI - 1 - i % NI : i % NI;
        acc[m][n] = multiply<T>(fb[s & 1][n], fa[s & 1][m], acc[m][n]);
#pragma unroll
        for (int r = i; r < (i + 1 == kProducts ? kReads : min(kReads, i + 1)); ++r) read_one(from, next, r);
        if (decltype(load)::value)
#pragma unroll
          for (int l = i * kLoads / kProducts; l < (i + 1) * kLoads / kProducts; ++l) issue_one(to, l);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // Slice t, whose first fragments are read already, from `cur`.  After its last ones are, one
    // barrier frees `cur` for slice t + kStages and opens slice t + 1, whose loads are kStages - 1
    // slices old by then.  What is read past the last slice is not used.
    const auto walk = [&](char* cur, char* nxt, int t) __attribute__((always_inline)) {
      prepare(t + kStages);
      if (!kDirect) issue(nxt);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < 3; ++s) step(s, cur, s + 1, std::false_type{}, cur);
      if (!kDirect) commit(nxt);
      barrier_after_loads<kDirect ? (kStages - 2) * kLoads : 0>();
      step(3, nxt, 0, std::integral_constant<bool, kDirect>{}, cur);
    };
    float bias[8] = {};
    {
      const int n = static_cast<int>(n0) + wn * TN + (lane % kVecs) * 8;
      if (a.bias != nullptr && n < a.N) load<8, false>(a.bias, n, a.N, bias);
    }
    commit(one);
    if (kDirect)
#pragma unroll
      for (int j = 1; j < kStages; ++j) {
        prepare(j);
        issue(ring + j * kStage);
      }
    // The first slice has come; the others, and what the epilogue before stored, may be under way.
    constexpr int kPending = kDirect ? (kStages - 1) * kLoads : 0;
    if (!whole) barrier_after_loads<kPending>();
    else if (a.z == nullptr) barrier_after_loads<kPending + kStores>();
    else barrier_after_loads<kPending + 2 * kStores>();
#pragma unroll
    for (int r = 0; r < MI + NI; ++r) read_one(one, 0, r);
    for (int t = 0, cur = 0; t < slices; ++t) {
      const int nxt = cur + kStage == kStages * kStage ? 0 : cur + kStage;
      walk(ring + cur, ring + nxt, t);
      cur = nxt;
    }
    barrier_after_loads<0>();

    // ---- epilogue, while the next tile's first slice is under way
    const int64_t me = m0 + wm * TM;
    const int n = static_cast<int>(n0) + wn * TN + (lane % kVecs) * 8;
    const int64_t part_row = static_cast<int64_t>(k0 / a.k_split) * a.M;
    whole = a.part == nullptr && m0 + BM <= a.M && n0 + BN <= a.N;
    id += gridDim.x;
    if (kDirect && id < total) open(id);
    asm volatile("" ::: "memory");   // the stores below are younger than those loads
    __builtin_amdgcn_sched_barrier(0);
    float* const turn = reinterpret_cast<float*>(two) + wave * 32 * TN;
#pragma unroll
    for (int k = 0; k < 8; ++k) asm volatile("" ::"v"(bias[k]));   // arrived long ago: nothing after has to wait for it
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const VecN<float, 4> v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          *reinterpret_cast<VecN<float, 4>*>(turn + turn_at<TN>(lane & 31, 8 * j + 2 * q + h)) = v;
        }
      __builtin_amdgcn_wave_barrier();
      float v[kPasses][8];
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int r = p * kRows + lane / kVecs, c = lane % kVecs * 2;
        __builtin_memcpy(v[p], turn + turn_at<TN>(r, c), 16);
        __builtin_memcpy(v[p] + 4, turn + turn_at<TN>(r, c + 1), 16);
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int64_t m = me + 32 * i + p * kRows + lane / kVecs;
        if (m >= a.M || n >= a.N) continue;
        if (a.part != nullptr) {
          store<8, false>(a.part + (part_row + m) * a.N, n, a.N, v[p]);
          continue;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) v[p][k] += bias[k];
        if (a.z != nullptr) stream<8>(static_cast<T*>(a.z) + m * a.ldz, n, a.N, v[p]);
        if (a.act != ETPC_ACT_NONE) activate<sizeof(T) == 4>(v[p], a.act);
        if (a.res != nullptr) {
          float w[8];
          load<8, false>(static_cast<const T*>(a.res) + m * a.ldres, n, a.N, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[p][k] += w[k];
        }
        stream<8>(static_cast<T*>(a.c) + m * a.ldc, n, a.N, v[p]);
      }
    }
    if (id >= total) break;
    barrier_after_reads();
    if (!kDirect) open(id);
  }
#endif
}

template <class T, int BM, int BN, int WM, int WN, int kStages, int kGrain>
hipError_t launch_tiles(MatmulArgs a, MatmulForm form, hipStream_t s) {
  const int64_t tiles_m = (static_cast<int64_t>(a.M) + BM - 1) / BM, tiles_n = (static_cast<int64_t>(a.N) + BN - 1) / BN;
  const int64_t total = tiles_m * tiles_n * a.splits;
  // as many workgroups as LDS holds at once, each walking its tiles
  static_assert(BM == BN, "one side");
  constexpr int resident = matmul_resident(BM, kStages);
  if (total > INT32_MAX - kCus * resident) return hipErrorInvalidValue;   // a workgroup steps past the last tile by that much
  a.tiles_m = static_cast<int32_t>(tiles_m), a.tiles_n = static_cast<int32_t>(tiles_n);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(total, kCus * resident))), block(64 * WM * WN);
  if (form == MatmulForm::kRowsCols)
    matmul_kernel<T, BM, BN, WM, WN, kStages, false, true, kGrain><<<grid, block, 0, s>>>(a);
  else if (form == MatmulForm::kRowsRows)
    matmul_kernel<T, BM, BN, WM, WN, kStages, false, false, kGrain><<<grid, block, 0, s>>>(a);
  else
    matmul_kernel<T, BM, BN, WM, WN, kStages, true, true, kGrain><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

template <class T>
hipError_t launch(const MatmulArgs& a, MatmulForm form, const MatmulShape& shape, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (shape.tile == 256) return launch_tiles<T, 256, 256, 2, 4, 2, 16>(a, form, s);
    if (shape.tile == 64 && shape.stages == 3) return launch_tiles<T, 64, 64, 2, 2, 3, 16>(a, form, s);
  }
  if (shape.grain == 16)
    return shape.tile >= 128 ? launch_tiles<T, 128, 128, 2, 2, 2, 16>(a, form, s) : launch_tiles<T, 64, 64, 2, 2, 2, 16>(a, form, s);
  if (shape.grain == 4)
    return shape.tile >= 128 ? launch_tiles<T, 128, 128, 2, 2, 2, 4>(a, form, s) : launch_tiles<T, 64, 64, 2, 2, 2, 4>(a, form, s);
  return shape.tile >= 128 ? launch_tiles<T, 128, 128, 2, 2, 2, 0>(a, form, s) : launch_tiles<T, 64, 64, 2, 2, 2, 0>(a, form, s);
}

}  // namespace mm
}  // namespace etpc

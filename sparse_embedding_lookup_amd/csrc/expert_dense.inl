// expert_dense.inl -- the experts' fully connected layers over rows sorted by expert, on the
// matrix cores.  Part of the translation unit of dense.hip.
//
// Expert e has the sorted positions p in [offsets[e], offsets[e+1]) and the weights W[e]
// [N, K].  With x(p) = X[p], or the token's row X[order[p] / k] read in place:
//   forward   Y[p, :]  = act(W[e] x(p) + b[e])
//   backward  dX[p, :] = W[e]^T dY[p, :], times [x(p) > 0] where x is a rectified output
//             dW[e]    = sum_p dY[p, :] x(p)^T,   db[e] = sum_p dY[p, :]        (fp32)
// Three products of one shape: rows by columns over a reduction, the rows cut at the experts'
// borders.  The row counts stay on the device: a grid is for every tile that n rows in E pieces
// can need, a block for each (loose_kernel) or as many blocks as run at once, which take the tiles
// there are in turn (wide_kernel); a block finds a tile's expert by a scan over the offsets.
// Positions from offsets[E] on belong to no expert; their rows of Y and dX are zero.
// Products are exact in the matrix cores (binary32 operands: rounded once), sums are fp32.
namespace ctr {
namespace experts {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

struct Product {
  const void* X;
  int64_t xs, x_rows;
  const int32_t* order;         // nullable: positions are X's rows
  uint32_t kmul;                // i / k = 2 i * kmul >> 32 + kshift for 0 <= i < 2^31
  int kshift;
  const int32_t* offsets;
  int64_t n;
  int E, K, N;
  const void* W;
  const float* b;               // forward, nullable
  int relu;                     // forward: act; backward: x is a rectified output
  const void* dY;
  int64_t dys;
  void* Y;                      // Y, or dX
  int64_t ys;
  float* dW;
  float* part;                  // partial sums of dW
  int64_t most;                 // how many of them there is room for
  const struct Plan* plan;      // who takes which tile of dW
  int64_t slice;                // positions a slice of dW's reduction
  bool big;                     // dW in 256 x 256 tiles
  int col_tiles, row_tiles;
};

// First and last position of expert e; e == E: the positions of no expert.  Clamped, so that
// bad offsets give bad numbers and no access outside the arrays.
__device__ __forceinline__ void bounds_of(const Product& g, int e, int64_t* lo, int64_t* hi) {
  const int64_t a = clamp64(g.offsets[e], 0, g.n);
  *lo = a;
  *hi = e < g.E ? clamp64(g.offsets[e + 1], a, g.n) : g.n;
}

// The expert of row tile `mt` (BM rows a tile, experts in order, then the positions of none)
// and its rows: every wave scans the tile counts, 64 experts at a time.  false: no such tile.
template <int BM>
__device__ __forceinline__ bool find_tile(const Product& g, int64_t mt, int* expert, int64_t* row0,
                                          int64_t* end) {
  const int lane = threadIdx.x & 63;
  int64_t run = 0;
  for (int e0 = 0; e0 <= g.E; e0 += 64) {
    const int e = e0 + lane;
    int64_t lo = 0, hi = 0;
    if (e <= g.E) bounds_of(g, e, &lo, &hi);
    const int tiles = (int)((hi - lo + BM - 1) / BM);
    int upto = tiles;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    const uint64_t past = __ballot(run + upto > mt);
    if (past) {
      const int at = __ffsll((unsigned long long)past) - 1;
      const int64_t first = run + __shfl(upto - tiles, at);
      *expert = e0 + at;
      *row0 = __shfl(lo, at) + (mt - first) * BM;
      *end = __shfl(hi, at);
      return true;
    }
    run += __shfl(upto, 63);
  }
  return false;
}

// Row of X of slot i (its token, i / k), or -1 (a slot outside X: its row reads as zeros).
__device__ __forceinline__ int32_t token_of(const Product& g, int32_t i) {
  const int32_t r = (int32_t)(__umulhi(2u * (uint32_t)i, g.kmul) >> g.kshift);
  return i >= 0 && r < (int32_t)g.x_rows ? r : -1;
}
// Row of X that position p reads, or -1.
__device__ __forceinline__ int64_t x_row(const Product& g, int64_t p) {
  if (!g.order) return p < g.x_rows ? p : -1;
  return token_of(g, g.order[p]);
}

enum Kind { kForward = 0, kInput = 1, kWeight = 2 };

// A value that is the same in the whole wave, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)x);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(x >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// Row tiles that the experts (and the positions of none) need.
template <int BM>
__device__ __forceinline__ int64_t count_tiles(const Product& g) {
  const int lane = threadIdx.x & 63;
  int tiles = 0;
  for (int e = lane; e <= g.E; e += 64) {
    int64_t lo, hi;
    bounds_of(g, e, &lo, &hi);
    tiles += (int)((hi - lo + BM - 1) / BM);
  }
  for (int d = 1; d < 64; d <<= 1) tiles += __shfl_xor(tiles, d);
  return tiles;
}

// The weight gradient's reduction is cut into slices of g.slice positions, so that an expert
// with many rows is many blocks' work: expert e has max(1, ceil(rows / slice)) of them.  One
// slice writes dW itself; the sums of several go to g.part, in order, and are added after.
struct Slice {
  int expert, count;            // slices of this expert
  int64_t lo, hi, partial;      // its positions; place among the partial sums, or -1
};
__device__ __forceinline__ int slices_of(const Product& g, int e, int64_t* lo, int64_t* hi) {
  bounds_of(g, e, lo, hi);
  const int c = (int)((*hi - *lo + g.slice - 1) / g.slice);
  return c > 1 ? c : 1;
}
__device__ __forceinline__ int64_t count_slices(const Product& g) {
  const int lane = threadIdx.x & 63;
  int c = 0;
  for (int e = lane; e < g.E; e += 64) {
    int64_t lo, hi;
    c += slices_of(g, e, &lo, &hi);
  }
  for (int d = 1; d < 64; d <<= 1) c += __shfl_xor(c, d);
  return c;
}
// Slice `unit` of all, or (expert >= 0) the first of that expert.  false: no such slice, or no
// room for its partial sums (or the expert's), which only offsets out of order can need.
__device__ __forceinline__ bool find_slice(const Product& g, int64_t unit, int expert, Slice* u) {
  const int lane = threadIdx.x & 63;
  int64_t run = 0, partials = 0;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    const int e = e0 + lane;
    int64_t lo = 0, hi = 0;
    const int c = e < g.E ? slices_of(g, e, &lo, &hi) : 0;
    const int m = c > 1 ? c : 0;
    int upto = c, mupto = m;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d), x = __shfl_up(mupto, d);
      if (lane >= d) {
        upto += v;
        mupto += x;
      }
    }
    const uint64_t hit = expert >= 0 ? __ballot(e == expert) : __ballot(run + upto > unit);
    if (hit) {
      const int at = __ffsll((unsigned long long)hit) - 1;
      const int64_t i = expert >= 0 ? 0 : unit - run - __shfl(upto - c, at);
      const int64_t first = __shfl(lo, at), last = __shfl(hi, at);
      u->expert = e0 + at;
      u->count = __shfl(c, at);
      u->lo = first + i * g.slice;
      u->hi = last < u->lo + g.slice ? last : u->lo + g.slice;
      u->partial = u->count > 1 ? partials + __shfl(mupto - m, at) + i : -1;
      return u->count == 1 || u->partial + (expert >= 0 ? u->count : 1) <= g.most;
    }
    run += __shfl(upto, 63);
    partials += __shfl(mupto, 63);
  }
  return false;
}

// The weight gradient's tiles are as long as their expert has rows, which differ widely.  One
// block lays out who takes which before the product: a unit's tiles in entries of about kNear
// neighbours, the entries sorted by the length of their tiles and dealt to the XCDs like cards,
// largest first, back and forth.  An XCD's blocks walk its tiles in strides to and fro, so that
// who begins with the longest tile ends with the shortest.  (Runs of tiles of equal cost an
// XCD, unsorted: dW of 16384 rows in 8 uneven experts of 2048 x 2048 175 us for 142 us.)
struct Entry {
  int32_t start;                // the entry's first tile in the XCD's order
  int32_t expert, lo, hi, partial;
  int32_t tile;                 // its first tile of the unit's
  int32_t pad[2];
};
constexpr int kEntries = 2048, kPlanThreads = 1024, kNear = 32;
struct Plan {
  int32_t tiles[8], count[8];   // of each XCD
  Entry entry[8][kEntries / 8];
};

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(Product g, Plan* plan) {
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  __shared__ int32_t units_to[kPlanThreads], partials_to[kPlanThreads];
  __shared__ int32_t begin[kPlanThreads], stop[kPlanThreads];
  __shared__ int32_t wave_sum[2][16], rounds[kEntries], many[8][kEntries / 8];
  int64_t lo = 0, hi = 0;
  const int c = t < g.E ? slices_of(g, t, &lo, &hi) : 0, m = c > 1 ? c : 0;
  int upto = c, mupto = m;
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d), x = __shfl_up(mupto, d);
    if (lane >= d) {
      upto += v;
      mupto += x;
    }
  }
  if (lane == 63) {
    wave_sum[0][w] = upto;
    wave_sum[1][w] = mupto;
  }
  begin[t] = (int32_t)lo;
  stop[t] = (int32_t)hi;
  __syncthreads();
  int units = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (i < w) {
      upto += wave_sum[0][i];
      mupto += wave_sum[1][i];
    }
    units += wave_sum[0][i];
  }
  units_to[t] = upto;
  partials_to[t] = mupto;
  const int tiles = g.row_tiles * g.col_tiles;
  int parts = (tiles + kNear - 1) / kNear, least = (2 * (int)kXcds + units - 1) / units;
  parts = parts > least ? parts : least;
  parts = parts < tiles ? parts : tiles;
  parts = parts < kEntries / units ? parts : kEntries / units;
  const int entries = units * parts;           // set_slices keeps the units below kEntries
  int top = kPlanThreads;                      // the experts, to a power of two
  while (top / 2 >= g.E) top >>= 1;
  __syncthreads();
  Entry x[kEntries / kPlanThreads];            // entry t and, if there are so many, t + 1024
  int size[kEntries / kPlanThreads];
#pragma unroll
  for (int i = 0; i < kEntries / kPlanThreads; ++i) {
    const int j = t + i * kPlanThreads;
    if (j >= entries) continue;
    const int u = j / parts, p = j % parts;
    int e = 0;
    for (int d = top / 2; d > 0; d >>= 1)
      if (units_to[e + d - 1] <= u) e += d;
    const int before = e > 0 ? units_to[e - 1] : 0, n = units_to[e] - before;
    x[i].start = 0;
    x[i].expert = e;
    x[i].lo = (int32_t)(begin[e] + (u - before) * g.slice);
    x[i].hi = stop[e] - x[i].lo < g.slice ? stop[e] : (int32_t)(x[i].lo + g.slice);
    const int partial = partials_to[e] - n + u - before;
    x[i].partial = n > 1 && partial < g.most ? partial : -1;   // all have room in ordered offsets
    x[i].tile = tiles * p / parts;
    size[i] = tiles * (p + 1) / parts - x[i].tile;
    rounds[j] = (x[i].hi - x[i].lo + 63) / 64;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEntries / kPlanThreads; ++i) {
    const int j = t + i * kPlanThreads;
    if (j >= entries) continue;
    const int mine = rounds[j];
    int rank = 0;
#pragma unroll 8
    for (int o = 0; o < entries; ++o) rank += rounds[o] > mine || (rounds[o] == mine && o < j);
    const int at = rank / (int)kXcds, in = rank % (int)kXcds;
    const int xcd = at & 1 ? (int)kXcds - 1 - in : in;
    many[xcd][at] = size[i];
    plan->entry[xcd][at] = x[i];               // without its start
  }
  __syncthreads();
  if (w < (int)kXcds) {                        // wave w: the starts of XCD w's entries
    const int full = entries / (int)kXcds, odd = entries % (int)kXcds;
    const int count = full + ((full & 1 ? (int)kXcds - 1 - w : w) < odd);
    int run = 0;
    for (int i = 0; i < count; i += 64) {
      const int n = i + lane < count ? many[w][i + lane] : 0;
      int s = n;
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(s, d);
        if (lane >= d) s += v;
      }
      if (i + lane < count) plan->entry[w][i + lane].start = run + s - n;
      run += __shfl(s, 63);
    }
    if (lane == 0) {
      plan->tiles[w] = run;
      plan->count[w] = count;
    }
  }
}

// Tile i of XCD x's.
__device__ __forceinline__ Entry find_entry(const Plan* plan, int x, int i) {
  const int lane = threadIdx.x & 63, count = plan->count[x];
  int at = -1;
  for (int k = 0; k < count; k += 64) {
    const uint64_t before = __ballot(k + lane < count && plan->entry[x][k + lane].start <= i);
    at += __popcll(before);
    if (before != ~0ull) break;
  }
  const auto* p = (const __attribute__((address_space(4))) int32_t*)(uintptr_t)
      &plan->entry[x][__builtin_amdgcn_readfirstlane(at < 0 ? 0 : at)];
  Entry e;
  e.start = p[0]; e.expert = p[1]; e.lo = p[2]; e.hi = p[3]; e.partial = p[4]; e.tile = p[5];
  return e;
}

// Four floats, aligned to one.
__device__ __forceinline__ f32x4 load4(const float* p) {
  f32x4 x;
  __builtin_memcpy(&x, p, 16);
  return x;
}
__device__ __forceinline__ void store4(float* p, f32x4 x) { __builtin_memcpy(p, &x, 16); }

// The 16-bit values of h where those of m are positive, else zero.
template <int TY>
__device__ __forceinline__ uint32_t keep_positive(uint32_t h, uint32_t m) {
  return (half_lo<TY>(m) > 0.f ? h & 0xFFFFu : 0u) | (half_hi<TY>(m) > 0.f ? h & 0xFFFF0000u : 0u);
}

// ------------------------------------------------------------------ 16-bit operands, staged
// The products of 16-bit operands in 16-byte pieces (widths and strides multiples of 8,
// 16-byte aligned arrays).  A block has a BM x BN output tile and a wave a WM x WN part of it
// in 32 x 32 matrix-core tiles.  The reduction advances in rounds of 64 values, so that a row
// is read 128 bytes at a time (half of that costs the first-level cache twice the requests,
// and the forward product 729 us instead of 603 at 65536 x 2208 x 2048).  Tiles go from
// memory to LDS directly (one 16-byte load a lane, 1 KB a wave, no registers in between); the
// loads' own bounds check gives zeros for rows and reduction values that are not there.
//
// LDS is a ring of five slots of one operand's round, in the order A0 B0 A1 B1 ...: while
// round j is read, B of round j + 1 and A of round j + 2 are on their way.  A round has two
// half steps, and a half step two parts: one that moves data (the wave's fragments from LDS
// to registers, its share of the loads of one operand) and one that computes (16 matrix-core
// instructions a wave in 256 x 256 tiles).  With eight waves, two on each SIMD, the second
// four run one part behind the first: while one of a SIMD's waves computes the other moves
// data.  Barriers end both parts.  With four waves there are two blocks a compute unit, which
// interleave by themselves, and one barrier a half step.
//
// An operand lies in LDS in one of two forms; the banks serve 256 bytes at a time:
//   by rows (64 reduction values of one row, 128 bytes): a fragment is one 16-byte read of 32
//     rows.  The 16-byte piece c of row r is at c ^ (r / 2 & 7), so that sixteen lanes that
//     read piece c of sixteen rows touch all banks.
//   by reduction (BM or BN values of one reduction index): a fragment is two transposing
//     reads, each giving a lane four reduction values of its row.  32 lanes read 64 bytes of
//     four reduction rows; piece c of reduction row q is at c ^ (4 (q & 3)), which spreads
//     the four over the banks.
// The matrix cores take the columns as their rows: a lane then holds four neighbouring
// columns of one output row, stored together.
//
// Blocks stay: each takes tiles of its XCD's part until there are none.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kRound = 64, kHalf = 32;         // reduction values
// An offset past every buffer: reads zeros, writes nothing.  Offsets are below 2^31, and so is
// what is added to them for all lanes, so that the sum never wraps; gathered rows, to which
// nothing is added, reach further.
constexpr uint32_t kNowhere = 0x80000000u, kFar = 0xFFFFFFF0u;

template <int TY>
__device__ __forceinline__ f32x16 mma(s16x8 a, s16x8 b, f32x16 c) {
  if constexpr (TY == kEltBF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// 16 bytes a lane from base + off + more to lds + 16 * lane (base, more and lds the same in the
// whole wave).
template <uint32_t END = kNowhere>
__device__ __forceinline__ void to_lds(const void* base, uint32_t off, uint32_t more,
                                       uint16_t* lds) {
  const __amdgpu_buffer_rsrc_t r =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)END, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16,
                                           (int)off, (int)more, 0, 0);
}

// 16 bytes a lane from base + off (base the same in the whole wave).
__device__ __forceinline__ uint4 load16(const void* base, uint32_t off) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<void*>(base), (short)0, (int)kFar, 0x00020000);
  const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// 16 bytes a lane to base + off (base the same in the whole wave).  No part of the address is
// in the instruction's scalar offset: with one the compiler lets the next instruction write the
// registers that are stored, and the store has been seen to take what that writes.
__device__ __forceinline__ void store16(void* base, uint32_t off, uint4 x) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const __amdgpu_buffer_rsrc_t r =
      __builtin_amdgcn_make_buffer_rsrc(base, (short)0, (int)kNowhere, 0x00020000);
  const u32x4 v = {x.x, x.y, x.z, x.w};
  __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)off, 0, 0);
}

// Ends a part: the wave's LDS reads are done and at most LOADS of its loads are in flight, in
// every wave (LOADS < 0: any number).
template <int LOADS>
__device__ __forceinline__ void arrive() {
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (LOADS < 0)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LOADS) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void arrive_only() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// ORDER: the weight gradient reads X's rows through g.order.
template <int TY, int KIND, int BM, int BN, int WM, int WN, bool ORDER>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, 2) void wide_kernel(Product g) {
  constexpr int WAVES = (BM / WM) * (BN / WN), WN_WAVES = BN / WN;
  constexpr bool AROW = KIND != kWeight, BROW = KIND == kForward, PAIRED = WAVES == 8;
  constexpr int TI = WM / 32, TJ = WN / 32;
  constexpr int AL = BM * kRound / 512 / WAVES, BL = BN * kRound / 512 / WAVES;
  constexpr int STORES = TI * (KIND == kWeight ? WN / 8 : WN / 16);
  constexpr int SLOT = (BM > BN ? BM : BN) * kRound;           // a ring slot holds either operand
  __shared__ __attribute__((aligned(16))) uint16_t R0[SLOT], R1[SLOT], R2[SLOT], R3[SLOT], R4[SLOT];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w / WN_WAVES, wn = w % WN_WAVES;
  const int rl = lane & 31, kg = lane >> 5;
  const int cols = KIND == kForward ? g.N : g.K;

  // A tile: the first of its rows and columns, the end of the rows, the reduction's range.
  struct Tile {
    int e, n0;
    int64_t row0, end, r0, r1;
    float* dW;
  };
  auto find = [&](int64_t at) {
    Tile n;
    n.r0 = 0;
    n.dW = g.dW;
    if constexpr (KIND == kWeight) {
      const Entry u = find_entry(g.plan, blockIdx.x % kXcds, (int)at);
      const uint32_t tile = (uint32_t)(u.tile + (int)at - u.start);
      n.e = u.expert;
      n.r0 = u.lo;
      n.r1 = u.hi;
      const int64_t part = u.partial;
      n.dW = part >= 0 ? g.part + part * g.N * g.K : g.dW + (int64_t)n.e * g.N * g.K;
      n.row0 = (int64_t)(tile / (uint32_t)g.col_tiles) * BM;
      n.n0 = (int)(tile % (uint32_t)g.col_tiles) * BN;
      n.end = g.N;
    } else {
      n.n0 = (int)((uint32_t)at % (uint32_t)g.col_tiles) * BN;
      n.e = g.E; n.row0 = n.end = g.n;
      find_tile<BM>(g, (uint32_t)at / (uint32_t)g.col_tiles, &n.e, &n.row0, &n.end);
      n.r1 = n.e < g.E ? (KIND == kForward ? g.K : g.N) : 0;
    }
    n.e = __builtin_amdgcn_readfirstlane(n.e);
    n.n0 = __builtin_amdgcn_readfirstlane(n.n0);
    n.row0 = uniform(n.row0);
    n.end = uniform(n.end);
    n.r0 = uniform(n.r0);
    n.r1 = uniform(n.r1);
    return n;
  };

  // A load takes 8 rows (by rows) or 512 / WIDE reduction rows (by reduction); load q of wave w
  // is number q * WAVES + w.  Where a lane's 16 bytes are: at `base` of the round, plus the
  // lane's offset, plus a number of rows that is the same in the wave.  By rows lane i has row
  // i / 8 and its piece (i % 8) ^ (row / 2 & 7).
  const uint16_t* abase;
  const uint16_t* bbase;
  int64_t astep, bstep;                                        // elements from round to round
  uint32_t aoff, boff, rowoff[AL];                             // bytes
  int arows, brows;                                            // rows that there are
  constexpr int APER = 512 / BM, BPER = 512 / BN;
  constexpr int ALANES = 64 / APER, BLANES = 64 / BPER;
  const int piece = ((lane & 7) ^ ((4 * w + (lane >> 4)) & 7)) * 8;   // first reduction value
  const int64_t ald = KIND == kForward ? g.xs : g.dys, bld = KIND == kWeight ? g.xs : g.K;
  auto aim = [&](const Tile& n) {
    const uint16_t* W =
        static_cast<const uint16_t*>(g.W) + (int64_t)(n.e < g.E ? n.e : 0) * g.N * g.K;
    arows = (int)(n.end - n.row0 < BM ? n.end - n.row0 : BM);
    brows = cols - n.n0 < BN ? cols - n.n0 : BN;
    if constexpr (KIND == kForward) {
      abase = static_cast<const uint16_t*>(g.X) + (g.order ? 0 : n.row0 * ald);
      astep = kRound;
#pragma unroll
      for (int q = 0; q < AL; ++q) {
        const int r = 8 * (q * WAVES + w) + (lane >> 3);
        int64_t x = r < arows ? r : -1;
        if (g.order && x >= 0) x = x_row(g, n.row0 + r);
        rowoff[q] = x >= 0 ? (uint32_t)(x * ald + piece) * 2 : kFar;
      }
    } else if constexpr (KIND == kInput) {
      abase = static_cast<const uint16_t*>(g.dY) + n.row0 * ald;
      astep = kRound;
      aoff = (uint32_t)((lane >> 3) * ald + piece) * 2;
    } else {
      abase = static_cast<const uint16_t*>(g.dY) + n.r0 * ald + n.row0;
      astep = kRound * ald;
      const int kr = w * APER + lane / ALANES, c = ((lane % ALANES) ^ (4 * (kr & 3))) * 8;
      aoff = c < arows ? (uint32_t)((lane / ALANES) * ald + c) * 2 : kNowhere;
    }
    if constexpr (BROW) {
      bbase = W + (int64_t)n.n0 * bld;
      bstep = kRound;
      boff = (uint32_t)((lane >> 3) * bld + piece) * 2;
    } else {
      bbase = (KIND == kInput ? W : static_cast<const uint16_t*>(g.X)) + n.n0;
      bstep = ORDER ? 0 : kRound * bld;
      if (!ORDER) bbase += n.r0 * bld;
      const int kr = w * BPER + lane / BLANES, c = ((lane % BLANES) ^ (4 * (kr & 3))) * 8;
      boff = c < brows ? (uint32_t)((ORDER ? 0 : (lane / BLANES) * bld) + c) * 2 : kNowhere;
    }
  };
  // with ORDER: the slots of the round after the last loaded one, ahead of their use
  // (scalar loads, which do not stand in line with the operands' loads)
  int32_t slot[BL];
  auto fetch_slots = [&](int64_t k) {
    if constexpr (ORDER) {
      const auto* o = (const __attribute__((address_space(4))) int32_t*)(uintptr_t)g.order;
      const int n1 = (int)g.n - 1;
#pragma unroll
      for (int q = 0; q < BL; ++q) {
        const int p = (int)k + (q * WAVES + w) * BPER;         // past the end: any slot, unused
        int32_t v[BPER], i = 0;
#pragma unroll
        for (int j = 0; j < BPER; ++j) v[j] = o[p + j < n1 ? p + j : n1];
#pragma unroll
        for (int j = 0; j < BPER; ++j) i = lane / BLANES == j ? v[j] : i;
        slot[q] = i;
      }
    }
  };

  // Load the next round of an operand, reduction values [k, k + 64).
  auto load_a = [&](uint16_t* A, int64_t k, int64_t r1) {
    const int left = (int)(r1 - k < kRound ? r1 - k : kRound);
#pragma unroll
    for (int q = 0; q < AL; ++q) {
      const int i = q * WAVES + w;
      if constexpr (KIND == kForward) {
        to_lds<kFar>(abase, piece < left ? rowoff[q] : kFar, 0, A + i * 512);
      } else if constexpr (KIND == kInput) {
        const bool in = piece < left && (lane >> 3) < arows - 8 * i;
        to_lds(abase, in ? aoff : kNowhere, (uint32_t)(8 * i * ald) * 2, A + i * 512);
      } else {
        const bool in = lane / ALANES < left - i * APER;
        to_lds(abase, in ? aoff : kNowhere, (uint32_t)(i * APER * ald) * 2, A + i * 512);
      }
    }
    abase += astep;
  };
  auto load_b = [&](uint16_t* B, int64_t k, int64_t r1) {
    const int left = (int)(r1 - k < kRound ? r1 - k : kRound);
#pragma unroll
    for (int q = 0; q < BL; ++q) {
      const int i = q * WAVES + w;
      if constexpr (BROW) {
        const bool in = piece < left && (lane >> 3) < brows - 8 * i;
        to_lds(bbase, in ? boff : kNowhere, (uint32_t)(8 * i * bld) * 2, B + i * 512);
      } else {
        bool in = lane / BLANES < left - i * BPER;
        if constexpr (ORDER) {
          const int32_t x = token_of(g, slot[q]);
          in = in && x >= 0 && boff != kNowhere;
          to_lds<kFar>(bbase, in ? boff + (uint32_t)x * (uint32_t)bld * 2 : kFar, 0, B + i * 512);
        } else {
          to_lds(bbase, in ? boff : kNowhere, (uint32_t)(i * BPER * bld) * 2, B + i * 512);
        }
      }
    }
    bbase += bstep;
    fetch_slots(k + kRound);
  };
  // The first loads of a tile: A0, B0 and A1.
  auto start = [&](const Tile& n) {
    if (n.r1 <= n.r0) return;
    fetch_slots(n.r0);
    load_a(R0, n.r0, n.r1);
    load_b(R1, n.r0, n.r1);
    load_a(R2, n.r0 + kRound, n.r1);
  };

  // Where a lane's fragments are in a slot, in bytes: those of the operand's 32-row tile i and
  // the reduction values 16 s + 8 kg .. + 8 are at `at` with a few bits flipped, plus a constant.
  // (By reduction: the 16 lanes of a group have reduction row + (lane & 15) / 4 and columns
  // 4 (lane & 3) ..)
  auto frag_at = [&](int row, bool byrow, int wide) -> uint32_t {
    if (byrow) return (row + rl) * kRound * 2 + ((kg ^ (rl >> 1 & 7)) * 16);
    const int kr = 8 * kg + ((lane & 15) >> 2);
    const int c = row + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    return kr * wide * 2 + ((c >> 3) ^ (4 * (kr & 3))) * 16 + (c & 7) * 2;
  };
  const uint32_t afrag = frag_at(WM * wm, AROW, BM), bfrag = frag_at(WN * wn, BROW, BN);
  auto frag = [&](const uint16_t* L, uint32_t at, int i, int s, auto byrow, auto wide) -> s16x8 {
    const char* p = reinterpret_cast<const char*>(L);
    if constexpr (decltype(byrow)::value) {
      return *reinterpret_cast<const s16x8*>(p + (at ^ (32 * s)) + 32 * i * kRound * 2);
    } else {
      constexpr int WIDE = decltype(wide)::value;
      typedef __attribute__((address_space(3))) s16x4* P;
      p += (at ^ (64 * i)) + 16 * s * WIDE * 2;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p + 4 * WIDE * 2));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  };

  f32x16 acc[TI][TJ];
  // Half step h of a round: `ahead` issues its loads and arrives.
  auto half = [&](const uint16_t* A, const uint16_t* B, auto h, auto ahead) {
    s16x8 a[2][TI], b[2][TJ];
    // the addresses are made here each time: kept for all slots they would take the registers
    // that the accumulators need
    uint32_t aat = afrag, bat = bfrag;
    asm volatile("" : "+v"(aat), "+v"(bat));
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        b[s][j] = frag(B, bat, j, 2 * decltype(h)::value + s,
                       std::integral_constant<bool, BROW>{}, std::integral_constant<int, BN>{});
#pragma unroll
      for (int i = 0; i < TI; ++i)
        a[s][i] = frag(A, aat, i, 2 * decltype(h)::value + s,
                       std::integral_constant<bool, AROW>{}, std::integral_constant<int, BM>{});
    }
    ahead();
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = mma<TY>(b[s][j], a[s][i], acc[i][j]);
    __builtin_amdgcn_s_setprio(0);
    if constexpr (PAIRED) arrive_only();
  };

  // The tile whose first loads are on their way: its sums into acc.  `stores`: of the tile
  // before, issued after the loads.
  auto multiply = [&](const Tile& n, bool stores) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const int64_t r0 = n.r0, r1 = n.r1;
    const int halves = (int)((r1 - r0 + kHalf - 1) / kHalf), rounds = (halves + 1) >> 1;
    if (halves <= 0) return;
    // (Loads past the last round read nowhere: the counts of loads in flight stay the same, and
  // all have ended when the last half step does.)
  // Round j on A and B; Bn takes B of round j + 1 (its slot held A of round j - 1), An takes A
    // of round j + 2 (its slot held B of round j - 1).
    auto round = [&](const uint16_t* A, const uint16_t* B, uint16_t* Bn, uint16_t* An, int j) {
      half(A, B, std::integral_constant<int, 0>{}, [&] {
        load_b(Bn, r0 + (int64_t)(j + 1) * kRound, r1);
        if (2 * j + 1 < halves) arrive<-1>();
        else arrive<0>();
      });
      if (2 * j + 1 < halves)
        half(A, B, std::integral_constant<int, 1>{}, [&] {
          // round j + 1 has landed when at most A of round j + 2 is in flight
          load_a(An, r0 + (int64_t)(j + 2) * kRound, r1);
          if (j + 1 < rounds) arrive<AL>();
          else arrive<0>();
        });
    };

    // A0 and B0 have landed when at most A1 and the stores after it are in flight
    if (stores) arrive<AL + STORES>();
    else arrive<AL>();
    if (PAIRED && w >= WAVES / 2) arrive_only();
    for (int j = 0; j < rounds; j += 5) {
      round(R0, R1, R3, R4, j);
      if (j + 1 < rounds) round(R2, R3, R0, R1, j + 1);
      if (j + 2 < rounds) round(R4, R0, R2, R3, j + 2);
      if (j + 3 < rounds) round(R1, R2, R4, R0, j + 3);
      if (j + 4 < rounds) round(R3, R4, R1, R2, j + 4);
    }
    if (PAIRED && w < WAVES / 2) arrive_only();
  };

  // acc[i][j][v] is row 32 i + rl, column 32 j + 8 (v / 4) + 4 kg + v % 4 of the wave's part.
  // 32 rows at a time go through 8 KB of LDS a wave (of the two slots that `start` leaves
  // free), so that a store is whole 16-byte pieces along rows.  Every store is issued, those
  // outside the tile to nowhere: `multiply` counts them.
  constexpr int EACH = SLOT * 2 / 8192;                        // waves a slot holds
  static_assert(2 * EACH >= WAVES, "the waves' parts fit");
  char* const out = reinterpret_cast<char*>(w < EACH ? R3 : R4) + (w % EACH) * 8192;
  auto finish = [&](const Tile& n, const f32x4 (&bias)[TJ][4]) {
    constexpr int SIZE = KIND == kWeight ? 4 : 2, PIECE = 16 / SIZE, LR = WN / PIECE;
    const int64_t ld = KIND == kWeight ? g.K : g.ys;
    const int64_t rw = n.row0 + WM * wm;                       // the wave's first row
    const int cw = n.n0 + WN * wn;                             // and column
    char* base = KIND == kWeight ? reinterpret_cast<char*>(n.dW) : static_cast<char*>(g.Y);
    base += (rw * ld + cw) * SIZE;
    // this lane's row and column in the 64 / LR rows of a store (from a lane number that the
    // compiler does not know: what it made of it would stay in registers over the products)
    int me = lane;
    asm volatile("" : "+v"(me));
    const int l = me % LR, rr = me / LR, rl = me & 31, kg = me >> 5;
    const bool in = cw + l * PIECE < cols;
    const int rows = (int)(n.end - rw < WM ? n.end - rw : WM);
    const uint32_t off = (uint32_t)(rr * ld + l * PIECE) * SIZE;
    // with x_relu: the input's values at the same places
    const bool masked = KIND == kInput && g.relu && n.e < g.E;
    const uint16_t* xbase = static_cast<const uint16_t*>(g.X) + cw + (g.order ? 0 : rw * g.xs);
#pragma unroll
    for (int i = 0; i < TI; ++i) {
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = 32 * j + 8 * q + 4 * kg;
          float x[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            x[v] = acc[i][j][4 * q + v];
            if constexpr (KIND == kForward) {
              x[v] += bias[j][q][v];
              if (g.relu) x[v] = x[v] > 0.f ? x[v] : 0.f;
            }
          }
          if constexpr (KIND == kWeight) {
            *reinterpret_cast<float4*>(out + rl * WN * 4 + ((c >> 2) ^ (rl & 15)) * 16) =
                make_float4(x[0], x[1], x[2], x[3]);
          } else {
            uint2 h;
            h.x = to_half<TY, false>(x[0], 0u) | (to_half<TY, false>(x[1], 0u) << 16);
            h.y = to_half<TY, false>(x[2], 0u) | (to_half<TY, false>(x[3], 0u) << 16);
            *reinterpret_cast<uint2*>(out + rl * (WN + 8) * 2 + c * 2) = h;
          }
        }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int t = 0; t < 32 * LR / 64; ++t) {
        const int r = t * (64 / LR) + rr;                      // of the 32 staged rows
        const bool here = in && 32 * i + r < rows;
        uint4 h;
        if constexpr (KIND == kWeight)
          h = *reinterpret_cast<const uint4*>(out + r * WN * 4 + (l ^ (r & 15)) * 16);
        else
          h = *reinterpret_cast<const uint4*>(out + r * (WN + 8) * 2 + l * 16);
        if constexpr (KIND == kInput) {
          if (masked) {
            int32_t x = 32 * i + r;
            if (g.order) x = here ? token_of(g, g.order[rw + x]) : -1;
            const uint32_t from = ((uint32_t)x * (uint32_t)g.xs + l * PIECE) * 2;
            const uint4 m = load16(xbase, here && x >= 0 ? from : kFar);
            h.x = keep_positive<TY>(h.x, m.x);
            h.y = keep_positive<TY>(h.y, m.y);
            h.z = keep_positive<TY>(h.z, m.z);
            h.w = keep_positive<TY>(h.w, m.w);
          }
        }
        const uint32_t more = (uint32_t)((32 * i + t * (64 / LR)) * ld) * SIZE;
        store16(base, here ? off + more : kNowhere, h);
      }
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // The next tile's first loads are issued before this tile's results are stored.  A block
  // takes every stride-th tile of its XCD's: of neighbouring tiles, which share operands, each
  // XCD, with an L2 of its own, has a run; blocks go to the 8 XCDs in turn.
  const int x = blockIdx.x % kXcds;
  const int64_t stride = gridDim.x / kXcds, mine = blockIdx.x / kXcds;
  int64_t at, last;
  if constexpr (KIND == kWeight) {
    at = mine;
    last = g.plan->tiles[x];
  } else {
    const int64_t total = uniform(count_tiles<BM>(g)) * g.col_tiles;
    at = total * x / kXcds + mine;
    last = total * (x + 1) / kXcds;
  }
  bool fro = false;
  auto next = [&](int64_t i) {
    if (KIND != kWeight) return i + stride;
    fro = !fro;                                // from mine in one stride to its mirror in the next
    return fro ? i + 2 * (stride - mine) - 1 : i + 2 * mine + 1;
  };
  if (at >= last) return;
  Tile n = find(at);
  aim(n);
  start(n);
  for (bool stores = false;; stores = true) {
    multiply(n, stores);
    f32x4 bias[TJ][4];
    if constexpr (KIND == kForward) {
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = n.n0 + WN * wn + 32 * j + 8 * q + 4 * kg;
          const bool in = g.b && n.e < g.E && c < cols;
#pragma unroll
          for (int v = 0; v < 4; ++v) bias[j][q][v] = in ? g.b[(int64_t)n.e * g.N + c + v] : 0.f;
        }
    }
    const Tile done = n;
    at = next(at);
    if (at < last) {
      n = find(at);
      aim(n);
      start(n);
    }
    finish(done, bias);
    if (at >= last) break;
  }
}

// ---------------------------------------------------- any type, width, stride and alignment
// What the staged kernel does not take: binary32, and 16-bit arrays in no whole 16-byte
// pieces.  A block of four waves has a BM x BM tile, a wave a quarter of it; operands go
// through registers, where what is past the end is cleared, into one of two LDS buffers, those
// of the next round while this round's products run.  A round is 128 bytes of a row: 64
// reduction values of 16 bits or 32 of binary32.  LDS holds them as above.  The binary32
// matrix instruction takes two reduction values a lane pair: lanes 0 to 31 have values
// 8 c + e and lanes 32 to 63 values 8 c + 4 + e of both operands, so that by rows a lane's
// next four values are one 16-byte read.
// 64 x 64 tiles where 128 x 128 would leave compute units without a tile.  Y, dX and dW of 4096
// x 479 x 257 in binary32, 8 uneven experts: 28, 23 and 50 us, a third of the matrix rate that
// this size leaves (350 tiles on 256 compute units).  Two sets of waves with every other round
// each: 28, 28 and 43 us.
template <int TY, int KIND, int BM>
__global__ __launch_bounds__(kThreads, 2) void loose_kernel(Product g) {
  using T = typename std::conditional<TY == kEltF32, float, uint16_t>::type;
  constexpr int SIZE = sizeof(T), PE = 16 / SIZE;              // elements a piece
  constexpr int ROUND = 128 / SIZE, PIECES = BM * 8 / kThreads; // pieces a thread and operand
  constexpr bool AROW = KIND != kWeight, BROW = KIND == kForward;
  constexpr int ACROSS = BM / PE;                              // pieces of a reduction row
  constexpr int TW = BM / 64;                                  // a wave's tiles each way
  __shared__ __attribute__((aligned(16))) char lds[2][2][BM * 128];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, wm = w >> 1, wn = w & 1;
  const int rl = lane & 31, kg = lane >> 5;
  const int cols = KIND == kForward ? g.N : g.K;

  // which tile: neighbours to one XCD
  const int64_t rows_of = KIND == kWeight ? count_slices(g) * g.row_tiles : count_tiles<BM>(g);
  const uint32_t total = (uint32_t)(rows_of * g.col_tiles), per = total / kXcds;
  if (blockIdx.x >= total) return;
  const uint32_t at = blockIdx.x < per * kXcds
                          ? blockIdx.x % kXcds * per + blockIdx.x / kXcds : blockIdx.x;
  const int n0 = (int)(at % (uint32_t)g.col_tiles) * BM;
  const uint32_t mt = at / (uint32_t)g.col_tiles;
  int e;
  int64_t row0, end, r0 = 0, r1;
  float* dW = g.dW;
  if constexpr (KIND == kWeight) {
    Slice u;
    if (!find_slice(g, mt / (uint32_t)g.row_tiles, -1, &u)) return;
    e = u.expert;
    row0 = (int64_t)(mt % (uint32_t)g.row_tiles) * BM;
    end = g.N;
    r0 = u.lo;
    r1 = u.hi;
    const int64_t part = uniform(u.partial);
    dW = part >= 0 ? g.part + part * g.N * g.K : dW + uniform(e) * g.N * g.K;
  } else {
    if (!find_tile<BM>(g, mt, &e, &row0, &end)) return;
    r1 = e < g.E ? (KIND == kForward ? g.K : g.N) : 0;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  row0 = uniform(row0);
  end = uniform(end);
  r0 = uniform(r0);
  r1 = uniform(r1);
  const T* X = static_cast<const T*>(g.X);
  const T* dY = static_cast<const T*>(g.dY);
  const T* W = static_cast<const T*>(g.W) + (int64_t)(e < g.E ? e : 0) * g.N * g.K;

  // A thread's pieces: by rows row t / 8 + 32 q and piece t % 8; by reduction number
  // kThreads q + t of ACROSS to a reduction row, so always the same piece t % ACROSS.
  typedef T Piece __attribute__((ext_vector_type(PE)));
  Piece a[PIECES], b[PIECES];
  const int kp = (t & 7) * PE, kr = t / ACROSS, c = t % ACROSS * PE;
  constexpr int STEP = kThreads / ACROSS;                      // reduction rows from q to q + 1
  // A whole round reads whole pieces, all inside their rows.  Rows and columns past the tile's
  // last are not stored, so any in their place will do: rows the tile's first, and a column piece
  // that is not all there the row's last whole one, moved down (by `down` elements) to where it
  // belongs if part of it is.  What is read for a row outside X is cleared: forward W's piece, in
  // the weight gradient X's first row, where X has any (without, the way by elements is taken,
  // which reads none; dY's piece in its place: dW 53 us for 50 at the size above).
  const int64_t atop = AROW ? end - row0 : end, btop = cols;
  const PieceAt ap = AROW ? PieceAt{0, 0} : piece_at(row0 + c, atop, PE);
  const PieceAt bp = BROW ? PieceAt{0, 0} : piece_at(n0 + c, btop, PE);
  const int64_t acol = ap.column, bcol = bp.column;
  const int adown = ap.down, bdown = bp.down;
  const bool aedge = !AROW && row0 + BM > atop, bedge = !BROW && n0 + BM > btop;
  const bool narrow = (!AROW && atop < PE) || (!BROW && btop < PE) ||
                      (KIND == kWeight && g.x_rows == 0);
  auto moved = [](Piece x, int down) {
    if constexpr (TY == kEltF32) {
      if (down & 1) x = __builtin_shufflevector(x, x, 1, 2, 3, 3);
      if (down & 2) x = __builtin_shufflevector(x, x, 2, 3, 3, 3);
    } else {
      if (down & 1) x = __builtin_shufflevector(x, x, 1, 2, 3, 4, 5, 6, 7, 7);
      if (down & 2) x = __builtin_shufflevector(x, x, 2, 3, 4, 5, 6, 7, 7, 7);
      if (down & 4) x = __builtin_shufflevector(x, x, 4, 5, 6, 7, 7, 7, 7, 7);
    }
    return x;
  };
  auto all = [](const T* p) {
    Piece x;
    __builtin_memcpy(&x, p, 16);
    return x;
  };
  auto some = [&](const T* p, int64_t there) {                 // `there` elements, then zeros
    if (there >= PE) return all(p);
    Piece x;
#pragma unroll
    for (int i = 0; i < PE; ++i) x[i] = i < there ? p[i] : T(0);
    return x;
  };
  int64_t xrow[PIECES];                                        // X's rows of the pieces
  auto look = [&](int64_t k) {                                 // the weight gradient's next
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const int64_t p = k + kr + q * STEP;
      xrow[q] = p < r1 ? x_row(g, p) : -1;
    }
  };
  if constexpr (KIND == kForward) {
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const int64_t r = row0 + q * 32 + (t >> 3);
      xrow[q] = r < end ? x_row(g, r) : -1;
    }
  } else if constexpr (KIND == kWeight) {
    look(r0);
  }
  const Piece zero = {};
  auto load = [&](int64_t k) {
    if (k + ROUND <= r1 && !narrow) {
#pragma unroll
      for (int q = 0; q < PIECES; ++q) {
        const int r = q * 32 + (t >> 3);
        const int64_t ar = row0 + (r < atop ? r : 0), br = n0 + r < btop ? n0 + r : n0;
        const int64_t kk = k + kr + q * STEP;
        if constexpr (KIND == kForward) {
          const T* w = W + br * g.K + k + kp;
          a[q] = all(xrow[q] >= 0 ? X + xrow[q] * g.xs + k + kp : w);
          if (xrow[q] < 0) a[q] = zero;
          b[q] = all(w);
        } else if constexpr (KIND == kInput) {
          a[q] = all(dY + ar * g.dys + k + kp);
          b[q] = all(W + kk * g.K + bcol);
        } else {
          a[q] = all(dY + kk * g.dys + acol);
          b[q] = all(X + (xrow[q] >= 0 ? xrow[q] : 0) * g.xs + bcol);
          if (xrow[q] < 0) b[q] = zero;
        }
        if (aedge) a[q] = moved(a[q], adown);
        if (bedge) b[q] = moved(b[q], bdown);
      }
    } else {
#pragma unroll
      for (int q = 0; q < PIECES; ++q) {
        const int r = q * 32 + (t >> 3);
        const int64_t kk = k + kr + q * STEP;
        if constexpr (KIND == kForward) {
          a[q] = some(X + xrow[q] * g.xs + k + kp, xrow[q] >= 0 ? r1 - k - kp : 0);
          b[q] = some(W + (int64_t)(n0 + r) * g.K + k + kp, n0 + r < cols ? r1 - k - kp : 0);
        } else if constexpr (KIND == kInput) {
          a[q] = some(dY + (row0 + r) * g.dys + k + kp, row0 + r < end ? r1 - k - kp : 0);
          b[q] = some(W + kk * g.K + n0 + c, kk < r1 ? cols - n0 - c : 0);
        } else {
          a[q] = some(dY + kk * g.dys + row0 + c, kk < r1 ? end - row0 - c : 0);
          b[q] = some(X + xrow[q] * g.xs + n0 + c, xrow[q] >= 0 ? cols - n0 - c : 0);
        }
      }
    }
    if constexpr (KIND == kWeight) look(k + ROUND);
  };
  // Bytes from a buffer's start of piece c of row r, and of piece c of reduction row q.
  auto by_row = [](int r, int c) { return r * 128 + (c ^ (r >> 1 & 7)) * 16; };
  auto by_red = [](int q, int c) {
    if constexpr (TY == kEltF32) return q * BM * 4 + (c ^ (q & 4 ? 8 : 0)) * 16;
    else if constexpr (BM == 64) return q * 128 + (c ^ (q & 2 ? 4 : 0)) * 16;
    else return q * BM * 2 + (c ^ (4 * (q & 3))) * 16;
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const int r = by_row(q * 32 + (t >> 3), t & 7), red = by_red(kr + q * STEP, t % ACROSS);
      *reinterpret_cast<Piece*>(lds[buf][0] + (AROW ? r : red)) = a[q];
      *reinterpret_cast<Piece*>(lds[buf][1] + (BROW ? r : red)) = b[q];
    }
  };

  f32x16 acc[TW][TW];
#pragma unroll
  for (int i = 0; i < TW; ++i)
#pragma unroll
    for (int j = 0; j < TW; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  // 16 bits: 8 reduction values of 32 rows; binary32: four (the e of above)
  auto frag = [&](const char* L, int row, int s, auto byrow) {
    if constexpr (decltype(byrow)::value) {
      return *reinterpret_cast<const Piece*>(L + by_row(row + rl, 2 * s + kg));
    } else if constexpr (TY == kEltF32) {
      const int c = row + rl;
      Piece x;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = *reinterpret_cast<const float*>(L + by_red(8 * s + 4 * kg + i, c >> 2) + (c & 3) * 4);
      return x;
    } else {
      const int kr = 16 * s + 8 * kg + ((lane & 15) >> 2);
      const int c = row + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
      typedef __attribute__((address_space(3))) s16x4* P;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(L + by_red(kr, c >> 3) + (c & 7) * 2));
      const s16x4 hi =
          __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(L + by_red(kr + 4, c >> 3) + (c & 7) * 2));
      return __builtin_bit_cast(Piece, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  };
  auto multiply = [&](int buf) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      Piece x[TW], y[TW];
#pragma unroll
      for (int i = 0; i < TW; ++i) {
        x[i] = frag(lds[buf][0], BM / 2 * wm + 32 * i, s, std::integral_constant<bool, AROW>{});
        y[i] = frag(lds[buf][1], BM / 2 * wn + 32 * i, s, std::integral_constant<bool, BROW>{});
      }
#pragma unroll
      for (int i = 0; i < TW; ++i)
#pragma unroll
        for (int j = 0; j < TW; ++j) {
          if constexpr (TY == kEltF32) {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(y[j][v], x[i][v], acc[i][j], 0, 0, 0);
          } else {
            acc[i][j] = mma<TY>(__builtin_bit_cast(s16x8, y[j]), __builtin_bit_cast(s16x8, x[i]),
                                acc[i][j]);
          }
        }
    }
  };
  if (r0 < r1) {
    // (Loads two rounds ahead give nothing: 29 us for 28.)
    load(r0);
    put(0);
    __syncthreads();
    int buf = 0;
    for (int64_t k = r0 + ROUND; k < r1; k += ROUND, buf ^= 1) {
      load(k);
      multiply(buf);
      put(buf ^ 1);
      __syncthreads();
    }
    multiply(buf);
  }

  // acc[i][j][v]: row 32 i + rl, column 32 j + 8 (v / 4) + 4 kg + v % 4 of the wave's part.  The
  // biases, or the input's values that decide over dX, are loaded together before they are
  // needed, those past the last column from the last.
  const bool biased = KIND == kForward && g.b && e < g.E, masked = KIND == kInput && g.relu && e < g.E;
#pragma unroll
  for (int i = 0; i < TW; ++i) {
    const int64_t r = row0 + BM / 2 * wm + 32 * i + rl;
    float with[TW][4][4];
    const int first = n0 + BM / 2 * wn + 4 * kg;
    const int64_t xr = masked && r < end ? x_row(g, r) : -1;
    const bool open = xr >= 0;
    if (biased || open) {
      const int64_t from = biased ? (int64_t)e * g.N : xr * g.xs;
#pragma unroll
      for (int j = 0; j < TW; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int c = first + 32 * j + 8 * q + v;
            const int64_t at = from + (c < cols ? c : cols - 1);
            with[j][q][v] = KIND == kForward ? g.b[at] : rows::load1<TY>(g.X, at);
          }
    }
    if (r >= end) continue;
#pragma unroll
    for (int j = 0; j < TW; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = first + 32 * j + 8 * q;
        if (c >= cols) continue;
        float x[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          x[v] = acc[i][j][4 * q + v];
          if constexpr (KIND == kForward) {
            if (biased) x[v] += with[j][q][v];
            if (g.relu) x[v] = x[v] > 0.f ? x[v] : 0.f;
          } else if constexpr (KIND == kInput) {
            if (masked && !(open && with[j][q][v] > 0.f)) x[v] = 0.f;
          }
        }
        if constexpr (KIND == kWeight || TY == kEltF32) {
          float* out = KIND == kWeight ? dW + r * g.K + c : static_cast<float*>(g.Y) + r * g.ys + c;
          if (c + 4 <= cols) {
            store4(out, f32x4{x[0], x[1], x[2], x[3]});
          } else {
#pragma unroll
            for (int v = 0; v < 3; ++v)
              if (c + v < cols) out[v] = x[v];
          }
        } else {
          uint16_t* out = static_cast<uint16_t*>(g.Y) + r * g.ys + c;
          uint16_t h[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) h[v] = (uint16_t)to_half<TY, false>(x[v], 0u);
          if (c + 4 <= cols) {
            __builtin_memcpy(out, h, 8);
          } else {
#pragma unroll
            for (int v = 0; v < 3; ++v)
              if (c + v < cols) out[v] = h[v];
          }
        }
      }
  }
}

// ------------------------------------------------------------------------ few rows an expert
// The forward product of a small request: its time is that of reading the weights of the
// experts that have rows.  A block of four waves has 16 columns of one expert, a wave every
// fourth 32 reduction values of them; weights and inputs go from memory to registers in the
// form that the 16 x 16 matrix instruction takes (a lane 16 bytes of one row), eight loads of
// weights in flight a wave, up to 64 rows of the expert against them.  The waves' sums are
// added in order through LDS.  (96 rows, 16 experts of 1024 x 1024: 11.7 us, of which about 5 are
// the launch and the chain of loads before the weights'; eight waves a block 15.7 us.)  An expert
// with more rows than that has its weights read again for every 64 of them, one after the other.
constexpr int kFewRows = 64;
template <int TY>
__device__ __forceinline__ f32x4 mma16(s16x8 a, s16x8 b, f32x4 c) {
  if constexpr (TY == kEltBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <int TY, int RT>                                      // RT tiles of 16 rows
__device__ __forceinline__ void few_rows(const Product& g, int e, int n0, int64_t row0,
                                         int64_t end, f32x4 (*red)[4][64]) {
  constexpr int DEEP = 8;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, l = lane & 15, kg = lane >> 4;
  const uint16_t* W = static_cast<const uint16_t*>(g.W) + (int64_t)e * g.N * g.K;
  const uint16_t* wrow = W + (int64_t)(n0 + l < g.N ? n0 + l : g.N - 1) * g.K + 8 * kg;
  const uint16_t* xrow[RT];
  bool there[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t r = row0 + 16 * i + l, x = r < end ? x_row(g, r) : -1;
    there[i] = x >= 0;
    xrow[i] = static_cast<const uint16_t*>(g.X) + (x >= 0 ? x : 0) * g.xs + 8 * kg;
  }
  f32x4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const s16x8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int k0 = 32 * w; k0 < g.K; k0 += 4 * 32 * DEEP) {
    s16x8 a[DEEP], b[DEEP][RT];
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      const int k = k0 + 128 * d;
      const bool in = k + 8 * kg < g.K;                        // K is a multiple of 8
      a[d] = in ? *reinterpret_cast<const s16x8*>(wrow + k) : zero;
#pragma unroll
      for (int i = 0; i < RT; ++i)
        b[d][i] = in && there[i] ? *reinterpret_cast<const s16x8*>(xrow[i] + k) : zero;
    }
#pragma unroll
    for (int d = 0; d < DEEP; ++d)
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[i] = mma16<TY>(a[d], b[d][i], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) red[w][i][lane] = acc[i];
  __syncthreads();
  // a lane has columns 4 kg .. + 4 of row l; wave w finishes tile w
  if (w < RT) {
    const f32x4 s = ((red[0][w][lane] + red[1][w][lane]) + red[2][w][lane]) + red[3][w][lane];
    const int64_t r = row0 + 16 * w + l;
    const int c = n0 + 4 * kg;
    if (r < end && c < g.N) {
      uint32_t h[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float x = s[v];
        if (g.b) x += g.b[(int64_t)e * g.N + c + v];
        if (g.relu) x = x > 0.f ? x : 0.f;
        h[v] = to_half<TY, false>(x, 0u);
      }
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.Y) + r * g.ys + c) =
          make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    }
  }
  __syncthreads();
}

template <int TY>
__global__ __launch_bounds__(kThreads) void few_kernel(Product g) {
  __shared__ f32x4 red[4][4][64];
  const int e = (int)(blockIdx.x / (uint32_t)g.col_tiles);
  const int n0 = (int)(blockIdx.x % (uint32_t)g.col_tiles) * 16;
  int64_t lo, hi;
  bounds_of(g, e, &lo, &hi);
  lo = uniform(lo);
  hi = uniform(hi);
  if (e == g.E) {                                              // positions of no expert
    const int64_t c = n0 + (threadIdx.x & 1) * 8;
    if (c < g.N)
      for (int64_t r = lo + threadIdx.x / 2; r < hi; r += kThreads / 2)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(g.Y) + r * g.ys + c) = make_uint4(0, 0, 0, 0);
    return;
  }
  for (; lo < hi; lo += kFewRows) {
    if (hi - lo <= 16) few_rows<TY, 1>(g, e, n0, lo, hi, red);
    else if (hi - lo <= 32) few_rows<TY, 2>(g, e, n0, lo, hi, red);
    else few_rows<TY, 4>(g, e, n0, lo, hi, red);
  }
}

// db[e, c] = sum of dY over the expert's rows.  Like the weight gradient's reduction it is cut
// into slices (of g.slice rows here), which write db itself or, where an expert has several,
// partial sums [unit, N] that join_kernel adds in order.  A block has one slice and
// LR lanes along the columns, VW columns each, times 256 / LR rows, four of them in flight.
// Bound by reading dY once: 16384 x 1024 in 16 bits 11.4 us, 65536 x 2048 94 us after the weight
// gradient's product, whose stores are still on their way to memory.  (In one launch with the
// plan, in blocks of 1024 threads: 17.2 us for 11.4 + 5.9.)
template <int TY, int VW>
__global__ __launch_bounds__(kThreads) void bias_grad_kernel(Product g, int LR,
                                                             float* __restrict__ db) {
  __shared__ float red[kThreads * VW];
  const int t = threadIdx.x, l = t & (LR - 1), r = t / LR, R = kThreads / LR;
  const int c = ((int)(blockIdx.x % g.col_tiles) * LR + l) * VW;
  Slice u;
  if (!find_slice(g, blockIdx.x / g.col_tiles, -1, &u)) return;
  float s[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) s[e] = 0.f;
  using P = rows::Piece<TY, (VW > 1)>;
  if (c < g.N) {
    int64_t p = u.lo + r;
    for (; p + 3 * R < u.hi; p += 4 * R) {
      P x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i].load(g.dY, (p + i * R) * g.dys + c);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < VW; ++e) s[e] += x[i].v[e];
    }
    for (; p < u.hi; p += R) {
      P x;
      x.load(g.dY, p * g.dys + c);
#pragma unroll
      for (int e = 0; e < VW; ++e) s[e] += x.v[e];
    }
  }
#pragma unroll
  for (int e = 0; e < VW; ++e) red[t * VW + e] = s[e];
  for (int d = kThreads / 2; d >= LR; d >>= 1) {
    __syncthreads();
    if (t < d)
#pragma unroll
      for (int e = 0; e < VW; ++e) red[t * VW + e] += red[(t + d) * VW + e];
  }
  if (t >= LR || c >= g.N) return;
  float* out = u.partial >= 0 ? g.part + u.partial * g.N : db + (int64_t)u.expert * g.N;
#pragma unroll
  for (int e = 0; e < VW; ++e) out[c + e] = red[t * VW + e];
}

// The gradients of the experts with several slices: their partial sums added in order.  The
// first dw_blocks blocks have kJoin elements of one expert's dW each, the others kThreads of one
// expert's db, whose slices (those of h) are shorter.  Bound by reading the partial sums (16 uneven
// experts of 1024 x 1024 13 us, 32 of 2208 x 2048 80 us).
constexpr int kJoin = 16 * kThreads;
__global__ __launch_bounds__(kThreads) void join_kernel(Product g, Product h, int64_t dw_blocks,
                                                        float* __restrict__ db) {
  Slice u;
  if (blockIdx.x >= dw_blocks) {
    const int64_t at = blockIdx.x - dw_blocks;
    const int e = (int)(at / h.col_tiles), c = (int)(at % h.col_tiles) * kThreads + threadIdx.x;
    if (!find_slice(h, 0, e, &u) || u.count < 2 || c >= h.N) return;
    const float* part = h.part + u.partial * h.N + c;
    float s = 0.f;
    int z = 0;
    for (; z + 8 <= u.count; z += 8) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = part[(int64_t)(z + i) * h.N];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += x[i];
    }
    for (; z < u.count; ++z) s += part[(int64_t)z * h.N];
    db[(int64_t)e * h.N + c] = s;
    return;
  }
  const int64_t count = (int64_t)g.N * g.K;
  const int64_t each = (count + kJoin - 1) / kJoin;
  const int e = (int)(blockIdx.x / each);
  if (!find_slice(g, 0, e, &u) || u.count < 2) return;
  const float* part = g.part + u.partial * count;
  float* out = g.dW + e * count;
  int64_t i = (blockIdx.x % each) * kJoin + threadIdx.x * 4;
#pragma unroll
  for (int q = 0; q < kJoin / (4 * kThreads); ++q, i += 4 * kThreads) {
    if (i + 4 <= count) {
      f32x4 s = load4(part + i);
      for (int z = 1; z < u.count; ++z) s += load4(part + z * count + i);
      store4(out + i, s);
    } else {
      for (int64_t j = i; j < count; ++j) {
        float s = part[j];
        for (int z = 1; z < u.count; ++z) s += part[z * count + j];
        out[j] = s;
      }
    }
  }
}

}  // namespace experts

static experts::Product expert_product(const void* X, int64_t xs, int64_t x_rows,
                                       const int32_t* order, int k, const int32_t* offsets,
                                       int64_t n, int E, int K, const void* W, int N) {
  experts::Product g{};
  g.X = X; g.xs = xs; g.x_rows = x_rows; g.order = order;
  // with 2^b >= k: kmul = floor(2^(31 + b) / k) + 1 exceeds the quotient by at most 1, which
  // moves i * kmul / 2^(31 + b) by less than 2^-b <= 1 / k: never past the next integer
  while (((int64_t)1 << g.kshift) < k) ++g.kshift;
  g.kmul = (uint32_t)((((uint64_t)1 << (31 + g.kshift)) / (uint64_t)(k > 0 ? k : 1)) + 1);
  g.offsets = offsets; g.n = n; g.E = E; g.K = K; g.N = N; g.W = W;
  return g;
}

// Rows up to which the few-rows kernel takes the forward product: 16 an expert, and 64.  Times
// of that many rows, and of one more in tiles, of 1024 x 1024 in 16 bits, back to back:
//   experts  rows  even              half in one expert  all in one
//      1       80    9.4 and 15 us
//     16      320   12.1 and 16 us    18 and 16 us         29 and 15 us
//     32      576   21.5 and 17 us    30 and 18 us         51 and 15 us
//    128     2112     76 and 49 us   100 and 61 us        184 and 16 us
//   1024    16448    601 and 570 us  767 and 590 us      1410 and 65 us
// The rule fits up to 16 experts with even rows; beyond, and the more uneven the rows are (which
// the host does not know), fewer rows would do better in tiles already.
static int64_t few_most(int E) { return 16 * (int64_t)E + 64; }

// Row tiles that n rows in E + 1 pieces can need.
static int64_t most_tiles(int64_t n, int E, int BM) { return n / BM + E + 1; }

// Whether a product takes the staged 16-bit kernel: everything in whole 16-byte pieces, and a
// block's rows within 32-bit byte offsets of its first (of X's first, where rows are gathered).
static bool wide_ok(const experts::Product& g, int dtype) {
  auto ok = [](const void* p, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride % 8 == 0 &&
           stride < ((int64_t)1 << 21);          // 256 rows: 2^30 bytes
  };
  if (dtype == kEltF32 || g.K % 8 || g.N % 8) return false;
  if (!ok(g.X, g.xs) || !ok(g.W, g.K) || !ok(g.Y, g.ys) || !ok(g.dY, g.dys)) return false;
  return !g.order || g.x_rows * g.xs < ((int64_t)1 << 31) - ((int64_t)1 << 20);
}

template <int TY, int KIND, int BM, int BN, int WM, int WN>
static hipError_t launch_wide(experts::Product g, hipStream_t s) {
  const int cols = KIND == experts::kForward ? g.N : g.K;
  g.col_tiles = (cols + BN - 1) / BN;
  g.row_tiles = (g.N + BM - 1) / BM;
  const int64_t blocks = KIND == experts::kWeight
                             ? (g.n / g.slice + g.E) * (int64_t)g.row_tiles * g.col_tiles
                             : most_tiles(g.n, g.E, BM) * g.col_tiles;
  // as many blocks as run at once, or the tiles there can be
  const int64_t most = 256 * (BM == 256 ? 1 : 2);
  const int64_t grid = (blocks < most ? blocks : most) + kXcds - 1;
  if constexpr (KIND == experts::kWeight)
    experts::plan_kernel<<<1, experts::kPlanThreads, 0, s>>>(g, const_cast<experts::Plan*>(g.plan));
  const unsigned whole = (unsigned)(grid / kXcds * kXcds), threads = (BM / WM) * (BN / WN) * 64;
  if (KIND == experts::kWeight && g.order)
    experts::wide_kernel<TY, KIND, BM, BN, WM, WN, KIND == experts::kWeight>
        <<<whole, threads, 0, s>>>(g);
  else
    experts::wide_kernel<TY, KIND, BM, BN, WM, WN, false><<<whole, threads, 0, s>>>(g);
  return hipGetLastError();
}

// 256 x 256 tiles, or 128 x 128 ones, two blocks of which share a compute unit.  A round of
// 256 large tiles takes 1 / 0.7 of a round of 512 small ones (1024 x 1024, 16 experts: 25 and
// 16 us), so the choice is by rounds: 8192 rows 29 and 35 us (1 round and 2), 4096 rows 26 and
// 20 us (1 and 1), 65536 rows 162 and 214 us (5 and 9).
static bool big_tiles(int64_t n, int E, int cols) {
  const int64_t big = (n / 256 + E / 2 + 1) * ((cols + 255) / 256);
  const int64_t small = (n / 128 + E / 2 + 1) * ((cols + 127) / 128);
  return (big + 255) / 256 * 10 <= (small + 511) / 512 * 7;
}

template <int TY, int KIND>
static hipError_t launch_product(experts::Product g, bool wide, hipStream_t s) {
  const int cols = KIND == experts::kForward ? g.N : g.K;
  if constexpr (TY != kEltF32) {
    if constexpr (KIND == experts::kForward) {
      if (wide && g.n <= few_most(g.E)) {
        g.col_tiles = (g.N + 15) / 16;
        experts::few_kernel<TY><<<(unsigned)((g.E + 1) * g.col_tiles), experts::kThreads, 0, s>>>(g);
        return hipGetLastError();
      }
    }
    if (wide) {
      if (KIND == experts::kWeight ? g.big : big_tiles(g.n, g.E, cols))
        return launch_wide<TY, KIND, 256, 256, 128, 64>(g, s);
      return launch_wide<TY, KIND, 128, 128, 64, 64>(g, s);
    }
  }
  auto tiles = [&](int BM) {
    g.col_tiles = (cols + BM - 1) / BM;
    g.row_tiles = (g.N + BM - 1) / BM;
    const int64_t units = KIND == experts::kWeight ? (g.n / g.slice + g.E) * g.row_tiles
                                                   : most_tiles(g.n, g.E, BM);
    return units * g.col_tiles;
  };
  if (tiles(128) >= 512) {
    experts::loose_kernel<TY, KIND, 128><<<(unsigned)tiles(128), experts::kThreads, 0, s>>>(g);
  } else {
    experts::loose_kernel<TY, KIND, 64><<<(unsigned)tiles(64), experts::kThreads, 0, s>>>(g);
  }
  return hipGetLastError();
}

static int64_t most_partials(const experts::Product& g) {
  // experts with several slices have more than `slice` rows each
  const int64_t a = 2 * (g.n / g.slice), b = g.n / g.slice + g.E;
  return a < b ? a : b;
}

// Positions a slice of the weight gradient's reduction.  Where every expert once around gives
// the compute units a tile each, only experts well above the mean rows are cut, for a slice
// more costs writing and reading N K sums: above twice the mean, or, where there are fewer than
// two tiles a compute unit, one and a half (product and join of 16384 rows in 16 uneven experts
// of 1024 x 1024, 256 tiles: 96 us with twice, 81 us; 8 experts of 2048 x 2048, 512 tiles: 147
// and 161 us).  Else as many slices as fill the chip.  The two steps are measured at those tile
// counts alone.  With many more tiles a compute unit the cuts still cost their sums: 32 uneven
// experts of 2208 x 2048, nine tiles a compute unit, 80 us for the join beside 622 us for the
// product, and room for up to as many sums as dW has elements.
static void set_slices(experts::Product& g, bool wide) {
  auto across = [&](int64_t t) { return (g.N + t - 1) / t * ((g.K + t - 1) / t); };
  g.big = across(256) * g.E >= 256;
  const int64_t tiles = across(wide ? (g.big ? 256 : 128) : 64);
  int64_t slice = tiles * g.E >= 512 ? 2 * g.n / g.E
                  : tiles * g.E >= 256 ? 3 * g.n / (2 * g.E) : g.n * tiles / 512;
  slice = slice < 512 ? 512 : slice;
  g.slice = (slice + 63) / 64 * 64;
  g.most = most_partials(g);
}

hipError_t launch_expert_dense_fwd(const void* X, int dtype, int64_t xs, int64_t x_rows,
                                   const int32_t* order, int k, const int32_t* offsets, int64_t n,
                                   int E, int K, const void* W, const float* b, int N, bool relu,
                                   void* Y, int64_t ys, hipStream_t s) {
  if (n == 0) return hipSuccess;
  experts::Product g = expert_product(X, xs, x_rows, order, k, offsets, n, E, K, W, N);
  g.b = b; g.relu = relu; g.Y = Y; g.ys = ys;
  return by_type(dtype, [&](auto ty) {
    return launch_product<decltype(ty)::value, experts::kForward>(g, wide_ok(g, dtype), s);
  });
}

// Rows a slice of the bias gradient: at least 256, at most about 1024 slices.
static int64_t bias_slice(int64_t n) {
  const int64_t s = (n + 1023) / 1024;
  return s < 256 ? 256 : s;
}

// The plan of the weight gradient's tiles, at the workspace's start.
constexpr int64_t kPlanFloats = (sizeof(experts::Plan) + 255) / 256 * 64;

size_t expert_dense_bwd_workspace_bytes(int64_t n, int E, int K, int N, int dtype) {
  experts::Product g = expert_product(nullptr, K, n, nullptr, 1, nullptr, n, E, K, nullptr, N);
  // arrays that are not in whole 16-byte pieces may take the other kernel, and its slices
  set_slices(g, false);
  int64_t need = g.most * N * K + kPlanFloats;
  if (dtype != kEltF32 && K % 8 == 0 && N % 8 == 0) {
    set_slices(g, true);
    const int64_t wide = g.most * N * K + kPlanFloats;
    need = wide > need ? wide : need;
  }
  g.slice = bias_slice(n);
  return (size_t)(need + most_partials(g) * N) * sizeof(float) + 256;
}

hipError_t launch_expert_dense_bwd(const void* X, int dtype, int64_t xs, int64_t x_rows,
                                   const int32_t* order, int k, const int32_t* offsets, int64_t n,
                                   int E, int K, const void* W, int N, bool x_relu,
                                   const void* dY, int64_t dys, void* dX, int64_t dxs, float* dW,
                                   float* db, void* workspace, hipStream_t s) {
  experts::Product g = expert_product(X, xs, x_rows, order, k, offsets, n, E, K, W, N);
  g.relu = x_relu; g.dY = dY; g.dys = dys;
  return by_type(dtype, [&](auto ty) {
    constexpr int TY = decltype(ty)::value;
    hipError_t e = hipSuccess;
    if (dX && n > 0) {
      experts::Product h = g;
      if (!x_relu) {                   // X is not read
        h.X = nullptr; h.xs = 0; h.x_rows = 0; h.order = nullptr;
      }
      h.Y = dX; h.ys = dxs;
      e = launch_product<TY, experts::kInput>(h, wide_ok(h, dtype), s);
    }
    // partial sums: the weight gradient's, then the bias gradient's
    float* part = static_cast<float*>(workspace) + kPlanFloats;
    experts::Product h = g, f = g;
    int64_t dw_blocks = 0, db_blocks = 0;
    if (e == hipSuccess && dW) {
      h.W = nullptr;
      h.dW = dW;
      const bool wide = wide_ok(h, dtype) && (reinterpret_cast<uintptr_t>(dW) & 15u) == 0;
      set_slices(h, wide);
      h.plan = static_cast<const experts::Plan*>(workspace);
      h.part = part;
      part += h.most * N * K;
      e = launch_product<TY, experts::kWeight>(h, wide, s);
      if (n > h.slice) dw_blocks = E * (((int64_t)N * K + experts::kJoin - 1) / experts::kJoin);
    }
    if (e == hipSuccess && db) {
      f.slice = bias_slice(n);
      f.most = most_partials(f);
      f.part = part;
      const int VW = TY == kEltF32 ? 4 : 8;
      const bool vec = whole_pieces(reinterpret_cast<uintptr_t>(dY), dys, N, TY == kEltF32 ? 4 : 2);
      const int LR = row_lanes(vec ? N / VW : N), wide = LR * (vec ? VW : 1);
      f.col_tiles = (N + wide - 1) / wide;
      const unsigned blocks = (unsigned)((n / f.slice + E) * f.col_tiles);
      if (vec)
        experts::bias_grad_kernel<TY, VW><<<blocks, experts::kThreads, 0, s>>>(f, LR, db);
      else
        experts::bias_grad_kernel<TY, 1><<<blocks, experts::kThreads, 0, s>>>(f, LR, db);
      e = hipGetLastError();
      f.col_tiles = (N + experts::kThreads - 1) / experts::kThreads;
      if (n > f.slice) db_blocks = (int64_t)E * f.col_tiles;
    }
    if (e == hipSuccess && dw_blocks + db_blocks > 0) {
      experts::join_kernel<<<(unsigned)(dw_blocks + db_blocks), experts::kThreads, 0, s>>>(
          h, f, dw_blocks, db);
      e = hipGetLastError();
    }
    return e;
  });
}

}  // namespace ctr

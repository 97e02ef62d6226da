// Work units of the grouped products: rows sorted by group (expert), group g
// holding the rows [offsets[g], offsets[g + 1]) of the token-side matrices and
// its own weight (or weight-gradient) matrix.
//
//   forward         Y[r,:]  = X[r,:] . W[g]^T       r in group g
//   input gradient  dX[r,:] = dY[r,:] . W[g]
//   weight gradient dW[g]   = sum over r in group g of dY[r,:]^T X[r,:]
//
// The group sizes are known on the device only, so the host launches a
// persistent grid for the largest possible number of units, and every wave
// finds its units by itself: lane l of a wave sums the tile rows of the groups
// [l c, (l + 1) c), c = ceil(groups / 64), and a prefix sum over the lanes,
// held in one register, answers "which lane holds unit u" with one ballot; the
// group among that lane's c is found with scalar loads.  No table in memory
// and no launch before the product.  The rows past the last group form one
// more group without a reduction, whose output rows are written as zeros.
//
// The offsets come from device memory unseen by the host: every use clamps
// them to [0, rows] and a group's end to its start or later, so wrong ones
// give wrong results but no access outside the matrices.  Offsets that descend
// would let groups overlap and the sum of their units pass 32 bits, so forward
// and input gradient write nothing then.
//
// Included by gemm_fast.h inside namespace dpg.
#pragma once

struct GroupedParams : GemmParams {
  const int* offsets;  // groups + 1, on the device; offsets[0] is taken as 0
  int groups;
  int rows;            // rows of the token-side matrices
  int ordered;         // weight gradient: groups by descending size
  int stream;          // outputs of whole 64-byte pieces: non-temporal stores
};

typedef __attribute__((address_space(4))) const int const_int_t;

// rows [first, end) of a group, clamped
__device__ __forceinline__ void group_rows(const int* offsets, int rows, int g, int& first, int& end) {
  const const_int_t* o = (const const_int_t*)(uintptr_t)offsets;
  first = g == 0 ? 0 : min(max(o[g], 0), rows);
  end = min(max(o[g + 1], first), rows);
}

// Weight gradient: a workgroup's units should take equally long in sum, and
// the groups' sizes differ (by 15 times among 64 groups of a skewed router).
// The groups are taken by descending size, each round of the grid going
// through the workgroups in the opposite direction of the one before, so that
// the large and small ones of neighbouring rounds even out.  The order of up
// to kOrderGroups groups is found at the start of every workgroup: each thread
// counts the groups before its own, and lane l of a wave keeps the four groups
// of ranks 4 l .. 4 l + 3 in one register.  65536 rows of 64 skewed groups, 1024 x
// 4096: 566 us in order of size, 631 as they come; of 256 groups, 512 x 2048, 234
// and 233: so many are even enough as they come, and more of them are not ordered.
constexpr int kOrderGroups = 256;

struct GroupMap {
  int per_lane;   // groups of one lane
  int lane_end;   // units of this lane's groups and all before (one value per lane)
  int grouped;    // units of all groups
  int total;      // with those of the rows past the last group
  int tail0;      // first row past the last group
  unsigned order; // weight gradient: four groups by rank
  int place;      // weight gradient: this workgroup's place in a round
};

// `scratch`: (NT + 64) dwords of LDS, free until the call returns
template <int NT>
__device__ __forceinline__ unsigned group_order(const GroupedParams& p, int tid, int* scratch) {
  constexpr int SHARE = NT / kOrderGroups;  // threads of one group
  int* count = scratch;                     // kOrderGroups
  unsigned char* ranked = (unsigned char*)(scratch + NT);
  const int g = tid % kOrderGroups, part = tid / kOrderGroups;
  if (tid < kOrderGroups) {
    int n = -1;
    if (g < p.groups) {
      const int first = g == 0 ? 0 : min(max(p.offsets[g], 0), p.rows);
      n = max(min(max(p.offsets[g + 1], 0), p.rows) - first, 0);
    }
    count[g] = n;
    if (SHARE > 1) count[kOrderGroups + g] = 0;
  }
  __syncthreads();
  const int mine = count[g];
  int before = 0;
  for (int o = part * (kOrderGroups / SHARE); o < min(p.groups, (part + 1) * (kOrderGroups / SHARE)); ++o) {
    const int n = count[o];
    before += n > mine || (n == mine && o < g);
  }
  if (SHARE > 1) {
    atomicAdd(&count[kOrderGroups + g], before);
    __syncthreads();
    before = count[kOrderGroups + g];
  }
  if (tid < kOrderGroups && g < p.groups) ranked[before] = (unsigned char)g;
  __syncthreads();
  const unsigned order = ((const unsigned*)ranked)[tid & 63];
  __syncthreads();  // the LDS becomes the pipeline's
  return order;
}

template <int BM, bool ROWS>
__device__ __forceinline__ GroupMap group_map(const GroupedParams& p, int lane) {
  GroupMap m = {};
  if constexpr (!ROWS) {
    m.total = m.grouped = p.groups * p.tiles_m * p.tiles_n * p.splits;
    return m;
  }
  m.per_lane = (p.groups + 63) >> 6;
  int units = 0;
  int at = 0;
  bool ascending = true;
  const int g0 = lane * m.per_lane;
  if (p.groups > 0 && g0 > 0) at = min(max(p.offsets[min(g0, p.groups)], 0), p.rows);
  for (int i0 = 0; p.groups > 0 && i0 < m.per_lane; i0 += 4) {
    int next[4];  // four loads in flight
#pragma unroll
    for (int i = 0; i < 4; ++i) next[i] = p.offsets[min(g0 + i0 + i + 1, p.groups)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i0 + i >= m.per_lane || g0 + i0 + i >= p.groups) continue;
      const int end = min(max(next[i], 0), p.rows);
      ascending &= end >= at;
      units += (max(end, at) - at + BM - 1) / BM;
      at = end;
    }
  }
  if (__ballot(!ascending) != 0) return m;  // no units
  units *= p.tiles_n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(units, d);
    if (lane >= d) units += v;
  }
  m.lane_end = units;
  m.grouped = __builtin_amdgcn_readlane(units, 63);
  const const_int_t* o = (const const_int_t*)(uintptr_t)p.offsets;
  m.tail0 = p.groups == 0 ? 0 : min(max(o[p.groups], 0), p.rows);
  m.total = (m.grouped + (p.rows - m.tail0 + BM - 1) / BM * p.tiles_n) * p.splits;
  return m;
}

// The K tiles of the unit's split, at least one (which reads zeros).
__device__ __forceinline__ void group_split(const GroupedParams& p, StepCursor& c, int k_tiles) {
  if (p.splits > 1) {
    const SplitParts sp = split_parts(p.splits, k_tiles);
    c.kt0 = split_begin(c.split, sp);
    c.nkt = max(1, split_begin(c.split + 1, sp) - c.kt0);
    // an empty split starts past the reduction
    if (split_begin(c.split + 1, sp) == c.kt0) c.kt0 = k_tiles;
  } else {
    c.nkt = max(1, k_tiles);
  }
}

constexpr int kNoUnit = -(1 << 30);  // past the stream's end, and so is the unit after it

// Unit u of the stream: the units of one group are consecutive, rastered in
// bands of group_m tile rows, and the XCD remap gives each XCD consecutive
// units, so that a group's weight is read into one XCD's L2.
template <int BM, int BN, bool ROWS>
__device__ __forceinline__ StepCursor group_cursor(const GroupedParams& p, const GroupMap& m, int unit) {
  StepCursor c;
  c.kt = c.kt0 = c.split = 0;
  int id;
  if constexpr (ROWS) {
    c.u = unit < m.total ? unit : kNoUnit;
    id = __builtin_amdgcn_readfirstlane(xcd_remap(min(unit, m.total - 1), m.total));
  } else {
    const int round = unit / (int)gridDim.x;
    id = round * (int)gridDim.x + ((round & 1) ? (int)gridDim.x - 1 - m.place : m.place);
    c.u = unit >= 0 && id < m.total ? unit : kNoUnit;
    id = __builtin_amdgcn_readfirstlane(min(max(id, 0), m.total - 1));
  }
  if (p.splits > 1) {
    const int per_split = m.total / p.splits;
    c.split = id / per_split;
    id -= c.split * per_split;
  }
  int t, tiles_m;
  if constexpr (ROWS) {
    const int l = __builtin_popcountll(__ballot(m.lane_end <= id));
    if (l < 64) {
      t = id - (l > 0 ? __builtin_amdgcn_readlane(m.lane_end, l - 1) : 0);
      c.b = l * m.per_lane;
      for (int i = 0;; ++i) {
        int end;
        group_rows(p.offsets, p.rows, c.b, c.base, end);
        c.count = end - c.base;
        tiles_m = (c.count + BM - 1) / BM;
        if (t < tiles_m * p.tiles_n || i + 1 >= m.per_lane || c.b + 1 >= p.groups) break;
        t -= tiles_m * p.tiles_n;
        ++c.b;
      }
      group_split(p, c, p.kt_total);
    } else {
      t = id - m.grouped;
      c.b = p.groups;
      c.base = m.tail0;
      c.count = p.rows - m.tail0;
      tiles_m = (c.count + BM - 1) / BM;
      c.nkt = 1;
    }
  } else {
    c.b = id / (p.tiles_m * p.tiles_n);
    t = id - c.b * (p.tiles_m * p.tiles_n);
    if (p.ordered) c.b = (__builtin_amdgcn_readlane(m.order, c.b >> 2) >> (8 * (c.b & 3))) & 255;
    int end;
    group_rows(p.offsets, p.rows, c.b, c.base, end);
    c.count = end - c.base;
    tiles_m = p.tiles_m;
    group_split(p, c, (c.count + 63) >> 6);
  }
  const int per_band = p.group_m * p.tiles_n;
  const int band = t / per_band;
  const int first_m = band * p.group_m;
  const int band_rows = max(min(tiles_m - first_m, p.group_m), 1);
  const int r = t - band * per_band;
  c.row0 = (first_m + r % band_rows) * BM;
  c.col0 = (r / band_rows) * BN;
  return c;
}

// Where a step's operands lie: element offsets of the group's parts of A and
// B, the rows of A, the step's first reduction index and the reduction's end.
// Steps past the last unit, of the rows past the last group and of an empty
// reduction get kk = K, i.e. empty descriptors.
struct GroupStep {
  int64_t a, b;
  int rows, kk, K;
};

template <bool ROWS>
__device__ __forceinline__ GroupStep group_step(const GroupedParams& p, const StepCursor& c, bool ok) {
  GroupStep s;
  if constexpr (ROWS) {
    const bool live = ok && c.b < p.groups;
    s.a = (int64_t)c.base * p.lda;
    s.b = live ? (int64_t)c.b * p.batch_b : 0;
    s.rows = live ? c.count : c.row0 + 1;
    s.K = p.K;
    s.kk = live ? min((c.kt0 + c.kt) * 64, p.K) : p.K;
  } else {
    s.a = (int64_t)c.base * p.lda;
    s.b = (int64_t)c.base * p.ldb;
    s.rows = p.M;
    s.K = c.count;
    s.kk = ok ? min((c.kt0 + c.kt) * 64, c.count) : c.count;
  }
  return s;
}

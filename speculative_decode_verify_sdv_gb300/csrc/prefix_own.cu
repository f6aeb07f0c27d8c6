// Attention of a batch's window rows to each sequence's own positions, behind a shared prefix.
//
// Per query row r of a kv head and own position p, as everywhere here:
//   s = q_r . k_p;  m = running max of scale s;  P = 2^((scale s - m) log2 e)
//   l += sum P;  O = O 2^(m_old - m) + P V
// What follows a shared prefix is short and there is a lot of it: reading it bounds the kernel,
// and a unit is over before a deep pipeline has filled.  So a CTA of few warps, 16 rows each, takes a
// part of one sequence's positions for one kv head in slices of 32, which come by TMA: the next
// slice's keys while this one's softmax and second product run, its values during the next first
// product.  What is start and end for one CTA is not for the others of its SM.
//
// 256 sequences of 100 to 1001 positions, five rows, 8 heads of 128 (417 MB): 123 us with the join; 64 of
// up to 2001, one row (134 MB): 38 us, 3.5 TB/s, each alone.  Three warps a scheduler, as many as their outputs leave
// registers for, wait for products, copies and one another.  Up to 64 rows have a warp for 16: with two
// row tiles in one warp and groups of 32 rows 256 windows of five rows took 364 us a call for 358,
// one of nine rows 21.7 for 15.5, 64 of them 58.5 for 53.1 (100 positions of their own).  Heads of
// 256, whose outputs fill a warp's registers, have a CTA for 16 rows: 24 tree windows 59.6 us, by four
// warps 61.5.  Loads without TMA were slower, more and shorter parts and two slices ahead no faster.
//
// The products are m16n8k16 MMAs whose operands are read as they lie, 16 bytes a lane.  A dot
// product does not ask for the order of its terms: a lane's 16 bytes of a key row are the reduction
// indices of two MMAs, the queries being taken in the same order.  Nor does an output ask for
// the order of its columns: a lane's 16 bytes of four value rows are one column each of eight
// MMAs, after the halves of two rows have been put side by side.
//
// Window positions that a row does not see have weight 0, their values what is not finite taken
// out; what is not finite among seen ones is told from the values at the end (as in the paged
// attention's kernels).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "attn_tc.h"
#include "prefix_attn.cuh"
#include "prefix_own.cuh"
#include "sdv.h"
#include "sdv_device.cuh"
#include "tc_util.cuh"

namespace sdv {

namespace {

// Positions of a table up to which this kernel is taken.  The paged attention deals any lengths evenly
// and takes some 10 us more in launches; here a part is a chain of slices, 1.2 us each for 128
// columns, and several row groups read everything several times.  Full tables of 32 heads over 8 of
// 128 behind a prefix of 1000, this kernel against the paged attention, us a call: one sequence of
// one row, 4000 positions 20 against 30, 8000 30 against 32, 16,000 50 against 37, eight of them
// 16,000 91 against 102; five rows (two warps), one sequence 2000 22 against 28, 4000 29 against 31,
// sixteen 2000 53 against 57, 4000 81 against 77; 16 rows (four warps), one 1000 22 against 27, 2000
// 27 against 28, 64 of them 500 124 against 142, 1000 161 against 155.
// How full the tables are is known on the device alone: half empty ones (lengths spread evenly) speak for this
// kernel, mostly empty ones more so.  1000 positions, full, half and mostly empty, this kernel's time over
// the paged attention's: 16 rows of 32 heads over 8 of 128, one sequence 0.78, 16 of them 0.97, 0.81, 0.66,
// 64 1.03, 0.85, 0.64; 32 rows (two row groups), four 1.18, 0.89, 0.72, 64 1.16, 0.92, 0.64.
//
// Heads of more than 128 columns have one warp a CTA, and every group of 16 rows reads the sequence
// again.  16 heads over 2 of 256, one group, 16 rows: one sequence of 3000 positions 0.91, 24 of them 0.89, 0.86,
// 0.82, 64 0.97, 0.91, 0.88.  Several groups, by how many there are of all sequences and heads: 40 (four
// sequences of nine rows) 1000 positions 1.05, 0.83, 0.69, 72 1.23, 0.99, 0.68; 96 1.20, 0.96, 0.84; 144 1.32,
// 1.06, 0.86; 160 1.52, 1.12, 0.79; 240 1.17, 1.04, 0.78; 288 1.20, 0.97, 0.78; 640 1.11, 0.96, 0.71; 2000 1.00,
// 0.82, 0.53.  Up to half as many as SMs all parts run at once, from some 1.5 an SM on their rounds
// are full; between, where the mean of the three passes 1, tables of 500: 96 0.86, 0.83, 0.71, 144 0.99, 0.80,
// 0.80, 160 1.00, 0.91, 0.74.
constexpr int kOwnMostOne = 4800;   // one warp, 128 columns, up to 16 cache heads of sequences; more by their number
constexpr int kOwnMostTwo = 3000;   // two warps
constexpr int kOwnMostFour = 1000;  // four, or several row groups
constexpr int kOwnMostWide = 500;   // several of more than 128 columns, half as many in all as SMs to 1.5 an SM
constexpr int kOwnMost = 2048;      // of a part, of a single long sequence
constexpr uint64_t kOwnDrainNs = 100000000ull;  // 0.1 s: copies under way at the end

// What is not finite in column d of the values that a row sees among positions from .. to - 1.
template <typename T>
__device__ __noinline__ uint32_t own_odd(const AttnArgs& a, const int32_t* table, int h, int ctx, int from, int to,
                                         uint32_t word, int d) {
  uint32_t odd = 0;
  for (int p = from; p < to; ++p) {
    if (p >= ctx && !(word >> (p - ctx) & 1u)) continue;
    const int id = __ldcg(table + p / a.page);
    if (id < 0 || id >= a.n_pages) continue;
    const float x = (float)static_cast<const T*>(a.v)[(((long long)id * a.Hkv + h) * a.page + p % a.page) * a.D + d];
    if (!(fabsf(x) < INFINITY)) odd |= x != x ? kOddNan : x > 0.f ? kOddPlus : kOddMinus;
  }
  return odd;
}

// As attn_word, by a coherent load.
__device__ __forceinline__ uint32_t own_word(const AttnArgs& a, int b, int i, int n) {
  if (i >= n) return 0u;
  const uint32_t live = n >= 32 ? 0xffffffffu : (1u << n) - 1u;
  return a.mask != nullptr ? __ldcg(a.mask + (size_t)b * a.S + i) & live : (2u << i) - 1u;
}

constexpr int kSlice = 32;  // positions

// Values of a slice from row `first` on: 0 in rows that are not there, and for what is not finite;
// whether there was any of that.  (A loop of its own: what a warp does once a slice or once a part
// is kept out of the straight code around it, whose instructions come late enough as it is.)
template <typename T, int D, int WARPS>
__device__ __forceinline__ bool own_clean(uint8_t* values, int first, uint32_t there) {
  bool odd = false;
#pragma unroll 1
  for (int e = first * (D / 8) + threadIdx.x; e < kSlice * (D / 8); e += 32 * WARPS) {
    const int row = e / (D / 8), ch = e % (D / 8);
    uint4* const at = reinterpret_cast<uint4*>(values + (ch >> 3) * (kSlice * 128) + row * 128 + (((ch ^ row) & 7) << 4));
    if (!(there >> row & 1u)) {
      *at = make_uint4(0, 0, 0, 0);
      continue;
    }
    uint4 x = *at;
    uint32_t* const w = reinterpret_cast<uint32_t*>(&x);
    bool any = false;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const uint32_t bad = nonfinite16<T>(w[y]);
      any |= bad != 0;
      w[y] &= (bad & 1u ? 0xffff0000u : 0xffffffffu) & (bad & 2u ? 0x0000ffffu : 0xffffffffu);
    }
    if (any) *at = x;
    odd |= any;
  }
  return odd;
}

// A lane's outputs of a row, 16 columns of every 64 from `first` on, once more where they are not
// finite (`all`: where they are, too): what the row's values say.
template <typename T>
__device__ __noinline__ void own_mend(const AttnArgs& a, const int32_t* table, int h, int ctx, int from, int to,
                                      uint32_t word, float* row, int first, bool all) {
  for (int d = first; d < a.D; d = (d & 15) == 15 ? d + 49 : d + 1) {
    if (!all && fabsf(row[d]) < INFINITY) continue;
    const uint32_t odd = own_odd<T>(a, table, h, ctx, from, to, word, d);
    if (odd) row[d] = odd_value(odd);
  }
}

template <int D, int WARPS>
struct OwnPlan {
  static constexpr int R = 16 * WARPS;
  static constexpr int kHalf = kSlice * D * 2;    // a slice's keys, its values
  static constexpr int LQ = D * 2 + 64;           // bytes between query rows: eight lanes' 16-byte reads meet no bank twice
  static constexpr int kSmem = 1024 + 2 * kHalf + R * LQ + 16;
};

struct OwnMaps {
  CUtensorMap k, v;
};

// The CTA's warps, and whether the condition holds in all (one) of them.
template <int WARPS>
__device__ __forceinline__ bool all_of(bool x) {
  if constexpr (WARPS > 1) return __syncthreads_and(x);
  __syncwarp();
  return x;
}
template <int WARPS>
__device__ __forceinline__ bool one_of(bool x) {
  if constexpr (WARPS > 1) return __syncthreads_or(x);
  return __any_sync(0xffffffffu, x);
}

template <typename T, int D, int WARPS, bool LAST>
__global__ void __launch_bounds__(32 * WARPS, (D > 128 ? 8 : 12) / WARPS)
    prefix_own_kernel(const __grid_constant__ OwnMaps maps, const __grid_constant__ JoinArgs join) {
  using PL = OwnPlan<D, WARPS>;
  constexpr int R = PL::R, DB = D / 64, KB = D / 32, LQ = PL::LQ, NT = kSlice / 8, BLOCK = kSlice * 128;
  constexpr float kLift = std::is_same<T, __nv_bfloat16>::value ? -kPrefixDrop : 6.f;  // P's power of two
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const sb = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  uint8_t* const mem = sb + 2 * PL::kHalf + warp * 16 * LQ;  // the warp's queries
  const uint32_t bars = base + 2 * PL::kHalf + R * LQ;  // of the keys' place, then the values'
  const OwnArgs& o = join.own;
  const AttnArgs& a = o.attn;
  // the prefix's parts first; of a sequence all first parts, then all second ones
  const int prefix_ctas = a.Hkv * o.prefix_parts, cta = (int)blockIdx.x - prefix_ctas;
  const bool shared = cta < 0;
  const int units = shared ? a.Hkv : a.B * a.Hkv * o.row_groups, at = shared ? (int)blockIdx.x : cta;
  const int y = at / units, unit = at - y * units;
  const int rg = shared ? 0 : unit % o.row_groups, bh = shared ? unit : unit / o.row_groups, h = bh % a.Hkv,
            b = bh / a.Hkv;  // (the rows of all sequences are those of "sequence" 0, were it that long)
  if (threadIdx.x == 0) {
    set_wait_limit(a.fault);
    mbar_init(bars, 1);
    mbar_init(bars + 8, 1);
    fence_barrier_init();
  }
  // Queries, lengths, tables and pages may be what launches in front of this call have written: they are read
  // behind the wait, or, beside the prefix's launch, behind the word that passes its wait on, by coherent
  // loads; then that launch is waited for at the end, for its partials and for the launch behind.
  unsigned* const word = join.prefix.passed;
  bool beside = false;
  if (o.prefix_parts == 0) {
    beside = passed_on(word);
    if constexpr (WARPS > 1) beside = __syncthreads_and(beside);
    else beside = __all_sync(0xffffffffu, beside);
  }
  if (!beside) griddep_wait();
  if (o.prefix_parts > 0 && blockIdx.x + 1 == gridDim.x) {  // the first launch: to the join
    if (threadIdx.x == 0) pass_on(word);
    all_of<WARPS>(true);
  }
  griddep_launch_dependents();
  AttnSeq seq;
  if (shared) {
    seq.ctx = prefix_length(o.prefix_length, o.prefix_pages, a.page, seq.bad);
    seq.n = a.B * a.S;
    seq.tiles = (seq.ctx + kOwnTile - 1) / kOwnTile;
  } else {
    seq = attn_seq(a, b);
  }
  const int ctx = seq.ctx, n = seq.n, total = shared ? ctx : ctx + n;
  const int per = own_per_part(seq.tiles, shared ? o.prefix_parts : o.parts);
  const int from = y * per * kOwnTile, to = min(from + per * kOwnTile, total);
  if (y > 0 && from >= total) return;
  if (seq.bad && threadIdx.x == 0) atomicOr(o.status, kDevErrIndex);
  all_of<WARPS>(true);
  const int r0 = rg * R + warp * 16, rows = shared ? n * a.G : a.rows;
  const int32_t* const table = shared ? o.prefix_table : a.table + (size_t)b * a.max_pages;
  // ---- the copies: slice i is positions from + 32 i .. + 31 ----
  const int page_log = 31 - __clz(a.page), box = min(a.page, kSlice), boxes = kSlice / box;
  const int slices = rg * R < n * a.G ? (to - from + kSlice - 1) / kSlice : 0;  // none for rows behind the window's end
  const bool busy = WARPS == 1 || r0 < min(n * a.G, rows);  // whether the warp has a row (of a CTA with some)
  const int beyond = a.n_pages * a.Hkv * a.page;  // a row past the tensor map's end: zeros
  const uint64_t policy = l2_policy_evict_first();
  // a lane's copy: a block of 64 elements, a page's part of the slice
  const int cb = lane % DB, bx = lane / DB;
  const bool mine = warp == 0 && bx < boxes;
  const uint32_t dst = base + cb * BLOCK + bx * box * 128;
  auto page_of = [&](int i) {  // of the lane's copy in slice i; -1 past the end
    const int p = from + kSlice * i + bx * box;
    return mine && i < slices && p < to ? __ldcg(table + (p >> page_log)) : -1;
  };
  auto row_of = [&](int i, int id) {
    const int p = from + kSlice * i + bx * box;
    return id >= 0 && id < a.n_pages ? (id * a.Hkv + h) * a.page + (p & (a.page - 1)) : beyond;
  };
  auto issue = [&](int i, int values, int row) {
    if (!values && i + 1 == a.fault.withhold) return;  // (the timeout path's test)
    if (lane == 0) mbar_arrive_expect_tx(bars + 8u * values, PL::kHalf);
    __syncwarp();
    if (mine) tma_load_2d(dst + values * PL::kHalf, values ? &maps.v : &maps.k, cb * 64, row, bars + 8u * values, policy);
  };
  int row_next = beyond, id_after = page_of(1);
  if (slices > 0 && warp == 0) {
    fence_proxy_async_global();
    const int row = row_of(0, page_of(0));
    issue(0, 0, row);
    issue(0, 1, row);
  }
  for (int e = lane; e < 16 * (D / 8); e += 32) {
    const int r = e / (D / 8), ch = e % (D / 8), row = r0 + r;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (row < rows && row / a.G < n)
      x = __ldcg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + ((long long)b * a.S + row / a.G) * a.q_stride +
                                                (h * a.G + row % a.G) * D) + ch);
    *reinterpret_cast<uint4*>(mem + r * LQ + ch * 16) = x;
  }
  uint32_t words[2];  // visibility of rows g and g + 8
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = r0 + half * 8 + g;
    words[half] = row < rows && !shared ? own_word(a, b, row / a.G, n) : 0u;
  }
  auto live = [&](int half) {
    const int row = r0 + half * 8 + g;
    return row < rows && row / a.G < n;
  };
  // Pages of the part that cannot be followed make every slice look for them.
  bool some_absent = false;
  if (from < to)
    for (int e = (from >> page_log) + lane; e <= (to - 1) >> page_log; e += 32) {
      const int id = __ldcg(table + e);
      some_absent |= id < 0 || id >= a.n_pages;
    }
  some_absent = __any_sync(0xffffffffu, some_absent);
  if (some_absent && threadIdx.x == 0) atomicOr(o.status, kDevErrIndex);
  __syncwarp();
  float out[8 * DB][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  bool odd_values = false, ok = true, next_keys = false;
#pragma unroll
  for (int j = 0; j < 8 * DB; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) out[j][e] = 0.f;
  // operands' places: key row g, value row 2 c, under the 128-byte swizzle
  const uint8_t* const ks = sb + g * 128;
  const uint8_t* const vs = sb + PL::kHalf + c * 256;
  const int k_chunk[2] = {(c ^ g) << 4, ((4 + c) ^ g) << 4};
  const int v_chunk[2] = {(g ^ (2 * c)) << 4, (g ^ (2 * c + 1)) << 4};
  const uint8_t* const qs = mem + g * LQ + c * 16;
  int i = 0;
  for (; i < slices; ++i) {
    const int p0 = from + kSlice * i;
    const bool more = i + 1 < slices;
    row_next = row_of(i + 1, id_after);
    id_after = page_of(i + 2);
    next_keys = false;
    ok = mbar_wait_warp(bars, i & 1, o.status);
    const bool edge = p0 + kSlice > ctx || some_absent;
    float s[NT][4];
    if (busy) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        uint4 kx[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
          kx[j] = *reinterpret_cast<const uint4*>(ks + (kb >> 1) * BLOCK + j * 1024 + k_chunk[kb & 1]);
        const uint4 lo = *reinterpret_cast<const uint4*>(qs + kb * 64);
        const uint4 hi = *reinterpret_cast<const uint4*>(qs + 8 * LQ + kb * 64);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma16816<T>(s[j], lo.x, hi.x, lo.y, hi.y, kx[j].x, kx[j].y);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma16816<T>(s[j], lo.z, hi.z, lo.w, hi.w, kx[j].z, kx[j].w);
      }
    }
    ok = all_of<WARPS>(ok);  // every lane has read the keys
    if (!ok) break;
    if (more && warp == 0) issue(i + 1, 0, row_next);
    next_keys = more;
    uint32_t there = 0xffffffffu;  // positions that are there
    if (edge) {
      there = to - p0 >= 32 ? 0xffffffffu : (1u << (to - p0)) - 1u;
      if (some_absent) {
        int e = -1;
        if (p0 + lane < to) e = __ldcg(table + ((p0 + lane) >> page_log));
        there &= __ballot_sync(0xffffffffu, e >= 0 && e < a.n_pages);
      }
    }
    uint32_t p16[2][NT];  // packed pairs
    if (busy) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x[2 * NT];
#pragma unroll
        for (int e = 0; e < 2 * NT; ++e) x[e] = s[e >> 1][half * 2 + (e & 1)] * a.scale_log2;
        if (edge) {
          const uint32_t see = live(half) ? there & attn_visible(p0, ctx, words[half]) : 0u;
#pragma unroll
          for (int e = 0; e < 2 * NT; ++e)
            if (!(see >> ((e >> 1) * 8 + c * 2 + (e & 1)) & 1u)) x[e] = -INFINITY;
        }
        float mx = x[0];
#pragma unroll
        for (int e = 1; e < 2 * NT; ++e) mx = fmaxf(mx, x[e]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const bool grow = mx > m[half] + 8.f;  // also from -inf to any number
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow && m[half] != -INFINITY ? exp2_approx(m[half] - mx) : 1.f;
          if (grow) m[half] = mx;
          l[half] *= f;
#pragma unroll
          for (int j = 0; j < 8 * DB; ++j) {
            out[j][half * 2] *= f;
            out[j][half * 2 + 1] *= f;
          }
        }
        const float ref = m[half] == -INFINITY ? -kLift : m[half] - kLift;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 2 * NT; e += 2) {
          const float y0 = exp2_approx(x[e] - ref), y1 = exp2_approx(x[e + 1] - ref);
          sum += y0 + y1;
          p16[half][e >> 1] = pack16<T>(y0, y1);
        }
        l[half] += sum;
      }
    }
    ok = mbar_wait_warp(bars + 8, i & 1, o.status);
    if (edge && p0 + kSlice > ctx) {  // what is not finite must not meet a weight of 0
      odd_values |= own_clean<T, D, WARPS>(sb + PL::kHalf, max(ctx - p0, 0), there);
      fence_proxy_async_smem();  // before the next values' copy
      all_of<WARPS>(true);
    }
    if (busy) {
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int k = 0; k < NT / 2; ++k) {
          uint4 vx[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int row = k * 16 + (z & 1) + (z >> 1) * 8;  // + 2 c
            vx[z] = *reinterpret_cast<const uint4*>(vs + d * BLOCK + row * 128 + v_chunk[z & 1]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t sel = e & 1 ? 0x7632u : 0x5410u;
            uint32_t v[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) v[z] = reinterpret_cast<const uint32_t*>(&vx[z])[e >> 1];
            const uint32_t b0 = __byte_perm(v[0], v[1], sel), b1 = __byte_perm(v[2], v[3], sel);
            mma16816<T>(out[d * 8 + e], p16[0][2 * k], p16[1][2 * k], p16[0][2 * k + 1], p16[1][2 * k + 1], b0, b1);
          }
        }
    }
    ok = all_of<WARPS>(ok);  // every lane has read the values
    if (!ok) break;
    if (more && warp == 0) issue(i + 1, 1, row_next);
  }
  if (!ok) {  // the copies under way have to land before the CTA ends: this slice's, and the next keys
    if (i + 1 != a.fault.withhold) mbar_wait_bounded(bars, i & 1, kOwnDrainNs);
    mbar_wait_bounded(bars + 8, i & 1, kOwnDrainNs);
    if (next_keys && i + 2 != a.fault.withhold) mbar_wait_bounded(bars, (i + 1) & 1, kOwnDrainNs);
  }
  odd_values = one_of<WARPS>(odd_values);
  const size_t part = (size_t)y * a.B * a.S * a.Hq;
  float* const part_o = shared ? o.prefix_o : o.part_o;
  float2* const part_ml = shared ? o.prefix_ml : o.part_ml;
  // with the join: where the prefix's partials of a row lie
  const PrefixArgs& pre = join.prefix;
  long long pre_total = 0;
  int pre_tiles = 0, pre_live = 0;
  if constexpr (LAST) {
    if (beside) griddep_wait();
    bool bad;  // (reported by that launch)
    pre_tiles = prefix_tiles(pre, prefix_length(pre, bad));
    pre_total = (long long)pre_tiles * pre.units;
    pre_live = attn_live_ctas(pre.ctas, pre_total);
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float sum = l[half];
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    const int row = r0 + half * 8 + g;
    if (LAST ? row >= rows : !live(half)) continue;  // (nor does the join read these)
    const long long orow = ((long long)b * a.S + row / a.G) * a.Hq + h * a.G + row % a.G;
    float* const dst = part_o + (part + orow) * D;
    // (a row that saw nothing has weights 0 only: its O is 0, or NaN by 0 * inf)
    const bool none = sum == 0.f;
    float top = m[half] == -INFINITY || none ? -INFINITY : m[half] - kLift;
    bool finite = true;
#pragma unroll
    for (int e = 0; e < 8 * DB; ++e)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        if (none) out[e][half * 2 + z] = 0.f;
        finite &= fabsf(out[e][half * 2 + z]) < INFINITY;
      }
    const bool odd = sum > 0.f && (odd_values || !finite);  // (NaN scores, a padding row's for one, leave NaN)
    if (!LAST || (odd && live(half))) {
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int e = 0; e < 16; e += 4) {  // a lane's 16 columns of a row lie side by side
          const int col = half * 2 + (e >> 3), j = d * 8 + (e & 7);
          *reinterpret_cast<float4*>(dst + d * 64 + c * 16 + e) =
              make_float4(out[j][col], out[j + 1][col], out[j + 2][col], out[j + 3][col]);
        }
      if (odd) own_mend<T>(a, table, h, ctx, from, to, words[half], dst, c * 16, odd_values);
    }
    if constexpr (!LAST) {
      if (c == 0) part_ml[part + orow] = make_float2(top, sum);
    } else {
      if (odd && live(half)) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) out[d * 8 + (e & 7)][half * 2 + (e >> 3)] = dst[d * 64 + c * 16 + e];
      }
      const int at = (b * a.S + row / a.G) * a.G + row % a.G;  // among all rows of the kv head
      const int rt = at / pre.row_tile, r = at - rt * pre.row_tile;
      const int unit = h * ((pre.row_tiles + pre.unit_tiles - 1) / pre.unit_tiles) + rt / pre.unit_tiles;
      const long long first = (long long)unit * pre_tiles;
      const int count = live(half) && pre_tiles > 0 ? attn_owner(pre_total, pre_live, first + pre_tiles - 1) -
                                                          attn_owner(pre_total, pre_live, first) + 1
                                                    : 0;
      const long long step = (long long)pre.unit_tiles * pre.row_tile;
      const long long place = ((long long)unit * pre.sharers * pre.unit_tiles + rt % pre.unit_tiles) * pre.row_tile + r;
#pragma unroll 1
      for (int k = 0; k < count; ++k) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(pre.part_ml) + place + k * step);
        const float4* const po = reinterpret_cast<const float4*>(pre.part_o + (place + k * step) * D) + c * 4;
        if (ml.x == -INFINITY && ml.y == 0.f) continue;
        const float mn = fmaxf(top, ml.x), f = exp2f(top - mn), f2 = exp2f(ml.x - mn);
        top = mn;
        sum = sum * f + ml.y * f2;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 x = __ldcg(po + d * 16 + e / 4);
            const int col = half * 2 + (e >> 3), j = d * 8 + (e & 7);
            out[j][col] = weighted<true>(out[j][col], f) + weighted<true>(x.x, f2);
            out[j + 1][col] = weighted<true>(out[j + 1][col], f) + weighted<true>(x.y, f2);
            out[j + 2][col] = weighted<true>(out[j + 2][col], f) + weighted<true>(x.z, f2);
            out[j + 3][col] = weighted<true>(out[j + 3][col], f) + weighted<true>(x.w, f2);
          }
      }
      const bool empty = !live(half) || sum == 0.f;
      const float inv = 1.f / sum;
      uint4* const to16 = reinterpret_cast<uint4*>(static_cast<T*>(join.out) + orow * D) + c * 2;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int col = half * 2 + z;
          auto two = [&](int e) { return empty ? 0u : pack16<T>(out[d * 8 + e][col] * inv, out[d * 8 + e + 1][col] * inv); };
          to16[d * 8 + z] = make_uint4(two(0), two(2), two(4), two(6));
        }
      if (c == 0 && join.lse != nullptr)
        join.lse[orow] = empty ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    }
  }
  if (!LAST && beside) griddep_wait();
  // (whoever starts from here on finds the prefix's launch ended; where a join follows, it does this)
  if (LAST && cta == 0 && threadIdx.x == 0) *word = 0;
}

template <typename T, int D, int WARPS, bool LAST>
cudaError_t own_launch(const OwnMaps& m, const JoinArgs& j, cudaStream_t st) {
  auto kernel = prefix_own_kernel<T, D, WARPS, LAST>;
  constexpr int smem = OwnPlan<D, WARPS>::kSmem;
  static std::atomic<unsigned long long> ready{0};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  const OwnArgs& a = j.own;
  const unsigned ctas = (unsigned)a.attn.Hkv * a.prefix_parts + (unsigned)a.attn.B * a.attn.Hkv * a.row_groups * a.parts;
  return launch_pdl(kernel, dim3(ctas), dim3(32 * WARPS), smem, st, m, j);
}

template <typename T, int D, int WARPS>
cudaError_t own_dispatch(const OwnMaps& m, const JoinArgs& j, bool last, cudaStream_t st) {
  if constexpr (D <= 128)
    if (last) return own_launch<T, D, WARPS, true>(m, j, st);
  return own_launch<T, D, WARPS, false>(m, j, st);
}
template <typename T>
cudaError_t own_dispatch(const OwnMaps& m, const JoinArgs& j, bool last, cudaStream_t st) {
  switch (j.own.attn.D + j.own.warps) {  // (heads of 256 have one warp)
    case 64 + 1: return own_dispatch<T, 64, 1>(m, j, last, st);
    case 64 + 2: return own_dispatch<T, 64, 2>(m, j, last, st);
    case 64 + 4: return own_dispatch<T, 64, 4>(m, j, last, st);
    case 128 + 1: return own_dispatch<T, 128, 1>(m, j, last, st);
    case 128 + 2: return own_dispatch<T, 128, 2>(m, j, last, st);
    case 128 + 4: return own_dispatch<T, 128, 4>(m, j, last, st);
    case 256 + 1: return own_dispatch<T, 256, 1>(m, j, last, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

bool own_takes(const OwnArgs& o, int sms) {
  const AttnArgs& a = o.attn;
  const long long positions = (long long)a.max_pages * a.page, units = (long long)a.B * a.Hkv;
  const long long groups = units * o.row_groups;
  const bool wide = a.D > 128 && 2 * groups > sms && 2 * groups < 3 * sms;
  const long long most = o.row_groups > 1 ? (wide ? kOwnMostWide : kOwnMostFour)
                         : o.warps == 4   ? kOwnMostFour
                         : o.warps == 2   ? kOwnMostTwo
                                          : kOwnMostOne * 128 / a.D * (units > 16 ? units : 16) / 16;
  return positions <= most && positions <= (long long)kOwnMost * o.parts;
}

cudaError_t launch_prefix_own(int dtype, const JoinArgs& j, bool last, cudaStream_t st) {
  OwnMaps m;
  const AttnArgs& t = j.own.attn;
  const uint64_t rows = (uint64_t)t.n_pages * t.Hkv * t.page;
  const int box = t.page < kSlice ? t.page : kSlice;
  const bool bf = dtype == SDV_BF16;
  if (!attn_page_map(t.k, bf, rows, t.D, box, &m.k) || !attn_page_map(t.v, bf, rows, t.D, box, &m.v))
    return cudaErrorUnknown;
  return bf ? own_dispatch<__nv_bfloat16>(m, j, last, st) : own_dispatch<__half>(m, j, last, st);
}

}  // namespace sdv

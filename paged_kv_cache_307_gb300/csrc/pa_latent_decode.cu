// pa_latent_decode.cu — attention over a paged cache of one latent vector a token, in the
// absorbed form (pa_latent_decode), on the 5th-generation tensor cores: the cached rows are
// the keys, and their latent part the values.
//
// Rows of a sequence are (query position, head) pairs.  A CTA takes NR = 16, 32 or 64 of them
// against tiles of 128 tokens, tokens in the accumulators' lanes:
//   S^T[128 tokens x NR] = C[128 x (R + P)] Q^T     A = the tile (K-major), B = Q rows
//   O^T[R dims x NR]    += C^T[R x 128] P^T         A = the same bytes (MN-major), B = P
// so a tile is read into shared memory once for both products, and few heads cost few
// columns and not padded rows.  R = 512 with 64 rows: O^T takes 256 columns of tensor
// memory, S^T two buffers of 64.
//
// Bound by HBM up to 64 rows a sequence: 64 requests x 16 heads over U[1024, 16384] take 108 to
// 112 us in a replayed graph (644 MB; 6.5 TB/s, 96 % of the copy rate, while all CTAs have tiles; 5.8
// with the start, the last tiles and the join), 116 through the call with inputs that change.  With 128 heads two CTAs read the same tiles (DRAM traffic
// is that of one: 340 MB) and the chain of a tile bounds them: 64 requests over U[1024, 8192]
// take 126 us (654 TFLOP/s), about 6500 clocks a tile, of which the 68 MMAs are 3700 (an MMA of
// M = 128 costs 48 clocks whatever is below 64 columns: its A operand's way out of shared
// memory), the softmax between them 1500, waits for the copies into the slots that the second
// product leaves 900.  Shared memory (Q 72 KB, a tile 144 KB) holds no second tile to fill those.
// A short call (2 contexts of up to 300 tokens, 9.6 us) is latency: of a CTA's 11000 clocks 3000 go
// until the first copy (lengths, cuts; mostly code met for the first time), 3500 until the first
// scores, 2500 in softmax and values, 1500 to 2000 until the rows are out; the join takes 2 us.
//
//  * The batch is a line of (sequence, row groups, tile) units, cut into equal parts for one
//    CTA an SM (Walk): no tail of long contexts, at most two partial results a CTA, and a
//    second kernel joins what a cut divides.
//  * Copies: a warp gets a TMA copy out in about 60 clocks whatever its size, and a tile is 72 boxes
//    of 2 KB (its chunks are apart in shared memory, so that the scores may begin with the first
//    pair of chunks): three warps share them (one warp: 153 us where 117 came of four).
//  * A slot of the ring is the 128 latent elements of one M = 128 product of O^T: it is free
//    again when that product is done, while the other products still run.
//  * The MMA warp keeps its descriptors in uniform registers (99 clocks an MMA where 49 do).
//  * The references of the softmax are common to the 128 threads of a column, 2^8 above the maximum that
//    set them, and move only when a score exceeds one: a barrier with a vote a tile; then O^T is scaled
//    in tensor memory.
//  * P lies over the rotated keys' chunk, which the scores are done with, where a tile is large.  It is
//    bf16, as the cached rows are that it meets (both operands have one type), 2^-9 of a weight on
//    average beside the output's own 2^-9; the sum that divides keeps the weights in 32 bits.
//  * Every wait is bounded (2 s); a timeout sets PA_DEV_TIMEOUT, and the roles wind down.
#include <stddef.h>

#include "pa_mma.cuh"
#include "pa_tc.cuh"

namespace pa {
namespace {

__device__ unsigned g_status_latent;

constexpr int kTile = 128;                   // tokens per tile
// Warps: softmax, SUB for each quarter of the accumulators' lanes (the columns divided among them),
// then three of TMA and one of MMA.
constexpr int subs(int nr) { return nr == 64 ? 4 : 2; }
constexpr int threads(int nr) { return 128 * subs(nr) + 128; }
constexpr uint32_t kChunk = 16384;           // 128 tokens x 64 elements
constexpr uint32_t kPair = 2 * kChunk;       // 128 elements: one M = 128 product of O^T
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;                // log2 units that a new reference is above its score
constexpr float kUnset = 3e38f;              // minus a reference that is not there yet
constexpr uint32_t kSmemMax = 232448;        // 227 KB
constexpr int kMaxSlots = 6;

struct LatentParams {
  __nv_bfloat16* out;
  const __nv_bfloat16* cache;                // for values that are not finite; the tiles go by the tensor map
  const int32_t* query_start;                // null: one row a sequence
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* ws_o;                               // [2 * CTAs, R / 128, NR / 4, 128, 4] partial sums
  float* ws_ml;                              // [2 * CTAs, NR, 2] their maximum and sum
  int4* ws_join;                             // [CTAs] what the CTA begins and others go on with: first row, rows, those others, its slot
  int B, H, R, P, rows, max_blocks, bs, num_blocks;
  int cl;                                    // CTAs that take neighbouring row groups over the same tokens
  float qscale;
};

template <int NR>
struct Shared {
  uint64_t full[kMaxSlots], empty[kMaxSlots], full_r[2], empty_r[2];
  uint64_t q_full, q_empty, s[2], p, pv, o_free, drain;
  alignas(16) float neg_m[NR];               // minus the reference of every row
  alignas(16) float f[NR];
  alignas(16) float red[4][NR];              // per warp: maxima, at the end sums
  alignas(16) uint4 turn[4 * subs(NR)][32];  // per warp: 8 columns of 32 dims on their way out
  int scan[threads(NR) / 32];
  unsigned first_off;
  int first_b;
  uint32_t tmem_base;
  int abort;
  unsigned odd;                              // the row group that values were taken out for: its first unit's place + 1
};

// Shared memory: Q [NC chunks][NR rows][128 B], a ring of SLOTS pairs, the rotated keys' chunk
// (P behind it where two of them and P's own 16 KB leave no room for a second tile's first pair).
template <int NR, int RC>
struct Layout {
  static constexpr int NC = RC + 1, NP = RC / 2;
  static constexpr bool kAlias = RC >= 6;
  static constexpr uint32_t kQ = NC * NR * 128u;
  static constexpr uint32_t kFixed = kQ + (kAlias ? kChunk : 3 * kChunk) + (uint32_t)sizeof(Shared<NR>) + 1024u;
  static constexpr int kFit = (int)((kSmemMax - kFixed) / kPair);
  static constexpr int kSlots = kFit < kMaxSlots ? kFit : kMaxSlots;
  static constexpr uint32_t kOffRing = kQ, kOffRope = kOffRing + kSlots * kPair;
  static constexpr uint32_t kOffP = kAlias ? kOffRope : kOffRope + 2 * kChunk;
  static constexpr uint32_t kOffShared = kOffP + kChunk;
  static constexpr uint32_t kBytes = kOffShared + (uint32_t)sizeof(Shared<NR>) + 1024u;
  static constexpr uint32_t kCols = 2 * NR + NP * NR;
  static constexpr uint32_t kTmem = kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kSlots >= NP && kBytes <= kSmemMax, "shared memory");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// Barrier 2 of the N softmax threads, true for all if true for any.
template <int N>
__device__ __forceinline__ bool vote(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 2, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(x ? 1u : 0u), "n"(N) : "memory");
  return r != 0;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(smem_u32(bar), parity)) return true;
  if (*abort_flag) return false;
  if (mbar_wait(bar, parity)) return true;
  atomicOr(&g_status_latent, PA_DEV_TIMEOUT);
  *abort_flag = 1;
  return false;
}

// A sequence: its first row, rows, context, and tiles (one at least, which writes the zeros).
struct Seq {
  int q0, n, L, tiles;
};
__device__ __forceinline__ Seq seq_of(const LatentParams& p, int b, bool flag) {
  Seq s{b, 1, 0, 1};
  if (p.query_start) {
    s.q0 = __ldg(&p.query_start[b]);
    const int e = __ldg(&p.query_start[b + 1]);
    s.n = s.q0 >= 0 && e >= s.q0 && e <= p.rows ? e - s.q0 : -1;
  }
  const int L = __ldg(&p.context_lens[b]), most = p.max_blocks * p.bs;
  s.L = L < 0 ? 0 : min(L, most);
  if (flag && (s.n < 0 || s.L != L)) atomicOr(&g_status_latent, PA_DEV_BAD_LEN);
  if (s.n < 0) s.n = 0;
  s.tiles = max(1, (s.L + kTile - 1) / kTile);
  return s;
}
__device__ __forceinline__ int supers_of(const LatentParams& p, const Seq& s, int nr) {
  return ((s.n * p.H + nr - 1) / nr + p.cl - 1) >> (p.cl - 1);               // (cl is 1 or 2)
}

// The line of `total` units in at most `parts` parts, none of them empty: the first `longer` of
// `len` + 1 units, the rest of `len`.  (The host refuses what could be 2^31 units.)
struct Cuts {
  unsigned len, longer, n;
  Cuts() = default;
  __device__ __forceinline__ Cuts(unsigned total, unsigned parts) {
    n = min(parts, total);
    len = n > 0 ? total / n : 0;
    longer = total - len * n;
  }
  __device__ __forceinline__ unsigned begin(unsigned part) const { return len * min(part, n) + min(min(part, n), longer); }
  __device__ __forceinline__ int part_of(unsigned unit) const {
    const unsigned first = longer * (len + 1);
    return (int)(unit < first ? unit / (len + 1) : longer + (unit - first) / len);
  }
};

// A CTA's work: consecutive units of the line of all (sequence, cl row groups, tile).  The
// line is cut into equal parts, so that every CTA has as many tiles whatever the lengths are;
// what a cut leaves in two CTAs is joined by the second kernel.
struct Item {
  int b, r0, rows;                           // row group: first row of the sequence's, rows of it
  int tile, nt, tiles;                       // first tile, tiles with something to see, tiles of the whole group
  unsigned unit;                             // the first tile's place in the line
  int end, L, n, q0;                         // tokens that any of its rows sees
  bool whole;
  int slot;
};
template <int NR>
struct Walk {
  int b, half, part;
  unsigned off, left, at;
  Cuts cuts;
  bool first;
  __device__ __forceinline__ bool next(const LatentParams& p, Item& it) {
    while (left > 0 && b < p.B) {            // (starts that go back and forth may name more than 2^31 units)
      const Seq s = seq_of(p, b, false);
      const unsigned supers = supers_of(p, s, NR);
      if (off >= supers * s.tiles) {
        ++b;
        off = 0;
        continue;
      }
      const unsigned sg = off < (unsigned)s.tiles ? 0u : off / (unsigned)s.tiles;
      const int t = (int)(off - sg * s.tiles);
      const int cnt = (int)min((unsigned)(s.tiles - t), left);
      it.unit = at;
      off += cnt;
      left -= cnt;
      at += cnt;
      const bool was_first = first;
      first = false;
      it.b = b;
      it.r0 = ((int)sg * p.cl + half) * NR;
      it.rows = min(NR, s.n * p.H - it.r0);
      if (it.rows <= 0) continue;
      it.end = s.n == 1 ? s.L : min(s.L, max(0, s.L - s.n + (int)((unsigned)(it.r0 + it.rows - 1) / (unsigned)p.H) + 1));
      it.tile = t;
      it.tiles = s.tiles;
      it.nt = max(0, min(t + cnt, (it.end + kTile - 1) / kTile) - t);
      it.L = s.L;
      it.n = s.n;
      it.q0 = s.q0;
      it.whole = cnt == s.tiles;
      it.slot = (part * p.cl + half) * 2 + (was_first ? 0 : 1);
      return true;
    }
    return false;
  }
};

// NaN in the elements of the calling softmax thread (dims r of every 128, its columns) that see a value
// which is not finite, among the part's tokens that some row of the group does not see: NR / H + 1 at
// most.  The rows of the output, or the partial sums, have been written.
template <int NR, int RC>
__device__ __noinline__ void put_nans(const LatentParams& p, const Item it) {
  constexpr int SUB = subs(NR), CW = NR / SUB, R = RC * 64, NP = RC / 2;
  const int r = (int)threadIdx.x & 127, c0 = (int)(threadIdx.x >> 7) * CW;
  const int past = it.L - it.n, cols = min(CW, it.rows - c0);
  const int first = max(it.tile * kTile, past + it.r0 / p.H + 1), stop = min(it.end, (it.tile + it.nt) * kTile);
  for (int i = 0; i < NP; ++i) {
    long long seen = cols;                   // rows from here on
    for (int t = first; t < stop; ++t) {
      int block = __ldg(&p.block_tables[(size_t)it.b * p.max_blocks + t / p.bs]);
      if ((unsigned)block >= (unsigned)p.num_blocks) block = 0;      // (as it was copied)
      const float x = __bfloat162float(p.cache[((size_t)block * p.bs + t % p.bs) * (R + p.P) + i * 128 + r]);
      if (x - x != 0.f) seen = min(seen, max(0ll, (long long)(t - past) * p.H - it.r0 - c0));
    }
    for (int c = (int)seen; c < cols; ++c) {
      if (it.whole) p.out[((size_t)it.q0 * p.H + it.r0 + c0 + c) * R + i * 128 + r] = __float2bfloat16_rn(NAN);
      else p.ws_o[((((size_t)it.slot * NP + i) * (NR / 4) + (c0 + c) / 4) * 128 + r) * 4 + (c & 3)] = NAN;
    }
  }
}

// Sum of every x[i] over the warp, N <= 32: x[0] is that of the column whose bits the lane's
// upper bits spell.
template <int N>
__device__ __forceinline__ void warp_sums(float (&x)[N], int lane) {
  int n = N;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    if (n > 1) {
      n /= 2;
      const bool up = lane & off;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i < n) {
          const float keep = up ? x[i + n] : x[i], give = up ? x[i] : x[i + n];
          x[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
        }
      }
    } else {
      x[0] += __shfl_xor_sync(0xffffffffu, x[0], off);
    }
  }
}
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[8]) { tmem_ld(taddr, r); }
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }

template <int NR, int RC>
__global__ void __launch_bounds__(threads(NR), 1)
latent_decode_kernel(const __grid_constant__ CUtensorMap mapC, const __grid_constant__ CUtensorMap mapQ,
                     const __grid_constant__ LatentParams p) {
  using Lay = Layout<NR, RC>;
  constexpr int NC = Lay::NC, NP = Lay::NP, SLOTS = Lay::kSlots;
  constexpr bool kAlias = Lay::kAlias;
  constexpr int kThreads = threads(NR), SUB = subs(NR), kSoft = 128 * SUB, kTma = 4 * SUB, kMma = kTma + 3;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  Shared<NR>* sh = reinterpret_cast<Shared<NR>*>(smem + Lay::kOffShared);
  volatile int* abort_flag = &sh->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;");

  if (threadIdx.x == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->full_r[i], 3);          // the TMA warps, with copies to do or without
      mbar_init(&sh->empty_r[i], 1);
      mbar_init(&sh->s[i], 1);
    }
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, 1);
    mbar_init(&sh->p, 4 * SUB);
    mbar_init(&sh->pv, 1);
    mbar_init(&sh->o_free, 4 * SUB);
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    sh->odd = 0;
    sh->first_b = p.B;
    fence_mbar_init();
    prefetch_tensormap(&mapC);
    prefetch_tensormap(&mapQ);
  }
  if (warp == kMma) {
    tmem_alloc(&sh->tmem_base, Lay::kTmem);
    tmem_relinquish();
  }

  // ---- this CTA's part of the line
  const int parts = gridDim.x >> (p.cl - 1), part = blockIdx.x >> (p.cl - 1);
  Walk<NR> walk;
  {
    const int per = p.B <= kThreads ? 1 : (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    const bool note = blockIdx.x == 0;
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
      const Seq s = seq_of(p, b, note);
      sum += supers_of(p, s, NR) * s.tiles;
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) sh->scan[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int mine = lane < kThreads / 32 ? sh->scan[lane] : 0;
    const int total = __reduce_add_sync(0xffffffffu, mine);
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0) + incl - sum;
    // (no empty parts: a line shorter than the grid leaves its last CTAs without work)
    const Cuts cuts(total, parts);
    const unsigned u0 = cuts.begin(part), u1 = cuts.begin(part + 1);
    if (u0 - (unsigned)before < (unsigned)sum) {     // (one thread, where there is anything)
      unsigned off = u0 - (unsigned)before;
      int b = b0;
      for (; b + 1 < b1; ++b) {
        const Seq s = seq_of(p, b, false);
        const unsigned u = (unsigned)(supers_of(p, s, NR) * s.tiles);
        if (off < u) break;
        off -= u;
      }
      sh->first_b = b;
      sh->first_off = off;
    }
    __syncthreads();
    walk.b = sh->first_b;
    walk.off = sh->first_off;
    walk.left = walk.b < p.B ? u1 - u0 : 0;
    walk.half = blockIdx.x & (p.cl - 1);
    walk.part = part;
    walk.at = u0;
    walk.cuts = cuts;
    walk.first = true;
    // (what stays where the CTA begins nothing that goes on)
    if (threadIdx.x == 0) p.ws_join[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  const uint32_t tmem = sh->tmem_base;
  const uint32_t tO = tmem + 2 * NR;
  Item it;

  if (warp >= kTma && warp < kMma) {
    // ------------------------------------------------------------ TMA producers
    // A warp gets a copy out in about 60 clocks, whatever its size, and a tile is 72 of 2 KB:
    // three warps share them, every third copy of a pair each.
    const uint64_t pol = policy_evict_first();
    const int w = warp - kTma;
    const int bsh = 31 - __clz(p.bs);
    const uint32_t box = (uint32_t)p.bs * 128u;
    const int blocks = kTile >> bsh;
    const int copy = lane * 3 + w;           // the lane's copy of a pair: a chunk of a block
    const int chunk = copy >= blocks ? 1 : 0, mine = copy - chunk * blocks;
    const bool used = copy < 2 * blocks;
    int kp = 0, kr = 0, kq = 0;              // pairs, rotated chunks and query groups requested
    bool ok = true;
    while (ok && walk.next(p, it)) {
      if (it.nt == 0) continue;
      const int32_t* row = p.block_tables + (size_t)it.b * p.max_blocks;
      auto id_of = [&](int j) -> int {
        const int t = (it.tile + j) * kTile + (mine << bsh);
        return j < it.nt && used && t < it.end ? __ldg(&row[t >> bsh]) : 0;
      };
      int blk = id_of(0);
      ok = __all_sync(0xffffffffu, wait(&sh->q_empty, (uint32_t)(kq & 1) ^ 1u, abort_flag));
      if (!ok) break;
      if (w == 0 && lane == 0) mbar_arrive_expect_tx(&sh->q_full, (uint32_t)NC * NR * 128u);   // (every warp has a chunk)
      __syncwarp();
      if (copy < NC) tma_load_4d(smem + copy * NR * 128, &mapQ, &sh->q_full, copy * 64, it.q0 * p.H + it.r0, 0, 0, pol);
      ++kq;
      for (int j = 0; j < it.nt; ++j) {
        const int next = id_of(j + 1);
        const int nb = (min(kTile, it.end - (it.tile + j) * kTile) + p.bs - 1) >> bsh;
        const bool has = used && mine < nb;
        if (has && (unsigned)blk >= (unsigned)p.num_blocks) {
          atomicOr(&g_status_latent, PA_DEV_BAD_BLOCK);
          blk = 0;                           // keep every copy inside the pool
        }
        for (int i = 0; i < NP; ++i, ++kp) {
          const int sl = kp % SLOTS;
          ok = __all_sync(0xffffffffu, wait(&sh->empty[sl], ((uint32_t)(kp / SLOTS) & 1u) ^ 1u, abort_flag));
          if (!ok) break;
          // (a warp may be ahead of the one that names the bytes: the phase waits for that one)
          if (w == 0 && lane == 0) mbar_arrive_expect_tx(&sh->full[sl], 2u * nb * box);
          __syncwarp();
          if (has)
            tma_load_4d(smem + Lay::kOffRing + sl * kPair + chunk * kChunk + mine * box, &mapC, &sh->full[sl],
                        i * 128 + chunk * 64, 0, blk, 0, pol);
        }
        if (!ok) break;
        const int sr = kAlias ? 0 : kr & 1;
        const uint32_t use = kAlias ? (uint32_t)kr : (uint32_t)kr >> 1;
        ok = __all_sync(0xffffffffu, wait(&sh->empty_r[sr], (use & 1u) ^ 1u, abort_flag));
        if (!ok) break;
        // All three arrive, once a tile: one without anything to copy would else be free to look at a
        // slot a turn late, when its parity has come round.  (A tile's slots are not used up before
        // its scores are done, and those wait for this.  An arrival for every pair took 2 %.)
        if (lane == 0) {
          if (w == 0) mbar_arrive_expect_tx(&sh->full_r[sr], (uint32_t)nb * box);
          else mbar_arrive(&sh->full_r[sr]);
        }
        __syncwarp();
        if (chunk == 0 && has)
          tma_load_4d(smem + Lay::kOffRope + sr * kChunk + mine * box, &mapC, &sh->full_r[sr], RC * 64, 0, blk, 0, pol);
        ++kr;
        blk = next;
      }
    }
    // no TMA write may land after the CTA has left
    if (lane == 0) {
      for (int k = max(0, kp - SLOTS); k < kp; ++k) mbar_wait(&sh->full[k % SLOTS], (uint32_t)(k / SLOTS) & 1u);
      for (int k = max(0, kr - (kAlias ? 1 : 2)); k < kr; ++k)
        mbar_wait(&sh->full_r[kAlias ? 0 : k & 1], (uint32_t)(kAlias ? k : k >> 1) & 1u);
      if (kq > 0) mbar_wait(&sh->q_full, (uint32_t)(kq - 1) & 1u);
    }
  } else if (warp == kMma) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks, with values that are the same in all lanes, and one lane issues: the
    // descriptors then stay in uniform registers (moved there for every MMA, 57 clocks an MMA and not 47).
    constexpr uint32_t idS = idesc_bf16_f32(kTile, NR, false, false);
    constexpr uint32_t idO = idesc_bf16_f32(kTile, NR, true, true);
    const bool lead = elect_one();
    const uint32_t t0 = __shfl_sync(0xffffffffu, tmem, 0), tO0 = t0 + 2 * NR;
    const uint32_t sb = __shfl_sync(0xffffffffu, sbase, 0);
    const uint64_t dk = sdesc_sw128(sb + Lay::kOffRing, 16, 1024);               // the tile as K
    const uint64_t dv = sdesc_sw128(sb + Lay::kOffRing, kChunk, 1024);           // the tile as V^T
    const uint64_t dr = sdesc_sw128(sb + Lay::kOffRope, 16, 1024);
    const uint64_t dq = sdesc_sw128(sb, 16, 1024);
    const uint64_t dp = sdesc_sw128(sb + Lay::kOffP, kChunk, 1024);
    constexpr int kEarly = SLOTS - NP < NP ? SLOTS - NP : NP;     // pairs of the next tile that a tile leaves room for
    constexpr bool kAllEarly = kEarly == NP && !kAlias;
    const int rope_steps = p.P / 16;
    int kt = 0, kq = 0;                      // tiles, query groups
    int u0 = 0;                              // slot of tile kt's first pair, and how often the ring has turned
    uint32_t turn = 0;
    // pairs [a, b) of tile k's scores, its pairs from slot `at` on in turn `tn`
    auto scores = [&](int k, int at, uint32_t tn, int a, int b) -> bool {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (i < a || i >= b) continue;
        const bool over = at + i >= SLOTS;
        const int sl = over ? at + i - SLOTS : at + i;
        if (!wait(&sh->full[sl], (tn + (over ? 1u : 0u)) & 1u, abort_flag)) return false;
        tc_fence_after();
        if (lead) {
          const uint64_t da = sdesc_at(dk, sl * kPair), db = sdesc_at(dq, i * 2 * NR * 128);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16(t0 + (k & 1) * NR, sdesc_at(da, (kk >> 2) * kChunk + (kk & 3) * 32),
                      sdesc_at(db, (kk >> 2) * NR * 128 + (kk & 3) * 32), idS, i > 0 || kk > 0 ? 1u : 0u);
        }
        __syncwarp();
      }
      return true;
    };
    auto scores_end = [&](int k, bool last) -> bool {
      const int sr = kAlias ? 0 : k & 1;
      if (!wait(&sh->full_r[sr], (uint32_t)(kAlias ? k : k >> 1) & 1u, abort_flag)) return false;
      tc_fence_after();
      if (lead) {
        const uint64_t da = sdesc_at(dr, sr * kChunk), db = sdesc_at(dq, RC * NR * 128);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (kk < rope_steps) umma_bf16(t0 + (k & 1) * NR, sdesc_at(da, kk * 32), sdesc_at(db, kk * 32), idS, 1u);
        umma_commit(&sh->s[k & 1]);
        if (!kAlias) umma_commit(&sh->empty_r[sr]);
        if (last) umma_commit(&sh->q_empty);
      }
      __syncwarp();
      return true;
    };
    bool ok = true;
    while (ok && walk.next(p, it)) {
      const int nt = __shfl_sync(0xffffffffu, it.nt, 0);
      if (nt == 0) continue;
      ok = wait(&sh->q_full, (uint32_t)kq & 1u, abort_flag) && scores(kt, u0, turn, 0, NP) && scores_end(kt, nt == 1);
      for (int j = 0; ok && j < nt; ++j, ++kt) {
        const bool more = j + 1 < nt;
        const bool over = u0 + NP >= SLOTS;
        const int u1 = over ? u0 + NP - SLOTS : u0 + NP;
        const uint32_t turn1 = turn + (over ? 1u : 0u);
        if (more && kEarly > 0) {
          if (!(ok = scores(kt + 1, u1, turn1, 0, kEarly))) break;
          if (kAllEarly && !(ok = scores_end(kt + 1, j + 2 == nt))) break;
        }
        if (!(ok = wait(&sh->p, (uint32_t)kt & 1u, abort_flag))) break;
        if (j == 0 && !(ok = wait(&sh->o_free, ((uint32_t)kq & 1u) ^ 1u, abort_flag))) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int sl = u0 + i >= SLOTS ? u0 + i - SLOTS : u0 + i;
          if (lead) {
            const uint64_t da = sdesc_at(dv, sl * kPair);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)   // 16 tokens each
              umma_bf16(tO0 + i * NR, sdesc_at(da, kk * 2048), sdesc_at(dp, kk * 2048), idO, j > 0 || kk > 0 ? 1u : 0u);
            umma_commit(&sh->empty[sl]);
            if (i == NP - 1) {
              umma_commit(&sh->pv);
              if (kAlias) umma_commit(&sh->empty_r[0]);
            }
          }
          __syncwarp();
        }
        if (more && !kAllEarly) {
          if (!(ok = scores(kt + 1, u1, turn1, kEarly, NP))) break;
          if (!(ok = scores_end(kt + 1, j + 2 == nt))) break;
        }
        u0 = u1;
        turn = turn1;
      }
      ++kq;
    }
    if (lead) umma_commit(&sh->drain);       // every MMA has completed before TMEM is freed
    mbar_wait(&sh->drain, 0);
  } else {
    // ------------------------------------------------------------ softmax
    // Thread = token; the tile's columns are divided among SUB warps a lane quarter.
    constexpr int CW = NR / SUB;
    const int r = (int)threadIdx.x & 127;    // token of the tile, latent dim at the end; TMEM lane
    const int sub = warp >> 2, c0 = sub * CW;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    int kt = 0;
    float l[CW];
    while (walk.next(p, it)) {
      const int past = it.L - it.n;          // position of the sequence's first row
#pragma unroll
      for (int c = 0; c < CW; ++c) l[c] = 0.f;
      for (int j = 0; j < it.nt; ++j, ++kt) {
        const int st = kt & 1;
        const int t = (it.tile + j) * kTile + r;
        wait(&sh->s[st], (uint32_t)(kt >> 1) & 1u, abort_flag);
        __syncwarp();
        tc_fence_after();
        // rows (t - past) H and on of the sequence see token t
        const int hide = t >= it.end ? NR : (int)max(-1ll, min((long long)NR, (long long)(t - past) * p.H - it.r0));
        const bool any_hidden = __any_sync(0xffffffffu, hide > c0);
        float x[CW];
        auto scores = [&]() {
          uint32_t v[CW];
          tmem_load(tmem + st * NR + c0 + lane_off, v);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < CW; ++c) x[c] = __uint_as_float(v[c]);
          if (any_hidden) {
#pragma unroll
            for (int c = 0; c < CW; ++c)
              if (c0 + c < hide) x[c] = -INFINITY;
          }
        };
        // exponents, against the references as they are
        auto exponents = [&]() {
#pragma unroll
          for (int c = 0; c < CW; c += 4) {
            const float4 m = *reinterpret_cast<const float4*>(&sh->neg_m[c0 + c]);
            x[c] = fmaf(x[c], p.qscale, m.x);
            x[c + 1] = fmaf(x[c + 1], p.qscale, m.y);
            x[c + 2] = fmaf(x[c + 2], p.qscale, m.z);
            x[c + 3] = fmaf(x[c + 3], p.qscale, m.w);
          }
        };
        bool need = j == 0;
        if (j > 0) {
          scores();
          exponents();
          float top[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) top[i] = fmaxf(x[2 * i], x[2 * i + 1]);
#pragma unroll
          for (int c = 8; c < CW; c += 2) top[(c >> 1) & 3] = fmax3(top[(c >> 1) & 3], x[c], x[c + 1]);
          need = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) > 0.f;
        }
        need = vote<kSoft>(need);
        if (need) {
          // new references: 2^8 above the tile's maxima, where those are above the references there are.
          // (No weight is above 1 then, and sums of large values stay finite.)
          scores();
#pragma unroll
          for (int c = 0; c < CW; ++c) {
            const float y = warp_max(x[c]);
            if (lane == 0) sh->red[warp & 3][c0 + c] = y;
          }
          named_sync(1, kSoft);
          if (threadIdx.x < NR) {
            const int c = (int)threadIdx.x;
            const float y = fmaxf(fmaxf(sh->red[0][c], sh->red[1][c]), fmaxf(sh->red[2][c], sh->red[3][c])) * p.qscale;
            const float old = j > 0 ? -sh->neg_m[c] : -INFINITY;
            const float m = y > old ? y + kSlack : old;
            sh->f[c] = old == -INFINITY ? 0.f : exp2f(old - m);
            // No reference yet (nothing seen, or scores of -inf alone): one that every finite score exceeds.
            sh->neg_m[c] = m == -INFINITY ? kUnset : -m;
          }
          named_sync(1, kSoft);
          exponents();
        }
        // P, and with it the rotated keys' chunk, is free; O holds the tile before
        if (kt > 0) wait(&sh->pv, (uint32_t)(kt - 1) & 1u, abort_flag);
        __syncwarp();
        if (need && j > 0) {
#pragma unroll
          for (int c = 0; c < CW; ++c) l[c] *= sh->f[c0 + c];
          tc_fence_after();
#pragma unroll 1
          for (int i = 0; i < NP; ++i) {
#pragma unroll 1
            for (int c = c0; c < c0 + CW; c += 8) {
              uint32_t v[8];
              tmem_ld(tO + i * NR + c + lane_off, v);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * sh->f[c + k]);
              tmem_st(tO + i * NR + c + lane_off, v);
            }
          }
          tmem_st_wait();
        }
        // P: row r of an MN-major tile, 8 columns a 16-byte piece
        unsigned char* prow = smem + Lay::kOffP + r * 128;
#pragma unroll
        for (int c = 0; c < CW; c += 8) {
          float e[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            e[i] = ex2(x[c + i]);
            l[c + i] += e[i];
          }
          *reinterpret_cast<uint4*>(prow + ((((c0 + c) >> 3) ^ (r & 7)) << 4)) =
              make_uint4(pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]), pack_bf16(e[4], e[5]), pack_bf16(e[6], e[7]));
        }
        if (t >= it.end || hide > 0) {
          // A slot that no row sees may hold anything, and 0 * NaN would reach O: its values are
          // zeroed.  Of a token that some rows see and others do not, what is not finite: most
          // rows that see it have a NaN from their score, and one whose score is -inf gets its NaN
          // in those elements when they are written.
          const bool drop = t >= it.end;
          bool odd = false;
#pragma unroll 1
          for (int i = 0; i < NP; ++i) {
            unsigned char* at = smem + Lay::kOffRing + ((kt * NP + i) % SLOTS) * kPair + r * 128;
            auto piece = [&](int k) {        // (another one in each row of eight)
              k += sub * (16 / SUB);
              return reinterpret_cast<uint4*>(at + (k >> 3) * kChunk + (((k + r) & 7) << 4));
            };
            if (drop) {
#pragma unroll
              for (int k = 0; k < 16 / SUB; ++k) *piece(k) = make_uint4(0u, 0u, 0u, 0u);
            } else {
#pragma unroll 1
              for (int k = 0; k < 16 / SUB; ++k) {
                const uint4 v = *piece(k);
                auto clean = [](uint32_t y) {
                  if ((y & 0x7f80u) == 0x7f80u) y &= 0xffff0000u;
                  if ((y & 0x7f800000u) == 0x7f800000u) y &= 0xffffu;
                  return y;
                };
                const uint4 w = make_uint4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
                odd |= w.x != v.x || w.y != v.y || w.z != v.z || w.w != v.w;
                *piece(k) = w;
              }
            }
          }
          if (odd) *static_cast<volatile unsigned*>(&sh->odd) = it.unit + 1;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->p);
      }

      // ---------------------------------------------------------- output of the row group
      warp_sums(l, lane);
      __syncwarp();
      named_sync(1, kSoft);
      {
        // the column that the halvings left in this lane
        int col = 0, spare = 31;
#pragma unroll
        for (int off = 16, n = CW / 2; n > 0; off >>= 1, n /= 2) {
          if (lane & off) col += n;
          spare &= ~off;
        }
        if ((lane & spare) == 0) sh->red[warp & 3][c0 + col] = l[0];
      }
      named_sync(1, kSoft);
      if (!it.whole && it.tile == 0 && threadIdx.x == 0) {
        // the CTAs after this one, as far as the group goes (it is the CTA's last: there is one at most)
        p.ws_join[blockIdx.x] = make_int4(it.q0 * p.H + it.r0, it.rows, max(0, min(walk.cuts.part_of(it.unit + it.tiles - 1), parts - 1) - part),
                                          it.slot & 1);
      }
      if (threadIdx.x < NR) {
        const int c = (int)threadIdx.x;
        const float sum = (sh->red[0][c] + sh->red[1][c]) + (sh->red[2][c] + sh->red[3][c]);
        if (it.whole) {
          sh->f[c] = it.nt > 0 && sum != 0.f ? 1.f / sum : 0.f;
        } else {
          float* ml = p.ws_ml + ((size_t)it.slot * NR + c) * 2;
          // (a part whose scores are all -inf has a sum of 0, marked by a maximum of -inf, and elements to be joined)
          ml[0] = it.nt > 0 && sum != 0.f ? -sh->neg_m[c] : -INFINITY;
          ml[1] = it.nt == 0 ? 0.f : sum != 0.f ? sum : 1.f;
        }
      }
      named_sync(1, kSoft);
      const int R = RC * 64;
#pragma unroll 1
      for (int i = 0; i < NP; ++i) {
        uint32_t v[CW];
        if (it.nt > 0) {
          // the last tile's values have left their slot: these dims are done
          const int u = (kt - 1) * NP + i;
          wait(&sh->empty[u % SLOTS], (uint32_t)(u / SLOTS) & 1u, abort_flag);
          __syncwarp();
          tc_fence_after();
          tmem_load(tO + i * NR + c0 + lane_off, v);
          tmem_ld_wait();
        }
        if (it.whole) {
          // Lanes hold a dim of 8 columns and write 8 dims of one: matrix k of the transposition is dims
          // 8 x + 2 k + {0, 1} of every x.  (A row group of 16 takes 2000 clocks; elements of 2 bytes 3000,
          // by shuffles 2300, by 256 bytes a row, which four warps put together, 3200.)
          const int dim = ((lane & 6) << 2) + ((lane >> 3) << 1) + (lane & 1);
          const int col = c0 + (lane >> 2);
          __nv_bfloat16* o = p.out + ((size_t)it.q0 * p.H + it.r0 + col) * R + i * 128 + (warp & 3) * 32 + (lane & 3) * 8;
#pragma unroll
          for (int g = 0; g < CW; g += 8) {
            const float4 f0 = *reinterpret_cast<const float4*>(&sh->f[c0 + g]);
            const float4 f1 = *reinterpret_cast<const float4*>(&sh->f[c0 + g + 4]);
            uint4 y = make_uint4(0u, 0u, 0u, 0u);
            if (it.nt > 0)
              y = make_uint4(pack_bf16(__uint_as_float(v[g]) * f0.x, __uint_as_float(v[g + 1]) * f0.y),
                             pack_bf16(__uint_as_float(v[g + 2]) * f0.z, __uint_as_float(v[g + 3]) * f0.w),
                             pack_bf16(__uint_as_float(v[g + 4]) * f1.x, __uint_as_float(v[g + 5]) * f1.y),
                             pack_bf16(__uint_as_float(v[g + 6]) * f1.z, __uint_as_float(v[g + 7]) * f1.w));
            sh->turn[warp][lane] = y;
            __syncwarp();
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                         : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w) : "r"(smem_u32(&sh->turn[warp][dim])) : "memory");
            __syncwarp();
            if (col + g < it.rows) st_v4(o + (size_t)g * R, y);
          }
        } else if (it.nt > 0) {
          // four columns of a dim side by side, as the join takes them
          uint4* o = reinterpret_cast<uint4*>(p.ws_o) + (((size_t)it.slot * NP + i) * (NR / 4) + c0 / 4) * 128 + r;
#pragma unroll
          for (int c = 0; c < CW; c += 4)
            if (c0 + c < it.rows) o[(c / 4) * 128] = make_uint4(v[c], v[c + 1], v[c + 2], v[c + 3]);
        }
      }
      if (it.nt > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->o_free);
        if (*static_cast<volatile unsigned*>(&sh->odd) == it.unit + 1) put_nans<NR, RC>(p, it);
      }
      named_sync(1, kSoft);                    // f and red are free again
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, Lay::kTmem);
}

// Joins the row groups that a cut left in several CTAs.  grid (CTAs, blocks of 8 warps): a warp takes
// four rows x 128 dims of the group that the CTA begins, if it begins one.  Bound by latency: what the
// CTA began, then maxima and sums together, four parts ahead (two: 11 drafts of 32 heads 25.5 us for
// 23.9 with the kernel before; a row a warp, one part after the other: 2 short contexts 12.7 for 10.9).
template <int NR, int RC>
__global__ void __launch_bounds__(256) latent_join_kernel(const LatentParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int R = RC * 64, NP = RC / 2;
  const int lane = threadIdx.x & 31;
  const int4 j = p.ws_join[blockIdx.x];
  const int u = blockIdx.y * 8 + (threadIdx.x >> 5), c = u / NP * 4, piece = u % NP;
  if (c >= j.y) return;
  const int parts = j.z + 1;                 // the CTA's slot, and the first slots of so many CTAs of its kind
  auto slot_of = [&](int q) -> size_t { return (size_t)(q == 0 ? (int)blockIdx.x * 2 + j.w : ((int)blockIdx.x + q * p.cl) * 2); };
  const float4* src = reinterpret_cast<const float4*>(p.ws_o) + ((size_t)piece * (NR / 4) + c / 4) * 128 + lane * 2;
  // (a part whose rows saw nothing has no sums: they are read and not used)
  float4 x[4][4];
  auto fetch = [&](int q0) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q0 + q >= parts) break;
      const float4* s = src + slot_of(q0 + q) * (NP * (NR / 4) * 128);
#pragma unroll
      for (int d = 0; d < 4; ++d) x[q][d] = s[(d >> 1) * 64 + (d & 1)];
    }
  };
  fetch(0);
  // maxima and sums: lane = (part, row)
  const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + c + (lane & 3);
  float m = -INFINITY;
  for (int q = lane >> 2; q < parts; q += 8) m = fmaxf(m, ml[slot_of(q) * NR].x);
#pragma unroll
  for (int off = 16; off > 2; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  float l = 0.f, w = 0.f, o[4][4] = {};
  uint32_t live = 0;
  for (int q0 = 0; q0 < parts; q0 += 4) {
    if ((q0 & 7) == 0) {
      const int mine = q0 + (lane >> 2);
      float2 y = make_float2(-INFINITY, 0.f);
      if (mine < parts) y = ml[slot_of(mine) * NR];
      live = __ballot_sync(0xffffffffu, y.y != 0.f);
      w = y.x != -INFINITY ? exp2f(y.x - m) : 0.f;
      if (y.x != -INFINITY) l = fmaf(y.y, w, l);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int from = ((q0 & 7) + q) * 4 + k;
        const float wk = __shfl_sync(0xffffffffu, w, from);
        if (!((live >> from) & 1u)) continue;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const float4 y = x[q][d];
          o[d][k] = fmaf(k == 0 ? y.x : k == 1 ? y.y : k == 2 ? y.z : y.w, wk, o[d][k]);
        }
      }
    }
    fetch(q0 + 4);
  }
#pragma unroll
  for (int off = 16; off > 2; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  const float inv = l != 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* out = p.out + ((size_t)j.x + c) * R + piece * 128 + lane * 2;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float f = __shfl_sync(0xffffffffu, inv, k);
    if (c + k < j.y) {
      *reinterpret_cast<uint32_t*>(out + k * R) = pack_bf16(o[0][k] * f, o[1][k] * f);
      *reinterpret_cast<uint32_t*>(out + k * R + 64) = pack_bf16(o[2][k] * f, o[3][k] * f);
    }
  }
}

bool good_sizes(int total, int num_seqs, int num_heads, int latent_dim, int max_blocks, int bs) {
  return total >= 0 && num_seqs >= 0 && num_heads > 0 && latent_shape(latent_dim, 16, bs) && max_blocks > 0 &&
         (long long)max_blocks * bs <= kMaxRowTokens && (long long)total * num_heads <= 0x7fffffffll;
}

// How the rows are taken: NR rows a CTA (what most sequences have, as far as it is known here),
// and two CTAs side by side over the same tokens where that is less than a sequence's rows.
struct Plan {
  int nr, cl, parts;
  size_t ml, join, bytes;                    // workspace offsets
};
Plan plan_of(int total, int num_seqs, int num_heads, int latent_dim) {
  Plan w = {};
  const long long rows = ((long long)total + num_seqs - 1) / num_seqs * num_heads;
  w.nr = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  w.cl = rows > w.nr ? 2 : 1;
  w.parts = kTunedSms / w.cl;
  const size_t slots = 2 * (size_t)w.parts * w.cl;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  w.ml = up(slots * w.nr * latent_dim * 4);
  w.join = w.ml + up(slots * w.nr * 8);
  w.bytes = w.join + up(slots * 16);
  return w;
}

struct Pick {
  const void *kernel, *join;
  size_t smem;
  int threads;
};
template <int NR, int RC>
Pick pick1() {
  return {reinterpret_cast<const void*>(&latent_decode_kernel<NR, RC>),
          reinterpret_cast<const void*>(&latent_join_kernel<NR, RC>), Layout<NR, RC>::kBytes, threads(NR)};
}
template <int NR>
Pick pick2(int rc) {
  return rc == 2 ? pick1<NR, 2>() : rc == 4 ? pick1<NR, 4>() : rc == 6 ? pick1<NR, 6>() : pick1<NR, 8>();
}
Pick pick(int nr, int rc) { return nr == 16 ? pick2<16>(rc) : nr == 32 ? pick2<32>(rc) : pick2<64>(rc); }

}  // namespace

unsigned* status_word_latent_decode() { return device_word(g_status_latent); }

}  // namespace pa

using namespace pa;

extern "C" int pa_latent_decode(void* out, const void* query, const int32_t* query_start, int total_queries,
                                const void* cache, const int32_t* block_tables, int max_blocks_per_seq,
                                const int32_t* context_lens, int num_seqs, int num_heads, int latent_dim,
                                int rope_dim, int block_size, int num_blocks, float scale, void* workspace,
                                size_t workspace_bytes, pa_dtype dtype, void* stream) {
  if (dtype != PA_BF16) return PA_ERR_DTYPE;
  if (!good_sizes(total_queries, num_seqs, num_heads, latent_dim, max_blocks_per_seq, block_size) ||
      !latent_shape(latent_dim, rope_dim, block_size) || num_blocks <= 0 || !(scale > 0.f) ||
      (!query_start && total_queries != num_seqs))
    return PA_ERR_SHAPE;
  if (num_seqs == 0 || total_queries == 0) return PA_OK;
  if (!out || !query || !cache || !block_tables || !context_lens) return PA_ERR_NULL;
  if (!aligned16(out) || !aligned16(query) || !aligned16(cache) || !aligned16(workspace)) return PA_ERR_ALIGN;
  const Plan w = plan_of(total_queries, num_seqs, num_heads, latent_dim);
  // units of (row groups, tile): 31 bits
  if (((long long)total_queries * num_heads / w.nr + num_seqs) * (((long long)max_blocks_per_seq * block_size + kTile - 1) / kTile) > 0x7fffffffll)
    return PA_ERR_SHAPE;
  if (!workspace || workspace_bytes < w.bytes) return PA_ERR_WORKSPACE;
  CUtensorMap mapC, mapQ;
  const uint64_t width = (uint64_t)latent_dim + rope_dim;
  {
    const uint64_t dims[4] = {width, (uint64_t)block_size, (uint64_t)num_blocks, 1};
    const uint64_t str[3] = {width * 2, width * 2 * block_size, width * 2 * block_size * num_blocks};
    const uint32_t box[4] = {64, (uint32_t)block_size, 1, 1};
    if (!encode_map(&mapC, cache, PA_BF16, 4, dims, str, box, true)) {
      note_host_error("cuTensorMapEncodeTiled failed for the latent pool");
      return PA_ERR_CUDA;
    }
  }
  {
    const uint64_t rows = (uint64_t)total_queries * num_heads;
    const uint64_t dims[4] = {width, rows, 1, 1};
    const uint64_t str[3] = {width * 2, width * 2 * rows, width * 2 * rows};
    const uint32_t box[4] = {64, (uint32_t)w.nr, 1, 1};
    if (!encode_map(&mapQ, query, PA_BF16, 4, dims, str, box, true)) {
      note_host_error("cuTensorMapEncodeTiled failed for the queries");
      return PA_ERR_CUDA;
    }
  }
  int dev = 0;
  if (!ck(cudaGetDevice(&dev), "cudaGetDevice")) return PA_ERR_CUDA;
  const Pick k = pick(w.nr, latent_dim / 64);
  if (!raise_smem_limit(k.kernel, dev)) return PA_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  LatentParams p = {};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.cache = static_cast<const __nv_bfloat16*>(cache);
  p.query_start = query_start;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.ws_o = reinterpret_cast<float*>(ws);
  p.ws_ml = reinterpret_cast<float*>(ws + w.ml);
  p.ws_join = reinterpret_cast<int4*>(ws + w.join);
  p.B = num_seqs;
  p.H = num_heads;
  p.R = latent_dim;
  p.P = rope_dim;
  p.rows = total_queries;
  p.max_blocks = max_blocks_per_seq;
  p.bs = block_size;
  p.num_blocks = num_blocks;
  p.cl = w.cl;
  p.qscale = scale * kLog2e;
  const unsigned ctas = (unsigned)(w.parts * w.cl);
  void* args[] = {&mapC, &mapQ, &p};
  if (!ck(cudaLaunchKernel(k.kernel, dim3(ctas), dim3(k.threads), args, k.smem, (cudaStream_t)stream),
          "cudaLaunchKernel(latent_decode_kernel)"))
    return PA_ERR_CUDA;
  if ((long long)max_blocks_per_seq * block_size <= kTile) return PA_OK;    // a tile a row group: nothing is cut
  void* join[] = {&p};
  return ck(launch_after(k.join, dim3(ctas, (unsigned)(w.nr / 4 * latent_dim / 128 + 7) / 8), dim3(256), join, (cudaStream_t)stream),
            "cudaLaunchKernel(latent_join_kernel)")
             ? PA_OK
             : PA_ERR_CUDA;
}

extern "C" size_t pa_latent_decode_workspace_bytes(int total_queries, int num_seqs, int num_heads, int latent_dim) {
  if (!good_sizes(total_queries, num_seqs, num_heads, latent_dim, 1, 8) || num_seqs == 0 || total_queries == 0) return 0;
  return plan_of(total_queries, num_seqs, num_heads, latent_dim).bytes;
}

// pa_latent_prefill.cu — ragged causal attention over expanded latent vectors
// (pa_latent_prefill) on the 5th-generation tensor cores: keys of key_dim elements a head,
// one rotated key for all heads, values of value_dim.
//
// Two chains in a CTA, each with 128 query rows of a head, a softmax warpgroup and an issuing warp:
//   S_x = Q_x [K | K_rope]^T   M = 128, N = 128 keys, K = key_dim + rope_dim (12 MMAs of 192)
//   O_x += P_x V               M = 128, N = value_dim, K = 128 keys, P from tensor memory
// Tensor memory holds S_0, S_1 (128 columns each, P_x over the first half of its S_x) and
// O_0, O_1: all 512 columns.  The products of one chain run while the other's softmax does.
//
// Bound by the chain of a tile and the tensor pipe: 4 prompts of 4096 tokens x 32 heads of 128 + 64
// take 465 to 475 us in a replayed graph (1460 TFLOP/s, 76 % of the burst GEMM rate; tensor pipe 66 %
// active) and 505 through the call with inputs that change (1360 TFLOP/s, 71 %).  A step
// of both chains takes 3600 clocks, of which the 40 MMAs are 2600 (65 each at N = 128: operands of
// 8 KB for a score's, at 128 bytes a clock), a chain's softmax 1500 and its products' way through
// the pipe, with the waits around them, 1900.  What was tried and lost: 2^x by a polynomial for some
// elements (the issue slots, not the special functions, bound the softmax), P in quarters, loading S
// in two parts.  K and V are kept in L2 for the other row tiles (5 % slower without).
//
//  * One CTA an SM walks the items, so the next one's Q and K arrive during the last tiles.
//  * K chunks and V halves share one ring of 16 KB slots, in the order in which they are needed.
//  * P is handed over by halves; the second half and the next scores go out in one turn.  It is bf16, as
//    the values are that it meets (both operands have one type): 2^-9 of a weight on average, beside
//    the output's own 2^-9; the sum that divides keeps the weights in 32 bits.  The call's error against
//    64 bits is 0.0020 to 0.0022 of the output's size, 0.0017 of it the output's rounding.
//  * The softmax reference moves only when a maximum exceeds it by 2^8.
//  * Values that are not finite are not looked for, though one reaches the rows of a tile that do not see
//    it, as 0 * NaN.  An item with a row that is not finite while its weights are is noted, and
//    done once more when the CTA's line is through: a warp of its own then takes such values out of
//    the key tiles that some row does not see whole, and the rows that see them get them back as
//    they are written.  That costs an item's time again, whatever the values are, and nobody waits
//    for it (rows done by themselves, key by key and among the items, held the other warps' waits up
//    for seconds in a long context).
//  * Every wait is bounded (2 s); a timeout sets PA_DEV_TIMEOUT, and the roles wind down.
#include "pa_mma.cuh"
#include "pa_tc.cuh"

namespace pa {
namespace {

__device__ unsigned g_status_latent;

constexpr int kThreads = 384;                // warps 0-3 and 4-7: softmax of a tile each; 8 TMA, 9 and 10 MMA of a tile each, 11 values
constexpr int kRows = 128;                   // query rows of a tile
constexpr int kKT = 128;                     // keys per tile
constexpr uint32_t kChunk = 16384;           // 128 rows x 64 elements
// Q: 2 tiles x 3 chunks; then a ring of 16 KB slots, which a key tile after the other takes for its
// K chunks (128 keys x 64 elements) and its two halves of V (64 keys x up to 128 elements).  One
// ring: a tile's last K then has the place of the V before it (a ring of two K and one V held
// every tile up by its V, about 1000 clocks).
constexpr int kSlots = 8;
constexpr uint32_t kOffRing = 6 * kChunk;
constexpr uint32_t kOffBar = kOffRing + kSlots * kChunk;
constexpr uint32_t kColO = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;                // log2 units a score may exceed its reference by
constexpr int kMaxSeqs = 2048;
// A chain without keys in an item waits for the other's (some 2 us for 128 keys): 1.3 s at most.
constexpr int kMaxContext = 1 << 26;
constexpr int kMostItems = 0x7fff0000;       // (and a round of every CTA more fits 31 bits)
// Registers: 384 x 168 at launch, then 2 x 128 x 208 for the softmax and 128 x 88 for the rest.
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split");

struct PrefillParams {
  __nv_bfloat16* out;
  const __nv_bfloat16* kv;                   // for values that are not finite; the tiles go by tensor maps
  const int32_t *query_start, *kv_start;
  int B, H, Dk, P, Dv, rows, kv_rows;
  float qscale;
};

constexpr int kNoted = 1024;                 // rounds that are told apart where items are done again (others go along)
struct Shared {
  uint64_t empty[kSlots], full_k[4], full_v[4], raw_v[4], q[2], q_empty[2], s[2], p[2][2], pv[2], o_free[2], drain[2], ml_full;
  float ml[128][2];                          // SPLIT: maximum and sum of the second half's rows
  uint32_t tmem_base;
  int abort;
  int turn;                                  // 1 while one row tile's products go out
  int redo;                                  // rounds up to the last one whose item is to be done again
  uint32_t noted[kNoted / 32];               // those rounds, modulo kNoted
};
constexpr uint32_t kSmemBytes = kOffBar + (uint32_t)sizeof(Shared) + 1024u;
static_assert(kSmemBytes <= 232448, "shared memory");

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
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(smem_u32(bar), parity)) return true;
  if (*abort_flag) return false;
  if (mbar_wait(bar, parity)) return true;
  atomicOr(&g_status_latent, PA_DEV_TIMEOUT);
  *abort_flag = 1;
  return false;
}

// One row tile's products go out together: let in among each other, both tiles' scores would be
// ready at the same time, and the tensor cores idle while both softmaxes run.  (Only the order is
// at stake: a turn that does not come is taken after a while.)
__device__ __forceinline__ void take_turn(int* turn) {
  for (int i = 0; i < 4096 && atomicCAS(turn, 0, 1) != 0; ++i) {}
}

// Query rows of sequence b, -1 for an inconsistent one.
__device__ __forceinline__ int rows_of(const PrefillParams& p, int b) {
  const int a = __ldg(&p.query_start[b]), e = __ldg(&p.query_start[b + 1]);
  const int u = __ldg(&p.kv_start[b]), v = __ldg(&p.kv_start[b + 1]);
  return a >= 0 && e >= a && e <= p.rows && u >= 0 && v >= u && v <= p.kv_rows && v - u <= kMaxContext ? e - a : -1;
}

// Two chains of softmax and products run side by side in a CTA.  They are two row tiles over the
// same keys or, SPLIT, the even and the odd key tiles of one row tile, joined at the end: half the
// time for an item, where the rows are too few to give every CTA 256 of them.
//
// The work: (unit, head) pairs, heads innermost, a unit being 256 (128) rows of a sequence; the units
// of all sequences in order, every sequence's last, and longest, unit first.  The CTAs take
// them in rounds, forth and back, so that no CTA has the longer ones of every round; a warp walks
// its CTA's by itself, 32 sequences a step.
struct Item {
  int h, q0, n, k0, L, first, past;          // head; rows; keys; the item's first row of the sequence's, its position
  int nt[2], most;                           // key tiles of each chain, of the item
  // key tiles that all its rows see whole
  __device__ __forceinline__ int whole() const { return max(0, past + 1) / kKT; }
};
template <bool SPLIT>
struct Walk {
  static constexpr int kUnit = SPLIT ? kRows : 2 * kRows;      // rows of a unit
  int round, b, base;                        // next round; a sequence at or before its unit's, units before that
  int last;                                  // the second time: rounds up to the last noted one
  __device__ __forceinline__ bool next(const PrefillParams& p, const Shared* sh, int lane, Item& it) {
    if (last > 0) {
      while (round < last && !((sh->noted[(round / 32) & (kNoted / 32 - 1)] >> (round & 31)) & 1u)) ++round;
      if (round >= last) return false;
    }
    const int item = round * (int)gridDim.x + (int)((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    ++round;
    if (item >= kMostItems) return false;    // (starts that go back and forth may name more than the host allows)
    const int unit = item / p.H;
    it.h = item - unit * p.H;
    for (; b < p.B; b += 32) {
      const int k = b + lane < p.B ? (max(rows_of(p, b + lane), 0) + kUnit - 1) / kUnit : 0;
      int incl = k;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
      }
      const uint32_t beyond = __ballot_sync(0xffffffffu, (unsigned)base + (unsigned)incl > (unsigned)unit);
      if (beyond) {
        const int at = __ffs(beyond) - 1;
        base += __shfl_sync(0xffffffffu, incl - k, at);
        const int units = __shfl_sync(0xffffffffu, k, at);
        b += at;
        it.q0 = __ldg(&p.query_start[b]);
        it.n = __ldg(&p.query_start[b + 1]) - it.q0;
        it.k0 = __ldg(&p.kv_start[b]);
        it.L = __ldg(&p.kv_start[b + 1]) - it.k0;
        it.first = (base + units - 1 - unit) * kUnit;
        it.past = it.L - it.n + it.first;
        auto tiles = [&](int x) -> int {
          const int r = min(it.n - it.first - x * kRows, kRows);
          const int end = r > 0 ? min(it.L, max(0, it.past + x * kRows + r)) : 0;
          return (end + kKT - 1) / kKT;
        };
        if constexpr (SPLIT) {
          const int all = tiles(0);
          it.nt[0] = (all + 1) / 2;
          it.nt[1] = all / 2;
          it.most = all;
        } else {
          it.nt[0] = tiles(0);
          it.nt[1] = tiles(1);
          it.most = max(it.nt[0], it.nt[1]);
        }
        return true;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
  }
};

// The values that are not finite, of the tokens after `past`, for a warp's rows from `row` on (at
// position `pos`) of the sequence whose rows begin at q0 and whose keys begin at k0: added to what the
// rows that see them hold (infinities of both signs make a NaN, as in the sum that they belong to).
// 255 tokens and 32 rows at most.
__device__ __noinline__ void put_back(const PrefillParams& p, int q0, int n, int k0, int h, int past, int row, int pos,
                                      int lane) {
  const int each = p.Dv / 32;                // a lane's elements, next to each other: 1, 2 or 4
  const __nv_bfloat16* v = p.kv + ((size_t)k0 * p.H + h) * (p.Dk + p.Dv) + p.Dk + lane * each;
  const size_t step = (size_t)p.H * (p.Dk + p.Dv);
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  int t = max(0, past + 1);
  for (int r = 0; r < 32 && row + r < n; ++r) {
#pragma unroll 4
    for (; t <= pos + r; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = e < each ? __bfloat162float(v[t * step + e]) : 0.f;
        if (x - x != 0.f) sum[e] += x;       // (NaN, not 0, for what is not finite)
      }
    }
    __nv_bfloat16* o = p.out + ((size_t)(q0 + row + r) * p.H + h) * p.Dv + lane * each;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < each && sum[e] != 0.f) o[e] = __float2bfloat16_rn(__bfloat162float(o[e]) + sum[e]);
  }
}

// f0 O of a warp's 32 rows, and f1 of the next chain's if there are two, as bf16 (zeros if there is
// none); returns the carries of exponents that are all ones.
__device__ __forceinline__ uint32_t write_rows(const PrefillParams& p, uint32_t tO, bool have, float f0, bool two,
                                               float f1, int q0, int row, int n, int h, int lane) {
  uint32_t full = 0;
  auto packed = [&](const uint32_t* w) -> uint4 {
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = have ? pack_bf16(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])) : 0u;
      full |= (y[i] & 0x7f807f80u) + 0x00800080u;
    }
    return make_uint4(y[0], y[1], y[2], y[3]);
  };
  // 32 elements of 4 rows change places among 4 lanes, which then write 64 bytes of a row together
  const int row4 = row - (lane & 3);                         // the lanes' first row
  __nv_bfloat16* o = p.out + ((size_t)(q0 + row4) * p.H + h) * p.Dv + (lane & 3) * 8;
#pragma unroll 1
  for (int c = 0; c < p.Dv; c += 32) {
    uint4 y[4];
    {
      uint32_t w[32];
      if (have) {
        tmem_ld32(tO + c, w);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f0);
      }
      if (two) {
        uint32_t z[32];
        tmem_ld32(tO + 128 + c, z);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(fmaf(__uint_as_float(z[i]), f1, __uint_as_float(w[i])));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = packed(w + k * 8);
    }
#pragma unroll
    for (int s = 1; s < 4; s *= 2) {
      const bool up = lane & s;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k & s) continue;
        uint4 give = up ? y[k] : y[k | s];
        give.x = __shfl_xor_sync(0xffffffffu, give.x, s);
        give.y = __shfl_xor_sync(0xffffffffu, give.y, s);
        give.z = __shfl_xor_sync(0xffffffffu, give.z, s);
        give.w = __shfl_xor_sync(0xffffffffu, give.w, s);
        if (up) y[k] = give;
        else y[k | s] = give;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (row4 + k < n) st_v4(o + (size_t)k * p.H * p.Dv + c, y[k]);
  }
  return full;
}

template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
latent_prefill_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapQr,
                      const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapKr,
                      const __grid_constant__ CUtensorMap mapV, const __grid_constant__ PrefillParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  Shared* sh = reinterpret_cast<Shared*>(smem + kOffBar);
  volatile int* abort_flag = &sh->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 8 && lane == 0) {
    prefetch_tensormap(&mapQ);
    prefetch_tensormap(&mapQr);
    prefetch_tensormap(&mapK);
    prefetch_tensormap(&mapKr);
    prefetch_tensormap(&mapV);
  }
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.B; b += kThreads)
      if (rows_of(p, b) < 0) atomicOr(&g_status_latent, PA_DEV_BAD_LEN);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->q[i], 1);
      mbar_init(&sh->q_empty[i], SPLIT ? 2 : 1);
      mbar_init(&sh->s[i], 1);
      mbar_init(&sh->p[i][0], 4);
      mbar_init(&sh->p[i][1], 4);
      mbar_init(&sh->pv[i], 1);
      mbar_init(&sh->o_free[i], 4);
      mbar_init(&sh->drain[i], 1);
    }
    for (int i = 0; i < kSlots; ++i) mbar_init(&sh->empty[i], SPLIT ? 1 : 2);    // chains that use a key tile
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh->full_k[i], 1);
      mbar_init(&sh->full_v[i], 1);
      mbar_init(&sh->raw_v[i], 1);
    }
    mbar_init(&sh->ml_full, 4);
    sh->abort = 0;
    sh->turn = 0;
    sh->redo = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < kNoted / 32) sh->noted[threadIdx.x] = 0u;
  if (warp == 9) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const int ncd = (p.Dk + 63) / 64, ncv = (p.Dv + 63) / 64;    // chunks of the keys' own part, of the values
  const int per = ncd + 3;                   // slots of a key tile: ncd + 1 of K, 2 of V
  Walk<SPLIT> walk{0, 0, 0, 0};
  Item it = {};
  // When a role has walked the line: true where all of them walk it again, for the noted items.  (All
  // twelve warps come here once, whatever has become of their waits.)
  auto once_more = [&]() -> bool {
    if (walk.last > 0) return false;
    __syncwarp();
    named_sync(1, kThreads);
    const int redo = *static_cast<volatile int*>(&sh->redo);
    if (redo == 0 || *abort_flag) return false;
    walk = Walk<SPLIT>{0, 0, 0, redo};
    return true;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // ------------------------------------------------------------ TMA producer
    if (warp == 8) {
      const uint64_t once = policy_evict_first(), keep = policy_evict_last();   // (K, V: other row tiles read them too)
      int u = 0, k = 0, m = 0, nq[2] = {0, 0};  // slots, key tiles, those to be looked through, row tiles requested
      bool ok = true;
      auto load_q = [&](int x) {
        if (it.nt[x] == 0) return;
        ok = ok && wait(&sh->q_empty[x], ((uint32_t)nq[x] & 1u) ^ 1u, abort_flag);
        if (!ok) return;
        mbar_arrive_expect_tx(&sh->q[x], (uint32_t)(ncd + 1) * kChunk);
        const int row = it.q0 + it.first + x * kRows;
        for (int c = 0; c < ncd; ++c) tma_load_4d(smem + (x * 3 + c) * kChunk, &mapQ, &sh->q[x], c * 64, it.h, row, 0, once);
        tma_load_4d(smem + (x * 3 + ncd) * kChunk, &mapQr, &sh->q[x], 0, it.h, row, 0, once);
        ++nq[x];
      };
      // the next slot, once it is free
      auto slot = [&]() -> unsigned char* {
        const int sl = u & (kSlots - 1);
        ok = ok && wait(&sh->empty[sl], ((uint32_t)(u / kSlots) & 1u) ^ 1u, abort_flag);
        ++u;
        return smem + kOffRing + sl * kChunk;
      };
      do {
        while (ok && walk.next(p, sh, lane, it)) {
          const int most = it.most, whole = walk.last > 0 ? it.whole() : most;
          if (lane == 0 && most > 0) {
            load_q(0);
            for (int j = 0; ok && j < most; ++j, ++k) {
              const int row = it.k0 + j * kKT;
              // Key tile k uses full_k[k & 3] and full_v[k & 3].  Each is armed once the first slot is
              // free, and not before: the slot's last user, or one after it, has waited for what the
              // barrier announced four tiles ago (a tile takes 4 or 5 of the 8 slots, so that every slot
              // of tile k - 4 has been free since).  Values to be looked through are announced to the
              // warp that does so, which arrives on full_v in the copy's place.
              uint64_t* full = &sh->full_k[k & 3];
              for (int c = 0; c <= ncd; ++c) {
                unsigned char* dst = slot();
                if (!ok) break;
                if (c == 0) mbar_arrive_expect_tx(full, (uint32_t)(ncd + 1) * kChunk);
                if (c < ncd) tma_load_4d(dst, &mapK, full, c * 64, it.h, row, 0, keep);
                else tma_load_4d(dst, &mapKr, full, 0, row, 0, 0, keep);
              }
              if (!ok) break;
              if (!SPLIT && j == 0) load_q(1);
              full = j < whole ? &sh->full_v[k & 3] : &sh->raw_v[m++ & 3];
              for (int v = 0; v < 2; ++v) {
                unsigned char* dst = slot();
                if (ok && v == 0) mbar_arrive_expect_tx(full, (uint32_t)ncv * kChunk);
                for (int c = 0; ok && c < ncv; ++c)
                  tma_load_4d(dst + c * (kChunk / 2), &mapV, full, c * 64, it.h, row + v * 64, 0, keep);
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
        // no TMA write may land after the CTA has left
        if (lane == 0 && ok) {
          for (int x = 0; x < 2; ++x)
            if (nq[x] > 0) mbar_wait(&sh->q[x], (uint32_t)(nq[x] - 1) & 1u);
          for (int i = max(0, k - 4); i < k; ++i) {
            mbar_wait(&sh->full_k[i & 3], (uint32_t)(i >> 2) & 1u);
            mbar_wait(&sh->full_v[i & 3], (uint32_t)(i >> 2) & 1u);
          }
        }
        // (given up: a millisecond for what is still on its way)
        if (lane == 0 && !ok)
          for (const unsigned long long t = globaltimer_ns(); globaltimer_ns() - t < 1000000ull;) {}
        __syncwarp();
      } while (once_more());
    }
    // ------------------------------------------------------------ values that are not finite
    // In items done again: zeros in their place, in the tokens that some row of the item does not see.
    if (warp == 11) {
      int k = 0, m = 0;                      // key tiles, those looked through
      bool ok = true;
      do {
        while (ok && walk.next(p, sh, lane, it)) {
          const int whole = walk.last > 0 ? it.whole() : it.most;
          for (int j = whole; ok && j < it.most; ++j, ++m) {
            ok = __all_sync(0xffffffffu, wait(&sh->raw_v[m & 3], (uint32_t)(m >> 2) & 1u, abort_flag));
            if (!ok) break;
            const int lo = it.past + 1 - j * kKT, hi = it.L - j * kKT;   // rows to look at: lo <= row < hi
            for (int part = 0; part < 4; ++part) {                       // 64 rows x 64 elements, 4 rows at a time
              const int v = part >> 1, c = part & 1;
              if (c >= ncv) continue;
              unsigned char* at = smem + kOffRing + (((k + j) * per + ncd + 1 + v) & (kSlots - 1)) * kChunk + c * (kChunk / 2) + lane * 16;
#pragma unroll 4
              for (int i = 0; i < 16; ++i) {
                const int row = v * 64 + i * 4 + (lane >> 3);
                if (row < lo || row >= hi) continue;
                auto clean = [](uint32_t x) {
                  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
                  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
                  return x;
                };
                uint4* y = reinterpret_cast<uint4*>(at + i * 512);
                const uint4 x = *y;
                *y = make_uint4(clean(x.x), clean(x.y), clean(x.z), clean(x.w));
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->full_v[(k + j) & 3]);
          }
          k += it.most;
        }
      } while (once_more());
    }
    // ------------------------------------------------------------ MMA issuers
    // A warp for each row tile x: P_x V of a key tile, then S_x of the next.  (One warp for both
    // was busy for longer than the products: a wait costs it about 190 clocks, an MMA 50.)  A whole
    // warp walks, with values that are the same in all lanes, and one lane issues: the descriptors
    // then stay in uniform registers.
    if (warp == 9 || warp == 10) {
      const int x = __shfl_sync(0xffffffffu, warp - 9, 0);
      const bool lead = elect_one();
      const uint32_t sb = __shfl_sync(0xffffffffu, sbase, 0), t0 = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t idS = idesc_bf16_f32(kRows, kKT, false, false);
      const uint32_t idO = idesc_bf16_f32(kRows, p.Dv, false, true);
      const int qx = SPLIT ? 0 : x;          // whose Q
      const uint64_t da = sdesc_sw128(sb + qx * 3 * kChunk, 16, 1024), dk = sdesc_sw128(sb + kOffRing, 16, 1024);
      const uint64_t dv = sdesc_sw128(sb + kOffRing, kChunk / 2, 1024);
      const uint32_t tS = t0 + x * 128, tO = t0 + kColO + x * 128;
      const int own_steps = p.Dk / 16, rope_steps = p.P / 16;
      bool ok = true;
      int k = 0, nq = 0, no = 0, np = 0;     // key tiles; Q tiles, outputs and P tiles of x
      // S_x against key tile k
      auto scores = [&](int k, bool last) {
        if (!ok) return;
        const int v = k * per;
        if (lead) {
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            if (c > ncd) break;
            const int sl = (v + c) & (kSlots - 1);
            const int steps = c == ncd ? rope_steps : min(4, own_steps - c * 4);
            const uint64_t a = sdesc_at(da, c * kChunk), b = sdesc_at(dk, sl * kChunk);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (kk < steps) umma_bf16(tS, sdesc_at(a, kk * 32), sdesc_at(b, kk * 32), idS, c > 0 || kk > 0 ? 1u : 0u);
            umma_commit(&sh->empty[sl]);
          }
          umma_commit(&sh->s[x]);
          if (last) umma_commit(&sh->q_empty[qx]);
        }
        __syncwarp();
      };
      do {
        bool more = walk.next(p, sh, lane, it);
        while (ok && more) {
          const int n = __shfl_sync(0xffffffffu, it.nt[x], 0);
          const int most = __shfl_sync(0xffffffffu, it.most, 0);
          constexpr int kStep = SPLIT ? 2 : 1;
          int kk = SPLIT ? k + x : k;          // the chain's key tile
          if (n > 0 || (SPLIT && most > 0)) ok = ok && wait(&sh->q[qx], (uint32_t)nq & 1u, abort_flag);
          if (n > 0) {
            ok = ok && wait(&sh->full_k[kk & 3], (uint32_t)(kk >> 2) & 1u, abort_flag);
            tc_fence_after();
            scores(kk, n == 1);
          } else if (SPLIT && most > 0 && lead && ok) {
            mbar_arrive(&sh->q_empty[0]);      // (no key tile for this chain)
          }
          more = walk.next(p, sh, lane, it);   // (while the softmax has work)
          // the last output of the chain has been read
          if (n > 0) ok = ok && wait(&sh->o_free[x], ((uint32_t)no & 1u) ^ 1u, abort_flag);
          for (int j = 0; ok && j < n; ++j, kk += kStep) {
            // O_x += P_x V, half a tile of keys at a time
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const int sl = (kk * per + ncd + 1 + v) & (kSlots - 1), kn = kk + kStep;
              ok = ok && wait(&sh->p[x][v], (uint32_t)(np + j) & 1u, abort_flag);
              if (v == 0) ok = ok && wait(&sh->full_v[kk & 3], (uint32_t)(kk >> 2) & 1u, abort_flag);
              if (!SPLIT && v == 1 && j + 1 < n) ok = ok && wait(&sh->full_k[kn & 3], (uint32_t)(kn >> 2) & 1u, abort_flag);
              if (!ok) break;
              tc_fence_after();
              if (v == 1 && lead) take_turn(&sh->turn);
              if (lead) {
                const uint64_t db = sdesc_at(dv, sl * kChunk);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  umma_bf16_ts(tO, tS + v * 32 + i * 8, sdesc_at(db, i * 2048), idO, j > 0 || v > 0 || i > 0 ? 1u : 0u);
                umma_commit(&sh->empty[sl]);
                if (v == 1) umma_commit(&sh->pv[x]);
              }
              __syncwarp();
            }
            if (SPLIT && j + 1 < n) {
              // (the chain's next keys may need the place of the values that just went out)
              const int kn = kk + kStep;
              if (lead) *static_cast<volatile int*>(&sh->turn) = 0;
              ok = ok && wait(&sh->full_k[kn & 3], (uint32_t)(kn >> 2) & 1u, abort_flag);
              tc_fence_after();
              if (lead) take_turn(&sh->turn);
            }
            if (j + 1 < n) scores(kk + kStep, j + 2 == n);
            if (lead) *static_cast<volatile int*>(&sh->turn) = 0;
          }
          if constexpr (!SPLIT) {
            // key tiles that only the other row tile sees
            for (int j = n; ok && j < most; ++j) {
              ok = wait(&sh->full_k[(k + j) & 3], (uint32_t)((k + j) >> 2) & 1u, abort_flag) &&
                   wait(&sh->full_v[(k + j) & 3], (uint32_t)((k + j) >> 2) & 1u, abort_flag);
              if (lead && ok)
                for (int c = 0; c < per; ++c) mbar_arrive(&sh->empty[((k + j) * per + c) & (kSlots - 1)]);
              __syncwarp();
            }
          }
          k += most;
          nq += SPLIT ? most > 0 : n > 0;
          no += n > 0;
          np += n;
        }
        if (lead) umma_commit(&sh->drain[x]);  // every MMA has completed before TMEM is freed
        mbar_wait(&sh->drain[x], walk.last > 0 ? 1u : 0u);
        __syncwarp();
      } while (once_more());
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2;                 // row tile
    const int r = (int)threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lane_off, tO = tmem + kColO + x * 128 + lane_off;
    int kc = 0, np = 0, np1 = 0, joins = 0;  // key tiles, tiles of P (of the second chain's, items that have any) before this item
    do {
      bool more = walk.next(p, sh, lane, it);
      while (more) {
        const int row = it.first + (SPLIT ? 0 : x * kRows) + r;  // of the sequence
        const int pos = it.past + (SPLIT ? 0 : x * kRows) + r;
        const int mine = x == 0 ? it.nt[0] : it.nt[1], other = SPLIT && x == 0 ? it.nt[1] : 0;
        float m_ref = -INFINITY, lsum = 0.f;
        for (int j = 0; j < mine; ++j) {
          wait(&sh->s[x], (uint32_t)(np + j) & 1u, abort_flag);
          __syncwarp();
          tc_fence_after();
          uint32_t v[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(tS + i * 32, v[i]);
          tmem_ld_wait();
          const int jt = SPLIT ? 2 * j + x : j;                  // key tile of the item
          const int seen = min(pos, it.L - 1) - jt * kKT;        // last key of the tile that the row sees
          if (__any_sync(0xffffffffu, seen < kKT - 1)) {
#pragma unroll
            for (int c = 0; c < kKT; ++c)
              if (c > seen) v[c >> 5][c & 31] = __float_as_uint(-INFINITY);
          }
          float mx8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) mx8[i] = __uint_as_float(v[0][i]);
#pragma unroll
          for (int c = 8; c < kKT; c += 2)
            mx8[(c >> 1) & 7] = fmax3(mx8[(c >> 1) & 7], __uint_as_float(v[c >> 5][c & 31]), __uint_as_float(v[c >> 5][(c + 1) & 31]));
          float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])) * p.qscale;
          const bool need = mx > m_ref + kSlack;
          const float alpha = need ? exp2f(m_ref - mx) : 1.f;    // (m_ref = -inf gives 0)
          if (need) m_ref = mx;
          if (j > 0 && __any_sync(0xffffffffu, need)) {
            // O holds P V of the tile before
            wait(&sh->pv[x], (uint32_t)(np + j - 1) & 1u, abort_flag);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < p.Dv; c += 16) {
              uint32_t w[16];
              tmem_ld16(tO + c, w);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
              tmem_st16(tO + c, w);
            }
            tmem_st_wait();
          }
          lsum *= alpha;
          // (weights of 2^-8 where the reference is, so that none is above 1, and sums of large values stay finite)
          const float negm = m_ref == -INFINITY ? 0.f : -m_ref - kSlack;
          const uint64_t qs2 = f2pack(p.qscale, p.qscale), nm2 = f2pack(negm, negm);
          uint64_t ls2[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) ls2[i] = f2pack(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t pw[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              float x0, x1;
              f2unpack(ffma2(f2pack(__uint_as_float(v[i][2 * c]), __uint_as_float(v[i][2 * c + 1])), qs2, nm2), x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              ls2[c & 3] = fadd2(ls2[c & 3], f2pack(p0, p1));
              pw[c] = pack_bf16(p0, p1);
            }
            tmem_st16(tS + i * 16, pw);
            if (i == 1 && (jt + 1) * kKT > it.L) {
              // Rows behind the context may hold anything, and 0 * NaN would reach O: zeros, before
              // any of P is handed over (by every chain that uses them: either's P V may come first).
              const int u = (kc + jt) * per + ncd + 1 + (r >> 6);
              wait(&sh->full_v[(kc + jt) & 3], (uint32_t)((kc + jt) >> 2) & 1u, abort_flag);
              if (jt * kKT + r >= it.L) {
                unsigned char* vrow = smem + kOffRing + (u & (kSlots - 1)) * kChunk + (r & 63) * 128;
                for (int c = 0; c < ncv * 8; ++c)  // (each row in another order: the banks are all in use)
                  *reinterpret_cast<uint4*>(vrow + (c >> 3) * (kChunk / 2) + (((c + r) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
              }
              __syncwarp();
            }
            if (i & 1) {
              // half a tile of P: its product may begin
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sh->p[x][i >> 1]);
            }
          }
          float ls[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) f2unpack(ls2[i], ls[2 * i], ls[2 * i + 1]);
          lsum += ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
        }

        // ---- O / l as bf16 rows
        const int q0 = it.q0, n = it.n, k0 = it.k0, h = it.h;
        kc += it.most;
        more = walk.next(p, sh, lane, it);     // (its loads run beside the last product)
        if (SPLIT && x == 1) {
          if (mine > 0) {
            // (its last product waited for the item before to be read)
            wait(&sh->pv[1], (uint32_t)(np + mine - 1) & 1u, abort_flag);
            __syncwarp();
            sh->ml[r][0] = m_ref;
            sh->ml[r][1] = lsum;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->ml_full);
          }
          np += mine;
          continue;
        }
        if (mine > 0) {
          wait(&sh->pv[x], (uint32_t)(np + mine - 1) & 1u, abort_flag);
          __syncwarp();
          tc_fence_after();
        }
        float f0 = 1.f, f1 = 0.f;              // of O_x, and of the other half's
        if (other > 0) {
          wait(&sh->ml_full, (uint32_t)joins & 1u, abort_flag);
          wait(&sh->pv[1], (uint32_t)(np1 + other - 1) & 1u, abort_flag);
          __syncwarp();
          tc_fence_after();
          const float m1 = sh->ml[r][0], l1 = sh->ml[r][1], m = fmaxf(m_ref, m1);
          f0 = m_ref == -INFINITY ? 0.f : exp2f(m_ref - m);
          f1 = m1 == -INFINITY ? 0.f : exp2f(m1 - m);
          lsum = fmaf(lsum, f0, l1 * f1);
          if (l1 != l1) lsum = l1;             // (a row of NaN scores has no maximum)
          ++joins;
        }
        const float inv = lsum != 0.f ? 1.f / lsum : 0.f;
        const uint32_t full = write_rows(p, tO, mine > 0, inv * f0, SPLIT && other > 0, inv * f1, q0, row, n, h, lane);
        if (mine > 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh->o_free[x]);
            if (other > 0) mbar_arrive(&sh->o_free[1]);
          }
        }
        if (walk.last > 0) {
          // (all of the warp's rows are written)
          __syncwarp();
          put_back(p, q0, n, k0, h, pos - r - (SPLIT ? 0 : x * kRows), row - lane, pos - lane, lane);
        } else if (__builtin_expect((full & 0x80008000u) && lsum - lsum == 0.f && row < n, 0)) {
          const int round = walk.round - 2;    // (the next item's has been looked up)
          atomicOr(&sh->noted[(round / 32) & (kNoted / 32 - 1)], 1u << (round & 31));
          atomicMax(&sh->redo, round + 1);
        }
        np += mine;
        np1 += other;
      }
    } while (once_more());
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }

}  // namespace

unsigned* status_word_latent_prefill() { return device_word(g_status_latent); }

}  // namespace pa

using namespace pa;

extern "C" int pa_latent_prefill(void* out, const void* query, const int32_t* query_start, int total_queries,
                                 const void* kv, const void* key_rope, long long key_rope_stride,
                                 const int32_t* kv_start, int total_kv, int num_seqs, int num_heads, int key_dim,
                                 int rope_dim, int value_dim, float scale, pa_dtype dtype, void* stream) {
  if (dtype != PA_BF16) return PA_ERR_DTYPE;
  if (total_queries < 0 || total_kv < 0 || num_seqs < 0 || num_seqs > kMaxSeqs || num_heads <= 0 || !dim_ok(key_dim) ||
      !dim_ok(value_dim) || rope_dim <= 0 || rope_dim > 64 || rope_dim % 16 || key_rope_stride < rope_dim ||
      !(scale > 0.f) || (long long)total_queries * num_heads > 0x7fffffffll)
    return PA_ERR_SHAPE;
  // units of 256 rows at most, and of 128
  const long long units2 = (long long)total_queries / (2 * kRows) + num_seqs;
  const long long units1 = (long long)total_queries / kRows + num_seqs;
  if (units1 * num_heads > kMostItems) return PA_ERR_SHAPE;
  if (num_seqs == 0 || total_queries == 0) return PA_OK;
  if (!out || !query || !query_start || !kv_start || (total_kv && (!kv || !key_rope))) return PA_ERR_NULL;
  if (!aligned16(out) || !aligned16(query) || !aligned16(kv) || !aligned16(key_rope) || key_rope_stride % 8)
    return PA_ERR_ALIGN;
  CUtensorMap mapQ, mapQr, mapK, mapKr, mapV;
  // (with no keys at all the maps are never read, and point at the queries)
  const char* kvb = static_cast<const char*>(total_kv ? kv : query);
  const char* krb = static_cast<const char*>(total_kv ? key_rope : query);
  const uint64_t T = (uint64_t)(total_kv ? total_kv : 1), H = (uint64_t)num_heads;
  auto rows_map = [&](CUtensorMap* m, const void* base, int dim, uint64_t width, uint64_t rows, uint32_t box_rows) {
    const uint64_t dims[4] = {(uint64_t)dim, H, rows, 1};
    const uint64_t str[3] = {width * 2, width * 2 * H, width * 2 * H * rows};
    const uint32_t box[4] = {64, 1, box_rows, 1};
    return encode_map(m, base, PA_BF16, 4, dims, str, box, true);
  };
  const uint64_t qw = (uint64_t)key_dim + rope_dim, kw = (uint64_t)key_dim + value_dim;
  const uint64_t kr_dims[4] = {(uint64_t)rope_dim, T, 1, 1};
  const uint64_t kr_str[3] = {(uint64_t)key_rope_stride * 2, (uint64_t)key_rope_stride * 2 * T,
                              (uint64_t)key_rope_stride * 2 * T};
  const uint32_t kr_box[4] = {64, kKT, 1, 1};
  if (!rows_map(&mapQ, query, key_dim, qw, total_queries, kRows) ||
      !rows_map(&mapQr, static_cast<const char*>(query) + key_dim * 2, rope_dim, qw, total_queries, kRows) ||
      !rows_map(&mapK, kvb, key_dim, kw, T, kKT) || !rows_map(&mapV, kvb + key_dim * 2, value_dim, kw, T, 64) ||
      !encode_map(&mapKr, krb, PA_BF16, 4, kr_dims, kr_str, kr_box, true)) {
    note_host_error("cuTensorMapEncodeTiled failed for the queries, keys or values");
    return PA_ERR_CUDA;
  }
  int dev = 0;
  if (!ck(cudaGetDevice(&dev), "cudaGetDevice")) return PA_ERR_CUDA;
  const int sms = device_sm_count();
  // The chains of a CTA divide one row tile's keys where the sequences have no second row tile, or
  // where 256 rows a CTA would leave SMs without work.
  const bool split = total_queries <= (long long)kRows * num_seqs || units2 * num_heads <= 2ll * sms;
  const long long items = (split ? units1 : units2) * num_heads;
  const void* kernel = split ? reinterpret_cast<const void*>(&latent_prefill_kernel<true>)
                             : reinterpret_cast<const void*>(&latent_prefill_kernel<false>);
  if (!raise_smem_limit(kernel, dev)) return PA_ERR_CUDA;
  PrefillParams p = {};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.kv = static_cast<const __nv_bfloat16*>(kv);
  p.query_start = query_start;
  p.kv_start = kv_start;
  p.B = num_seqs;
  p.H = num_heads;
  p.Dk = key_dim;
  p.P = rope_dim;
  p.Dv = value_dim;
  p.rows = total_queries;
  p.kv_rows = total_kv;
  p.qscale = scale * kLog2e;
  void* args[] = {&mapQ, &mapQr, &mapK, &mapKr, &mapV, &p};
  return ck(cudaLaunchKernel(kernel, dim3((unsigned)(items < sms ? items : sms)), dim3(kThreads), args, kSmemBytes,
                             (cudaStream_t)stream),
            "cudaLaunchKernel(latent_prefill_kernel)")
             ? PA_OK
             : PA_ERR_CUDA;
}

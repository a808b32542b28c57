// pa_latent_prefill.cu — ragged causal attention over expanded latent vectors
// (pa_latent_prefill) on the 5th-generation tensor cores: keys of key_dim elements a head,
// one rotated key for all heads, values of value_dim.
//
// One CTA per (256 queries of a sequence, head), as two tiles of 128 rows:
//   S_x = Q_x [K | K_rope]^T   M = 128, N = 128 keys, K = key_dim + rope_dim (12 MMAs of 192)
//   O_x += P_x V               M = 128, N = value_dim, K = 128 keys, P from tensor memory
// Tensor memory holds S_0, S_1 (128 columns each, P_x over the first half of its S_x) and
// O_0, O_1.  The products of one tile run while the other's softmax does:
//   ... P_0 V, S_0', P_1 V, S_1', P_0' V, ...
#include "pa_mma.cuh"
#include "pa_tc.cuh"

namespace pa {
namespace {

__device__ unsigned g_status_latent;

constexpr int kThreads = 384;                // warps 0-3 and 4-7: softmax of a tile each; 8 TMA, 9 MMA, 10-11 none
constexpr int kRows = 128;                   // query rows of a tile
constexpr int kKT = 128;                     // keys per tile
constexpr uint32_t kChunk = 16384;           // 128 rows x 64 elements
constexpr uint32_t kOffK = 6 * kChunk;       // Q: 2 tiles x 3 chunks; K: 2 stages x 3 chunks
constexpr uint32_t kOffV = kOffK + 6 * kChunk;   // V: 2 halves of 64 keys x 2 chunks of 8 KB
constexpr uint32_t kOffBar = kOffV + 2 * kChunk;
constexpr uint32_t kColO = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;                // log2 units a score may exceed its reference by
constexpr int kMaxSeqs = 2048;
// Registers: 384 x 168 at launch, then 2 x 128 x 200 for the softmax and 128 x 104 for the rest.
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 200, kOtherRegs = 104;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split");

struct PrefillParams {
  __nv_bfloat16* out;
  const int32_t *query_start, *kv_start;
  int B, H, Dk, P, Dv, rows, kv_rows;
  float qscale;
};

struct Shared {
  uint64_t q[2], full_k[2], empty_k[2], full_v[2], empty_v[2], s[2], p[2], pv[2], drain;
  int bad_from[128];                         // per value element: first key that is not finite, of the masked ones
  int any_bad;
  uint32_t tmem_base;
  int abort;
  int scan[kThreads / 32];
  int unit[3];                               // sequence, tile of it, units in all
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

// Query rows of sequence b, -1 for an inconsistent one.
__device__ __forceinline__ int rows_of(const PrefillParams& p, int b) {
  const int a = __ldg(&p.query_start[b]), e = __ldg(&p.query_start[b + 1]);
  const int u = __ldg(&p.kv_start[b]), v = __ldg(&p.kv_start[b + 1]);
  return a >= 0 && e >= a && e <= p.rows && u >= 0 && v >= u && v <= p.kv_rows ? e - a : -1;
}

__global__ void __launch_bounds__(kThreads, 1)
latent_prefill_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapQr,
                      const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapKr,
                      const __grid_constant__ CUtensorMap mapV, const PrefillParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  Shared* sh = reinterpret_cast<Shared*>(smem + kOffBar);
  volatile int* abort_flag = &sh->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- work item: the units (256 rows) of all sequences in order, every sequence's last, and
  // longest, unit first; heads innermost
  const int unit = (int)(blockIdx.x / p.H), h = (int)(blockIdx.x % p.H);
  {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
      const int n = rows_of(p, b);
      if (n < 0 && blockIdx.x == 0) atomicOr(&g_status_latent, PA_DEV_BAD_LEN);
      sum += (max(n, 0) + 2 * kRows - 1) / (2 * kRows);
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) sh->scan[warp] = incl;
    __syncthreads();
    int before = incl - sum, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sh->scan[w];
      total += sh->scan[w];
    }
    if (unit >= total) return;               // nothing allocated yet
    if (unit >= before && unit < before + sum) {
      for (int b = b0; b < b1; ++b) {
        const int k = (max(rows_of(p, b), 0) + 2 * kRows - 1) / (2 * kRows);
        if (unit < before + k) {
          sh->unit[0] = b;
          sh->unit[1] = before + k - 1 - unit;
          break;
        }
        before += k;
      }
    }
    if (threadIdx.x < 128) sh->bad_from[threadIdx.x] = 0x7fffffff;
    if (threadIdx.x == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh->q[i], 1);
        mbar_init(&sh->full_k[i], 1);
        mbar_init(&sh->empty_k[i], 1);
        mbar_init(&sh->full_v[i], 1);
        mbar_init(&sh->empty_v[i], 1);
        mbar_init(&sh->s[i], 1);
        mbar_init(&sh->p[i], 128);
        mbar_init(&sh->pv[i], 1);
      }
      mbar_init(&sh->drain, 1);
      sh->abort = 0;
      sh->any_bad = 0;
      fence_mbar_init();
    }
    if (warp == 9) {
      tmem_alloc(&sh->tmem_base, 512);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const int b = sh->unit[0];
  const int q0 = __ldg(&p.query_start[b]), n = __ldg(&p.query_start[b + 1]) - q0;
  const int k0 = __ldg(&p.kv_start[b]), L = __ldg(&p.kv_start[b + 1]) - k0;
  const int first = sh->unit[1] * 2 * kRows;   // first row of the sequence's
  const int past = L - n + first;              // its position
  // tiles of keys that each row tile sees
  int nt[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = min(n - first - x * kRows, kRows);           // rows of the tile
    const int end = r > 0 ? min(L, max(0, past + x * kRows + r)) : 0;
    nt[x] = (end + kKT - 1) / kKT;
  }
  const int most = max(nt[0], nt[1]);
  const uint32_t tmem = sh->tmem_base;
  const int ncd = (p.Dk + 63) / 64, ncv = (p.Dv + 63) / 64;    // chunks of the keys' own part, of the values

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // ------------------------------------------------------------ TMA producer
    if (warp == 8 && lane == 0 && most > 0) {
      const uint64_t once = policy_evict_first(), keep = policy_evict_last();   // (K, V: other row tiles read them too)
      auto load_q = [&](int x) {
        if (nt[x] == 0) return;
        mbar_arrive_expect_tx(&sh->q[x], (uint32_t)(ncd + 1) * kChunk);
        for (int c = 0; c < ncd; ++c)
          tma_load_4d(smem + (x * 3 + c) * kChunk, &mapQ, &sh->q[x], c * 64, h, q0 + first + x * kRows, 0, once);
        tma_load_4d(smem + (x * 3 + ncd) * kChunk, &mapQr, &sh->q[x], 0, h, q0 + first + x * kRows, 0, once);
      };
      int nk = 0, nv = 0;
      auto load_k = [&](int j) -> bool {
        const int st = j & 1;
        if (!wait(&sh->empty_k[st], ((uint32_t)(j >> 1) & 1u) ^ 1u, abort_flag)) return false;
        mbar_arrive_expect_tx(&sh->full_k[st], (uint32_t)(ncd + 1) * kChunk);
        unsigned char* dst = smem + kOffK + st * 3 * kChunk;
        for (int c = 0; c < ncd; ++c)
          tma_load_4d(dst + c * kChunk, &mapK, &sh->full_k[st], c * 64, h, k0 + j * kKT, 0, keep);
        tma_load_4d(dst + ncd * kChunk, &mapKr, &sh->full_k[st], 0, k0 + j * kKT, 0, 0, keep);
        nk = j + 1;
        return true;
      };
      load_q(0);
      bool ok = load_k(0);
      load_q(1);
      for (int j = 0; ok && j < most; ++j) {
        if (j + 1 < most && !(ok = load_k(j + 1))) break;
        for (int v = 0; v < 2; ++v) {
          if (!(ok = wait(&sh->empty_v[v], ((uint32_t)j & 1u) ^ 1u, abort_flag))) break;
          mbar_arrive_expect_tx(&sh->full_v[v], (uint32_t)ncv * kChunk / 2);
          for (int c = 0; c < ncv; ++c)
            tma_load_4d(smem + kOffV + v * kChunk + c * (kChunk / 2), &mapV, &sh->full_v[v], c * 64, h,
                        k0 + j * kKT + v * 64, 0, keep);
          nv = 2 * j + v + 1;
        }
      }
      // no TMA write may land after the CTA has left
      for (int x = 0; x < 2; ++x)
        if (nt[x] > 0) mbar_wait(&sh->q[x], 0);
      for (int j = max(0, nk - 2); j < nk; ++j) mbar_wait(&sh->full_k[j & 1], (uint32_t)(j >> 1) & 1u);
      for (int i = max(0, nv - 2); i < nv; ++i) mbar_wait(&sh->full_v[i & 1], (uint32_t)(i >> 1) & 1u);
    }
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks, with values that are the same in all lanes, and one lane issues: the
    // descriptors then stay in uniform registers.
    if (warp == 9 && most > 0) {
      const bool lead = elect_one();
      const uint32_t sb = __shfl_sync(0xffffffffu, sbase, 0), t0 = __shfl_sync(0xffffffffu, tmem, 0);
      const int n0 = __shfl_sync(0xffffffffu, nt[0], 0), n1 = __shfl_sync(0xffffffffu, nt[1], 0);
      const uint32_t idS = idesc_bf16_f32(kRows, kKT, false, false);
      const uint32_t idO = idesc_bf16_f32(kRows, p.Dv, false, true);
      const uint64_t dq = sdesc_sw128(sb, 16, 1024), dk = sdesc_sw128(sb + kOffK, 16, 1024);
      const uint64_t dv = sdesc_sw128(sb + kOffV, kChunk / 2, 1024);
      const int own_steps = p.Dk / 16, rope_steps = p.P / 16;
      bool ok = true;
      auto scores = [&](int x, int j) {
        if (j == 0) ok = ok && wait(&sh->q[x], 0, abort_flag);
        ok = ok && wait(&sh->full_k[j & 1], (uint32_t)(j >> 1) & 1u, abort_flag);
        if (!ok) return;
        tc_fence_after();
        if (lead) {
          const uint64_t da = sdesc_at(dq, x * 3 * kChunk), db = sdesc_at(dk, (j & 1) * 3 * kChunk);
          const uint32_t d = t0 + x * 128;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            if (kk >= own_steps) break;
            umma_bf16(d, sdesc_at(da, (kk >> 2) * kChunk + (kk & 3) * 32), sdesc_at(db, (kk >> 2) * kChunk + (kk & 3) * 32), idS,
                      kk > 0 ? 1u : 0u);
          }
          const uint64_t ra = sdesc_at(da, ncd * kChunk), rb = sdesc_at(db, ncd * kChunk);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk >= rope_steps) break;
            umma_bf16(d, sdesc_at(ra, kk * 32), sdesc_at(rb, kk * 32), idS, 1u);
          }
          umma_commit(&sh->s[x]);
        }
        __syncwarp();
      };
      auto values = [&](int x, int j, bool frees) {
        ok = ok && wait(&sh->p[x], (uint32_t)j & 1u, abort_flag);
        for (int v = 0; v < 2; ++v) {
          ok = ok && wait(&sh->full_v[v], (uint32_t)j & 1u, abort_flag);
          if (!ok) return;
          tc_fence_after();
          if (lead) {
            const uint64_t db = sdesc_at(dv, v * kChunk);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16_ts(t0 + kColO + x * 128, t0 + x * 128 + v * 32 + kk * 8, sdesc_at(db, kk * 2048), idO,
                           j > 0 || v > 0 || kk > 0 ? 1u : 0u);
            if (frees) umma_commit(&sh->empty_v[v]);
            if (v == 1) umma_commit(&sh->pv[x]);
          }
          __syncwarp();
        }
      };
      // (the row tile that sees a key tile last frees it)
      if (n0 > 0) scores(0, 0);
      if (n1 > 0) scores(1, 0);
      if (ok && lead) umma_commit(&sh->empty_k[0]);
      for (int j = 0; ok && j < max(n0, n1); ++j) {
        if (j < n0) values(0, j, j >= n1);
        if (j + 1 < n0) scores(0, j + 1);
        if (j < n1) values(1, j, true);
        if (j + 1 < n1) scores(1, j + 1);
        if (ok && lead && j + 1 < max(n0, n1)) umma_commit(&sh->empty_k[(j + 1) & 1]);
        __syncwarp();
      }
      if (lead) umma_commit(&sh->drain);     // every MMA has completed before TMEM is freed
      mbar_wait(&sh->drain, 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2;                 // row tile
    const int r = (int)threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lane_off, tO = tmem + kColO + x * 128 + lane_off;
    const int row = first + x * kRows + r;   // of the sequence
    const int pos = past + x * kRows + r;
    const int mine = x == 0 ? nt[0] : nt[1];
    float m_ref = -INFINITY, lsum = 0.f;
    for (int j = 0; j < mine; ++j) {
      wait(&sh->s[x], (uint32_t)j & 1u, abort_flag);
      __syncwarp();
      tc_fence_after();
      uint32_t v[4][32];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(tS + i * 32, v[i]);
      tmem_ld_wait();
      const int seen = min(pos, L - 1) - j * kKT;              // last key of the tile that the row sees
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
      const float alpha = need ? exp2f(m_ref - mx) : 1.f;      // (m_ref = -inf gives 0)
      if (need) m_ref = mx;
      if (j > 0 && __any_sync(0xffffffffu, need)) {
        // O holds P V of the tile before
        wait(&sh->pv[x], (uint32_t)(j - 1) & 1u, abort_flag);
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
      const float negm = m_ref == -INFINITY ? 0.f : -m_ref;
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
      }
      float ls[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) f2unpack(ls2[i], ls[2 * i], ls[2 * i + 1]);
      lsum += ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
      // Values that not every row of the CTA sees: rows behind the context may hold anything, and
      // 0 * NaN would reach O, so they are zeroed; of the others what is not finite, and the rows
      // that do see it are told so at the end.  The row tile whose P V comes first does it.
      if ((x == 0 || j >= nt[0]) && j * kKT + kKT - 1 > past) {
        const int key = j * kKT + r;
        wait(&sh->full_v[r >> 6], (uint32_t)j & 1u, abort_flag);
        if (key > past) {
          unsigned char* vrow = smem + kOffV + (r >> 6) * kChunk + (r & 63) * 128;
          for (int c = 0; c < ncv * 8; ++c) {
            uint4* w = reinterpret_cast<uint4*>(vrow + (c >> 3) * (kChunk / 2) + (c & 7) * 16);
            if (key >= L) {
              *w = make_uint4(0u, 0u, 0u, 0u);
              continue;
            }
            uint32_t y[4] = {w->x, w->y, w->z, w->w};
            bool bad = false;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              bad = bad || (y[i] & 0x7f80u) == 0x7f80u || (y[i] & 0x7f800000u) == 0x7f800000u;
            if (bad) {
              const int d = (c >> 3) * 64 + (((c & 7) ^ (r & 7)) << 3);     // first element of the piece
              sh->any_bad = 1;
              for (int i = 0; i < 4; ++i) {
                if ((y[i] & 0x7f80u) == 0x7f80u) {
                  atomicMin(&sh->bad_from[d + 2 * i], key);
                  y[i] &= 0xffff0000u;
                }
                if ((y[i] & 0x7f800000u) == 0x7f800000u) {
                  atomicMin(&sh->bad_from[d + 2 * i + 1], key);
                  y[i] &= 0xffffu;
                }
              }
              *w = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&sh->p[x]);
    }

    // ---- O / l as bf16 rows
    if (mine > 0) {
      wait(&sh->pv[x], (uint32_t)(mine - 1) & 1u, abort_flag);
      __syncwarp();
      tc_fence_after();
    }
    const float inv = lsum != 0.f ? 1.f / lsum : 0.f;
    const bool bad = *static_cast<volatile int*>(&sh->any_bad) != 0;   // (written before the last P this tile used)
    __nv_bfloat16* o = p.out + ((size_t)(q0 + row) * p.H + h) * p.Dv;
    for (int c = 0; c < p.Dv; c += 32) {
      uint32_t w[32];
      if (mine > 0) {
        tmem_ld32(tO + c, w);
        tmem_ld_wait();
      }
      if (row >= n) continue;
      if (bad) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (pos >= sh->bad_from[c + i]) w[i] = 0x7fc00000u;
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          y[i] = mine > 0 ? pack_bf16(__uint_as_float(w[g * 8 + 2 * i]) * inv, __uint_as_float(w[g * 8 + 2 * i + 1]) * inv) : 0u;
        st_v4(o + c + g * 8, make_uint4(y[0], y[1], y[2], y[3]));
      }
    }
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
  const long long units = (long long)total_queries / (2 * kRows) + num_seqs;
  if (units * num_heads > 0x7fffffffll) return PA_ERR_SHAPE;
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
  if (!raise_smem_limit(reinterpret_cast<const void*>(&latent_prefill_kernel), dev)) return PA_ERR_CUDA;
  PrefillParams p = {};
  p.out = static_cast<__nv_bfloat16*>(out);
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
  return ck(cudaLaunchKernel(reinterpret_cast<const void*>(&latent_prefill_kernel), dim3((unsigned)(units * num_heads)),
                             dim3(kThreads), args, kSmemBytes, (cudaStream_t)stream),
            "cudaLaunchKernel(latent_prefill_kernel)")
             ? PA_OK
             : PA_ERR_CUDA;
}

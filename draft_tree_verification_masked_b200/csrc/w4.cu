// w4.cu -- products with 4-bit weights and group scales on tcgen05 / TMEM (sm_100a).
//
// Single-request verification moves weights rather than computing ("EAGLE-4 是什麼？...",
// aiposthub.com, opening section), and a tree of drafted tokens shares one pass over them, so a
// target held in 4 bits reads a quarter of the bytes:
//
//   y[m][n] = sum_g s[n][g] * (sum_{k in g} (q[n][k] - z[n][g]) x[m][k]) + b[n]
//
// The weights are the MMA's A operand (128 rows a tile), the tokens its N dimension: even one
// token fills the tensor core's rows.  The inner sums take the integers q - z, which bf16 holds
// exactly; the tensor core multiplies them with x exactly and adds in fp32.  Each group's sum is
// read back from TMEM and enters an fp32 register accumulator times its scale, so no weight is
// ever rounded.
//
//   q -> bf16   a thread owns one row: (w >> 4 p) & 0x000f000f | 0x43004300 is the pair
//               (128 + q_p, 128 + q_{p+4}), and subtracting 128 + z is exact.  The pairs go to
//               TMEM as A.  x is copied once per call with every eight values in the matching
//               order 0 4 1 5 2 6 3 7.
//   D = A x^T   tcgen05.mma M=128 x N=NT x K=16, A from TMEM, x from shared memory.
//
// One CTA per SM walks its equal share of a flat list of work units, so that any N and K fill all
// SMs.  A unit is four 128 x 128 weight blocks: two row tiles of two
// k blocks where there are many rows (x is then read once for 256 rows), or four k blocks of one
// row tile (few rows).  Row tiles whose units lie on several
// CTAs are summed from partials in the workspace by the CTA that arrives last, in the order of k,
// so results do not depend on timing.
#include <algorithm>

#include "kernels.cuh"

namespace etree {

namespace {
constexpr int kWThreads = 32 * 20;          // TMA, two MMA, one idle, 8 unpacking, 8 summing warps
constexpr int kWBox = 128 * 64;             // [128 rows][64 bytes]
constexpr int kWMaxStages = 5;
constexpr int kWSmem = 226 * 1024;

struct W4Smem {
  uint64_t full[kWMaxStages], empty[kWMaxStages];
  uint64_t a_full[4], a_free[4], d_full[4], d_free[4], s_full[4][2], drain[2];
  uint32_t tmem;
  int last;
};

__device__ __forceinline__ void w4_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// First unit of CTA c, and the CTA that holds unit u.
__device__ __forceinline__ int w4_first(int units, int grid, int c) {
  return (int)((int64_t)units * c / grid);
}
__device__ __forceinline__ int w4_owner(int units, int grid, int u) {
  return (int)(((int64_t)(u + 1) * grid - 1) / units);
}

// A CTA's walk over its units: the tile, its row and token chunk, and the unit's place in depth.
struct W4Walk {
  int tile, kb, rowt, chunk;
  __device__ __forceinline__ W4Walk(const W4Params& p, int u) {
    tile = u / p.kbu;
    kb = u - tile * p.kbu;
    rowt = tile / p.chunks;
    chunk = tile - rowt * p.chunks;
  }
  __device__ __forceinline__ void next(const W4Params& p) {
    if (++kb < p.kbu) return;
    kb = 0;
    ++tile;
    if (++chunk < p.chunks) return;
    chunk = 0;
    ++rowt;
  }
};

__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// The bf16 pair (128 + q, 128 + q') of the nibbles at bits 0 and 16: (w & 0x000f000f) | magic in one
// operation, with the second constant in a register.
__device__ __forceinline__ uint32_t nibble_pair(uint32_t w, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xEA;" : "=r"(r) : "r"(w), "r"(magic));
  return r;
}

// a - b on bf16 pairs (exact here: integers of magnitude below 256).
__device__ __forceinline__ uint32_t sub_pair(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                   *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Sums of two tokens in one 64-bit register: acc += (v0, v1) s, each lane rounded as in fmaf.
__device__ __forceinline__ void ffma2_acc(uint64_t& acc, float v0, float v1, float s) {
  uint64_t x, ss;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(v0), "f"(v1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(x), "l"(ss));
}
__device__ __forceinline__ float half_of(uint64_t acc, int i) {
  return __uint_as_float((uint32_t)(acc >> (32 * i)));
}
}  // namespace

// x [M][K] (rows x_stride apart) -> xp [rows][K], every eight values as 0 4 1 5 2 6 3 7 and rows
// behind M zero; the tiles' arrival counters are cleared.
__global__ void __launch_bounds__(256) w4_prepare_kernel(W4Params p, int rows) {
  pdl_trigger();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int c8 = p.K / 8;
  for (int64_t t = i; t < p.tiles; t += (int64_t)gridDim.x * 256) p.count[t] = 0;
  if (i >= (int64_t)rows * c8) return;
  const int m = (int)(i / c8), c = (int)(i - (int64_t)m * c8);
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (m < p.M) {
    const uint4 x = *reinterpret_cast<const uint4*>(p.x + (int64_t)m * p.x_stride + c * 8);
    v.x = __byte_perm(x.x, x.z, 0x5410);
    v.y = __byte_perm(x.x, x.z, 0x7632);
    v.z = __byte_perm(x.y, x.w, 0x5410);
    v.w = __byte_perm(x.y, x.w, 0x7632);
  }
  reinterpret_cast<uint4*>(p.xp)[i] = v;
}

// What the roles share: pieces of shared memory, the first unit and the TMEM base.
struct W4Cta {
  uint8_t* smem;
  float *red, *scale_s;
  W4Smem* sh;
  int u0;
  uint32_t tmem;
};

// The two roles with many live registers are functions of their own, so that each is allocated
// apart (inlined side by side they spilled in the inner loops).
template <int NT, int KS>
__device__ __noinline__ void w4_unpack(const W4Params& p, const W4Cta& c, int nu) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int ks = KS, rpt = KS == 4 ? 128 : 256;
  W4Smem* const sh = c.sh;
  float* const scale_s = c.scale_s;
  const int u0 = c.u0, gpb = 128 / p.group, ng = p.K / p.group;
  const uint32_t tmem = c.tmem;
  uint8_t* const smem = c.smem;
  constexpr int stage = 4 * kWBox + ks * NT * 256;
  const bool wide = (ng & 3) == 0;                      // four groups of a row in one load
  const int upc = max(1, 4 / (gpb * ks));               // units that four groups serve
  // ------------------------------------------------------------------------- q to A in TMEM
  const int wg = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
  const int wrow = (ks == 4 ? 0 : wg * 128) + row;    // the row in the tile
  const uint32_t la = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 128 * wg;
  const int sw = (row >> 1) & 3;
  // scales and zero points of four consecutive groups: `cur` serves upc units of a tile, `nxt`
  // the units after them
  struct Groups {
    uint32_t s01, s23, z;
  };
  // The loads are unconditional, at addresses kept inside the arrays, so that nothing waits for
  // them before they are used; rows and groups behind the end get the scale 0 there.
  auto fetch = [&](const W4Walk& at, int e) -> Groups {
    const int n = min(at.rowt * rpt + wrow, p.N - 1);
    const int g = ((at.kb * ks + (2 * wg + e) % ks) * gpb) & ~3;
    const int64_t o = (int64_t)n * ng + min(g, ng - (wide ? 4 : 1));
    Groups r;
    r.z = 0x08080808u;
    if (wide) {
      const uint2 s = __ldg(reinterpret_cast<const uint2*>(p.scales + o));
      r.s01 = s.x;
      r.s23 = s.y;
      if (p.zeros) r.z = __ldg(reinterpret_cast<const uint32_t*>(p.zeros + o));
    } else {
      uint32_t s[4], z[4] = {8u, 8u, 8u, 8u};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t oj = (int64_t)n * ng + min(g + j, ng - 1);
        s[j] = __ldg(p.scales + oj);
        if (p.zeros) z[j] = __ldg(p.zeros + oj);
      }
      r.s01 = s[0] | s[1] << 16;
      r.s23 = s[2] | s[3] << 16;
      r.z = z[0] | z[1] << 8 | z[2] << 16 | z[3] << 24;
    }
    return r;
  };
  Groups cur[2], nxt[2];
  W4Walk at(p, u0), pre = at;
  int pre_left = nu;                                  // units from `pre` to the end
  auto fetch_pre = [&]() {
    nxt[0] = fetch(pre, 0);
    nxt[1] = fetch(pre, 1);
    do {                                              // to the first unit of the next chunk
      pre.next(p);
      --pre_left;
    } while ((pre.kb & (upc - 1)) != 0 && pre_left > 0);
  };
  fetch_pre();
  uint32_t magic = 0x43004300u;
  asm volatile("" : "+r"(magic));                        // stays in a register
  bool ok = true;
  int st = 0;
  uint32_t ph = 0;
  for (int i = 0; ok && i < nu; ++i, at.next(p)) {
    if (i == 0 || (at.kb & (upc - 1)) == 0) {
      cur[0] = nxt[0];
      cur[1] = nxt[1];
      if (pre_left > 0) fetch_pre();
    }
    if (!mbar_wait(&sh->full[st], ph)) { ok = false; break; }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int w = 2 * wg + e;
      const int g0 = ((at.kb * ks + w % ks) * gpb) & 3;
      const uint8_t* src = smem + st * stage + w * kWBox + row * 64;
      uint32_t qw[16];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 q = *reinterpret_cast<const uint4*>(src + ((c ^ sw) << 4));
        qw[4 * c] = q.x;
        qw[4 * c + 1] = q.y;
        qw[4 * c + 2] = q.z;
        qw[4 * c + 3] = q.w;
      }
      // A is free again; this also says that the summing warps are done with unit i - 2, whose
      // scales lie where unit i's go
      if (i > 0 && !mbar_wait(&sh->a_free[w], (i - 1) & 1)) { ok = false; break; }
      tc_fence_after();
      float* sc = scale_s + ((i & 1) * 4 + w) * gpb * 128 + row;
      const int gb = (at.kb * ks + w % ks) * gpb;       // the block's first group
      const bool in = at.rowt * rpt + wrow < p.N;
      for (int g = 0; g < gpb; ++g) {
        const uint32_t sv = ((g0 + g) & 2) ? cur[e].s23 : cur[e].s01;
        sc[g * 128] = in && gb + g < ng
                          ? __uint_as_float(((g0 + g) & 1) ? (sv & 0xffff0000u) : (sv << 16))
                          : 0.f;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t z = (cur[e].z >> (8 * (g0 + (c * gpb >> 2)))) & 15u;
        const uint32_t zz = 0x43004300u | z | z << 16;
        uint32_t v[16];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int b = 0; b < 4; ++b)
            v[4 * j + b] = sub_pair(nibble_pair(qw[4 * c + j] >> (4 * b), magic), zz);
        tmem_st16_async(la + 64 * e + 16 * c, v);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh->s_full[w][i & 1]);
        mbar_arrive(&sh->a_full[w]);
        if (e == 1) mbar_arrive(&sh->empty[st]);
      }
    }
    if (++st == p.stages) { st = 0; ph ^= 1; }
  }
  if (!ok && lane == 0) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_W4);
}

template <int NT, int KS>
__device__ __noinline__ void w4_sum(const W4Params& p, const W4Cta& c, int nu) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int ks = KS, rpt = KS == 4 ? 128 : 256;
  W4Smem* const sh = c.sh;
  float* const scale_s = c.scale_s;
  const int u0 = c.u0, gpb = 128 / p.group;
  const uint32_t tmem = c.tmem;
  float* const red = c.red;
  const int per_round = NT == 64 ? 1 : min(gpb, 64 / NT), rounds = gpb / per_round;
  // ------------------------------------------------------- the scaled sums of the groups
  const int wg = (warp - 12) >> 2, row = (warp & 3) * 32 + lane, tid = threadIdx.x - 12 * 32;
  const int wrow = (ks == 4 ? 0 : wg * 128) + row;
  const uint32_t ld = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256 + 128 * wg;
  pdl_wait();
  W4Walk at(p, u0);
  uint64_t acc[NT / 2];                               // tokens 2 c and 2 c + 1
  auto clear = [&]() {
#pragma unroll
    for (int c = 0; c < NT / 2; ++c) acc[c] = 0ull;
  };
  clear();
  bool ok = true;
  uint32_t use = 0;
  for (int i = 0; i < nu; ++i, at.next(p)) {
    for (int rd = 0; ok && rd < rounds; ++rd, ++use) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int w = 2 * wg + e;
        const float* sc = scale_s + (((i & 1) * 4 + w) * gpb + rd * per_round) * 128 + row;
        if (ok && !mbar_wait(&sh->s_full[w][i & 1], (i >> 1) & 1)) ok = false;
        if (ok && !mbar_wait(&sh->d_full[w], use & 1)) ok = false;
        tc_fence_after();
        for (int g = 0; g < per_round; ++g) {
          const float s = sc[g * 128];
#pragma unroll
          for (int c = 0; c < NT; c += 16) {
            float d[16];
            tmem_ld16(ld + 64 * e + NT * g + c, d);
#pragma unroll
            for (int b = 0; b < 16; b += 2)
              ffma2_acc(acc[(c + b) / 2], d[b], d[b + 1], s);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->d_free[w]);
      }
    }

    // ------------------------------------------------ the end of this CTA's part of a tile
    const bool tile_end = at.kb + 1 == p.kbu;
    if (!tile_end && i + 1 < nu) continue;
    const int tile = at.tile;
    const int m0 = at.chunk * NT, mv = min(NT, p.M - m0);
    if constexpr (KS == 4) {                          // add the other warpgroup's sums
      if (wg == 1) {
#pragma unroll
        for (int c = 0; c < NT; ++c) red[c * 128 + row] = half_of(acc[c / 2], c & 1);
      }
      w4_sync();
      if (wg == 0) {
#pragma unroll
        for (int c = 0; c < NT; c += 2)
          ffma2_acc(acc[c / 2], red[c * 128 + row], red[(c + 1) * 128 + row], 1.f);
      }
    }
    const bool mine = ks == 2 || wg == 0;
    const int t0 = u0 + i - at.kb, t1 = t0 + p.kbu;
    auto bias_of = [&](int n) {
      return p.bias ? __uint_as_float((uint32_t)__ldg(p.bias + n) << 16) : 0.f;
    };
    if (u0 <= t0 && tile_end) {                       // the whole tile
      const int n = at.rowt * rpt + wrow;
      if (mine && n < p.N) {
        const float b = bias_of(n);
        // one running pointer: 64 row offsets at once would push the sums out of the registers
        const int64_t step = p.out_stride * (p.out_f32 ? 4 : 2);
        char* dst = reinterpret_cast<char*>(p.out) +
                    ((int64_t)m0 * p.out_stride + n) * (p.out_f32 ? 4 : 2);
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          if (c < mv) {
            const float v = half_of(acc[c / 2], c & 1) + b;
            if (p.out_f32) *reinterpret_cast<float*>(dst) = v;
            else *reinterpret_cast<__nv_bfloat16*>(dst) = __float2bfloat16_rn(v);
          }
          dst += step;
          asm volatile("" : "+l"(dst));
        }
      }
    } else {
      const int64_t part = (int64_t)NT * rpt;         // a CTA has room for two parts of tiles
      if (mine) {
        float* dst = p.part + (2 * blockIdx.x + (u0 >= t0 ? 0 : 1)) * part + wrow;
#pragma unroll
        for (int c = 0; c < NT; ++c)
          if (c < mv) dst[c * rpt] = half_of(acc[c / 2], c & 1);
      }
      __threadfence();
      w4_sync();
      const int c0 = w4_owner(p.units, gridDim.x, t0), c1 = w4_owner(p.units, gridDim.x, t1 - 1);
      if (tid == 0) sh->last = atomicAdd(p.count + tile, 1) == c1 - c0;
      w4_sync();
      if (sh->last) {
        __threadfence();
        // this thread's rows at every step'th token; the loads of 8 tokens are in flight at once
        constexpr int step = 256 / rpt;
        const int rr = tid & (rpt - 1), n = at.rowt * rpt + rr;
        const float b = n < p.N ? bias_of(n) : 0.f;
        for (int m = tid / rpt; m < mv; m += 8 * step) {
          float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          for (int c = c0; c <= c1; ++c) {
            const bool first = w4_first(p.units, gridDim.x, c) >= t0;
            const float* src = p.part + (2 * c + (first ? 0 : 1)) * part + rr;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              x[e] = m + e * step < mv ? __ldcg(src + (m + e * step) * rpt) : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += x[e];
          }
          if (n < p.N) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (m + e * step < mv) {
                const int64_t o = (int64_t)(m0 + m + e * step) * p.out_stride + n;
                if (p.out_f32) reinterpret_cast<float*>(p.out)[o] = v[e] + b;
                else reinterpret_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v[e] + b);
              }
          }
        }
      }
    }
    if constexpr (KS == 4) w4_sync();                 // `red` is free again
    clear();
  }
  if (!ok && lane == 0) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_W4);
}

template <int NT, int KS>
__global__ void __launch_bounds__(kWThreads, 1)
w4_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_x,
          const __grid_constant__ W4Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int ks = KS;                                // k blocks of a unit: 4 or 2
  constexpr int xbytes = NT * 256;                          // one k block of x: two boxes [NT][64]
  constexpr int stage = 4 * kWBox + ks * xbytes;
  float* red = reinterpret_cast<float*>(smem + p.stages * stage);      // [NT][128], ks = 4
  // scales of a unit's blocks: [unit parity][block][group][128 rows]
  const int gpb = 128 / p.group;                        // groups of a k block
  float* scale_s = red + (ks == 4 ? NT * 128 : 0);
  W4Smem* sh = reinterpret_cast<W4Smem*>(scale_s + 8 * 128 * gpb);
  const int u0 = w4_first(p.units, gridDim.x, blockIdx.x);
  const int nu = w4_first(p.units, gridDim.x, blockIdx.x + 1) - u0;
  constexpr int rpt = ks == 4 ? 128 : 256;                // rows of a tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 10);
    }
    for (int w = 0; w < 4; ++w) {
      mbar_init(&sh->a_full[w], 4);
      mbar_init(&sh->a_free[w], 1);
      mbar_init(&sh->s_full[w][0], 4);
      mbar_init(&sh->s_full[w][1], 4);
      mbar_init(&sh->d_full[w], 1);
      mbar_init(&sh->d_free[w], 4);
    }
    mbar_init(&sh->drain[0], 1);
    mbar_init(&sh->drain[1], 1);
    fence_barrier_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;                       // A of warpgroup w at 64 w, D at 256 + 64 w

  const int per_round = NT == 64 ? 1 : min(gpb, 64 / NT);          // groups that D holds at once
  const int rounds = gpb / per_round;

  const W4Cta c{smem, red, scale_s, sh, u0, tmem};
  if (warp == 0) {
    // ------------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      auto load_q = [&](const W4Walk& at, int st) {
        const int kb = at.kb * ks, row0 = at.rowt * rpt;
        uint8_t* dst = smem + st * stage;
        mbar_arrive_expect_tx(&sh->full[st], stage);
#pragma unroll
        for (int w = 0; w < 4; ++w)
          tma_load_2d(dst + w * kWBox, &tm_q, &sh->full[st], (kb + w % ks) * 64,
                      row0 + w / ks * 128);
      };
      auto load_x = [&](const W4Walk& at, int st) {
        uint8_t* dst = smem + st * stage + 4 * kWBox;
        for (int w = 0; w < ks; ++w)
          for (int h = 0; h < 2; ++h)
            tma_load_2d(dst + w * xbytes + h * (NT * 128), &tm_x, &sh->full[st],
                        (at.kb * ks + w) * 128 + h * 64, at.chunk * NT);
      };
      // the first weights do not depend on the kernel that reorders x
      const int ahead = min(nu, p.stages);
      W4Walk at(p, u0);
      for (int i = 0; i < ahead; ++i, at.next(p)) load_q(at, i);
      pdl_wait();
      bool ok = true;
      int issued = 0, st = 0;
      uint32_t ph = 0;
      at = W4Walk(p, u0);
      for (int i = 0; i < nu; ++i, at.next(p)) {
        if (i >= ahead) {
          if (!mbar_wait(&sh->empty[st], ph ^ 1)) { ok = false; break; }
          load_q(at, st);
        }
        load_x(at, st);
        issued = i + 1;
        if (++st == p.stages) { st = 0; ph ^= 1; }
      }
      // every copy has landed before the CTA may exit (bounded)
      for (int i = max(0, issued - p.stages); i < issued; ++i)
        ok = mbar_wait(&sh->full[i % p.stages], (i / p.stages) & 1) && ok;
      if (!ok) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_W4);
    }
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------- MMA issuers, two of the four blocks each
    const uint32_t id = idesc_bf16_f32(128, NT);
    const uint64_t dx0 = smem_desc_sw128(smem + 4 * kWBox);
    const int kg = p.group / 16, kg_log = 31 - __clz(kg);           // MMAs of a group
    bool ok = true;
    int st = 0;
    uint32_t ph = 0, use = 0;                           // `use` counts the fillings of D
    for (int i = 0; ok && i < nu; ++i) {
      ok = mbar_wait(&sh->full[st], ph);
      tc_fence_after();
      const uint64_t dx = dx0 + (uint64_t)((uint32_t)(st * stage) >> 4);
      for (int rd = 0; rd < rounds; ++rd, ++use) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int w = 2 * (warp - 1) + e;
          if (use > 0) ok = ok && mbar_wait(&sh->d_free[w], (use - 1) & 1);
          if (rd == 0) ok = ok && mbar_wait(&sh->a_full[w], i & 1);
          tc_fence_after();
          const uint64_t dxw = dx + w % ks * (xbytes >> 4);
          const uint32_t aw = tmem + 64 * w, dw = aw + 256;
          if (ok && elect_one()) {
            if (kg == 8) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                tc_mma_bf16_ts(dw, aw + 8 * k, dxw + (k >> 2) * (NT * 128 >> 4) + 2 * (k & 3), id,
                               k > 0 ? 1u : 0u);
            } else {
              const int k0 = rd * per_round * kg;
#pragma unroll 2
              for (int k = 0; k < per_round * kg; ++k)
                tc_mma_bf16_ts(dw + ((k >> kg_log) * NT), aw + 8 * (k0 + k),
                               dxw + ((k0 + k) >> 2) * (NT * 128 >> 4) + 2 * ((k0 + k) & 3), id,
                               k & (kg - 1));
            }
            tc_commit(&sh->d_full[w]);
            if (rd == rounds - 1) {
              tc_commit(&sh->a_free[w]);
              if (e == 1) tc_commit(&sh->empty[st]);
            }
          }
          __syncwarp();
        }
      }
      if (++st == p.stages) { st = 0; ph ^= 1; }
    }
    if (elect_one()) tc_commit(&sh->drain[warp - 1]);
    __syncwarp();
    if (!mbar_wait(&sh->drain[warp - 1], 0)) ok = false;
    if (!ok && lane == 0) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_W4);
  } else if (warp >= 4 && warp < 12) {
    w4_unpack<NT, KS>(p, c, nu);
  } else if (warp >= 12) {
    w4_sum<NT, KS>(p, c, nu);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

static int w4_stages(int nt, int ks, int group) {
  const int stage = 4 * kWBox + ks * nt * 256;
  const int fixed = 1024 + (ks == 4 ? nt * 512 : 0) + 8 * 512 * (128 / group) + (int)sizeof(W4Smem);
  return std::min(kWMaxStages, (kWSmem - fixed) / stage);
}

cudaError_t launch_w4(const CUtensorMap& q, const CUtensorMap& x, W4Params p, int nt, int grid,
                      cudaStream_t s) {
  p.stages = w4_stages(nt, p.ks, p.group);
  const int rows = p.chunks * nt;
  const int64_t items = (int64_t)rows * (p.K / 8);
  w4_prepare_kernel<<<(unsigned)((items + 255) / 256), 256, 0, s>>>(p, rows);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  auto go = [&](auto kernel) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(grid), dim3(kWThreads), (size_t)kWSmem, s, q, x, p);
  };
  if (p.ks == 4)
    return nt == 16 ? go(w4_kernel<16, 4>) : go(w4_kernel<32, 4>);
  return nt == 16 ? go(w4_kernel<16, 2>) : nt == 32 ? go(w4_kernel<32, 2>) : go(w4_kernel<64, 2>);
}

}  // namespace etree

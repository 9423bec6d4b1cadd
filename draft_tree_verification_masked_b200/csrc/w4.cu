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
constexpr int kWThreads = 32 * 12;          // TMA, MMA, two idle, eight consumer warps
constexpr int kWBox = 128 * 64;             // [128 rows][64 bytes]
constexpr int kWMaxStages = 5;
constexpr int kWSmem = 220 * 1024;

struct W4Smem {
  uint64_t full[kWMaxStages], empty[kWMaxStages];
  uint64_t a_full[4], d_full[4], d_free[4], drain;
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

// a - b on bf16 pairs (exact here: integers of magnitude below 256).
__device__ __forceinline__ uint32_t sub_pair(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                   *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// (a0, a1) += (v0, v1) s
__device__ __forceinline__ void ffma2_acc(float& a0, float& a1, float v0, float v1, float s) {
  uint64_t x, ss, a;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(v0), "f"(v1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(x), "l"(ss));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(a));
}

// Scales and zero points of four consecutive groups of one row.
struct W4Groups {
  uint32_t s01, s23, z;
};
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

template <int NT, int KS>
__global__ void __launch_bounds__(kWThreads, 1)
w4_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_x,
          W4Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int ks = KS;                                // k blocks of a unit: 4 or 2
  constexpr int xbytes = NT * 256;                          // one k block of x: two boxes [NT][64]
  constexpr int stage = 4 * kWBox + ks * xbytes;
  float* red = reinterpret_cast<float*>(smem + p.stages * stage);      // [NT][128], ks = 4
  W4Smem* sh = reinterpret_cast<W4Smem*>(reinterpret_cast<uint8_t*>(red) +
                                         (ks == 4 ? NT * 128 * 4 : 0));
  const int u0 = w4_first(p.units, gridDim.x, blockIdx.x);
  const int nu = w4_first(p.units, gridDim.x, blockIdx.x + 1) - u0;
  constexpr int rpt = ks == 4 ? 128 : 256;                // rows of a tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 9);
    }
    for (int w = 0; w < 4; ++w) {
      mbar_init(&sh->a_full[w], 4);
      mbar_init(&sh->d_full[w], 1);
      mbar_init(&sh->d_free[w], 4);
    }
    mbar_init(&sh->drain, 1);
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

  const int gpb = 128 / p.group;                       // groups of a k block
  const int per_round = min(gpb, 64 / NT);             // groups that D holds at once
  const int rounds = gpb / per_round;

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
  } else if (warp == 1) {
    // -------------------------------------------------------------------------- MMA issuer
    const uint32_t id = idesc_bf16_f32(128, NT);
    const uint64_t dx0 = smem_desc_sw128(smem + 4 * kWBox);
    const int kg = p.group / 16;                        // MMAs of a group
    bool ok = true;
    int st = 0;
    uint32_t ph = 0, dph = 0;
    for (int i = 0; ok && i < nu; ++i) {
      ok = mbar_wait(&sh->full[st], ph);
      tc_fence_after();
      const uint64_t dx = dx0 + (uint64_t)((uint32_t)(st * stage) >> 4);
      for (int rd = 0; ok && rd < rounds; ++rd) {
        for (int w = 0; ok && w < 4; ++w) {
          ok = rd == 0 ? mbar_wait(&sh->a_full[w], i & 1) : mbar_wait(&sh->d_free[w], dph);
          tc_fence_after();
          const uint64_t dxw = dx + w % ks * (xbytes >> 4);
          if (ok && elect_one()) {
            for (int g = 0; g < per_round; ++g) {
              const uint32_t d = tmem + 256 + 64 * w + NT * g;
              const int k0 = (rd * per_round + g) * kg;
              for (int k = k0; k < k0 + kg; ++k)
                tc_mma_bf16_ts(d, tmem + 64 * w + 8 * k,
                               dxw + (k >> 2) * (NT * 128 >> 4) + 2 * (k & 3), id, k > k0 ? 1u : 0u);
            }
            tc_commit(&sh->d_full[w]);
            if (rd == rounds - 1 && w == 3) tc_commit(&sh->empty[st]);
          }
          __syncwarp();
        }
        if (rd > 0) dph ^= 1;
      }
      if (++st == p.stages) { st = 0; ph ^= 1; }
    }
    if (elect_one()) tc_commit(&sh->drain);
    __syncwarp();
    if (!mbar_wait(&sh->drain, 0)) ok = false;
    if (!ok && lane == 0) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_W4);
  } else if (warp >= 4) {
    // ------------------------------------------- consumers: q to A, and the scaled group sums
    // A warpgroup serves two of the unit's four blocks: the tensor core works on one while the
    // other is unpacked or read back.
    const int wg = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t la = tmem + ((uint32_t)(quarter * 32) << 16) + 128 * wg, ld = la + 256;
    const int ng = p.K / p.group;
    const bool wide = (ng & 3) == 0;
    constexpr int kLd = NT == 16 ? 16 : 32;
    const int wrow = ks == 4 ? 0 : wg * 128;            // this warpgroup's rows in the tile
    float acc[NT];
    bool ok = true;
    int st = 0;
    uint32_t ph = 0, dph = 0;
    W4Groups cur[2], nxt[2];
    auto fetch = [&](int n, int chunk) -> W4Groups {    // groups [4 chunk, 4 chunk + 4)
      W4Groups r{0u, 0u, 0x08080808u};
      if (n >= p.N || 4 * chunk >= ng) return r;
      const int64_t at = (int64_t)n * ng + 4 * chunk;
      if (wide) {
        const uint2 s = __ldg(reinterpret_cast<const uint2*>(p.scales + at));
        r.s01 = s.x;
        r.s23 = s.y;
        if (p.zeros) r.z = __ldg(reinterpret_cast<const uint32_t*>(p.zeros + at));
      } else {
        uint32_t s[4] = {0u, 0u, 0u, 0u}, z[4] = {8u, 8u, 8u, 8u};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * chunk + i < ng) {
            s[i] = __ldg(p.scales + at + i);
            if (p.zeros) z[i] = __ldg(p.zeros + at + i);
          }
        r.s01 = s[0] | s[1] << 16;
        r.s23 = s[2] | s[3] << 16;
        r.z = z[0] | z[1] << 8 | z[2] << 16 | z[3] << 24;
      }
      return r;
    };
    // `cur` serves upc consecutive units of a tile (4 / gpb k blocks), `nxt` the units after them
    const int upc = max(1, 4 / (gpb * ks));
    W4Walk at(p, u0), pre = at;
    int pre_left = nu;                                  // units from `pre` to the end
    auto fetch_pre = [&]() {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int kb = pre.kb * ks + (2 * wg + e) % ks;
        nxt[e] = fetch(pre.rowt * rpt + wrow + row, kb * gpb >> 2);
      }
      do {                                              // to the first unit of the next chunk
        pre.next(p);
        --pre_left;
      } while (pre.kb % upc != 0 && pre_left > 0);
    };
    fetch_pre();
    pdl_wait();
    auto clear = [&]() {
#pragma unroll
      for (int c = 0; c < NT; ++c) acc[c] = 0.f;
    };
    clear();
    for (int i = 0; i < nu; ++i, at.next(p)) {
      if (i == 0 || at.kb % upc == 0) {
        cur[0] = nxt[0];
        cur[1] = nxt[1];
        if (pre_left > 0) fetch_pre();
      }
      if (ok && !mbar_wait(&sh->full[st], ph)) ok = false;
      if (ok) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int w = 2 * wg + e;
          const int g0 = ((at.kb * ks + w % ks) * gpb) & 3;
          const uint8_t* src = smem + st * stage + w * kWBox + row * 64;
          const int sw = (row >> 1) & 3;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 q4 = *reinterpret_cast<const uint4*>(src + ((c ^ sw) << 4));
            const uint32_t qw[4] = {q4.x, q4.y, q4.z, q4.w};
            const uint32_t z = (cur[e].z >> (8 * (g0 + (c * gpb >> 2)))) & 15u;
            const uint32_t zz = 0x43004300u | z | z << 16;
            uint32_t v[16];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int b = 0; b < 4; ++b)
                v[4 * j + b] = sub_pair(((qw[j] >> (4 * b)) & 0x000f000fu) | 0x43004300u, zz);
            tmem_st16_async(la + 64 * e + 16 * c, v);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh->a_full[w]);
            if (e == 1) mbar_arrive(&sh->empty[st]);
          }
        }
        for (int rd = 0; ok && rd < rounds; ++rd) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int w = 2 * wg + e;
            const int g0 = ((at.kb * ks + w % ks) * gpb) & 3;
            if (ok && !mbar_wait(&sh->d_full[w], dph)) ok = false;
            tc_fence_after();
            for (int g = 0; g < per_round; ++g) {
              const int gi = g0 + rd * per_round + g;
              const uint32_t sv = (gi & 2) ? cur[e].s23 : cur[e].s01;
              const float s = __uint_as_float((gi & 1) ? (sv & 0xffff0000u) : (sv << 16));
#pragma unroll
              for (int c = 0; c < NT; c += kLd) {
                float d[kLd];
                if constexpr (kLd == 32) tmem_ld32(ld + 64 * e + NT * g + c, d);
                else tmem_ld16(ld + 64 * e + NT * g + c, d);
#pragma unroll
                for (int b = 0; b < kLd; b += 2)
                  ffma2_acc(acc[c + b], acc[c + b + 1], d[b], d[b + 1], s);
              }
            }
            tc_fence_before();
            __syncwarp();
            if (rd + 1 < rounds && lane == 0) mbar_arrive(&sh->d_free[w]);
          }
          dph ^= 1;
        }
      }
      if (++st == p.stages) { st = 0; ph ^= 1; }

      // ------------------------------------------------ the end of this CTA's part of a tile
      const bool tile_end = at.kb + 1 == p.kbu;
      if (!tile_end && i + 1 < nu) continue;
      const int tile = at.tile;
      const int m0 = at.chunk * NT, mv = min(NT, p.M - m0);
      if constexpr (KS == 4) {                          // add the other warpgroup's sums
        if (wg == 1) {
#pragma unroll
          for (int c = 0; c < NT; ++c) red[c * 128 + row] = acc[c];
        }
        w4_sync();
        if (wg == 0) {
#pragma unroll
          for (int c = 0; c < NT; ++c) acc[c] += red[c * 128 + row];
        }
      }
      const bool mine = ks == 2 || wg == 0;
      const int t0 = u0 + i - at.kb, t1 = t0 + p.kbu;
      auto put = [&](int m, int nn, float v) {
        if (p.bias) v += __uint_as_float((uint32_t)__ldg(p.bias + nn) << 16);
        const int64_t o = (int64_t)(m0 + m) * p.out_stride + nn;
        if (p.out_f32) reinterpret_cast<float*>(p.out)[o] = v;
        else reinterpret_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v);
      };
      if (u0 <= t0 && tile_end) {                       // the whole tile
        const int n = at.rowt * rpt + wrow + row;
        if (mine && n < p.N) {
#pragma unroll
          for (int c = 0; c < NT; ++c)
            if (c < mv) put(c, n, acc[c]);
        }
      } else {
        const int c0 = w4_owner(p.units, gridDim.x, t0), c1 = w4_owner(p.units, gridDim.x, t1 - 1);
        auto slot = [&](int c) {                        // CTA c's part of this tile
          const bool first = w4_first(p.units, gridDim.x, c) >= t0;
          return p.part + ((int64_t)2 * c + (first ? 0 : 1)) * NT * rpt;
        };
        if (mine) {
          float* dst = slot(blockIdx.x) + wrow + row;
#pragma unroll
          for (int c = 0; c < NT; ++c)
            if (c < mv) dst[c * rpt] = acc[c];
        }
        __threadfence();
        w4_sync();
        if (threadIdx.x == 128) sh->last = atomicAdd(p.count + tile, 1) == c1 - c0;
        w4_sync();
        if (sh->last) {
          __threadfence();
          for (int o = threadIdx.x - 128; o < mv * rpt; o += 256) {
            const int rr = o & (rpt - 1), nn = at.rowt * rpt + rr;
            float v = 0.f;
            for (int c = c0; c <= c1; ++c) v += __ldcg(slot(c) + o);
            if (nn < p.N) put(o / rpt, nn, v);
          }
        }
      }
      if constexpr (KS == 4) w4_sync();                 // `red` is free again
      clear();
    }
    if (!ok && lane == 0) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_W4);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

int w4_stages(int nt, int ks) {
  const int stage = 4 * kWBox + ks * nt * 256;
  const int fixed = 1024 + (ks == 4 ? nt * 512 : 0) + (int)sizeof(W4Smem);
  return std::min(kWMaxStages, (kWSmem - fixed) / stage);
}

cudaError_t launch_w4(const CUtensorMap& q, const CUtensorMap& x, W4Params p, int nt, int grid,
                      cudaStream_t s) {
  p.stages = w4_stages(nt, p.ks);
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
    return nt == 16 ? go(w4_kernel<16, 4>) : nt == 32 ? go(w4_kernel<32, 4>) : go(w4_kernel<64, 4>);
  return nt == 16 ? go(w4_kernel<16, 2>) : nt == 32 ? go(w4_kernel<32, 2>) : go(w4_kernel<64, 2>);
}

}  // namespace etree

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
//               (128 + q_p, 128 + q_{p+4}), and subtracting 128 + z is exact (integers made from bit
//               patterns: Kim et al., "Who Says Elephants Can't Run", 2022).  The pairs go to
//               TMEM as A.  x is copied once per call with every eight values in the matching
//               order 0 4 1 5 2 6 3 7.
//   D = A x^T   tcgen05.mma M=128 x N=NT x K=16, A from TMEM, x from shared memory.
//
// A unit of work is four 128 x 128 weight blocks: two row tiles of two k blocks where there are many
// rows (x is then read once for 256 rows), or four k blocks of one row tile (few rows).  One CTA per
// SM takes whole tiles in turn; the tiles left over are shared unit by unit, and a second kernel adds
// their parts in the order of k, so results do not depend on timing.  Inside a CTA one warp issues
// the loads, two the MMAs, one brings scales and zero points, eight unpack and eight add.
//
// Floor of 64 tokens x 151,936 x 5,120 with fp32 output: 447 MB, 69 us at the copy rate.  Measured
// 210 us after a rest, at 1,965 MHz (2.1 TB/s), and 218 us in a loop, which meets the power limit at
// about 1,800 MHz; no pipe is above 40%, so it is the hand-overs between the roles that bound it.
// 16 tokens of the same, bf16 output, 130 us and 32 tokens 137 (floors 64 and 65); 512 tokens x 7,168
// x 5,120 85 us and 4,096 tokens 561 us, 536 TFLOP/s: each 64 tokens unpack the weights anew.
#include <algorithm>

#include "kernels.cuh"

namespace etree {

namespace {
constexpr int kWThreads = 32 * 20;          // TMA, two MMA, one scale, 8 unpacking, 8 summing warps
constexpr int kWBox = 128 * 64;             // [128 rows][64 bytes]
constexpr int kWMaxStages = 5;
constexpr int kWSmem = 226 * 1024;

struct W4Smem {
  uint64_t full[kWMaxStages], empty[kWMaxStages];
  uint64_t a_full[4], a_free[4], d_full[4], d_free[4], drain[2];
  uint32_t tmem;
};

// NT tokens a tile, KS k blocks a unit (of 4 / KS row tiles), GPB groups a k block of 128.
template <int NT, int KS, int GPB>
struct W4Shape {
  static constexpr int kRows = 512 / KS;                // rows of a tile
  static constexpr int kX = NT * 256;                   // one k block of x: two boxes [NT][64]
  // scales and zero points of a unit: a warpgroup's 2 GPB groups of its 128 rows, as 32-bit words
  // [word][256]
  static constexpr int kSWords = GPB, kZWords = (2 * GPB + 3) / 4;
  static constexpr int kTx = 4 * kWBox + KS * kX;       // bytes that TMA brings
  static constexpr int kStage = kTx + (kSWords + kZWords) * 1024;
  static constexpr int kRed = KS == 4 ? NT * 512 : 0;   // one warpgroup's sums
  static constexpr int kFixed = 1024 + kRed + (int)sizeof(W4Smem);
  static constexpr int kFit = (kWSmem - kFixed) / kStage;
  static constexpr int kStages = kFit < kWMaxStages ? kFit : kWMaxStages;
  static constexpr int kPerRound = GPB < 64 / NT ? GPB : 64 / NT;   // groups that D holds at once
  static constexpr int kRounds = GPB / kPerRound;
  static_assert(kStages >= 2, "two stages at least");
};

__device__ __forceinline__ void w4_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The units of the shared tiles are dealt to the first share_grid CTAs, share_base each and one more
// to the first share_rem: CTA c's first unit, and the CTA that holds unit u.
__device__ __forceinline__ int w4_first(const W4Params& p, int c) {
  return c * p.share_base + min(c, p.share_rem);
}
__device__ __forceinline__ int w4_owner(const W4Params& p, int u) {
  const int longer = p.share_rem * (p.share_base + 1);
  return u < longer ? u / (p.share_base + 1) : p.share_rem + (u - longer) / p.share_base;
}

// A CTA's segments in order: its share of the shared tiles' units, at most the end of one tile and
// the start of the next, then `whole` tiles of its own.  Every role walks the same list.
struct W4Segment {
  int rowt, chunk, tile, kb, n, unit0;                  // n units from kb; unit0: the shared unit
  bool part;
};
__device__ __forceinline__ bool w4_segment(const W4Params& p, int s, W4Segment& at) {
  if ((int)blockIdx.x < p.share_grid) {
    int u = w4_first(p, blockIdx.x);
    const int end = w4_first(p, blockIdx.x + 1);
    int t = u / p.kbu;
    const int split = min(end, (t + 1) * p.kbu);
    if (s == 1 && split < end) {
      u = split;
      ++t;
    }
    if (s == 0 || (s == 1 && split < end)) {
      at.kb = u - t * p.kbu;
      at.n = (u < split ? split : end) - u;
      at.tile = p.tiles - p.share_units / p.kbu + t;
      at.unit0 = u;
      at.part = at.n < p.kbu;
      at.rowt = at.tile / p.chunks;
      at.chunk = at.tile - at.rowt * p.chunks;
      return true;
    }
    s -= split < end ? 2 : 1;
  }
  if (s >= p.whole) return false;
  at.kb = 0;
  at.n = p.kbu;
  at.tile = blockIdx.x * p.whole + s;
  at.unit0 = 0;
  at.part = false;
  at.rowt = at.tile / p.chunks;
  at.chunk = at.tile - at.rowt * p.chunks;
  return true;
}

// The units of this CTA.
__device__ __forceinline__ int units_of(const W4Params& p) {
  const int own = p.whole * p.kbu;
  if ((int)blockIdx.x >= p.share_grid) return own;
  return own + w4_first(p, blockIdx.x + 1) -
         w4_first(p, blockIdx.x);
}

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

// CNT consecutive elements of a row of ng scales (or zero points) from index g, packed into 32-bit
// words.  The addresses stay inside the row, so that the loads need no condition; the caller
// drops what lies behind the row's end.
template <int CNT, typename T>
struct W4Row {
  static constexpr int kBytes = CNT * (int)sizeof(T), kWords = (kBytes + 3) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void fetch(const T* row, int g, int ng, bool wide) {
    if (wide) {                                         // ng is a multiple of CNT
      const T* at = row + min(g, ng - CNT);
      if constexpr (kBytes == 2) w[0] = __ldg(reinterpret_cast<const uint16_t*>(at));
      else if constexpr (kBytes == 4) w[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
      else if constexpr (kBytes == 8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
        w[0] = v.x;
        w[1] = v.y;
      } else {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(at));
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = 0u;
#pragma unroll
      for (int i = 0; i < CNT; ++i)
        w[i * sizeof(T) / 4] |= (uint32_t)__ldg(row + min(g + i, ng - 1))
                                << (8 * sizeof(T) * (i % (4 / sizeof(T))));
    }
  }
};
}  // namespace

// x [M][K] (rows x_stride apart) -> xp [rows][K], every eight values as 0 4 1 5 2 6 3 7 and rows
// behind M zero.
__global__ void __launch_bounds__(256) w4_prepare_kernel(W4Params p, int rows) {
  pdl_trigger();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int c8 = p.K / 8;
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

// One warp brings the scales and zero points, a few bytes of each row: eight rows a lane.  With two
// row tiles a unit's groups lie behind the last one's, and eight groups are loaded at once, for 4 / GPB
// units.  The next units' loads are in flight while a stage is awaited.
template <int NT, int KS, int GPB>
__device__ __noinline__ void w4_scales(const W4Params& p, uint8_t* smem, W4Smem* sh) {
  using Sh = W4Shape<NT, KS, GPB>;
  constexpr int kU = KS == 2 ? 4 / GPB : 1, kGroups = 2 * GPB * kU;
  const int lane = threadIdx.x & 31, ng = p.K / p.group;
  const bool wide = ng % kGroups == 0;
  W4Row<kGroups, uint16_t> sc[8];
  W4Row<kGroups, uint8_t> zp[8];
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int j = 0; j < zp[r].kWords; ++j) zp[r].w[j] = 0x08080808u;
  int64_t base = 0;                                     // the tile's first row, in elements
  int off[8];                                           // this lane's rows behind it
  auto rows_of = [&](int rowt) {                        // once a segment
    base = (int64_t)rowt * Sh::kRows * ng;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int i = r * 32 + lane;                      // row i of the unit's 2 x 128
      off[r] = min(KS == 4 ? i & 127 : i, p.N - 1 - rowt * Sh::kRows) * ng;
    }
  };
  auto fetch = [&](int kb) {
    const uint16_t* s = p.scales + base;
    const uint8_t* z = p.zeros + base;
#pragma unroll
    for (int half = 0; half < 2; ++half) {              // rows of warpgroup 0, then of 1
      const int g = ((kb & ~(kU - 1)) * KS + (KS == 4 ? 2 * half : 0)) * GPB;
#pragma unroll
      for (int r = 4 * half; r < 4 * half + 4; ++r) sc[r].fetch(s + off[r], g, ng, wide);
      if (p.zeros) {
#pragma unroll
        for (int r = 4 * half; r < 4 * half + 4; ++r) zp[r].fetch(z + off[r], g, ng, wide);
      }
    }
  };
  // word i of an array in registers
  auto pick = [](const uint32_t* w, int n, int i) {
    uint32_t v = w[0];
#pragma unroll
    for (int j = 1; j < n; ++j) v = i == j ? w[j] : v;
    return v;
  };
  W4Segment at;
  int seg = 0;
  bool more = w4_segment(p, seg, at);
  int kb = at.kb, left = at.n, st = 0;
  uint32_t ph = 1;                                      // the first round of stages is free
  bool ok = true;
  if (more) {
    rows_of(at.rowt);
    fetch(kb);
  }
  while (more) {
    const int sub = kb & (kU - 1);                      // of the units loaded
    if (!mbar_wait(&sh->empty[st], ph)) { ok = false; break; }
    uint32_t* dst = reinterpret_cast<uint32_t*>(smem + st * Sh::kStage + Sh::kTx) + lane;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
#pragma unroll
      for (int j = 0; j < Sh::kSWords; ++j)
        dst[j * 256 + r * 32] = kU == 1 ? sc[r].w[j] : pick(sc[r].w, sc[r].kWords, sub * GPB + j);
#pragma unroll
      for (int j = 0; j < Sh::kZWords; ++j)
        dst[(Sh::kSWords + j) * 256 + r * 32] =
            kU == 1    ? zp[r].w[j]
            : GPB == 1 ? pick(zp[r].w, zp[r].kWords, sub >> 1) >> (16 * (sub & 1))
                       : pick(zp[r].w, zp[r].kWords, sub);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->full[st]);
    if (++st == Sh::kStages) { st = 0; ph ^= 1; }
    ++kb;
    bool load = (kb & (kU - 1)) == 0;
    if (--left == 0) {                                  // the next unit is another segment's
      more = w4_segment(p, ++seg, at);
      kb = at.kb;
      left = at.n;
      if (more) rows_of(at.rowt);
      load = true;
    }
    if (more && load) fetch(kb);
  }
  if (!ok && lane == 0) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_PRODUCT);
}

// The two roles with many live registers are functions of their own, so that each is allocated
// apart (inlined side by side they spilled in the inner loops).
//
// Unpacking: warpgroup wg turns blocks 2 wg and 2 wg + 1 of every unit into A in TMEM.
template <int NT, int KS, int GPB>
__device__ __noinline__ void w4_unpack(const W4Params& p, uint8_t* smem, W4Smem* sh, uint32_t tmem,
                                       int nu) {
  using Sh = W4Shape<NT, KS, GPB>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wg = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
  const uint32_t la = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 128 * wg;
  const int sw = (row >> 1) & 3;
  uint32_t magic = 0x43004300u;
  asm volatile("" : "+r"(magic));                       // stays in a register
  int st = 0;
  uint32_t ph = 0, done = 0;                            // units done, modulo 2 (as parity)
  const uint8_t* src0 = smem + 2 * wg * kWBox + row * 64;
  const uint8_t* src = src0;
  const uint8_t* zp0 = smem + Sh::kTx + Sh::kSWords * 1024 + (wg * 128 + row) * 4;
  bool ok = true;
  for (int i = 0; i < nu; ++i) {
    if (!mbar_wait(&sh->full[st], ph)) { ok = false; break; }
    uint32_t zw[Sh::kZWords];
#pragma unroll
    for (int j = 0; j < Sh::kZWords; ++j)
      zw[j] = *reinterpret_cast<const uint32_t*>(zp0 + st * Sh::kStage + j * 1024);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t qw[16];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 q = *reinterpret_cast<const uint4*>(src + e * kWBox + ((c ^ sw) << 4));
        qw[4 * c] = q.x;
        qw[4 * c + 1] = q.y;
        qw[4 * c + 2] = q.z;
        qw[4 * c + 3] = q.w;
      }
      if (i > 0 && !mbar_wait(&sh->a_free[2 * wg + e], done ^ 1)) { ok = false; break; }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int zi = e * GPB + c * GPB / 4;           // this group's byte
        const uint32_t z = (zw[zi / 4] >> (8 * (zi % 4))) & 15u;
        const uint32_t zz = z * 0x00010001u | magic;
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
      if (lane == 0) mbar_arrive(&sh->a_full[2 * wg + e]);
    }
    if (!ok) break;
    if (lane == 0) mbar_arrive(&sh->empty[st]);
    done ^= 1;
    src += Sh::kStage;
    if (++st == Sh::kStages) {
      st = 0;
      ph ^= 1;
      src = src0;
    }
  }
  if (!ok && lane == 0) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_PRODUCT);
}

// Summing: warpgroup wg adds the scaled group sums of blocks 2 wg and 2 wg + 1, and writes the tile.
template <int NT, int KS, int GPB>
__device__ __noinline__ void w4_sum(const W4Params& p, const uint8_t* smem, float* red, W4Smem* sh,
                                    uint32_t tmem) {
  using Sh = W4Shape<NT, KS, GPB>;
  constexpr int kRows = Sh::kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wg = (warp - 12) >> 2, row = (warp & 3) * 32 + lane;
  const int wrow = (KS == 4 ? 0 : wg * 128) + row;
  const uint32_t ld = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256 + 128 * wg;
  const int ng = p.K / p.group;
  const uint8_t* sp0 = smem + Sh::kTx + (wg * 128 + row) * 4;
  pdl_wait();
  uint64_t acc[NT / 2];                                 // tokens 2 c and 2 c + 1
  uint32_t use = 0, ph = 0;
  int st = 0;
  bool ok = true;
  W4Segment at;
  for (int seg = 0; w4_segment(p, seg, at); ++seg) {
#pragma unroll
    for (int c = 0; c < NT / 2; ++c) acc[c] = 0ull;
    for (int i = 0; i < at.n; ++i) {
      const int g0 = ((at.kb + i) * KS + (KS == 4 ? 2 * wg : 0)) * GPB;
      if (ok && !mbar_wait(&sh->full[st], ph)) ok = false;
      uint32_t sc[Sh::kSWords];
#pragma unroll
      for (int j = 0; j < Sh::kSWords; ++j)
        sc[j] = *reinterpret_cast<const uint32_t*>(sp0 + st * Sh::kStage + j * 1024);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->empty[st]);
      if (++st == Sh::kStages) { st = 0; ph ^= 1; }
#pragma unroll
      for (int rd = 0; rd < Sh::kRounds; ++rd) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (ok && !mbar_wait(&sh->d_full[2 * wg + e], (use + rd) & 1)) ok = false;
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < Sh::kPerRound; ++g) {
            const int si = e * GPB + rd * Sh::kPerRound + g;
            if (g0 + si >= ng) continue;                // behind the row's end
            const uint32_t sv = sc[si / 2];
            const float s = __uint_as_float((si & 1) ? (sv & 0xffff0000u) : (sv << 16));
#pragma unroll
            for (int c = 0; c < NT; c += 16) {
              float d[16];
              tmem_ld16(ld + 64 * e + NT * g + c, d);
#pragma unroll
              for (int b = 0; b < 16; b += 2) ffma2_acc(acc[(c + b) / 2], d[b], d[b + 1], s);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->d_free[2 * wg + e]);
        }
      }
      use += Sh::kRounds;
    }

    // ---------------------------------------------------------------- the segment's end
    int again = seg;                                    // the segment anew: it was not kept in
    asm volatile("" : "+r"(again));                     // registers beside the sums
    w4_segment(p, again, at);
    const int rowt = at.rowt;
    const int m0 = at.chunk * NT, mv = min(NT, p.M - m0);
    if constexpr (KS == 4) {                            // add the other warpgroup's sums
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
    const bool mine = KS == 2 || wg == 0;
    auto bias_of = [&](int n) {
      return p.bias ? __uint_as_float((uint32_t)__ldg(p.bias + n) << 16) : 0.f;
    };
    if (!at.part) {
      const int n = rowt * kRows + wrow;
      if (mine && n < p.N) {
        const float b = bias_of(n);
        // one running pointer: NT row offsets at once would push the sums out of the registers
        const int64_t step = p.out_stride * (p.out_f32 ? 4 : 2);
        char* dst = reinterpret_cast<char*>(p.out) +
                    ((int64_t)m0 * p.out_stride + n) * (p.out_f32 ? 4 : 2);
        if (p.out_f32) {
#pragma unroll
          for (int c = 0; c < NT; ++c) {
            if (c < mv) *reinterpret_cast<float*>(dst) = half_of(acc[c / 2], c & 1) + b;
            dst += step;
            asm volatile("" : "+l"(dst));
          }
        } else {
#pragma unroll
          for (int c = 0; c < NT; ++c) {
            if (c < mv)
              *reinterpret_cast<__nv_bfloat16*>(dst) =
                  __float2bfloat16_rn(half_of(acc[c / 2], c & 1) + b);
            dst += step;
            asm volatile("" : "+l"(dst));
          }
        }
      }
    } else {
      const int t0 = at.unit0 - at.kb;                  // the tile's first shared unit
      const int64_t part_size = (int64_t)NT * kRows;    // a CTA has room for two parts of tiles
      if (mine) {
        const int mine0 = w4_first(p, blockIdx.x);
        float* dst = p.part + (2 * blockIdx.x + (mine0 >= t0 ? 0 : 1)) * part_size + wrow;
#pragma unroll
        for (int c = 0; c < NT; ++c)
          if (c < mv) dst[c * kRows] = half_of(acc[c / 2], c & 1);
      }
    }
    if constexpr (KS == 4) w4_sync();                   // `red` is free again
  }
  if (!ok && lane == 0) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_PRODUCT);
}

template <int NT, int KS, int GPB>
__global__ void __launch_bounds__(kWThreads, 1)
w4_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_x,
          const __grid_constant__ W4Params p) {
  using Sh = W4Shape<NT, KS, GPB>;
  constexpr int kStages = Sh::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(smem + kStages * Sh::kStage);      // [NT][128], KS = 4
  W4Smem* sh = reinterpret_cast<W4Smem*>(reinterpret_cast<uint8_t*>(red) + Sh::kRed);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh->full[i], 2);                       // TMA, the scale warp
      mbar_init(&sh->empty[i], 18);                     // 8 unpacking and 8 summing warps, 2 MMA commits
    }
    for (int w = 0; w < 4; ++w) {
      mbar_init(&sh->a_full[w], 4);
      mbar_init(&sh->a_free[w], 1);
      mbar_init(&sh->d_full[w], 1);
      mbar_init(&sh->d_free[w], 4);
    }
    mbar_init(&sh->drain[0], 1);
    mbar_init(&sh->drain[1], 1);
    fence_barrier_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_x);
  }
  pdl_trigger();                                        // the join waits for this grid's end
  if (warp == 1) {
    tmem_alloc(&sh->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;                       // block w: A at 64 w, D at 256 + 64 w

  if (warp == 0) {
    // ------------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      auto load_q = [&](int rowt, int kb, int st) {
        uint8_t* dst = smem + st * Sh::kStage;
        mbar_arrive_expect_tx(&sh->full[st], Sh::kTx);
#pragma unroll
        for (int w = 0; w < 4; ++w)
          tma_load_2d(dst + w * kWBox, &tm_q, &sh->full[st], (kb * KS + w % KS) * 64,
                      rowt * Sh::kRows + w / KS * 128);
      };
      auto load_x = [&](int chunk, int kb, int st) {
        uint8_t* dst = smem + st * Sh::kStage + 4 * kWBox;
#pragma unroll
        for (int w = 0; w < 2 * KS; ++w)
          tma_load_2d(dst + w * (NT * 128), &tm_x, &sh->full[st], kb * KS * 128 + w * 64, chunk * NT);
      };
      // the first weights do not depend on the kernel that reorders x (an ordinary launch, before
      // which everything earlier on the stream has completed)
      int ahead = 0;
      W4Segment at;
      for (int seg = 0; ahead < kStages && w4_segment(p, seg, at); ++seg)
        for (int i = 0; i < at.n && ahead < kStages; ++i) load_q(at.rowt, at.kb + i, ahead++);
      pdl_wait();
      bool ok = true;
      int issued = 0, st = 0;
      uint32_t ph = 0;
      for (int seg = 0; ok && w4_segment(p, seg, at); ++seg)
        for (int i = 0; i < at.n; ++i) {
          if (issued >= ahead) {
            if (!mbar_wait(&sh->empty[st], ph ^ 1)) { ok = false; break; }
            load_q(at.rowt, at.kb + i, st);
          }
          load_x(at.chunk, at.kb + i, st);
          ++issued;
          if (++st == kStages) { st = 0; ph ^= 1; }
        }
      // every copy has landed before the CTA may exit (bounded); weights without their x as well
      // are none: the loop above reaches every unit that was loaded ahead
      for (int i = max(0, issued - kStages); i < issued; ++i)
        ok = mbar_wait(&sh->full[i % kStages], (i / kStages) & 1) && ok;
      if (!ok) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_PRODUCT);
    }
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------- MMA issuers, two of the four blocks each
    constexpr uint32_t id = idesc_bf16_f32(128, NT);
    constexpr int kg = 8 / GPB;                         // MMAs of a group
    const uint64_t dx0 = smem_desc_sw128(smem + 4 * kWBox);
    bool ok = true, any = false;
    int st = 0;
    uint32_t ph = 0, use = 0, unit = 0;                 // `use` counts the fillings of D
    const int nu = units_of(p);
      for (int i = 0; ok && i < nu; ++i) {
        ok = mbar_wait(&sh->full[st], ph);
        const uint64_t dx = dx0 + (uint64_t)((uint32_t)(st * Sh::kStage) >> 4);
#pragma unroll
        for (int rd = 0; rd < Sh::kRounds; ++rd) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int w = 2 * (warp - 1) + e;
            if (any || rd > 0) ok = ok && mbar_wait(&sh->d_free[w], (use + rd - 1) & 1);
            if (rd == 0) ok = ok && mbar_wait(&sh->a_full[w], unit & 1);
            tc_fence_after();
            const uint64_t dxw = dx + w % KS * (Sh::kX >> 4);
            const uint32_t aw = tmem + 64 * w, dw = aw + 256;
            if (ok && elect_one()) {
#pragma unroll
              for (int j = 0; j < Sh::kPerRound * kg; ++j) {
                const int k = rd * Sh::kPerRound * kg + j;
                tc_mma_bf16_ts(dw + j / kg * NT, aw + 8 * k,
                               dxw + (k >> 2) * (NT * 128 >> 4) + 2 * (k & 3), id,
                               j % kg > 0 ? 1u : 0u);
              }
              tc_commit(&sh->d_full[w]);
              if (rd == Sh::kRounds - 1) {
                tc_commit(&sh->a_free[w]);
                if (e == 1) tc_commit(&sh->empty[st]);
              }
            }
            __syncwarp();
          }
        }
        any = true;
        use += Sh::kRounds;
        ++unit;
        if (++st == kStages) { st = 0; ph ^= 1; }
      }
    if (elect_one()) tc_commit(&sh->drain[warp - 1]);
    __syncwarp();
    if (!mbar_wait(&sh->drain[warp - 1], 0)) ok = false;
    if (!ok && lane == 0) report(p.ws, ETREE_ETIMEOUT, DET_WAIT_PRODUCT);
  } else if (warp == 3) {
    w4_scales<NT, KS, GPB>(p, smem, sh);
  } else if (warp < 12) {
    w4_unpack<NT, KS, GPB>(p, smem, sh, tmem, units_of(p));
  } else {
    w4_sum<NT, KS, GPB>(p, smem, red, sh, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Row tiles whose units lie on several CTAs: their parts are added in the order of k, four rows of
// one token a thread.  One block row per shared tile.
template <int NT, int KS>
__global__ void __launch_bounds__(256) w4_join_kernel(const __grid_constant__ W4Params p) {
  constexpr int kRows = 512 / KS, kQuads = kRows / 4;
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.y * p.kbu;                    // the tile's first shared unit
  const int c0 = w4_owner(p, t0), c1 = w4_owner(p, t0 + p.kbu - 1);
  if (c0 == c1) return;                                 // one CTA's, already written
  const int tile = p.tiles - p.share_units / p.kbu + blockIdx.y;
  const int rowt = tile / p.chunks, m0 = (tile - rowt * p.chunks) * NT;
  const int o = blockIdx.x * 256 + threadIdx.x, m = o / kQuads, rr = o % kQuads * 4;
  const int n = rowt * kRows + rr;
  if (m0 + m >= p.M || n >= p.N) return;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const bool first = w4_first(p, c) >= t0;
    const float4 x = __ldcg(reinterpret_cast<const float4*>(
        p.part + (2 * c + (first ? 0 : 1)) * ((int64_t)NT * kRows) + m * kRows + rr));
    v.x += x.x;
    v.y += x.y;
    v.z += x.z;
    v.w += x.w;
  }
  const float y[4] = {v.x, v.y, v.z, v.w};
  const int64_t at = (int64_t)(m0 + m) * p.out_stride + n;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < p.N) {
      const float r = y[i] + (p.bias ? __uint_as_float((uint32_t)__ldg(p.bias + n + i) << 16) : 0.f);
      if (p.out_f32) reinterpret_cast<float*>(p.out)[at + i] = r;
      else reinterpret_cast<__nv_bfloat16*>(p.out)[at + i] = __float2bfloat16_rn(r);
    }
}

// Few tokens or small products: one launch, no tensor memory, no reordered x.  A warp takes MT x 16 rows
// at every eighth k block and multiplies with mma.sync m16n8k16 (weights as A, NTL x 8 tokens as
// B); the order of k inside a block is free as long as A and B agree, so a lane loads its rows'
// bytes and its token's values in runs, in words of eight weights whose k lie in one group:
//   word w of lane t (of the four that share a row) starts at k = first(w, t),
//   GPB = 1: 32 t + 8 w;   2: 64 (w / 2) + 16 t + 8 (w % 2);   4: 32 w + 8 t.
// Sums of a group leave the tensor core as they do above and are scaled in fp32; the eight warps'
// sums meet in shared memory in the order of the warps.
constexpr int kSmallWarps = 8;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int MT, int GPB>
struct W4SmallBlock {                                   // a lane's part of MT x 16 rows x 128 k
  uint32_t q[MT][2][4];                                 // [tile][row g or g + 8][word]
  uint16_t s[MT][2][GPB];
  uint8_t z[MT][2][GPB];
};

template <int MT, int NTL, int GPB>
__global__ void __launch_bounds__(32 * kSmallWarps) w4_small_kernel(const __grid_constant__ W4Params p) {
  constexpr int kRows = 16 * MT, kPart = NTL < 4 ? NTL : 4, kTok = 8 * kPart;
  constexpr bool kAhead = NTL <= 2;
  __shared__ float sums[kSmallWarps][kTok][kRows + 1];  // kPart of the NTL token tiles at once
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kRows, nkb = (p.K + 127) / 128, ng = p.K / p.group;
  uint32_t magic = 0x43004300u;
  asm volatile("" : "+r"(magic));                       // stays in a register
  auto first = [&](int w) {
    return GPB == 1 ? 32 * t + 8 * w : GPB == 2 ? 64 * (w / 2) + 16 * t + 8 * (w % 2) : 32 * w + 8 * t;
  };
  const uint8_t* qrow[MT][2];
  const uint16_t* srow[MT][2];
  const uint8_t* zrow[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = min(n0 + 16 * i + 8 * h + g, p.N - 1);     // rows behind the end: any row
      qrow[i][h] = p.wq + n * (p.K / 2);
      srow[i][h] = p.scales + n * ng;
      zrow[i][h] = p.zeros + n * ng;
    }
  auto load = [&](W4SmallBlock<MT, GPB>& blk, int kb) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        constexpr int kRun = 4 / GPB;                   // words that lie together
#pragma unroll
        for (int w = 0; w < 4; w += kRun) {
          const int k = kb * 128 + first(w);
          const uint8_t* at = qrow[i][h] + k / 2;
          uint32_t* dst = &blk.q[i][h][w];
          if (k < p.K) {
            if constexpr (GPB == 1) {
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(at));
              dst[0] = v.x;
              dst[1] = v.y;
              dst[2] = v.z;
              dst[3] = v.w;
            } else if constexpr (GPB == 2) {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
              dst[0] = v.x;
              dst[1] = v.y;
            } else {
              dst[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
            }
          } else {
#pragma unroll
            for (int j = 0; j < kRun; ++j) dst[j] = 0u;
          }
        }
#pragma unroll
        for (int j = 0; j < GPB; ++j) {
          const int at = min(kb * GPB + j, ng - 1);
          blk.s[i][h][j] = __ldg(srow[i][h] + at);
          blk.z[i][h][j] = p.zeros ? __ldg(zrow[i][h] + at) : 8;
        }
      }
  };
  float acc[MT][NTL][4] = {};
  const uint16_t* xrow = p.x + g * p.x_stride;          // token g, and every eighth after it
  auto token = [&](int j, int k) {
    return 8 * j + g < p.M && k < p.K
               ? __ldg(reinterpret_cast<const uint4*>(xrow + 8 * j * p.x_stride + k))
               : make_uint4(0u, 0u, 0u, 0u);
  };
  auto multiply = [&](const W4SmallBlock<MT, GPB>& blk, int kb) {
    uint4 xs[kAhead ? 4 : 1][NTL];                      // a block's tokens at once, if registers allow
    if constexpr (kAhead) {
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int j = 0; j < NTL; ++j) xs[w][j] = token(j, kb * 128 + first(w));
    }
#pragma unroll
    for (int gi = 0; gi < GPB; ++gi) {
      float d[MT][NTL][4] = {};
      uint32_t zz[MT][2];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) zz[i][h] = (blk.z[i][h][gi] & 15u) * 0x00010001u | magic;
#pragma unroll
      for (int w = gi * 4 / GPB; w < (gi + 1) * 4 / GPB; ++w) {
        uint4(&x)[NTL] = xs[kAhead ? w : 0];
        if constexpr (!kAhead) {
#pragma unroll
          for (int j = 0; j < NTL; ++j) x[j] = token(j, kb * 128 + first(w));
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {          // pairs (2 half, 2 half + 4), (.. + 1, .. + 5)
          uint32_t a[MT][4];
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t q = blk.q[i][h][w] >> (8 * half);
              a[i][h] = sub_pair(nibble_pair(q, magic), zz[i][h]);
              a[i][2 + h] = sub_pair(nibble_pair(blk.q[i][h][w] >> (8 * half + 4), magic), zz[i][h]);
            }
#pragma unroll
          for (int j = 0; j < NTL; ++j) {
            const uint32_t lo = half ? x[j].y : x[j].x, hi = half ? x[j].w : x[j].z;
            const uint32_t b0 = __byte_perm(lo, hi, 0x5410), b1 = __byte_perm(lo, hi, 0x7632);
#pragma unroll
            for (int i = 0; i < MT; ++i) mma_bf16(d[i][j], a[i], b0, b1);
          }
        }
      }
      if (kb * GPB + gi < ng) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const float s0 = __uint_as_float((uint32_t)blk.s[i][0][gi] << 16);
          const float s1 = __uint_as_float((uint32_t)blk.s[i][1][gi] << 16);
#pragma unroll
          for (int j = 0; j < NTL; ++j) {
            acc[i][j][0] += s0 * d[i][j][0];
            acc[i][j][1] += s0 * d[i][j][1];
            acc[i][j][2] += s1 * d[i][j][2];
            acc[i][j][3] += s1 * d[i][j][3];
          }
        }
      }
    }
  };
  W4SmallBlock<MT, GPB> even, odd;
  pdl_wait();                                           // the weights too may be fresh
  pdl_trigger();
  int kb = warp;
  if (kb < nkb) load(even, kb);
  while (kb < nkb) {
    if (kb + kSmallWarps < nkb) load(odd, kb + kSmallWarps);
    multiply(even, kb);
    kb += kSmallWarps;
    if (kb >= nkb) break;
    if (kb + kSmallWarps < nkb) load(even, kb + kSmallWarps);
    multiply(odd, kb);
    kb += kSmallWarps;
  }
#pragma unroll
  for (int j0 = 0; j0 < NTL; j0 += kPart) {
    if (j0 > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < kPart; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sums[warp][8 * j + 2 * t + (c & 1)][16 * i + g + 8 * (c >> 1)] = acc[i][j0 + j][c];
    __syncthreads();
    for (int o = threadIdx.x; o < kRows * kTok; o += 32 * kSmallWarps) {
      const int r = o % kRows, m = 8 * j0 + o / kRows, n = n0 + r;
      if (n >= p.N || m >= p.M) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kSmallWarps; ++w) v += sums[w][o / kRows][r];
      if (p.bias) v += __uint_as_float((uint32_t)__ldg(p.bias + n) << 16);
      const int64_t at = m * p.out_stride + n;
      if (p.out_f32) reinterpret_cast<float*>(p.out)[at] = v;
      else reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
    }
  }
}

template <int MT, int NTL>
static cudaError_t go_w4_small(const W4Params& p, cudaStream_t s) {
  const dim3 grid((p.N + 16 * MT - 1) / (16 * MT)), block(32 * kSmallWarps);
  if (p.group == 128) return launch_pdl(w4_small_kernel<MT, NTL, 1>, grid, block, 0, s, p);
  if (p.group == 64) return launch_pdl(w4_small_kernel<MT, NTL, 2>, grid, block, 0, s, p);
  return launch_pdl(w4_small_kernel<MT, NTL, 4>, grid, block, 0, s, p);
}

cudaError_t launch_w4_small(const W4Params& p, int mt, cudaStream_t s) {
  if (p.M <= 8) return mt == 1 ? go_w4_small<1, 1>(p, s) : go_w4_small<2, 1>(p, s);
  if (p.M <= 16) return mt == 1 ? go_w4_small<1, 2>(p, s) : go_w4_small<2, 2>(p, s);
  if (p.M <= 32) return mt == 1 ? go_w4_small<1, 4>(p, s) : go_w4_small<2, 4>(p, s);
  return mt == 1 ? go_w4_small<1, 8>(p, s) : go_w4_small<2, 8>(p, s);
}

template <int NT, int KS, int GPB>
static cudaError_t go_w4(const CUtensorMap& q, const CUtensorMap& x, const W4Params& p, int grid,
                         cudaStream_t s) {
  const cudaError_t e = raise_smem_once(w4_kernel<NT, KS, GPB>, kWSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(w4_kernel<NT, KS, GPB>, dim3(grid), dim3(kWThreads), (size_t)kWSmem, s, q, x, p);
}

template <int NT, int KS>
static cudaError_t go_w4(const CUtensorMap& q, const CUtensorMap& x, const W4Params& p, int grid,
                         cudaStream_t s) {
  cudaError_t e = p.group == 128  ? go_w4<NT, KS, 1>(q, x, p, grid, s)
                  : p.group == 64 ? go_w4<NT, KS, 2>(q, x, p, grid, s)
                                  : go_w4<NT, KS, 4>(q, x, p, grid, s);
  if (e != cudaSuccess || p.share_units == 0) return e;
  return launch_pdl(w4_join_kernel<NT, KS>, dim3(NT * (512 / KS) / 1024, p.share_units / p.kbu),
                    dim3(256), 0, s, p);
}

cudaError_t launch_w4(const CUtensorMap& q, const CUtensorMap& x, const W4Params& p, int nt, int ks,
                      int grid, cudaStream_t s) {
  const int rows = p.chunks * nt;
  const int64_t items = (int64_t)rows * (p.K / 8);
  w4_prepare_kernel<<<(unsigned)((items + 255) / 256), 256, 0, s>>>(p, rows);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (ks == 4) return nt == 16 ? go_w4<16, 4>(q, x, p, grid, s) : go_w4<32, 4>(q, x, p, grid, s);
  return nt == 16   ? go_w4<16, 2>(q, x, p, grid, s)
         : nt == 32 ? go_w4<32, 2>(q, x, p, grid, s)
                    : go_w4<64, 2>(q, x, p, grid, s);
}

}  // namespace etree

// Products with many rows: the matrix units bound them.
//
// Four waves, two by two, each with W x W tiles of 32 x 32 results in registers
// (W = 4: a workgroup has 256 x 256 results and a compute unit for itself; W = 2:
// 128 x 128, two workgroups a compute unit).  Every operand byte of a stage -- two
// steps of 64 columns of two E2M1 operands, one step where one has 8 bits -- goes
// from memory to LDS once for the workgroup and from LDS to registers once for each
// wave that multiplies it; W = 4 reads 8 operands of 32 x 64 for 16 matrix instructions.
//
// The copies into LDS are asynchronous and take no registers.  kMxRing stages of them
// are in flight in as many slots of LDS:
//
//   stage s:  start multiplying stage s, whose operands are in registers
//             wait until the copies of stage s + 1 have landed (all waves: barrier)
//             between the other products, one by one: read stage s + 1 from LDS into
//               the other set of registers, and start the copies of stage s + kMxRing
//               into the slot of stage s, which all waves had read before the barrier
//
// so the matrix units have work at the barrier and beside the reads, and a copy has
// kMxRing - 1 stages to arrive (8 slots of W = 2 in place of 4 gained nothing).  Issued
// in one go, the copies and reads of a stage held the products up for as long as
// memory took to accept them (8192^3 E4M3: 543 us, the matrix units busy for 49% of
// it).  Layout in LDS is that in memory, the instruction's order: a wave's reads are
// runs of 1 KiB and meet no bank twice.  Scales go the same way, a dword a lane and
// chunk, a chunk ahead of their codes.
//
// What bounds large ones is power, then what the matrix units wait for: counters give
// a clock of 1.6 to 1.75 GHz in place of 2.4 and matrix units that are busy for 64%
// (8192^3 E2M1), 78% (E4M3), 68% (to fp32 through bf16), 76% (4096 x 4096 x 65536 E2M1),
// 83% (4096 x 4096 x 16384 E5M2 x E4M3) of the cycles; 4096 x 11008 over 4096
// columns 47% at 1.89 GHz: the beginning and end of sixteen chunks weigh more, and the last
// of three rounds is not full.  With the products
// alone left in a copy of the kernel a stage of E2M1 takes 0.70 us of 0.96.  8192^3 once
// the power control has settled: E2M1 231 .. 247 us, 4.5 PFLOP/s; E4M3 375 .. 399, 2.8;
// to fp32 through bf16 890 .. 907.  The first 8 ms of a load: 274, 440, 990.
#pragma once

#include <type_traits>

#include "nc_mx_mul.h"

namespace nc {

constexpr int kMxRing = 4;         // stages in flight, and slots

// A wave's address, the same in every lane, which the compiler does not always see.
__device__ __forceinline__ const uint8_t* mx_uniform(const uint8_t* p) {
  const uint64_t b = (uint64_t)(uintptr_t)p;
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b), hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
  return reinterpret_cast<const uint8_t*>((uintptr_t)((uint64_t)hi << 32 | lo));
}
// A copy of one or two KiB from memory to LDS, 16 bytes a lane from base + off; at:
// byte of LDS of the first lane's.  Written as assembly because the compiler waits
// for all copies in flight before any read of LDS; waiting is the caller's.  It has
// no result that a register would have to be kept for.  M0 holds the LDS address; its
// write needs a wait state before the use.  It is named as clobbered, so that a value
// that the compiler puts there is written anew after it (M0 is never allocated, of which
// a warning would tell).  The instruction's offset counts in memory and in LDS.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int UNITS> __device__ __forceinline__ void mx_copy(const uint8_t* base, uint32_t off, uint32_t at) {
  const int m0 = __builtin_amdgcn_readfirstlane((int)at);
  if constexpr (UNITS == 2)
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\tglobal_load_lds_dwordx4 %1, %2 offset:1024"
                     ::"s"(m0), "v"(off), "s"(mx_uniform(base)) : "memory", "m0");
  else
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(m0), "v"(off), "s"(mx_uniform(base)) : "memory", "m0");
}
// 256 bytes, a dword a lane.
__device__ __forceinline__ void mx_copy_scales(const uint8_t* base, uint32_t off, uint32_t at) {
  __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(__builtin_amdgcn_readfirstlane((int)at)), "v"(off), "s"(mx_uniform(base)) : "memory", "m0");
}
#pragma clang diagnostic pop
template <int N> __device__ __forceinline__ void mx_wait() { __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory"); }
__device__ __forceinline__ void mx_barrier() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
}

template <int FA, int FB, int W> struct MxTile {
  static constexpr int STEPS = FA == NC_E2M1 && FB == NC_E2M1 ? 2 : 1;     // of a stage
  static constexpr int SPC = 4 / STEPS;                                    // stages of a chunk
  static constexpr int STRIPS = 2 * W;                                     // of either operand, of the workgroup
  static constexpr int UA = STEPS * mx_step_bytes(FA) / 1024, UB = STEPS * mx_step_bytes(FB) / 1024;   // KiB of a strip and stage
  static constexpr int STAGE = STRIPS * (UA + UB) * 1024;
  static constexpr int SCALES = 2 * STRIPS * kMxScaleBytes;                // of a chunk
  static constexpr int SLOTS = 4;                                          // chunks of scales: those of the stages in flight and more ahead
  static constexpr int LDS = kMxRing * STAGE + SLOTS * SCALES;
  static constexpr int COPIES_SC = (W + SPC - 1) / SPC;                    // copies of scales of a wave and stage
  static constexpr int COPIES = W / 2 * (UA + UB);                         // other copies of a wave and stage
  static constexpr int ROW_EPI = 4 * 32 * (32 * W + 4) * 4;                // a row of tiles of each wave, on its way out
  static constexpr int ROWS = W % 2 == 0 && 2 * ROW_EPI <= LDS ? 2 : 1;    // rows of tiles at a time
  static constexpr int EPI = ROWS * ROW_EPI;
  static_assert(EPI <= LDS, "results fit where the operands were");
};

template <int FA, int FB, bool WIDE, int W>
__global__ void __launch_bounds__(256, W == 4 ? 1 : 2) mx_many(MxProduct p) {
  using T = MxTile<FA, FB, W>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  const int lane = (int)(threadIdx.x & 63), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;

  // Workgroups follow each other over the eight XCDs: each XCD gets a run of
  // neighbouring tiles, in columns of four, whose operands its L2 holds.
  const uint32_t tiles_a = ((uint32_t)p.a.strips + T::STRIPS - 1) / T::STRIPS, tiles_b = ((uint32_t)p.b.strips + T::STRIPS - 1) / T::STRIPS;
  const uint32_t tiles = tiles_a * tiles_b;
  uint32_t tile = blockIdx.x % tiles;
  const uint32_t split = blockIdx.x / tiles;
  {
    const uint32_t each = tiles / 8, more = tiles % 8, xcd = tile % 8, i = tile / 8;
    tile = xcd * each + min(xcd, more) + i;
  }
  uint32_t ta, tb;
  {
    const uint32_t band = tile / (4 * tiles_b), first = band * 4, high = min(4u, tiles_a - first), in = tile - band * 4 * tiles_b;
    ta = first + in % high;
    tb = in / high;
  }
  const int32_t strip_a = (int32_t)ta * T::STRIPS, strip_b = (int32_t)tb * T::STRIPS;

  // this split's chunks
  const int32_t chunks = p.b.chunks;
  const int32_t c0 = (int32_t)((int64_t)chunks * split / p.splits), c1 = (int32_t)((int64_t)chunks * (split + 1) / p.splits);
  const int32_t stages = (c1 - c0) * T::SPC;

  // What this wave copies: W / 2 strips of a and of b, and their scales; strips
  // past the end are the last one's again.  The pointers go on with every copy.
  const uint8_t *ga[W / 2], *gb[W / 2], *gs[W];
#pragma unroll
  for (int i = 0; i < W / 2; ++i) {
    const int64_t sa = (int64_t)min(strip_a + wave * (W / 2) + i, p.a.strips - 1) * chunks + c0;
    const int64_t sb = (int64_t)min(strip_b + wave * (W / 2) + i, p.b.strips - 1) * chunks + c0;
    ga[i] = p.a.codes + sa * mx_chunk_bytes(FA);
    gb[i] = p.b.codes + sb * mx_chunk_bytes(FB);
    gs[i] = p.a.scales + sa * kMxScaleBytes;
    gs[W / 2 + i] = p.b.scales + sb * kMxScaleBytes;
  }
  const uint32_t off16 = (uint32_t)lane * 16, off4 = (uint32_t)lane * 4;
  const uint32_t codes0 = lds0 + (uint32_t)wave * (W / 2) * (T::UA * 1024), sc0 = lds0 + kMxRing * T::STAGE + (uint32_t)wave * (W / 2) * kMxScaleBytes;
  // the i-th of this wave's strips, of a, then of b, in the slot at `slot`
  const auto copy = [&](uint32_t slot, int i) {
    if (i < W / 2) {
      mx_copy<T::UA>(ga[i], off16, codes0 + slot + i * (T::UA * 1024));
      ga[i] += T::UA * 1024;
    } else {
      mx_copy<T::UB>(gb[i - W / 2], off16, codes0 + slot + T::STRIPS * T::UA * 1024 + (i - W / 2) * (T::UB * 1024) + (uint32_t)wave * (W / 2) * ((T::UB - T::UA) * 1024));
      gb[i - W / 2] += T::UB * 1024;
    }
  };
  // the scales of a chunk for the wave's j-th strip
  const auto copy_scales = [&](int32_t c, int j) {
    mx_copy_scales(gs[j] + (int64_t)min(c, c1 - c0 - 1) * kMxScaleBytes, off4,
                   sc0 + (uint32_t)(c % T::SLOTS) * T::SCALES + (uint32_t)(j < W / 2 ? j : T::STRIPS + j - W / 2) * kMxScaleBytes);
  };

  f32x16_t acc[W][W];
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  {
    const int wa = wave >> 1, wb = wave & 1;   // this wave's quarter of the results
    struct Set { u32x4 a[W][T::UA], b[W][T::UB]; } set[2];
    uint32_t xa[W], xb[W], na[W], nb[W];
    constexpr int READS = W * (T::UA + T::UB);
    // the i-th read of a stage: in the order in which the products take them
    const auto read = [&](int32_t t, Set& f, int i) {
      const uint8_t* at = lds + (t % kMxRing) * T::STAGE + lane * 16;
      if (i < W * T::UB) f.b[i % W][i / W] = *reinterpret_cast<const u32x4*>(at + T::STRIPS * T::UA * 1024 + (wb * W + i % W) * (T::UB * 1024) + i / W * 1024);
      else f.a[(i - W * T::UB) % W][(i - W * T::UB) / W] = *reinterpret_cast<const u32x4*>(at + (wa * W + (i - W * T::UB) % W) * (T::UA * 1024) + (i - W * T::UB) / W * 1024);
    };
    const auto frag_a = [&](const Set& f, int i, int s) {
      MxFrag<FA> r;
#pragma unroll
      for (int h = 0; h < T::UA / T::STEPS; ++h) r.w[h] = f.a[i][s * (T::UA / T::STEPS) + h];
      return r;
    };
    const auto frag_b = [&](const Set& f, int j, int s) {
      MxFrag<FB> r;
#pragma unroll
      for (int h = 0; h < T::UB / T::STEPS; ++h) r.w[h] = f.b[j][s * (T::UB / T::STEPS) + h];
      return r;
    };
    const auto read_scales = [&](int32_t c, uint32_t (&a)[W], uint32_t (&b)[W]) {
      const uint8_t* at = lds + kMxRing * T::STAGE + (c % T::SLOTS) * T::SCALES + lane * 4;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        a[i] = *reinterpret_cast<const uint32_t*>(at + (wa * W + i) * kMxScaleBytes);
        b[i] = *reinterpret_cast<const uint32_t*>(at + (T::STRIPS + wb * W + i) * kMxScaleBytes);
      }
    };

    // One stage's products, with `between` called after each (WIDE: each row) of them.
    const auto multiply = [&](const Set& f, int u, auto between) {
#pragma unroll
      for (int s = 0; s < T::STEPS; ++s) {
        const int byte = u * T::STEPS + s;
        if constexpr (WIDE) {
          MxWide b[W];
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const MxScales x = mx_scales<true>(xb[j], lane);
            b[j] = mx_widen<FB>(frag_b(f, j, s), (x.block0 >> (8 * byte)) & 255u, (x.block1 >> (8 * byte)) & 255u);
          }
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const MxScales x = mx_scales<true>(xa[i], lane);
            const MxWide a = mx_widen<FA>(frag_a(f, i, s), (x.block0 >> (8 * byte)) & 255u, (x.block1 >> (8 * byte)) & 255u);
#pragma unroll
            for (int j = 0; j < W; ++j) acc[i][j] = mx_mma_wide(a, b[j], acc[i][j]);
            between(s * W + i, T::STEPS * W);
          }
        } else {
#pragma unroll
          for (int i = 0; i < W; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) {
              const MxFrag<FA> a = frag_a(f, i, s);
              const MxFrag<FB> b = frag_b(f, j, s);
              if (byte == 0) acc[i][j] = mx_mma<FA, FB, 0>(a, b, acc[i][j], xa[i], xb[j]);
              else if (byte == 1) acc[i][j] = mx_mma<FA, FB, 1>(a, b, acc[i][j], xa[i], xb[j]);
              else if (byte == 2) acc[i][j] = mx_mma<FA, FB, 2>(a, b, acc[i][j], xa[i], xb[j]);
              else acc[i][j] = mx_mma<FA, FB, 3>(a, b, acc[i][j], xa[i], xb[j]);
              between((s * W + i) * W + j, T::STEPS * W * W);
            }
        }
      }
    };
    // One chunk.  Once no copies are left to start, the first wait is for all that
    // are in flight; the last stage then reads one that is not there, for nobody.
    const auto chunk = [&](int32_t c, auto more) {
      constexpr bool MORE = decltype(more)::value;
#pragma unroll
      for (int u = 0; u < T::SPC; ++u) {
        const int32_t t = c * T::SPC + u;
        const Set& now = set[u & 1];
        Set& next = set[(u & 1) ^ 1];
        multiply(now, u, [&](int k, int of) {
          const int first = WIDE ? 0 : of / 8;           // the barrier comes after this product
          if (k == first) {
            if (MORE) mx_wait<(kMxRing - 2) * T::COPIES>();   // and some scales, which a later stage needs
            else mx_wait<0>();
            mx_barrier();
            if (u == T::SPC - 1) read_scales(c + 1, na, nb);
          }
          if (k >= first) {
            const int at = k - first, n = of - first;
#pragma unroll
            for (int i = 0; i < READS; ++i)
              if (i * n / READS == at) read(t + 1, next, i);
            if (MORE) {                                  // stage t + kMxRing, and scales of the chunk after its own
              constexpr int ITEMS = W + T::COPIES_SC;
#pragma unroll
              for (int i = 0; i < ITEMS; ++i)
                if (i * n / ITEMS == at) {
                  if (i < W) copy((uint32_t)(t % kMxRing) * T::STAGE, i);
                  else copy_scales(c + kMxRing / T::SPC + 1, (u * T::COPIES_SC + i - W) % W);
                }
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        });
        if (u == T::SPC - 1) {
#pragma unroll
          for (int i = 0; i < W; ++i) {
            xa[i] = na[i];
            xb[i] = nb[i];
          }
        }
      }
    };

    // the scales of the chunks in flight and one more, then the ring
#pragma unroll 1
    for (int k = 0; k <= kMxRing / T::SPC; ++k)
#pragma unroll
      for (int j = 0; j < W; ++j) copy_scales(k, j);
#pragma unroll 1
    for (int t = 0; t < min(kMxRing, stages); ++t)
#pragma unroll
      for (int i = 0; i < W; ++i) copy((uint32_t)t * T::STAGE, i);
    if (stages >= kMxRing) mx_wait<(kMxRing - 1) * T::COPIES>();
    else mx_wait<0>();
    mx_barrier();
#pragma unroll
    for (int i = 0; i < READS; ++i) read(0, set[0], i);
    read_scales(0, xa, xb);
    int32_t c = 0;
#pragma unroll 1
    for (; c < c1 - c0 - kMxRing / T::SPC; ++c) chunk(c, std::true_type{});
    if constexpr (W == 4) {                      // as a loop of its own it takes more registers than there are
      static_assert(kMxRing / T::SPC <= 2, "the chunks in flight");
      if (kMxRing / T::SPC == 1 || c1 - c0 > 1) chunk(c++, std::false_type{});
      if (kMxRing / T::SPC == 2) chunk(c, std::false_type{});
    } else {
#pragma unroll 1
      for (; c < c1 - c0; ++c) chunk(c, std::false_type{});
    }
  }

  // Results through LDS, ROWS tiles' rows of a wave at a time, so that a row goes
  // out in runs of 16 bytes (bf16) a lane.  Each wave has a place of its own.
  mx_wait<0>();
  mx_barrier();
  constexpr int COLS = 32 * W, ROWS = T::ROWS, ACROSS = COLS / 8;
  float (*hold)[COLS + 4] = reinterpret_cast<float (*)[COLS + 4]>(lds + wave * (T::EPI / 4));
  const int64_t row0 = ((int64_t)strip_a + (wave >> 1) * W) * kMxRows, col0 = ((int64_t)strip_b + (wave & 1) * W) * kMxRows;
  MxProduct o = p;
  if (p.splits > 1) {
    o.out = p.part + (int64_t)split * p.a.rows * p.b.rows;
    o.out_stride = p.b.rows;
    o.out_dtype = NC_F32;
    o.bias = nullptr;
    o.accumulate = 0;
    o.stream = 0;                                // the join reads them
  }
  const int c = lane % ACROSS * 8;
  const MxStore<8> store(o, col0 + c);
  const bool inside = row0 + 32 * W <= p.a.rows && col0 + COLS <= p.b.rows;   // all of this wave's results
#pragma unroll
  for (int i = 0; i < W; i += ROWS) {
#pragma unroll
    for (int h = 0; h < ROWS; ++h)
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) hold[32 * h + 8 * (e / 4) + 4 * (lane >> 5) + e % 4][32 * j + (lane & 31)] = acc[i + h][j][e];
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const auto take = [&](int r, float (&y)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = hold[r][c + e];
    };
    if (inside) {
#pragma unroll 4
      for (int r = lane / ACROSS; r < 32 * ROWS; r += 64 / ACROSS) {
        float y[8];
        take(r, y);
        store.whole(row0 + 32 * i + r, y);
      }
    } else if (store.left > 0) {
#pragma unroll 1
      for (int r = lane / ACROSS; r < 32 * ROWS && row0 + 32 * i + r < p.a.rows; r += 64 / ACROSS) {
        float y[8];
        take(r, y);
        store(row0 + 32 * i + r, y);
      }
    }
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

template <int FA, int FB, bool WIDE, int W> hipError_t mx_many_run(const MxProduct& p, hipStream_t stream) {
  constexpr int S = 2 * W;
  const uint32_t tiles = ((uint32_t)p.a.strips + S - 1) / S * (((uint32_t)p.b.strips + S - 1) / S);
  mx_many<FA, FB, WIDE, W><<<dim3(tiles * (uint32_t)p.splits), dim3(256), 0, stream>>>(p);
  return hipGetLastError();
}
template <int FA, int FB> hipError_t mx_many_launch(const MxProduct& p, int w, hipStream_t stream) {
  if constexpr (FA != NC_E2M1 || FB != NC_E2M1) {
    // four times the operands' registers: no room for W = 4
    if (p.out_dtype == NC_F32) return mx_many_run<FA, FB, true, 2>(p, stream);
  }
  return w == 4 ? mx_many_run<FA, FB, false, 4>(p, stream) : mx_many_run<FA, FB, false, 2>(p, stream);
}

hipError_t mx_many_e2m1(const MxProduct& p, int fb, int w, hipStream_t stream);
hipError_t mx_many_e4m3(const MxProduct& p, int fb, int w, hipStream_t stream);
hipError_t mx_many_e5m2(const MxProduct& p, int fb, int w, hipStream_t stream);

}  // namespace nc

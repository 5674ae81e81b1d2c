// kv4.cu -- rows into a KV cache held in 4 bits, and back (the record: kv4.cuh).
//
// Writing a group of 32 channels x_0..x_31 (bf16): with x* the element of largest magnitude
// (the negative one where +|x*| and -|x*| both occur),
//   scale = -x* / 8,   n_i = clamp(round(x_i / scale), -8, 7) + 8,
// round to nearest, ties to even. Dividing a bf16 value by 8 is exact, so x* itself is held
// exactly (code -8). Groups with |x*| < 2^-100 are held as zeros (their scale
// would near the subnormals); a group with a NaN or an infinity gets a NaN scale, so that
// its values read back as NaN.
//
// The kernels write n without a division for each element: with r = 1 / scale to 2^-23,
// x r is within 2^-22 of x / scale in relative terms, and adding and taking away 1.5 * 2^11
// rounds it to a multiple of 2^-12; a tie comes out exactly, and anything else stays on its
// side of one (x / scale is at most 8 in magnitude and at least 2^-9 from a tie it does not
// meet, having two 8-bit significands). A second such constant then rounds to an integer.
//
// Both kernels move bytes, and what bounds the write of bf16 rows is still issue slots: 97
// instructions a record (65536 tokens x 8 heads, 60 us where the bytes need 53; 107 us with a
// warp to a record and 164 instructions, 76 us with 125; 74 us for as many records of 1, 2, 3 or 6
// heads, which share rows less and spill). Reading them takes 55 us, fp32 rows of
// 16384 tokens 26 us either way for 24 of bytes. A half-warp takes a record: lanes 0..7 its K
// row, 8..15 its V row, each lane channels 8 c .. 8 c + 7 and 64 more of them further on, so the
// rows are runs of 128 bytes and four lanes share a scale. A warp takes 2 STEPS records,
// neighbouring heads first and then the next tokens, with the loads of all in flight together.
#include "kv4.cuh"

namespace diffattn {

namespace {
constexpr int WARPS = 4;
// Pairs of records of a warp. Fewer make more blocks, of which a ragged batch leaves many without
// rows: 13 packed chunks of 1 to 1531 tokens x 8 heads took 21.7 us with fp32 rows (1 pair; 2: 15.2)
// and 12.0 read as bf16 (2 pairs; 4: 9.8), against 0.5 and 0.8 us gained on 16384 and 65536 tokens.
constexpr int kSteps = 4, kStepsF32 = 2;
}  // namespace

// The rows of entry b: their count and the first one's row in packed tensors. Offsets that
// are inconsistent give ok = false (the entry is skipped and reported).
struct Kv4Entry {
  int n, row0;
  bool ok;
};
__device__ __forceinline__ Kv4Entry kv4_entry(const Kv4RowsArgs& a, int b) {
  Kv4Entry e;
  if (!a.cu) {
    e.n = a.N; e.row0 = 0; e.ok = true;
    return e;
  }
  e.row0 = __ldg(a.cu + b);
  const int64_t n = (int64_t)__ldg(a.cu + b + 1) - e.row0;
  e.ok = e.row0 >= 0 && n >= 0 && n <= a.N && e.row0 + n <= a.total;
  e.n = e.ok ? (int)n : 0;
  return e;
}

// Where this lane's channels are: in the K or V tensor (elements) and in the cache (bytes). Of
// the warp's 2 STEPS records, half-warp `sub` takes 2 s + sub at step s; SHIFT is the log2 of the
// heads among them, so steps of one row share its position, page and offsets. (With SHIFT at run
// time they were computed for every record, and the write of 65536 x 8 bf16 rows took 76 us, not 64.)
template <int SHIFT>
struct Kv4Lane {
  const Kv4RowsArgs& a;
  int b, i0, c, v, sub;
  int64_t pos, base, cache_base, s1, s2;
  __device__ __forceinline__ Kv4Lane(const Kv4RowsArgs& args, const Kv4Entry& e, int entry, int lane, int recs)
      : a(args), b(entry) {
    const uint32_t item = blockIdx.x * WARPS + (threadIdx.x >> 5);
    const uint32_t head_items = (uint32_t)a.H >> SHIFT;
    const uint32_t row_item = item / head_items;
    i0 = (int)(row_item * (uint32_t)(recs >> SHIFT));
    c = lane & 7;
    v = (lane >> 3) & 1;
    sub = lane >> 4;
    const int h0 = ((int)(item - row_item * head_items) << SHIFT) + (SHIFT ? sub : 0);
    pos = a.pos ? __ldg(a.pos + b) : 0;
    s1 = v ? a.vs[1] : a.ks[1];
    s2 = v ? a.vs[2] : a.ks[2];
    base = (a.cu ? e.row0 * s1 : b * (v ? a.vs[0] : a.ks[0])) + h0 * s2 + c * 8;
    cache_base = h0 * a.cache.stride[2];
  }
  __device__ __forceinline__ int row(int s) const { return i0 + (SHIFT ? 2 * s >> SHIFT : 2 * s + sub); }
  static __device__ __forceinline__ bool new_row(int s) { return s == 0 || SHIFT == 0 || 2 * s % (1 << SHIFT) == 0; }
  // heads past the first step's
  static __device__ __forceinline__ int head(int s) { return 2 * s % (1 << SHIFT); }
  // the record of row i and the first step's head, or -1
  __device__ __forceinline__ int64_t record(int i) const {
    const int64_t t = pos + i;
    if (t < 0 || t >= a.cache.L) return -1;
    const int64_t at = kv4_page_offset(a.cache, b, (int)t);
    return at < 0 ? -1 : at + cache_base;
  }
};

// 1 / x to 2^-23 in relative terms
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 8 codes and the bf16 bits of the scale of 8 channels (bf16 pairs w), which with those of
// the three lanes beside it make a group
__device__ __forceinline__ uint32_t kv4_encode(const uint32_t (&w)[4], uint32_t& scale_bits) {
  // The largest magnitude among the group's positive values (low half) and among its
  // negative ones (high half), on bf16 bits: as signed 16-bit integers the largest is the
  // largest positive value, as unsigned ones the largest negative one.
  const uint32_t up = __vimax_s16x2_relu(__vimax3_s16x2(w[0], w[1], w[2]), w[3]);
  const uint32_t down = __vimax3_u16x2(__vimax3_u16x2(w[0], w[1], w[2]), w[3], 0x80008000u) ^ 0x80008000u;
  uint32_t most = __vmaxu2(__byte_perm(up, down, 0x5410), __byte_perm(up, down, 0x7632));
  most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 1));
  most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 2));
  const uint32_t p16 = most & 0xffffu, n16 = most >> 16, size = max(p16, n16);
  const bool finite = size < 0x7f80u;
  const bool held = finite && size >= (27u << 7);  // not under 2^-100
  const float peak = __uint_as_float(size << 16);
  const float scale = n16 >= p16 ? peak * 0.125f : peak * -0.125f;
  // kFine in [2^11, 2^12): units of 2^-12; adding kWhole - kFine, exact up to its own
  // rounding, then gives the integer on top of kWhole = 1.5 * 2^23
  constexpr float kFine = 1.5f * 2048.f, kWhole = 12582912.f;
  const float inv = rcp_approx(scale);
  float2 k[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 t = fma2(make_float2(bf16_low(w[i]), bf16_high(w[i])), make_float2(inv, inv), make_float2(kFine, kFine));
    t = make_float2(fminf(t.x, kFine + 7.f), fminf(t.y, kFine + 7.f));
    k[i] = add2(add2(t, make_float2(kWhole - kFine, kWhole - kFine)), make_float2(-kWhole, -kWhole));
  }
  // four codes as the digits of a number, 8 added to each, in the low 16 bits of a float
  const float2 even = fma2(k[1], make_float2(256.f, 256.f), k[0]), odd = fma2(k[3], make_float2(256.f, 256.f), k[2]);
  const float lo = __fmaf_rn(even.y, 16.f, even.x) + (kWhole + 34952.f);  // 0x8888
  const float hi = __fmaf_rn(odd.y, 16.f, odd.x) + (kWhole + 34952.f);
  scale_bits = !finite ? 0x7fc0u : (held ? __float_as_uint(scale) >> 16 : 0u);
  return held ? __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410) : 0x88888888u;
}

template <bool F32, int SHIFT>
__global__ void __launch_bounds__(WARPS * 32, 12) kv4_write_kernel(Kv4RowsArgs a) {
  constexpr int STEPS = F32 ? kStepsF32 : kSteps;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  kv4_wait();
  const Kv4Entry e = kv4_entry(a, b);
  if (!e.ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_status(a.cache.dev_status, DIFFATTN_ERR_INVALID_ARG);
    return;
  }
  const Kv4Lane<SHIFT> at(a, e, b, lane, 2 * STEPS);
  if (at.i0 >= e.n) return;
  const int64_t ext = at.v ? a.ext_v : a.ext_k;
  const void* src = at.v ? a.v : a.k;

  uint32_t raw[F32 ? 1 : STEPS][2][4];  // 8 channels and the 8 at 64 further on
  float4 wide[F32 ? STEPS : 1][2][2];
  int64_t dst[STEPS];  // byte offset of the record, -1: not written
  int64_t place = -1, from = 0;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    if (at.new_row(s)) {
      const int i = at.row(s);
      place = i < e.n ? at.record(i) : -1;
      if (i < e.n && place < 0 && (lane & 15) == 0) report_status(a.cache.dev_status, DIFFATTN_ERR_INVALID_ARG);
      from = at.base + min(i, e.n - 1) * at.s1;  // rows past the entry load its last one and are not written
    }
    dst[s] = place < 0 ? -1 : place + at.head(s) * a.cache.stride[2];
    const int64_t off = from + at.head(s) * at.s2;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const bool ok = in_bounds(off + 64 * q, 8, ext, a.cache.dev_status, a.cache.dbg_status);
      if constexpr (F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(src) + off + 64 * q);
        wide[s][q][0] = ok ? __ldcs(p) : make_float4(0.f, 0.f, 0.f, 0.f);
        wide[s][q][1] = ok ? __ldcs(p + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(src) + off + 64 * q);
        const uint4 x = ok ? __ldcs(p) : make_uint4(0u, 0u, 0u, 0u);
        raw[s][q][0] = x.x; raw[s][q][1] = x.y; raw[s][q][2] = x.z; raw[s][q][3] = x.w;
      }
    }
    if (dst[s] >= 0 && !in_bounds(dst[s], kKv4Record, a.cache.ext, a.cache.dev_status, a.cache.dbg_status)) dst[s] = -1;
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    uint32_t codes[2], bits[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if constexpr (F32) {
        const float4 x = wide[s][q][0], y = wide[s][q][1];
        const uint32_t w[4] = {pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y), pack_bf16(y.z, y.w)};
        codes[q] = kv4_encode(w, bits[q]);
      } else {
        codes[q] = kv4_encode(raw[s][q], bits[q]);
      }
      bits[q] |= __shfl_down_sync(0xffffffffu, bits[q], 4) << 16;  // lane c = 0: groups 2 q, 2 q + 1
    }
    if (dst[s] >= 0) {
      uint32_t* row = reinterpret_cast<uint32_t*>(a.cache.base + dst[s]) + at.v * 16 + at.c;
      row[0] = codes[0];
      row[8] = codes[1];
      if (at.c == 0)
        *reinterpret_cast<uint2*>(a.cache.base + dst[s] + kKv4Scales + at.v * 8) = make_uint2(bits[0], bits[1]);
    }
  }
}

// Channels 2 i and 2 i + 1 of a word of 8 codes, as two bf16 values n - 8 (exact: 128 + n - 136)
template <int I>
__device__ __forceinline__ __nv_bfloat162 kv4_pair(uint32_t w) {
  const uint32_t lo = w >> (8 * I), hi = I < 2 ? w << (12 - 8 * I) : w >> (8 * I - 12);
  const uint32_t x = (lo & 0xfu) | (hi & 0xf0000u) | 0x43004300u;
  return __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), __float2bfloat162_rn(136.f));
}

// Reading back: each lane turns 4 code bytes and their group's scale into 8 channels, twice:
// scale * (n - 8) has 12 significant bits, exact in fp32 and rounded once to bf16 (nearest).
template <bool F32, int SHIFT>
__global__ void __launch_bounds__(WARPS * 32) kv4_read_kernel(Kv4RowsArgs a) {
  constexpr int STEPS = F32 ? kStepsF32 : kSteps;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  kv4_wait();
  const Kv4Entry e = kv4_entry(a, b);
  if (!e.ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_status(a.cache.dev_status, DIFFATTN_ERR_INVALID_ARG);
    return;
  }
  const Kv4Lane<SHIFT> at(a, e, b, lane, 2 * STEPS);
  if (at.i0 >= e.n) return;
  const int64_t ext = at.v ? a.ext_v : a.ext_k;
  void* dst = at.v ? a.v : a.k;

  uint32_t codes[STEPS][2], scale[STEPS][2];  // scale: bf16 bits
  int64_t place = -1;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    if (at.new_row(s)) {
      const int i = at.row(s);
      place = i < e.n ? at.record(i) : -1;
      // outside the entry or the pool: the row reads as zeros
      if (i < e.n && place < 0 && (lane & 15) == 0) report_status(a.cache.dev_status, DIFFATTN_ERR_INVALID_ARG);
    }
    const int64_t from = place + at.head(s) * a.cache.stride[2];
    const bool ok = place >= 0 && in_bounds(from, kKv4Record, a.cache.ext, a.cache.dev_status, a.cache.dbg_status);
    const uint8_t* rec = a.cache.base + (ok ? from : 0);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      codes[s][q] = ok ? __ldcs(reinterpret_cast<const uint32_t*>(rec) + at.v * 16 + 8 * q + at.c) : 0u;
      scale[s][q] = ok ? __ldcs(reinterpret_cast<const uint16_t*>(rec + kKv4Scales) + at.v * 4 + 2 * q + (at.c >> 2)) : 0u;
    }
  }
  int64_t to = 0;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int odd = at.c & 1;
    if constexpr (F32) {
      // a pair of lanes swaps halves of its 16 channels, so that a store of 16 bytes per lane
      // fills whole 32-byte sectors: channels 4 odd .. and 8 + 4 odd .. of the pair's
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, codes[s][q], 1);
        codes[s][q] = odd ? __byte_perm(other, codes[s][q], 0x7632) : __byte_perm(codes[s][q], other, 0x5410);
      }
    }
    if (at.new_row(s)) to = at.base + at.row(s) * at.s1;
    if (at.row(s) >= e.n) continue;
    const int64_t off = to + at.head(s) * at.s2;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (!in_bounds(off + 64 * q, 8, ext, a.cache.dev_status, a.cache.dbg_status)) continue;
      const uint32_t w = codes[s][q];
      const __nv_bfloat162 n[4] = {kv4_pair<0>(w), kv4_pair<1>(w), kv4_pair<2>(w), kv4_pair<3>(w)};
      if constexpr (F32) {
        const float f = __uint_as_float(scale[s][q] << 16);
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(dst) + off + 64 * q - 4 * odd);
        const float2 x0 = __bfloat1622float2(n[0]), x1 = __bfloat1622float2(n[1]);
        const float2 x2 = __bfloat1622float2(n[2]), x3 = __bfloat1622float2(n[3]);
        __stcs(p, make_float4(f * x0.x, f * x0.y, f * x1.x, f * x1.y));
        __stcs(p + 2, make_float4(f * x2.x, f * x2.y, f * x3.x, f * x3.y));
      } else {
        const uint32_t both = scale[s][q] | scale[s][q] << 16;
        const __nv_bfloat162 f = *reinterpret_cast<const __nv_bfloat162*>(&both);
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 x = __hmul2(n[i], f);
          y[i] = *reinterpret_cast<const uint32_t*>(&x);
        }
        __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst) + off + 64 * q),
               make_uint4(y[0], y[1], y[2], y[3]));
      }
    }
  }
}

// A warp's records: 2^shift neighbouring heads (as many of its 2 STEPS as divide H) by rows.
template <size_t SHIFTS>
static cudaError_t kv4_launch(const Kv4RowsArgs& a, void (*const (&fns)[SHIFTS])(Kv4RowsArgs), int recs,
                              cudaStream_t stream) {
  int shift = 0;
  while (shift + 1 < (int)SHIFTS && a.H % (2 << shift) == 0) ++shift;
  const int64_t rows = recs >> shift;
  const int64_t items = ((int64_t)a.N + rows - 1) / rows * (a.H >> shift);
  return kv4_launch_early(fns[shift], dim3((unsigned)((items + WARPS - 1) / WARPS), (unsigned)a.B), dim3(WARPS * 32), 0,
                          stream, a);
}

using Kv4Kernel = void (*)(Kv4RowsArgs);

cudaError_t launch_kv4_write(const Kv4RowsArgs& a, cudaStream_t stream) {
  static const Kv4Kernel f32[] = {kv4_write_kernel<true, 0>, kv4_write_kernel<true, 1>, kv4_write_kernel<true, 2>};
  static const Kv4Kernel bf16[] = {kv4_write_kernel<false, 0>, kv4_write_kernel<false, 1>, kv4_write_kernel<false, 2>,
                                   kv4_write_kernel<false, 3>};
  return a.f32 ? kv4_launch(a, f32, 2 * kStepsF32, stream) : kv4_launch(a, bf16, 2 * kSteps, stream);
}

cudaError_t launch_kv4_read(const Kv4RowsArgs& a, cudaStream_t stream) {
  static const Kv4Kernel f32[] = {kv4_read_kernel<true, 0>, kv4_read_kernel<true, 1>, kv4_read_kernel<true, 2>};
  static const Kv4Kernel bf16[] = {kv4_read_kernel<false, 0>, kv4_read_kernel<false, 1>, kv4_read_kernel<false, 2>,
                                   kv4_read_kernel<false, 3>};
  return a.f32 ? kv4_launch(a, f32, 2 * kStepsF32, stream) : kv4_launch(a, bf16, 2 * kSteps, stream);
}

}  // namespace diffattn

// kv4.cu -- rows into a KV cache held in 4 bits, and back (the record: kv4.cuh).
//
// Writing a group of 32 channels x_0..x_31 (bf16): with x* the element of largest magnitude
// (the negative one where +|x*| and -|x*| both occur),
//   scale = -x* / 8,   n_i = clamp(round(x_i / scale), -8, 7) + 8,
// round to nearest, ties to even. Dividing a bf16 value by 8 is exact, so x* itself is held
// exactly (code -8), and x_i / scale is a quotient of two 8-bit significands: it is a tie or
// at least 2^-9 away from one in relative terms, so the rounded fp32 division decides every
// code as exact arithmetic would. Groups with |x*| < 2^-100 are held as zeros (their scale
// would near the subnormals); a group with a NaN or an infinity gets a NaN scale, so that
// its values read back as NaN.
//
// Both kernels move bytes: one warp takes one (token, head) at a time, lanes 0..15 its K
// row, lanes 16..31 its V row, 8 channels (4 code bytes) each, so the codes of a record are
// one 128-byte run of a warp's 4-byte accesses and four lanes share a scale. A warp holds
// RECS records in flight, because one 16-byte load per lane does not cover the latency.
#include "kv4.cuh"

namespace diffattn {

namespace {
constexpr int WARPS = 8;
constexpr int RECS = 4;                 // records of a warp in flight
constexpr int PER_BLOCK = WARPS * RECS;
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

// Element offset of this lane's 8 channels in the K or V tensor, for row i of entry b.
__device__ __forceinline__ int64_t kv4_row_offset(const Kv4RowsArgs& a, const Kv4Entry& e, int b, int i,
                                                  int h, int lane) {
  const int64_t* s = lane < 16 ? a.ks : a.vs;
  return (a.cu ? (int64_t)(e.row0 + i) * s[1] : b * s[0] + i * s[1]) + h * s[2] + (lane & 15) * 8;
}

template <bool F32>
__global__ void __launch_bounds__(WARPS * 32) kv4_write_kernel(Kv4RowsArgs a) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const Kv4Entry e = kv4_entry(a, b);
  if (!e.ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_status(a.cache.dev_status, DIFFATTN_ERR_INVALID_ARG);
    return;
  }
  const int64_t recs = (int64_t)e.n * a.H;
  const int64_t r0 = ((int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5)) * RECS;
  if (r0 >= recs) return;
  const int64_t pos = a.pos ? __ldg(a.pos + b) : 0;
  const int64_t ext = lane < 16 ? a.ext_k : a.ext_v;
  const void* src = lane < 16 ? a.k : a.v;

  uint32_t raw[RECS][4];  // 8 channels of each record in bf16
  int64_t dst[RECS];      // byte offset of the record, -1: not written
#pragma unroll
  for (int r = 0; r < RECS; ++r) {
    dst[r] = -1;
    if (r0 + r >= recs) continue;
    const int i = (int)((r0 + r) / a.H), h = (int)((r0 + r) - (int64_t)i * a.H);
    const int64_t t = pos + i;
    if (t >= 0 && t < a.cache.L) dst[r] = kv4_page_offset(a.cache, b, (int)t);
    if (dst[r] >= 0) {
      dst[r] += h * a.cache.stride[2];
      if (!in_bounds(dst[r], kKv4Record, a.cache.ext, a.cache.dev_status, a.cache.dbg_status)) dst[r] = -1;
    } else if (lane == 0) {
      report_status(a.cache.dev_status, DIFFATTN_ERR_INVALID_ARG);
    }
    const int64_t off = kv4_row_offset(a, e, b, i, h, lane);
    const bool ok = in_bounds(off, 8, ext, a.cache.dev_status, a.cache.dbg_status);
    if (F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(src) + off);
      const float4 x = ok ? p[0] : make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 y = ok ? p[1] : make_float4(0.f, 0.f, 0.f, 0.f);
      raw[r][0] = pack_bf16(x.x, x.y); raw[r][1] = pack_bf16(x.z, x.w);
      raw[r][2] = pack_bf16(y.x, y.y); raw[r][3] = pack_bf16(y.z, y.w);
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(src) + off);
      const uint4 x = ok ? *p : make_uint4(0u, 0u, 0u, 0u);
      raw[r][0] = x.x; raw[r][1] = x.y; raw[r][2] = x.z; raw[r][3] = x.w;
    }
  }
#pragma unroll
  for (int r = 0; r < RECS; ++r) {
    if (r0 + r >= recs) break;
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_low(raw[r][i]);
      x[2 * i + 1] = bf16_high(raw[r][i]);
    }
    // the group's largest and smallest value and whether all are finite, over its 4 lanes
    float hi = x[0], lo = x[0];
    bool finite = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi = fmaxf(hi, x[i]);
      lo = fminf(lo, x[i]);
      finite = finite && (__float_as_uint(x[i]) & 0x7f800000u) != 0x7f800000u;
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      finite = __shfl_xor_sync(0xffffffffu, (int)finite, o) && finite;
    }
    const float peak = hi > -lo ? hi : lo;
    const bool zero = fabsf(peak) < 7.888609052210118e-31f;  // 2^-100
    const float scale = peak * -0.125f;
    uint32_t codes = 0x88888888u;
    if (finite && !zero) {
      codes = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = fminf(fmaxf(rintf(__fdiv_rn(x[i], scale)), -8.f), 7.f);
        codes |= (uint32_t)((int)n + 8) << (4 * i);
      }
    }
    // bf16 bits of the scale (exact: a power of two times a bf16 value)
    const uint32_t sb = !finite ? 0x7fc0u : (zero ? 0u : __float_as_uint(scale) >> 16);
    const uint32_t pair = sb | (__shfl_down_sync(0xffffffffu, sb, 4) << 16);
    if (dst[r] >= 0) {
      uint8_t* rec = a.cache.base + dst[r];
      reinterpret_cast<uint32_t*>(rec)[lane] = codes;
      if ((lane & 7) == 0) reinterpret_cast<uint32_t*>(rec + kKv4Scales)[lane >> 3] = pair;
    }
  }
}

// Reading back: each lane turns 4 code bytes and its group's scale into 8 channels,
// scale * (n - 8): 12 significant bits, exact in fp32 and rounded once to bf16 (nearest).
template <bool F32>
__global__ void __launch_bounds__(WARPS * 32) kv4_read_kernel(Kv4RowsArgs a) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const Kv4Entry e = kv4_entry(a, b);
  if (!e.ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_status(a.cache.dev_status, DIFFATTN_ERR_INVALID_ARG);
    return;
  }
  const int64_t recs = (int64_t)e.n * a.H;
  const int64_t r0 = ((int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5)) * RECS;
  if (r0 >= recs) return;
  const int64_t pos = a.pos ? __ldg(a.pos + b) : 0;
  const int64_t ext = lane < 16 ? a.ext_k : a.ext_v;
  void* dst = lane < 16 ? a.k : a.v;

  uint32_t codes[RECS];
  float scale[RECS];
  int64_t off[RECS];  // element offset of this lane's 8 channels
#pragma unroll
  for (int r = 0; r < RECS; ++r) {
    codes[r] = 0u;
    scale[r] = 0.f;
    off[r] = -1;
    if (r0 + r >= recs) continue;
    const int i = (int)((r0 + r) / a.H), h = (int)((r0 + r) - (int64_t)i * a.H);
    off[r] = kv4_row_offset(a, e, b, i, h, lane);
    const int64_t t = pos + i;
    int64_t at = -1;
    if (t >= 0 && t < a.cache.L) at = kv4_page_offset(a.cache, b, (int)t);
    if (at < 0) {  // outside the entry or the pool: the row reads as zeros
      if (lane == 0) report_status(a.cache.dev_status, DIFFATTN_ERR_INVALID_ARG);
      continue;
    }
    at += h * a.cache.stride[2];
    if (!in_bounds(at, kKv4Record, a.cache.ext, a.cache.dev_status, a.cache.dbg_status)) continue;
    const uint8_t* rec = a.cache.base + at;
    codes[r] = reinterpret_cast<const uint32_t*>(rec)[lane];
    scale[r] = __uint_as_float(
        (uint32_t)reinterpret_cast<const uint16_t*>(rec + kKv4Scales)[lane >> 2] << 16);
  }
#pragma unroll
  for (int r = 0; r < RECS; ++r) {
    if (off[r] < 0 || !in_bounds(off[r], 8, ext, a.cache.dev_status, a.cache.dbg_status)) continue;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = scale[r] * (float)((int)((codes[r] >> (4 * i)) & 15u) - 8);
    if (F32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(dst) + off[r]);
      p[0] = make_float4(x[0], x[1], x[2], x[3]);
      p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst) + off[r]) =
          make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    }
  }
}

static dim3 kv4_grid(const Kv4RowsArgs& a) {
  return dim3((unsigned)(((int64_t)a.N * a.H + PER_BLOCK - 1) / PER_BLOCK), (unsigned)a.B);
}

cudaError_t launch_kv4_write(const Kv4RowsArgs& a, cudaStream_t stream) {
  if (a.f32) kv4_write_kernel<true><<<kv4_grid(a), WARPS * 32, 0, stream>>>(a);
  else kv4_write_kernel<false><<<kv4_grid(a), WARPS * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4RowsArgs& a, cudaStream_t stream) {
  if (a.f32) kv4_read_kernel<true><<<kv4_grid(a), WARPS * 32, 0, stream>>>(a);
  else kv4_read_kernel<false><<<kv4_grid(a), WARPS * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace diffattn

// Rotary positions and the paged key-value cache: the rotation table, the
// rotation, the quantising write and the read back.
//
// Cache layout.  A page holds `page_size` tokens of every kv head:
//   [heads][page_size / 16] units, one unit = 16 consecutive tokens of one head:
//     [K codes][V codes][K scales][V scales]
// so a unit is one contiguous piece of HBM that a single bulk copy brings in.
// The codes are stored as the attention kernel's 32 lanes consume them (the A
// fragments of a 16 x 16 x 16 MMA whose M side is the tokens for K and the
// channels for V).  The grain is an octet, 8 consecutive channels of one
// token (GS = 16, 8 or 4 bytes); every lane owns D / 16 octets of K and D / 16
// of V, its octets are laid out in 16-byte vectors, and vector v of all
// 32 lanes is one conflict-free 512-byte shared-memory load:
//   byte(lane, i) = ((i * GS / 16) * 32 + lane) * 16 + (i * GS) % 16
//   K octet o of token r:  lane (r % 8) * 4 + o % 4,  i = (o / 4) * 2 + r / 8
//   V octet o of token r:  lane (o / (D / 64)) * 4 + (r % 8) / 2,
//                          i = (o % (D / 64)) * 4 + (r / 8) * 2 + r % 2
// Scales: E4M3 fp32 [16 tokens] for K, then V; NVFP4 K [16 tokens][2][D / 32]
// (16-channel block 2b + h at [h][b]), V [D / 16 blocks][16 tokens].
#include <cuda_bf16.h>

#include <type_traits>

#include "hq_internal.cuh"

namespace hq {

// ---- the rotation table ------------------------------------------------------
// Frequency i of a rotation of R channels, radians per position, in 64 bits.
__device__ __forceinline__ double rope_freq(const hq_rope_desc &d, int i) {
  const double two_pi = 6.283185307179586476925;
  double f = pow(d.base, -2.0 * i / d.rot_dim);
  if (d.scaling == HQ_ROPE_LINEAR) f /= d.factor;
  if (d.scaling == HQ_ROPE_TURNS) {
    const double turns = d.context * f / two_pi;
    const double y = fmin(fmax((turns - d.low) / (d.high - d.low), 0.0), 1.0);
    f = f * (y + (1.0 - y) / d.factor);
  }
  if (d.scaling == HQ_ROPE_INDEX) {
    // index of the frequency that makes n turns over the context
    const double den = 2.0 * log(d.base);
    const double at_high = d.rot_dim * log(d.context / (two_pi * d.high)) / den;
    const double at_low = d.rot_dim * log(d.context / (two_pi * d.low)) / den;
    const double first = fmax(floor(at_high), 0.0), last = fmin(ceil(at_low), d.rot_dim - 1.0);
    const double y = 1.0 - fmin(fmax((i - first) / fmax(last - first, 0.001), 0.0), 1.0);
    f = f * (y + (1.0 - y) / d.factor);
  }
  return f;
}

// table[p] = amplitude * (cos(p f_0) .. cos(p f_{R/2-1}), sin(p f_0) ..).  The
// angle of a far position does not fit fp32 (position 131072 leaves 2^-7 of a
// radian there), so the product and the reduction are 64-bit: the angle is
// counted in turns and brought to [-1/8, 1/8] of one; what is left is at most
// pi/4 and goes through fp32 sine and cosine, an error of about one fp32 step.
__global__ void rope_table_kernel(hq_rope_desc d, long long P, float *__restrict__ table) {
  const int half = d.rot_dim / 2;
  const float amp = (float)d.amplitude;
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    const double per = rope_freq(d, i) / 6.283185307179586476925;  // turns per position
    for (long long p = blockIdx.x; p < P; p += gridDim.x) {
      const double turns = (double)p * per;
      const double quarters = rint(turns * 4.0);
      const float r = (float)((turns - quarters * 0.25) * 6.283185307179586476925);
      const int quad = (int)((long long)quarters & 3);
      const float s = sinf(r), c = cosf(r);
      float co = (quad & 1) ? s : c, si = (quad & 1) ? c : s;
      if (quad == 1 || quad == 2) co = -co;
      if (quad >= 2) si = -si;
      table[p * d.rot_dim + i] = amp * co;
      table[p * d.rot_dim + half + i] = amp * si;
    }
  }
}

hq_status launch_rope_table(const hq_rope_desc *d, int P, float *table, cudaStream_t st) {
  hq_rope_desc r = *d;
  if (r.amplitude == 0.0) r.amplitude = 1.0;
  const int half = r.rot_dim / 2;
  int threads = (half + 31) / 32 * 32;
  if (threads > 256) threads = 256;
  const int blocks = P < 148 * 8 ? P : 148 * 8;
  rope_table_kernel<<<blocks, threads, 0, st>>>(r, P, table);
  return check_launch();
}

// ---- the rotation --------------------------------------------------------------
// (a, b) -> (a c - b s, b c + a s), each step an fp32 IEEE operation.
__device__ __forceinline__ void rope_pair(float a, float b, float c, float s, float &x, float &y) {
  x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

__device__ __forceinline__ float bf16_at(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ uint16_t to_bf16(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
  return (uint32_t)to_bf16(lo) | ((uint32_t)to_bf16(hi) << 16);
}
__device__ __forceinline__ void unpack8(const uint4 v, float *f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float *f) {
  return make_uint4(to_bf16x2(f[0], f[1]), to_bf16x2(f[2], f[3]), to_bf16x2(f[4], f[5]), to_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void load8(const float *p, float *f) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Work of a head: chunks of 8 pairs, then chunks of 8 unrotated channels.  A
// chunk holds both channels of its pairs, so x and out may be the same.
// Widths that are a multiple of 16 move 16 bytes at a time; others (pairs
// that straddle 16-byte pieces) go channel by channel.
__host__ __device__ inline int rope_chunks(int D, int rot) { return (rot / 2 + 7) / 8 + (D - rot + 7) / 8; }

__device__ __forceinline__ void rope_chunk(int c, int D, int rot, int inter, const uint16_t *x,
                                           const float *tab, uint16_t *out) {
  const int half = rot / 2, npair = (half + 7) / 8;
  if (c >= npair) {  // past the rotated part: copied
    if (x == out) return;
    const int ch = rot + (c - npair) * 8;
    if ((rot & 7) == 0) {
      *reinterpret_cast<uint4 *>(out + ch) = *reinterpret_cast<const uint4 *>(x + ch);
    } else {
      for (int i = ch; i < ch + 8 && i < D; ++i) out[i] = x[i];
    }
    return;
  }
  if ((rot & 15) == 0) {
    const int i0 = inter ? 16 * c : 8 * c, i1 = inter ? 16 * c + 8 : 8 * c + half;
    float a[8], b[8], co[8], si[8];
    unpack8(*reinterpret_cast<const uint4 *>(x + i0), a);
    unpack8(*reinterpret_cast<const uint4 *>(x + i1), b);
    load8(tab + 8 * c, co);
    load8(tab + half + 8 * c, si);
    if (inter) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        rope_pair(a[2 * j], a[2 * j + 1], co[j], si[j], a[2 * j], a[2 * j + 1]);
        rope_pair(b[2 * j], b[2 * j + 1], co[4 + j], si[4 + j], b[2 * j], b[2 * j + 1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) rope_pair(a[j], b[j], co[j], si[j], a[j], b[j]);
    }
    *reinterpret_cast<uint4 *>(out + i0) = pack8(a);
    *reinterpret_cast<uint4 *>(out + i1) = pack8(b);
    return;
  }
  for (int i = 8 * c; i < 8 * c + 8 && i < half; ++i) {
    const int i0 = inter ? 2 * i : i, i1 = inter ? 2 * i + 1 : i + half;
    float u, v;
    rope_pair(bf16_at(x + i0), bf16_at(x + i1), tab[i], tab[half + i], u, v);
    out[i0] = to_bf16(u);
    out[i1] = to_bf16(v);
  }
}

struct RopeArgs {
  int T, H, D, rot, inter, P;
  const uint16_t *x;
  long long xt, xh;  // strides between tokens and heads, elements
  const int32_t *pos;
  const float *table;
  uint16_t *out;
  long long ot, oh;
};

__device__ __forceinline__ void rope_rows(const RopeArgs &a, size_t first, size_t step) {
  const int nc = rope_chunks(a.D, a.rot);
  const size_t total = (size_t)a.T * a.H * nc;
  for (size_t i = first; i < total; i += step) {
    const int c = (int)(i % nc);
    const size_t th = i / nc;
    const int h = (int)(th % a.H);
    const size_t t = th / a.H;
    const int p = a.pos[t];
    if (p < 0 || p >= a.P) {
      set_device_error(HQ_ERR_DEVICE_INDEX);
      continue;
    }
    rope_chunk(c, a.D, a.rot, a.inter, a.x + t * a.xt + h * a.xh, a.table + (size_t)p * a.rot,
               a.out + t * a.ot + h * a.oh);
  }
}

__global__ void rope_kernel(RopeArgs a) {
  rope_rows(a, blockIdx.x * (size_t)blockDim.x + threadIdx.x, (size_t)gridDim.x * blockDim.x);
}

hq_status launch_rope(const RopeArgs &a, cudaStream_t st) {
  const size_t total = (size_t)a.T * a.H * rope_chunks(a.D, a.rot);
  rope_kernel<<<quant_grid(total, 256), 256, 0, st>>>(a);
  return check_launch();
}

// ---- the cache layout ------------------------------------------------------------
__host__ __device__ constexpr int kv_granule(int fmt) { return fmt == A_BF16 ? 16 : fmt == A_FP8 ? 8 : 4; }
__host__ __device__ constexpr int kv_code_bytes(int fmt, int D) { return 2 * D * kv_granule(fmt); }  // 16 tokens of K or V
__host__ __device__ constexpr int kv_scale_bytes(int fmt, int D) { return fmt == A_BF16 ? 0 : fmt == A_FP8 ? 64 : D; }
__host__ __device__ constexpr int kv_unit_bytes(int fmt, int D) {
  return 2 * (kv_code_bytes(fmt, D) + kv_scale_bytes(fmt, D));
}

template <int GS>
__device__ __forceinline__ int lane_byte(int lane, int i) {
  return ((i * GS / 16) * 32 + lane) * 16 + (i * GS) % 16;
}
template <int GS>
__device__ __forceinline__ int k_octet(int o, int r) {
  return lane_byte<GS>((r & 7) * 4 + (o & 3), (o >> 2) * 2 + (r >> 3));
}
template <int GS, int D>
__device__ __forceinline__ int v_octet(int o, int r) {
  constexpr int NQ = D / 64;
  return lane_byte<GS>((o / NQ) * 4 + ((r & 7) >> 1), (o % NQ) * 4 + (r >> 3) * 2 + (r & 1));
}

struct KvArgs {
  int H, page_units;        // kv heads; units per page
  int page;                 // tokens per page
  long long slots_total;    // num_pages * page
  size_t page_bytes;
  uint8_t *pages;
  const float *glob;        // NVFP4: second-level scales of K and V
};

// The unit and the row inside it of (slot, head).
template <int FMT, int D>
__device__ __forceinline__ uint8_t *kv_unit(const KvArgs &a, long long slot, int h, int &r) {
  const long long pg = slot / a.page;
  const int off = (int)(slot - pg * a.page);
  r = off & 15;
  return a.pages + (size_t)pg * a.page_bytes + ((size_t)h * a.page_units + (off >> 4)) * kv_unit_bytes(FMT, D);
}

// Stores octet o of a token's key (IS_V = 0) or value.  The LPR lanes of a
// row call it together (`on`: the lane has an octet; D = 192 leaves a quarter
// of its 32 lanes idle).
template <int FMT, int D, int LPR>
__device__ __forceinline__ void kv_store(uint8_t *unit, int r, int o, bool on, bool is_v, const float *f,
                                         const float *glob) {
  constexpr int GS = kv_granule(FMT), CB = kv_code_bytes(FMT, D), SB = kv_scale_bytes(FMT, D);
  uint8_t *codes = unit + (is_v ? CB : 0) + (is_v ? v_octet<GS, D>(o, r) : k_octet<GS>(o, r));
  if constexpr (FMT == A_BF16) {
    if (on) *reinterpret_cast<uint4 *>(codes) = pack8(f);
  } else {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
    uint8_t *scales = unit + 2 * CB + (is_v ? SB : 0);
    if constexpr (FMT == A_FP8) {
      // hq_quant_act's per-token recipe on the head's D channels
#pragma unroll
      for (int k = LPR / 2; k > 0; k >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, k));
      const float s = (amax == 0.f) ? 1.f : __fdiv_rn(amax, 448.f);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = f32x2_to_e4m3x2(__fdiv_rn(f[2 * i], s), __fdiv_rn(f[2 * i + 1], s));
      if (on) *reinterpret_cast<uint2 *>(codes) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
      if (on && o == 0) reinterpret_cast<float *>(scales)[r] = s;
    } else {
      // hq_quant_act's NVFP4 recipe with a static tensor scale; a block is two lanes
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      const float g = glob[is_v ? 1 : 0];
      const uint32_t sb = f32x2_to_e4m3x2(__fdiv_rn(__fdiv_rn(amax, 6.f), g), 0.f) & 0xFFu;
      const float d = __fmul_rn(e4m3_to_f32(sb), g);
      uint32_t w = 0;
      if (d != 0.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w |= f32x2_to_e2m1x2(__fdiv_rn(f[2 * i], d), __fdiv_rn(f[2 * i + 1], d)) << (8 * i);
      }
      if (on) {
        *reinterpret_cast<uint32_t *>(codes) = w;
        const int b = o >> 1;
        if ((o & 1) == 0) scales[is_v ? b * 16 + r : r * (D / 16) + (b & 1) * (D / 32) + (b >> 1)] = (uint8_t)sb;
      }
    }
  }
}

// Octet o of a token's key or value as fp32.
template <int FMT, int D>
__device__ __forceinline__ void kv_load(const uint8_t *unit, int r, int o, bool is_v, const float *glob, float *f) {
  constexpr int GS = kv_granule(FMT), CB = kv_code_bytes(FMT, D), SB = kv_scale_bytes(FMT, D);
  const uint8_t *codes = unit + (is_v ? CB : 0) + (is_v ? v_octet<GS, D>(o, r) : k_octet<GS>(o, r));
  const uint8_t *scales = unit + 2 * CB + (is_v ? SB : 0);
  if constexpr (FMT == A_BF16) {
    unpack8(*reinterpret_cast<const uint4 *>(codes), f);
  } else if constexpr (FMT == A_FP8) {
    const uint2 w = *reinterpret_cast<const uint2 *>(codes);
    const float s = reinterpret_cast<const float *>(scales)[r];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(e4m3_to_f32(((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xFFu), s);
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(codes);
    const int b = o >> 1;
    const float s = e4m3_to_f32(scales[is_v ? b * 16 + r : r * (D / 16) + (b & 1) * (D / 32) + (b >> 1)]);
    const float g = glob[is_v ? 1 : 0];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(__fmul_rn(e2m1_to_f32((w >> (4 * i)) & 15u), s), g);
  }
}

// Eight channels from octet o of a row, rotated (rot > 0) in fp32.
__device__ __forceinline__ void rope_octet(const uint16_t *x, int o, int rot, int inter, const float *tab, float *f) {
  unpack8(*reinterpret_cast<const uint4 *>(x + 8 * o), f);
  const int half = rot / 2;
  if (8 * o >= rot) return;
  if ((rot & 15) == 0 && !inter) {
    const bool second = 8 * o >= half;
    float p[8], co[8], si[8], u;
    unpack8(*reinterpret_cast<const uint4 *>(x + (second ? 8 * o - half : 8 * o + half)), p);
    const float *t = tab + (second ? 8 * o - half : 8 * o);
    load8(t, co);
    load8(t + half, si);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (second) rope_pair(p[i], f[i], co[i], si[i], u, f[i]);
      else rope_pair(f[i], p[i], co[i], si[i], f[i], u);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ch = 8 * o + i;
    if (ch >= rot) break;
    const int j = inter ? ch >> 1 : (ch < half ? ch : ch - half);
    const bool second = inter ? (ch & 1) : ch >= half;
    const float mine = bf16_at(x + ch), other = bf16_at(x + (inter ? ch ^ 1 : second ? ch - half : ch + half));
    float u, v;
    if (second) rope_pair(other, mine, tab[j], tab[half + j], u, v);
    else rope_pair(mine, other, tab[j], tab[half + j], v, u);
    f[i] = v;
  }
}

struct KvRows {
  int T;
  const uint16_t *k, *v;
  long long ks, vs;         // strides between tokens, elements
  const long long *slots;
  uint16_t *k_out, *v_out;  // read back
};

template <int D>
__host__ __device__ constexpr int kv_lpr() { return D == 64 ? 8 : D == 128 ? 16 : 32; }

// LPR lanes per (token, head): each takes one octet of the key and one of the
// value.  Blocks past `kv_blocks` rotate the rope.H heads of q.
template <int FMT, int D>
__global__ void __launch_bounds__(256) kv_write_kernel(KvArgs a, KvRows w, RopeArgs rope, int kv_blocks) {
  if (blockIdx.x >= kv_blocks) {
    rope_rows(rope, (blockIdx.x - kv_blocks) * (size_t)blockDim.x + threadIdx.x,
              (size_t)(gridDim.x - kv_blocks) * blockDim.x);
    return;
  }
  constexpr int LPR = kv_lpr<D>();
  const int o = threadIdx.x % LPR;
  const bool on = o < D / 8;
  const size_t rows = (size_t)w.T * a.H, step = (size_t)kv_blocks * (256 / LPR);
  // whole warps stay together for the shuffles: a row past the end is clamped and not stored
  for (size_t base = blockIdx.x * (size_t)(256 / LPR); base < rows; base += step) {
    const size_t row = base + threadIdx.x / LPR;
    const size_t t = (row < rows ? row : rows - 1) / a.H;
    const int h = (int)((row < rows ? row : rows - 1) % a.H);
    const long long slot = w.slots[t];
    bool ok = row < rows && slot >= 0;
    const float *tab = nullptr;
    if (ok && slot >= a.slots_total) {
      set_device_error(HQ_ERR_DEVICE_INDEX);
      ok = false;
    }
    if (ok && rope.rot) {
      const int p = rope.pos[t];
      if (p < 0 || p >= rope.P) {
        set_device_error(HQ_ERR_DEVICE_INDEX);
        ok = false;
      } else {
        tab = rope.table + (size_t)p * rope.rot;
      }
    }
    float fk[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, fv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (ok && on) {
      const uint16_t *kr = w.k + t * w.ks + (size_t)h * D;
      if (rope.rot) rope_octet(kr, o, rope.rot, rope.inter, tab, fk);
      else unpack8(*reinterpret_cast<const uint4 *>(kr + 8 * o), fk);
      unpack8(*reinterpret_cast<const uint4 *>(w.v + t * w.vs + (size_t)h * D + 8 * o), fv);
    }
    int r = 0;
    uint8_t *unit = ok ? kv_unit<FMT, D>(a, slot, h, r) : a.pages;
    // the lanes of a row that is not stored still take part in the shuffles
    if (__any_sync(0xffffffffu, ok)) {
      kv_store<FMT, D, LPR>(unit, r, o, ok && on, false, fk, a.glob);
      kv_store<FMT, D, LPR>(unit, r, o, ok && on, true, fv, a.glob);
    }
  }
}

template <int FMT, int D>
__global__ void __launch_bounds__(256) kv_read_kernel(KvArgs a, KvRows w) {
  constexpr int LPR = kv_lpr<D>();
  const int o = threadIdx.x % LPR;
  if (o >= D / 8) return;
  const size_t rows = (size_t)w.T * a.H, step = (size_t)gridDim.x * (256 / LPR);
  for (size_t row = blockIdx.x * (size_t)(256 / LPR) + threadIdx.x / LPR; row < rows; row += step) {
    const size_t t = row / a.H;
    const int h = (int)(row % a.H);
    const long long slot = w.slots[t];
    if (slot < 0) continue;
    if (slot >= a.slots_total) {
      set_device_error(HQ_ERR_DEVICE_INDEX);
      continue;
    }
    int r;
    const uint8_t *unit = kv_unit<FMT, D>(a, slot, h, r);
    float f[8];
    if (w.k_out) {
      kv_load<FMT, D>(unit, r, o, false, a.glob, f);
      *reinterpret_cast<uint4 *>(w.k_out + t * w.ks + (size_t)h * D + 8 * o) = pack8(f);
    }
    if (w.v_out) {
      kv_load<FMT, D>(unit, r, o, true, a.glob, f);
      *reinterpret_cast<uint4 *>(w.v_out + t * w.vs + (size_t)h * D + 8 * o) = pack8(f);
    }
  }
}

// The activation-format constant of a cache description; false if it is not
// one that is built.
bool kv_format(const hq_kv_desc *d, int *fmt) {
  switch (d->dtype) {
    case HQ_BF16: *fmt = A_BF16; break;
    case HQ_E4M3: *fmt = A_FP8; break;
    case HQ_NVFP4: *fmt = A_NVFP4; break;
    default: return false;
  }
  return d->head_dim == 64 || d->head_dim == 128 || d->head_dim == 192 || d->head_dim == 256;
}

size_t kv_page_bytes(const hq_kv_desc *d, int fmt) {
  return (size_t)d->heads * (d->page_size / 16) * kv_unit_bytes(fmt, d->head_dim);
}

KvArgs kv_args(const hq_kv_desc *d, int fmt, int num_pages, const void *pages, const float *glob) {
  KvArgs a{};
  a.H = d->heads;
  a.page = d->page_size;
  a.page_units = d->page_size / 16;
  a.slots_total = (long long)num_pages * d->page_size;
  a.page_bytes = kv_page_bytes(d, fmt);
  a.pages = (uint8_t *)const_cast<void *>(pages);
  a.glob = glob;
  return a;
}

template <class F>
static hq_status kv_dispatch(int fmt, int D, F &&f) {
#define HQ_KV_CASE(FM, DD) \
  if (fmt == FM && D == DD) return f(std::integral_constant<int, FM>{}, std::integral_constant<int, DD>{});
#define HQ_KV_DIMS(FM) HQ_KV_CASE(FM, 64) HQ_KV_CASE(FM, 128) HQ_KV_CASE(FM, 192) HQ_KV_CASE(FM, 256)
  HQ_KV_DIMS(A_BF16)
  HQ_KV_DIMS(A_FP8)
  HQ_KV_DIMS(A_NVFP4)
#undef HQ_KV_DIMS
#undef HQ_KV_CASE
  return HQ_ERR_UNSUPPORTED;
}

hq_status launch_kv_write(int fmt, int D, const KvArgs &a, const KvRows &w, const RopeArgs &rope, cudaStream_t st) {
  return kv_dispatch(fmt, D, [&](auto F, auto DD) {
    const int kb = quant_grid((size_t)w.T * a.H * kv_lpr<DD>(), 256);
    const int qb = rope.H ? quant_grid((size_t)rope.T * rope.H * rope_chunks(rope.D, rope.rot), 256) : 0;
    kv_write_kernel<F, DD><<<kb + qb, 256, 0, st>>>(a, w, rope, kb);
    return check_launch();
  });
}

hq_status launch_kv_read(int fmt, int D, const KvArgs &a, const KvRows &w, cudaStream_t st) {
  return kv_dispatch(fmt, D, [&](auto F, auto DD) {
    kv_read_kernel<F, DD><<<quant_grid((size_t)w.T * a.H * kv_lpr<DD>(), 256), 256, 0, st>>>(a, w);
    return check_launch();
  });
}

}  // namespace hq

// Rotary positions in the layouts and scalings of pkv_rotary_spec, with the
// append of the rotated key and the value (pkv_rotary_append).
//
// Mathematics.  Pair i of a head at position p turns by p * f_i; f_i is made
// once on the host in double precision (pkv_rotary_init) and kept as a 64-bit
// fraction of a turn, so p * f_i mod 1 is one exact wrapping product for any
// 32-bit position, signed ones included, and only the reduced angle is rounded
// to float32.
//
// What bounds it: memory.  A token's rows are read and written once.  Two kernels:
// rotary_kernel moves 16-byte pieces and gives every thread the same place in head
// after head, so that a loop step costs no division; rotary_any_kernel takes any
// even sizes, strides and alignment an element at a time.
#include <cmath>
#include <cstdint>

#include "common.cuh"

namespace pkv {
namespace {

constexpr uint32_t kRotaryCheck = 0x526f7431u;
constexpr int kThreads = 256;

struct RotaryParams {
  const void *q, *k, *v;
  void *q_out, *k_out, *k_cache, *v_cache;
  const int32_t *positions;
  const int64_t *slots;
  int32_t *err;
  long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride, num_slots;
  int T, Hq, Hkv, d, rot, tb;   // tb: tokens per CTA
  int per_head;                 // rotary_kernel: 2 x 16-byte items of a head
  float amplitude;
  unsigned long long turns[128];
};

// The angles of the CTA's tokens, amplitude * (cos, sin): cs [tokens][rot/2], or with
// VEC > 1 [tokens][VEC/2][rot/2/VEC][2], so that threads of neighbouring items (VEC
// pairs each) read two pairs from neighbouring 16 bytes (pair after pair, eight
// threads met in the same banks four times over).
template <int VEC>
__device__ __forceinline__ void fill_angles(const RotaryParams &p, float2 *cs, int t0, int nt) {
  const int half = p.rot >> 1;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, c = i - t * half;
    const unsigned long long ph =
        static_cast<unsigned long long>(static_cast<long long>(p.positions[t0 + t])) * p.turns[c];
    float s, co;
    // the signed fraction of a turn times 2 pi / 2^64
    sincosf(static_cast<float>(static_cast<long long>(ph)) * 3.4061215800865545e-19f, &s, &co);
    const int at = VEC == 1 ? i : 2 * ((t * (VEC / 2) + c % VEC / 2) * (half / VEC) + c / VEC) + c % 2;
    cs[at] = make_float2(co * p.amplitude, s * p.amplitude);
  }
  if (p.slots && threadIdx.x < nt && p.slots[t0 + threadIdx.x] >= p.num_slots)
    set_dev_err(p.err, PKV_DEVERR_BAD_SLOT);
}

// The pairs of one item turned in place; w[i * step] holds the (cos, sin) of pairs 2i
// and 2i + 1.
template <typename T, bool IL>
__device__ __forceinline__ void rotate_item(uint4 &a, uint4 &b, const float4 *w, int step) {
  uint32_t *x = &a.x, *y = &b.x;
  if constexpr (sizeof(T) == 2) {   // a word holds two elements
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 c = w[i * step];
      float u1, u2, v1, v2;
      if constexpr (IL) {   // a pair is a word: the first four in a, the others in b
        uint32_t *p = i < 2 ? x + 2 * i : y + (2 * i - 4);
        rope_rotate(bf16_lo(p[0]), bf16_hi(p[0]), c.x, c.y, &u1, &u2);
        rope_rotate(bf16_lo(p[1]), bf16_hi(p[1]), c.z, c.w, &v1, &v2);
        p[0] = pack_bf16(u1, u2);
        p[1] = pack_bf16(v1, v2);
      } else {
        rope_rotate(bf16_lo(x[i]), bf16_lo(y[i]), c.x, c.y, &u1, &u2);
        rope_rotate(bf16_hi(x[i]), bf16_hi(y[i]), c.z, c.w, &v1, &v2);
        x[i] = pack_bf16(u1, v1);
        y[i] = pack_bf16(u2, v2);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 c = w[i * step];
      float *p = reinterpret_cast<float *>(x), *q = reinterpret_cast<float *>(y);
      if constexpr (IL) {
        float *r = i == 0 ? p : q;
        rope_rotate(r[0], r[1], c.x, c.y, &r[0], &r[1]);
        rope_rotate(r[2], r[3], c.z, c.w, &r[2], &r[3]);
      } else {
        rope_rotate(p[2 * i], q[2 * i], c.x, c.y, &p[2 * i], &q[2 * i]);
        rope_rotate(p[2 * i + 1], q[2 * i + 1], c.z, c.w, &p[2 * i + 1], &q[2 * i + 1]);
      }
    }
  }
}

// A CTA serves tb tokens.  An item is two 16-byte pieces of one head of one token: of
// a query or key head the two halves of VEC rotating pairs or 2 VEC elements behind
// them, of a value head (after the key heads) 2 VEC elements.  Every head has
// per_head items; a thread keeps its item number c within the head and goes through
// the CTA's (token, head) pairs kThreads / per_head at a time, kBatch of them with
// their loads in flight together; the first batch's go out before the angles are
// formed.  16384 tokens of 32 + 8 heads of 128 in bf16, whole heads turned: 64 us, 6.3
// TB/s (float32 119 us, 6.8 TB/s); four pairs at a time, with fewer CTAs on an SM, took
// 5 % longer.
template <typename T, bool IL>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  extern __shared__ float2 cs[];
  constexpr int VEC = 16 / static_cast<int>(sizeof(T)), kBatch = 2;
  pdl_wait();
  const int t0 = blockIdx.x * p.tb, nt = min(p.tb, p.T - t0);
  const int half = p.rot >> 1, H = p.Hq + p.Hkv, heads = H + (p.slots ? p.Hkv : 0);
  const int c = threadIdx.x % p.per_head, first = threadIdx.x / p.per_head;
  const int stride = kThreads / p.per_head;
  const bool rot = c < half / VEC;
  const int off = rot ? (IL ? 2 * VEC * c : VEC * c) : p.rot + 2 * VEC * (c - half / VEC);
  const int gap = rot && !IL ? half : VEC;
  const int voff = 2 * VEC * c;   // of a value head
  int t = 0, h = first < stride ? first : heads;   // (threads behind the last whole head: none)
  if (first >= stride) t = nt;
  auto settle = [&]() {
    while (h >= heads && t < nt) {
      h -= heads;
      ++t;
    }
  };
  settle();
  uint4 a[kBatch], b[kBatch];
  // loads of up to kBatch pairs from (t, h) on; returns how many
  auto load_batch = [&](int lt, int lh) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (lt < nt) {
        const long long tok = t0 + lt;
        const T *src;
        int g = gap;
        if (lh < p.Hq) {
          src = static_cast<const T *>(p.q) + tok * p.q_stride + lh * p.d + off;
        } else if (lh < H) {
          src = static_cast<const T *>(p.k) + tok * p.k_stride + (lh - p.Hq) * p.d + off;
        } else {
          src = static_cast<const T *>(p.v) + tok * p.v_stride + (lh - H) * p.d + voff;
          g = VEC;
        }
        a[u] = *reinterpret_cast<const uint4 *>(src);
        b[u] = *reinterpret_cast<const uint4 *>(src + g);
        lh += stride;
        while (lh >= heads && lt < nt) {
          lh -= heads;
          ++lt;
        }
      }
    }
  };
  load_batch(t, h);
  fill_angles<VEC>(p, cs, t0, nt);
  __syncthreads();
  bool again = false;
  while (t < nt) {
    if (again) load_batch(t, h);
    again = true;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (t < nt) {
        const long long tok = t0 + t;
        if (rot && h < H)
          rotate_item<T, IL>(a[u], b[u],
                             reinterpret_cast<const float4 *>(cs + t * half) + c, half / VEC);
        if (h < p.Hq) {
          T *dst = static_cast<T *>(p.q_out) + tok * p.q_out_stride + h * p.d + off;
          *reinterpret_cast<uint4 *>(dst) = a[u];
          *reinterpret_cast<uint4 *>(dst + gap) = b[u];
        } else {
          const bool val = h >= H;
          if (!val && p.k_out) {
            T *dst = static_cast<T *>(p.k_out) + tok * p.k_out_stride + (h - p.Hq) * p.d + off;
            *reinterpret_cast<uint4 *>(dst) = a[u];
            *reinterpret_cast<uint4 *>(dst + gap) = b[u];
          }
          const long long slot = p.slots ? p.slots[tok] : -1;
          if (slot >= 0 && slot < p.num_slots) {
            const long long blk = slot / kBlockTokens;
            const size_t row = (static_cast<size_t>(blk) * p.Hkv + (h - (val ? H : p.Hq))) *
                                   kBlockTokens + static_cast<size_t>(slot - blk * kBlockTokens);
            T *dst = static_cast<T *>(val ? p.v_cache : p.k_cache) + row * p.d + (val ? voff : off);
            *reinterpret_cast<uint4 *>(dst) = a[u];
            *reinterpret_cast<uint4 *>(dst + (val ? VEC : gap)) = b[u];
          }
        }
        h += stride;
        settle();
      }
    }
  }
}

// Any even sizes, an element at a time.  A CTA serves tb tokens; an item is a pair of
// elements of one head: a rotating pair, or two neighbours behind the pairs or in a
// value head.  Bound by its instructions (an element a load, the divisions of an item):
// 16384 tokens of 32 + 8 heads of 80, 20 rotated: 153 us in bf16 (1.6 TB/s), 151 us in
// float32 (3.3 TB/s).
template <typename T, bool IL>
__global__ void __launch_bounds__(kThreads) rotary_any_kernel(
    const __grid_constant__ RotaryParams p) {
  extern __shared__ float2 cs[];
  pdl_wait();
  const int t0 = blockIdx.x * p.tb, nt = min(p.tb, p.T - t0);
  const int half = p.rot >> 1, pairs = p.d >> 1;
  const int H = p.Hq + p.Hkv, heads = H + (p.slots ? p.Hkv : 0);
  fill_angles<1>(p, cs, t0, nt);
  __syncthreads();
  for (int e = threadIdx.x; e < nt * heads * pairs; e += kThreads) {
    const int t = e / (heads * pairs), r = e - t * heads * pairs, h = r / pairs, i = r - h * pairs;
    const long long tok = t0 + t;
    const bool val = h >= H, rot = !val && i < half;
    const int o1 = rot && !IL ? i : 2 * i, o2 = rot && !IL ? half + i : 2 * i + 1;
    const T *src = h < p.Hq ? static_cast<const T *>(p.q) + tok * p.q_stride + h * p.d
                   : !val   ? static_cast<const T *>(p.k) + tok * p.k_stride + (h - p.Hq) * p.d
                            : static_cast<const T *>(p.v) + tok * p.v_stride + (h - H) * p.d;
    T x1 = src[o1], x2 = src[o2];
    if (rot) {
      const float2 w = cs[t * half + i];
      float y1, y2;
      rope_rotate(to_f32(x1), to_f32(x2), w.x, w.y, &y1, &y2);
      x1 = from_f32<T>(y1);
      x2 = from_f32<T>(y2);
    }
    T *dst = h < p.Hq          ? static_cast<T *>(p.q_out) + tok * p.q_out_stride + h * p.d
             : !val && p.k_out ? static_cast<T *>(p.k_out) + tok * p.k_out_stride + (h - p.Hq) * p.d
                               : nullptr;
    if (dst) {
      dst[o1] = x1;
      dst[o2] = x2;
    }
    if (h >= p.Hq && p.slots) {
      const long long slot = p.slots[tok];
      if (slot >= 0 && slot < p.num_slots) {
        const long long blk = slot / kBlockTokens;
        const size_t row = (static_cast<size_t>(blk) * p.Hkv + (h - (val ? H : p.Hq))) *
                               kBlockTokens + static_cast<size_t>(slot - blk * kBlockTokens);
        T *to = static_cast<T *>(val ? p.v_cache : p.k_cache) + row * p.d;
        to[o1] = x1;
        to[o2] = x2;
      }
    }
  }
}

template <typename T>
cudaError_t launch(const RotaryParams &p, bool wide, bool il, unsigned grid, size_t smem,
                   cudaStream_t s) {
  auto kern = wide ? (il ? rotary_kernel<T, true> : rotary_kernel<T, false>)
                   : (il ? rotary_any_kernel<T, true> : rotary_any_kernel<T, false>);
  return launch_waiting(kern, grid, kThreads, smem, s, p);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_rotary_init(const pkv_rotary_spec *s, int32_t d, pkv_rotary *out) {
  clear_error();
  PKV_REQUIRE(s && out, PKV_ERR_INVALID_ARG, "NULL argument");
  PKV_REQUIRE(d >= 2 && d <= 256 && d % 2 == 0, PKV_ERR_UNSUPPORTED, "head_dim %d", d);
  const int r = s->rot_dim;
  PKV_REQUIRE(r >= 2 && r <= d && r % 2 == 0, PKV_ERR_INVALID_ARG,
              "rot_dim %d must be even, in [2, %d]", r, d);
  PKV_REQUIRE(s->layout == PKV_ROTARY_HALF || s->layout == PKV_ROTARY_INTERLEAVED,
              PKV_ERR_UNSUPPORTED, "layout %d", s->layout);
  PKV_REQUIRE(s->scaling >= PKV_ROTARY_PLAIN && s->scaling <= PKV_ROTARY_BANDS,
              PKV_ERR_UNSUPPORTED, "scaling %d", s->scaling);
  PKV_REQUIRE(s->base >= 1.0 && std::isfinite(s->base), PKV_ERR_INVALID_ARG, "base must be >= 1");
  const float amplitude = static_cast<float>(s->amplitude);
  PKV_REQUIRE(amplitude > 0.f && std::isfinite(amplitude), PKV_ERR_INVALID_ARG,
              "amplitude must be positive and finite in float32");
  PKV_REQUIRE(s->scaling == PKV_ROTARY_PLAIN || (s->factor >= 1.0 && std::isfinite(s->factor)),
              PKV_ERR_INVALID_ARG, "factor must be >= 1");
  double base = s->base;
  if (s->scaling == PKV_ROTARY_NTK) {
    PKV_REQUIRE(r > 2, PKV_ERR_INVALID_ARG, "this scaling needs rot_dim > 2");
    base *= std::pow(s->factor, static_cast<double>(r) / (r - 2));
    PKV_REQUIRE(std::isfinite(base), PKV_ERR_INVALID_ARG, "factor too large");
  }
  const double two_pi = 2.0 * 3.141592653589793238462643383279502884;
  const double N = s->original_len;
  double lo = 0.0, hi = 0.0;
  if (s->scaling == PKV_ROTARY_RAMP || s->scaling == PKV_ROTARY_BANDS) {
    PKV_REQUIRE(s->original_len > 0, PKV_ERR_INVALID_ARG, "original_len must be positive");
    PKV_REQUIRE(s->low > 0.0 && s->high > s->low && std::isfinite(s->high), PKV_ERR_INVALID_ARG,
                "0 < low < high must hold");
  }
  if (s->scaling == PKV_ROTARY_RAMP) {
    PKV_REQUIRE(base > 1.0, PKV_ERR_INVALID_ARG, "this scaling needs base > 1");
    lo = std::fmax(0.0, std::floor(r * std::log(N / (two_pi * s->high)) / (2 * std::log(base))));
    hi = std::fmin(r - 1.0, std::ceil(r * std::log(N / (two_pi * s->low)) / (2 * std::log(base))));
  }
  for (int i = 0; i < r / 2; ++i) {
    const double g = std::pow(base, -2.0 * i / static_cast<double>(r));
    double f = g;
    if (s->scaling == PKV_ROTARY_LINEAR) {
      f = g / s->factor;
    } else if (s->scaling == PKV_ROTARY_RAMP) {
      const double w = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 0.001)));
      f = g * (1.0 - w) + g / s->factor * w;
    } else if (s->scaling == PKV_ROTARY_BANDS) {
      const double t = N * g / two_pi;
      const double w = std::fmin(1.0, std::fmax(0.0, (t - s->low) / (s->high - s->low)));
      f = g * w + g / s->factor * (1.0 - w);
    }
    out->turns[i] = static_cast<uint64_t>(std::ldexp(f / two_pi, 64));   // f <= 1
  }
  for (int i = r / 2; i < 128; ++i) out->turns[i] = 0;
  out->d = d;
  out->rot_dim = r;
  out->layout = s->layout;
  out->amplitude = amplitude;
  out->check = kRotaryCheck;
  return PKV_OK;
}

extern "C" int pkv_rotary_append(const pkv_rotary_args *a, void *stream) {
  clear_error();
  PKV_REQUIRE(a && a->rotary, PKV_ERR_INVALID_ARG, "NULL argument");
  const pkv_rotary &r = *a->rotary;
  PKV_REQUIRE(r.check == kRotaryCheck, PKV_ERR_INVALID_ARG,
              "rotary was not filled by pkv_rotary_init");
  PKV_REQUIRE(a->T >= 0 && a->Hq >= 0 && a->Hkv >= 0, PKV_ERR_INVALID_ARG, "negative size");
  PKV_REQUIRE(dtype_ok(a->dtype), PKV_ERR_UNSUPPORTED, "dtype %d", a->dtype);
  PKV_REQUIRE(a->d == r.d, PKV_ERR_INVALID_ARG, "head_dim %d, but rotary was made for %d", a->d,
              r.d);
  PKV_REQUIRE(a->Hq <= 65536 && a->Hkv <= 65536, PKV_ERR_UNSUPPORTED, "too many heads");
  if (a->T == 0 || a->Hq + a->Hkv == 0) return PKV_OK;
  const bool append = a->slot_mapping != nullptr && a->Hkv > 0;
  PKV_REQUIRE(a->positions, PKV_ERR_INVALID_ARG, "positions is NULL");
  PKV_REQUIRE(a->Hq == 0 || (a->q && a->q_out), PKV_ERR_INVALID_ARG, "NULL query tensor");
  PKV_REQUIRE(a->Hkv == 0 || (a->k && (a->k_out || append)), PKV_ERR_INVALID_ARG,
              "NULL key tensor");
  const long long qrow = static_cast<long long>(a->Hq) * a->d;
  const long long krow = static_cast<long long>(a->Hkv) * a->d;
  PKV_REQUIRE(a->Hq == 0 || a->T == 1 || (a->q_stride >= qrow && a->q_out_stride >= qrow),
              PKV_ERR_INVALID_ARG, "a query token's heads overlap the next token's");
  PKV_REQUIRE(a->Hkv == 0 || a->T == 1 ||
                  (a->k_stride >= krow && (!a->k_out || a->k_out_stride >= krow) &&
                   (!append || a->v_stride >= krow)),
              PKV_ERR_INVALID_ARG, "a key or value token's heads overlap the next token's");
  PKV_REQUIRE((a->Hq == 0 || a->q != a->q_out || a->T == 1 || a->q_stride == a->q_out_stride) &&
                  (a->Hkv == 0 || !a->k_out || a->k != a->k_out || a->T == 1 ||
                   a->k_stride == a->k_out_stride),
              PKV_ERR_INVALID_ARG, "in place needs equal strides");
  const int elem = static_cast<int>(dtype_size(a->dtype));
  {
    // outputs may be their own inputs, and overlap nothing else
    const long long qs = a->q_stride * elem, ks = a->k_stride * elem, vs = a->v_stride * elem,
                    qos = a->q_out_stride * elem, kos = a->k_out_stride * elem;
    const long long ql = qrow * elem, kl = krow * elem, vl = append ? kl : 0,
                    kol = a->k_out ? kl : 0, T = a->T;
    const bool clash =
        (a->q_out != a->q && rows_overlap(a->q_out, qos, ql, a->q, qs, ql, T)) ||
        rows_overlap(a->q_out, qos, ql, a->k, ks, kl, T) ||
        rows_overlap(a->q_out, qos, ql, a->v, vs, vl, T) ||
        rows_overlap(a->q_out, qos, ql, a->k_out, kos, kol, T) ||
        (a->k_out != a->k && rows_overlap(a->k_out, kos, kol, a->k, ks, kl, T)) ||
        rows_overlap(a->k_out, kos, kol, a->q, qs, ql, T) ||
        rows_overlap(a->k_out, kos, kol, a->v, vs, vl, T);
    PKV_REQUIRE(!clash, PKV_ERR_INVALID_ARG, "an output overlaps another tensor");
  }
  const uintptr_t cache_addr =
      append ? reinterpret_cast<uintptr_t>(a->k_cache) | reinterpret_cast<uintptr_t>(a->v_cache) : 0;
  if (append) {
    PKV_REQUIRE(a->v && a->k_cache && a->v_cache && a->num_blocks >= 0, PKV_ERR_INVALID_ARG,
                "NULL append argument");
    PKV_REQUIRE(a->d * elem % 16 == 0 && cache_addr % 16 == 0, PKV_ERR_INVALID_ARG,
                "append needs 16-byte rows and 16-byte aligned caches");
    const long long bytes = static_cast<long long>(a->num_blocks) * kBlockTokens * krow * elem;
    PKV_REQUIRE(!rows_overlap(a->k_cache, 0, bytes, a->v_cache, 0, bytes, 1), PKV_ERR_INVALID_ARG,
                "the caches overlap");
  }
  uintptr_t addr = 0;
  long long strides = 0;
  if (a->Hq) {
    addr |= reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->q_out);
    strides |= a->T > 1 ? a->q_stride | a->q_out_stride : 0;
  }
  if (a->Hkv) {
    addr |= reinterpret_cast<uintptr_t>(a->k);
    strides |= a->T > 1 ? a->k_stride : 0;
    if (a->k_out) {
      addr |= reinterpret_cast<uintptr_t>(a->k_out);
      strides |= a->T > 1 ? a->k_out_stride : 0;
    }
    if (append) {
      addr |= reinterpret_cast<uintptr_t>(a->v);
      strides |= a->T > 1 ? a->v_stride : 0;
    }
  }
  PKV_REQUIRE(addr % elem == 0, PKV_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  const int vec16 = 16 / elem;
  // whole 16-byte items in every head
  const bool wide = addr % 16 == 0 && strides % vec16 == 0 && r.rot_dim % (2 * vec16) == 0 &&
                    a->d % (2 * vec16) == 0;
  RotaryParams p;
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.q_out = a->q_out;
  p.k_out = a->k_out;
  p.k_cache = a->k_cache;
  p.v_cache = a->v_cache;
  p.positions = a->positions;
  p.slots = append ? a->slot_mapping : nullptr;
  p.err = a->dev_err_flag;
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.v_stride = a->v_stride;
  p.q_out_stride = a->q_out_stride;
  p.k_out_stride = a->k_out_stride;
  p.num_slots = append ? static_cast<long long>(a->num_blocks) * kBlockTokens : 0;
  p.T = a->T;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.d = a->d;
  p.rot = r.rot_dim;
  p.amplitude = r.amplitude;
  for (int i = 0; i < 128; ++i) p.turns[i] = r.turns[i];
  p.per_head = a->d / (2 * vec16);
  const int heads = a->Hq + a->Hkv + (append ? a->Hkv : 0);
  // tokens per CTA: one while the tokens do not fill the GPU twice over, else
  // enough for kItems items a thread (4 to 8 measure alike, 16 loses 10 %)
  constexpr long long kItems = 6;
  const long long items = static_cast<long long>(heads) * (wide ? p.per_head : a->d / 2);
  long long tb = kItems * kThreads / items;
  if (tb < 1 || a->T <= 304) tb = 1;
  if (tb > 16) tb = 16;
  p.tb = static_cast<int>(tb);
  const unsigned grid = static_cast<unsigned>((a->T + tb - 1) / tb);
  const size_t smem = static_cast<size_t>(tb) * (r.rot_dim / 2) * sizeof(float2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool il = r.layout == PKV_ROTARY_INTERLEAVED;
  const cudaError_t e = a->dtype == PKV_BF16 ? launch<__nv_bfloat16>(p, wide, il, grid, smem, s)
                                             : launch<float>(p, wide, il, grid, smem, s);
  PKV_REQUIRE(e == cudaSuccess, PKV_ERR_CUDA, "rotary_kernel launch: %s", cudaGetErrorString(e));
  return PKV_OK;
}

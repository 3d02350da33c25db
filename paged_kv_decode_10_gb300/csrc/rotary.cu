// Rotary positions in the layouts and scalings of pkv_rotary_spec, with the
// append of the rotated key and the value (pkv_rotary_append).
//
// Mathematics.  Pair i of a head at position p turns by p * f_i; f_i is made
// once on the host in double precision (pkv_rotary_init) and kept as a 64-bit
// fraction of a turn, so p * f_i mod 1 is one exact wrapping product for any
// 32-bit position, signed ones included, and only the reduced angle is rounded
// to float32.
//
// What bounds it: memory.  A token's rows are read and written once.
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
  float amplitude;
  unsigned long long turns[128];
};

// VEC elements moved by one load or store (16 bytes, or one element where
// sizes, strides or addresses do not allow that).
template <typename T, int VEC>
struct Piece {
  T e[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Piece<T, VEC> load_piece(const T *p) {
  Piece<T, VEC> r;
  if constexpr (VEC == 1) {
    r.e[0] = *p;
  } else {
    static_assert(sizeof(r) == 16, "16-byte pieces");
    *reinterpret_cast<uint4 *>(r.e) = *reinterpret_cast<const uint4 *>(p);
  }
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void store_piece(T *p, const Piece<T, VEC> &r) {
  if constexpr (VEC == 1)
    *p = r.e[0];
  else
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(r.e);
}

// A CTA serves tb tokens.  Its work is a list of items: per token and q or k
// head, the head's rotated pairs VEC at a time (two pieces), then the elements
// behind them two pieces at a time; then, when appending, the values two pieces
// at a time.  A thread takes every kThreads-th item, kBatch of them at once so
// that their loads are in flight together; the first batch's go out before the
// angles are formed.
template <typename T, int VEC, bool IL>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  extern __shared__ float2 cs[];   // [tb][rot/2] (cos, sin), times the amplitude
  constexpr int kBatch = 4;
  using P = Piece<T, VEC>;
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * p.tb;
  const int nt = min(p.tb, p.T - t0);
  const int half = p.rot >> 1;
  const int rc = half / VEC;                          // rotating items of a head
  const int tc = ((p.d - p.rot) / VEC + 1) / 2;       // items of the rest of a head
  const int vc = p.slots ? (p.d / VEC + 1) / 2 : 0;   // items of a value head
  const int per_head = rc + tc, H = p.Hq + p.Hkv;
  const int per_token = H * per_head + p.Hkv * vc;
  const int items = nt * per_token;

  struct Item {
    const T *src;      // first piece
    int t, h, off, gap;   // token, head (H + value head), element offset, second piece's distance
    bool two, rot;
  };
  auto item_of = [&](int e) {
    Item it;
    it.t = e / per_token;
    int r = e - it.t * per_token;
    const long long t = t0 + it.t;
    int c;
    if (r < H * per_head) {
      it.h = r / per_head;
      c = r - it.h * per_head;
      const T *head = it.h < p.Hq
                          ? static_cast<const T *>(p.q) + t * p.q_stride + it.h * p.d
                          : static_cast<const T *>(p.k) + t * p.k_stride + (it.h - p.Hq) * p.d;
      it.rot = c < rc;
      if (it.rot) {
        it.off = IL ? 2 * VEC * c : VEC * c;
        it.gap = IL ? VEC : half;
        it.two = true;
      } else {
        it.off = p.rot + 2 * VEC * (c - rc);
        it.gap = VEC;
        it.two = it.off + VEC < p.d;
      }
      it.src = head + it.off;
    } else {
      r -= H * per_head;
      const int hv = r / vc;
      it.h = H + hv;
      it.rot = false;
      it.off = 2 * VEC * (r - hv * vc);
      it.gap = VEC;
      it.two = it.off + VEC < p.d;
      it.src = static_cast<const T *>(p.v) + t * p.v_stride + hv * p.d + it.off;
    }
    return it;
  };
  P a[kBatch], b[kBatch];
  auto load_batch = [&](int e0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int e = e0 + u * kThreads;
      if (e < items) {
        const Item it = item_of(e);
        a[u] = load_piece<T, VEC>(it.src);
        if (it.two) b[u] = load_piece<T, VEC>(it.src + it.gap);
      }
    }
  };
  load_batch(tid);
  for (int i = tid; i < nt * half; i += kThreads) {
    const int t = i / half, c = i - t * half;
    const unsigned long long ph =
        static_cast<unsigned long long>(static_cast<long long>(p.positions[t0 + t])) * p.turns[c];
    float s, co;
    // the signed fraction of a turn times 2 pi / 2^64
    sincosf(static_cast<float>(static_cast<long long>(ph)) * 3.4061215800865545e-19f, &s, &co);
    cs[i] = make_float2(co * p.amplitude, s * p.amplitude);
  }
  if (p.slots && tid < nt && p.slots[t0 + tid] >= p.num_slots)
    set_dev_err(p.err, PKV_DEVERR_BAD_SLOT);
  __syncthreads();
  for (int e0 = tid; e0 < items; e0 += kBatch * kThreads) {
    if (e0 != tid) load_batch(e0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int e = e0 + u * kThreads;
      if (e >= items) break;
      const Item it = item_of(e);
      if (it.rot) {
        const float2 *w = cs + it.t * half + (IL ? it.off / 2 : it.off);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          T *x1, *x2;
          if constexpr (IL && VEC > 1) {   // pairs lie side by side across the two pieces
            x1 = 2 * i < VEC ? &a[u].e[(2 * i) % VEC] : &b[u].e[(2 * i) % VEC];
            x2 = x1 + 1;
          } else {
            x1 = &a[u].e[i];
            x2 = &b[u].e[i];
          }
          float y1, y2;
          const float2 c = w[i];
          rope_rotate(to_f32(*x1), to_f32(*x2), c.x, c.y, &y1, &y2);
          *x1 = from_f32<T>(y1);
          *x2 = from_f32<T>(y2);
        }
      }
      const long long t = t0 + it.t;
      if (it.h < H) {
        T *dst = it.h < p.Hq ? static_cast<T *>(p.q_out) + t * p.q_out_stride + it.h * p.d
                 : p.k_out   ? static_cast<T *>(p.k_out) + t * p.k_out_stride + (it.h - p.Hq) * p.d
                             : nullptr;
        if (dst) {
          store_piece<T, VEC>(dst + it.off, a[u]);
          if (it.two) store_piece<T, VEC>(dst + it.off + it.gap, b[u]);
        }
      }
      if (p.slots && it.h >= p.Hq) {
        const long long slot = p.slots[t];
        if (slot >= 0 && slot < p.num_slots) {
          const bool val = it.h >= H;
          const long long blk = slot / kBlockTokens;
          const size_t row = (static_cast<size_t>(blk) * p.Hkv + (it.h - (val ? H : p.Hq))) *
                                 kBlockTokens + static_cast<size_t>(slot - blk * kBlockTokens);
          T *dst = static_cast<T *>(val ? p.v_cache : p.k_cache) + row * p.d + it.off;
          store_piece<T, VEC>(dst, a[u]);
          if (it.two) store_piece<T, VEC>(dst + it.gap, b[u]);
        }
      }
    }
  }
}

template <typename T, int VEC>
void launch(const RotaryParams &p, bool il, unsigned grid, size_t smem, cudaStream_t s) {
  if (il)
    rotary_kernel<T, VEC, true><<<grid, kThreads, smem, s>>>(p);
  else
    rotary_kernel<T, VEC, false><<<grid, kThreads, smem, s>>>(p);
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
  PKV_REQUIRE(s->amplitude > 0.0 && std::isfinite(s->amplitude), PKV_ERR_INVALID_ARG,
              "amplitude must be positive");
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
  out->amplitude = static_cast<float>(s->amplitude);
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
  const uintptr_t cache_addr =
      append ? reinterpret_cast<uintptr_t>(a->k_cache) | reinterpret_cast<uintptr_t>(a->v_cache) : 0;
  if (append) {
    PKV_REQUIRE(a->v && a->k_cache && a->v_cache && a->num_blocks >= 0, PKV_ERR_INVALID_ARG,
                "NULL append argument");
    PKV_REQUIRE(a->d * elem % 16 == 0 && cache_addr % 16 == 0, PKV_ERR_INVALID_ARG,
                "append needs 16-byte rows and 16-byte aligned caches");
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
  const bool wide = addr % 16 == 0 && strides % vec16 == 0 && (r.rot_dim / 2) % vec16 == 0 &&
                    a->d % vec16 == 0;
  const int vec = wide ? vec16 : 1;
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
  // tokens per CTA: one while the tokens do not fill the GPU twice over, else
  // enough for about four items a thread
  const long long per_token =
      static_cast<long long>(a->Hq + a->Hkv) * (r.rot_dim / 2 / vec + ((a->d - r.rot_dim) / vec + 1) / 2) +
      (append ? static_cast<long long>(a->Hkv) * ((a->d / vec + 1) / 2) : 0);
  PKV_REQUIRE(per_token < (1 << 24), PKV_ERR_UNSUPPORTED, "too many heads");
  long long tb = 4 * kThreads / per_token;
  if (tb < 1 || a->T <= 304) tb = 1;
  if (tb > 16) tb = 16;
  p.tb = static_cast<int>(tb);
  const unsigned grid = static_cast<unsigned>((a->T + tb - 1) / tb);
  const size_t smem = static_cast<size_t>(tb) * (r.rot_dim / 2) * sizeof(float2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool il = r.layout == PKV_ROTARY_INTERLEAVED;
  if (a->dtype == PKV_BF16)
    wide ? launch<__nv_bfloat16, 8>(p, il, grid, smem, s)
         : launch<__nv_bfloat16, 1>(p, il, grid, smem, s);
  else
    wide ? launch<float, 4>(p, il, grid, smem, s) : launch<float, 1>(p, il, grid, smem, s);
  PKV_LAUNCH_CHECK("rotary_kernel");
  return PKV_OK;
}

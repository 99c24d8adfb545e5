// MXFP4 decode GEMV for gfx950.
//
// Format (OCP microscaling, 4-bit floats): a codes plane where byte j of a row
// holds code 2j in bits 0-3 and code 2j+1 in bits 4-7 (sign, two exponent bits,
// one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6), then a scales plane of one byte
// p for every 32 columns.  w = 2^(p - 127) * value(code); p = 255 is NaN.
//
// Lane mapping: a wave covers 4096 columns = 2048 code bytes of a row.  Lane l
// owns code bytes [16l, 16l+16) and [1024+16l, 1024+16l+16): two whole blocks,
// read by load instructions of 1 KB of consecutive bytes each (nontemporal: no
// other instruction reads their lines), plus the scale byte of each.  The codes
// are decoded by the conversion instructions of the format, two at a time and
// exactly, so a block's sum is that of the decoded values
//   t = sum value(code) x,   partial += 2^(p - 127 + e) t
// with e the lane's power of two (below), applied by one ldexp, which neither
// overflows nor loses bits where the result does not.  fp32 activations: one
// conversion for two weights, one FMA a weight.  fp16 and bf16: one conversion
// and one v_dot2_f32_f16 for two weights against the activations as fp16 (fp16
// as given, bf16 scaled per lane by 2^-e; exact, half_scale_exp).
//
// Bound: HBM at one and two rows (17/32 byte a weight): 18944 x 3584 with one fp32
// row takes 9.5 us (3.8 TB/s with the start and end of the launch).
#include "gemv_skeleton.h"

namespace qmv {

struct Mxfp4Policy {
  static constexpr int kColsPerWave = 64 * 64;
  static constexpr int kXElems = 64;
  // shared-activation GEMV: one-row tiles, three in flight (SxShape), as INT4
  static constexpr int kSxRows = 1, kSxTiles = 3;
  struct XSliceF32 {
    float v[64];  // v[32 h + k]: activation of column col[h] + k, scaled by 2^-e (f32_slice_factor)
    int e;
  };
  struct XSliceHalf {
    h2_t h[32];  // h[16 hf + i]: fp16 activations 2i and 2i + 1 of half hf
    int e;
  };
  template <typename XT>
  using XSliceT = typename XSliceFor<XT, XSliceF32, XSliceHalf>::type;
  struct Frag {
    uint4 q[2];
    uint32_t p[2];
  };

  const uint8_t* codes[2];
  const uint8_t* scales[2];
  uint32_t code_row, scale_row;
  int col[2];
  bool okh[2];

  __device__ Mxfp4Policy(const uint8_t* w, uint64_t scales_offset, int cols, int kslot, int lane) {
    code_row = static_cast<uint32_t>(cols) / 2;
    scale_row = static_cast<uint32_t>(cols) / 32;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int c = kslot * kColsPerWave + 2048 * h + 32 * lane;
      okh[h] = c < cols;
      if (!okh[h]) c = cols - 32;  // past the row end: read valid columns, x zeroed
      col[h] = c;
      codes[h] = w + c / 2;
      scales[h] = w + scales_offset + c / 32;
    }
  }

  template <class XS>
  __device__ void load_x_raw(const XS& x, uint4* raw) const {
    constexpr int kPer = 32 * static_cast<int>(sizeof(typename XS::elem)) / 16;
    qmv::load_x_raw<32>(x, col[0], raw);
    qmv::load_x_raw<32>(x, col[1], raw + kPer);
  }

  template <typename XT>
  __device__ void finish_x(const uint4* raw, XSliceT<XT>& s) const {
    if constexpr (__is_same(XT, float)) {
      x_to_f32<64>(raw, s.v, static_cast<const float*>(nullptr));
      float xs, un;
      const float f = f32_slice_factor<64>(s.v, true, xs, un);
      s.e = __builtin_amdgcn_frexp_expf(un) - 1;
#pragma unroll
      for (int k = 0; k < 64; ++k) s.v[k] = okh[k / 32] ? s.v[k] * f : 0.f;
    } else {
      // dword i of the raw row: activations 2i and 2i + 1, as the codes' pairs are
      auto word = [&](int i) {
        const uint32_t w = (i & 3) == 0 ? raw[i / 4].x : (i & 3) == 1 ? raw[i / 4].y : (i & 3) == 2 ? raw[i / 4].z : raw[i / 4].w;
        return okh[i / 16] ? w : 0u;
      };
      if constexpr (__is_same(XT, _Float16)) {
        s.e = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) s.h[i] = __builtin_bit_cast(h2_t, word(i));
      } else {
        uint32_t top = 0;  // largest magnitude, as bits
#pragma unroll
        for (int i = 0; i < 32; ++i) top = max(top, max((word(i) << 16) & 0x7FFFFFFFu, word(i) & 0x7FFF0000u));
        const float mx[1] = {__uint_as_float(top)};
        // (beside an infinity finite numbers must not become one: the largest power)
        s.e = mx[0] == __builtin_inff() ? 103 : half_scale_exp<XT, 1>(mx);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint32_t w = word(i);
          s.h[i] = h2_t{scaled_f16(__uint_as_float(w << 16), s.e), scaled_f16(__uint_as_float(w & 0xFFFF0000u), s.e)};
        }
      }
    }
  }

  __device__ void load(int row, Frag& f) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f.q[h] = ld16_stream(codes[h] + static_cast<size_t>(row) * code_row);
      f.p[h] = scales[h][static_cast<size_t>(row) * scale_row];
    }
  }

  template <typename XT>
  __device__ float dot(const Frag& f, const XSliceT<XT>& s) const {
    float out;
    dot_rows<XT, 1>(f, &s, &out);
    return out;
  }

  // The codes are decoded once for all NBR rows; each row's sums follow the
  // same order whatever NBR is, so out[m] equals dot(f, s[m]) bit for bit.
  template <typename XT, int NBR>
  __device__ void dot_rows(const Frag& f, const XSliceT<XT>* s, float* out) const {
    typedef float f2_t __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int m = 0; m < NBR; ++m) out[m] = 0.f;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint32_t q[4] = {f.q[hf].x, f.q[hf].y, f.q[hf].z, f.q[hf].w};
      float t0[NBR], t1[NBR];
#pragma unroll
      for (int m = 0; m < NBR; ++m) t0[m] = t1[m] = 0.f;
      // byte b of dword i: codes 8i + 2b and 8i + 2b + 1
      auto pair = [&](int at, auto w, auto w1) {
#pragma unroll
        for (int m = 0; m < NBR; ++m) {
          if constexpr (__is_same(XT, float)) {
            t0[m] = fmaf(w.x, s[m].v[32 * hf + 2 * at], t0[m]);
            t1[m] = fmaf(w.y, s[m].v[32 * hf + 2 * at + 1], t1[m]);
            t0[m] = fmaf(w1.x, s[m].v[32 * hf + 2 * at + 2], t0[m]);
            t1[m] = fmaf(w1.y, s[m].v[32 * hf + 2 * at + 3], t1[m]);
          } else {
            t0[m] = __builtin_amdgcn_fdot2(w, s[m].h[16 * hf + at], t0[m], false);
            t1[m] = __builtin_amdgcn_fdot2(w1, s[m].h[16 * hf + at + 1], t1[m], false);
          }
        }
      };
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (__is_same(XT, float)) {
          const f2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 0);
          const f2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 1);
          const f2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 2);
          const f2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 3);
          pair(4 * i, a, b);
          pair(4 * i + 2, c, d);
        } else {
          const h2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q[i], 1.0f, 0);
          const h2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q[i], 1.0f, 1);
          const h2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q[i], 1.0f, 2);
          const h2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q[i], 1.0f, 3);
          pair(4 * i, a, b);
          pair(4 * i + 2, c, d);
        }
      }
      const int p = static_cast<int>(f.p[hf]);
#pragma unroll
      for (int m = 0; m < NBR; ++m) {
        const float t = __builtin_amdgcn_ldexpf(t0[m] + t1[m], p - 127 + s[m].e);
        out[m] += p == 255 ? __builtin_nanf("") : t;
      }
    }
  }
};

hipError_t gemv_mxfp4_rows(const GemvCall* calls, int n, int x_dtype, int64_t batch, hipStream_t s) {
  return launch_gemv_rows<Mxfp4Policy>(calls, n, x_dtype, batch, s);
}

hipError_t gemv_mxfp4(const GemvCall* calls, int n, int x_dtype, int64_t batch, hipStream_t s) {
  return launch_gemv<Mxfp4Policy>(calls, n, x_dtype, batch, s);
}

hipError_t gemv_mxfp4_pair(const GemvCall& a, const void* b_w, float* b_y, int x_dtype, int64_t batch, bool glu,
                           hipStream_t s) {
  return launch_gemv_pair<Mxfp4Policy>(a, b_w, b_y, x_dtype, batch, glu, s);
}

}  // namespace qmv

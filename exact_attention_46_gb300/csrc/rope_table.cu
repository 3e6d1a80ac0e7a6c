// rope_table.cu -- the rotary-embedding table read by the fused RoPE + rotation + quantiser.
//
// RoPE as in RoFormer (Su et al. 2021, section 3.2), the reading taken for the rotary embedding
// that the hada.io FA3 summary ("Niedrige FP8-Präzision und incoherent processing") names as
// the bandwidth-bound op to fuse the Hadamard rotation with: pair i of the row at position p
// turns by p * theta_i, theta_i = base^(-2i/D).  Entry (p, i) of the table is
// (cos, sin)(p * theta_i), evaluated in fp64 and rounded to nearest fp32, so that every entry
// is the fp32 value closest to the exact one (up to the fp64 library's last-bit error).  The
// table is built once per (n_pos, D, base) and reused across calls; its cost is not on the
// per-step path.
#include <cuda_runtime.h>

#include "cache.h"
#include "internal.h"

namespace ea46 {

namespace {

__global__ void rope_table_kernel(float2* cs, long long n, int D, double base) {
  const long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= n) return;
  const long long p = idx / (D / 2);
  const int i = static_cast<int>(idx % (D / 2));
  const double theta = pow(base, -2.0 * i / D);
  double s, c;
  sincos(static_cast<double>(p) * theta, &s, &c);
  cs[idx] = make_float2(__double2float_rn(c), __double2float_rn(s));
}

// The table for a context stretched by `factor`, theta_i in fp64:
//   linear  position interpolation: theta_i / factor;
//   ntk     base * factor^(rot / (rot - 2)) in place of base;
//   yarn    by parts (Peng et al. 2023, "YaRN", section 3.2-3.3): a pair that makes more than 32
//           turns within the original length keeps theta_i, one that makes fewer than 1 takes
//           theta_i / factor, in between linear in the number of turns; cos and sin times
//           0.1 ln(factor) + 1.
// The fp64 pipe bounds it, so a thread turns one pair through RUN positions by angle addition, 2 calls of
// sincos for RUN entries: off by 2^-48 at most after 16 turns, against the 2^-25 of the rounding to fp32.
constexpr int RUN = 16;

__global__ void rope_scaled_table_kernel(float2* cs, int n_pos, int rot, double base, int scaling, double factor,
                                         double original_length) {
  const long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long p0 = idx / (rot / 2) * RUN;
  const int i = static_cast<int>(idx % (rot / 2));
  if (p0 >= n_pos) return;
  if (scaling == ROPE_NTK) base *= pow(factor, static_cast<double>(rot) / (rot - 2));
  double theta = pow(base, -2.0 * i / rot), gain = 1.0;
  if (scaling == ROPE_LINEAR) theta /= factor;
  if (scaling == ROPE_YARN) {
    const double turns = original_length * theta / 6.283185307179586476925;
    const double keep = fmin(1.0, fmax(0.0, (turns - 1.0) / 31.0));
    theta = (1.0 - keep) * theta / factor + keep * theta;
    gain = 0.1 * log(factor) + 1.0;
  }
  double s, c, ds, dc;
  sincos(static_cast<double>(p0) * theta, &s, &c);
  sincos(theta, &ds, &dc);
  for (long long p = p0; p < p0 + RUN && p < n_pos; ++p) {
    cs[p * (rot / 2) + i] = make_float2(__double2float_rn(c * gain), __double2float_rn(s * gain));
    const double turned = c * dc - s * ds;
    s = s * dc + c * ds;
    c = turned;
  }
}

}  // namespace

cudaError_t launch_rope_scaled_table(float* cs, int n_pos, int rot, double base, int scaling, double factor,
                                     double original_length, cudaStream_t stream) {
  const long long n = (static_cast<long long>(n_pos) + RUN - 1) / RUN * (rot / 2);
  rope_scaled_table_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, stream>>>(
      reinterpret_cast<float2*>(cs), n_pos, rot, base, scaling, factor, original_length);
  return cudaGetLastError();
}

cudaError_t launch_rope_table(float* cs, int n_pos, int D, double base, cudaStream_t stream) {
  const long long n = static_cast<long long>(n_pos) * (D / 2);
  const int threads = 256;
  const long long blocks = (n + threads - 1) / threads;
  rope_table_kernel<<<static_cast<unsigned>(blocks), threads, 0, stream>>>(
      reinterpret_cast<float2*>(cs), n, D, base);
  return cudaGetLastError();
}

}  // namespace ea46

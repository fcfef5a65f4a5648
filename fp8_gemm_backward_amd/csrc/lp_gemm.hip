// Host side of the fused backward GEMMs: operand descriptors, tile-size
// choice and dispatch to the per-format kernel instantiations.
#include "lp_gemm_kernel.hpp"

namespace lp {
namespace gk {
namespace {

Op make_op(const lp_qtensor& t) {
  Op o{};
  o.codes = static_cast<const uint8_t*>(t.codes);
  o.scales = static_cast<const uint8_t*>(t.scales);
  o.tensor_scale = t.tensor_scale;
  o.rows = (int32_t)t.rows;
  const int64_t R = t.rows, Cc = t.cols;
  switch (t.fmt) {
    case LP_BF16:
      o.code_ld = (int32_t)(Cc * 2);
      break;
    case LP_MXFP4:
      o.code_ld = (int32_t)(Cc / 2);
      o.scale_ld = (int32_t)(Cc / 32);
      o.scale_bytes = R * (Cc / 32);
      break;
    case LP_NVFP4:
      o.code_ld = (int32_t)(Cc / 2);
      o.scale_ld = (int32_t)(Cc / 16);
      o.scale_bytes = R * (Cc / 16);
      break;
    case LP_FP8_B128:
      o.code_ld = (int32_t)Cc;
      o.scale_ld = (int32_t)(((Cc + 127) / 128) * 4);
      o.scale_bytes = ((R + 127) / 128) * ((Cc + 127) / 128) * 4;
      break;
    case LP_FP8T_E4M3:
    case LP_FP8T_E5M2:
      o.code_ld = (int32_t)Cc;
      break;
    case LP_FP8_R128:                                            // scale rows: one per run
      o.code_ld = (int32_t)Cc;
      o.scale_ld = (int32_t)((t.scale_axis == -1 ? R : Cc) * 4);
      o.scale_bytes = (((t.scale_axis == -1 ? Cc : R) + 127) / 128) * o.scale_ld;
      break;
    case LP_MXFP8:
      o.code_ld = (int32_t)Cc;
      if (t.scale_axis == -1) {
        o.scale_ld = (int32_t)(Cc / 32);
        o.scale_bytes = R * (Cc / 32);
      } else {
        o.scale_ld = (int32_t)Cc;
        o.scale_bytes = (R / 32) * Cc;
      }
      break;
  }
  o.code_batch = R * o.code_ld;
  o.scale_batch = o.scale_bytes;
  return o;
}


constexpr int kCUsPerXcd = 32;

// P-tile rows per group of the tile order (grouped_order): a group of g rows
// and kCUsPerXcd / g columns of tiles runs on one XCD at a time and fetches
// g * a + (kCUsPerXcd / g) * b bytes per slab into its L2 (a, b: bytes of one
// P-tile row and one Q-tile column of a slab), least at g = sqrt(32 b / a);
// the power of two nearest to it, ties to the smaller.
int32_t tile_group(int64_t a, int64_t b, int64_t np) {
  int32_t g = 1;
  while (g < kCUsPerXcd && (int64_t)(2 * g) * (2 * g) * a < (int64_t)kCUsPerXcd * b * 2) g *= 2;
  return (int32_t)(g < np ? g : (np > 0 ? np : 1));
}

// Bytes per element of an operand's codes, times 2.
int64_t code_bytes2(int fmt) {
  return fmt == LP_BF16 ? 4 : (fmt == LP_MXFP4 || fmt == LP_NVFP4) ? 1 : 2;
}

// Grouped grad_X and forward on 256 x 256 tiles (prm.ntiles: the host's
// bound on them) split by dispatch round: the whole rounds of kCUs tiles in
// this launch, a short last round as 256 x 128 tiles in a second launch
// (tail_params).  The group sizes live on the device, so the kernels count
// the tiles and both launches reach the same split, or none (the second
// launch then has no tile).  Returns whether to make the second launch.
// Only for contractions of at least kTailMinSlabs slabs: measured in steady
// state, the block-FP8 grouped forward (4096-long contraction, 544 tiles)
// went from 342.5 to 316.3 us, while the MXFP4 grouped grad_X (2048-long,
// 1088 tiles) went from 268.0 to 271.7 us; a short tile's fixed costs and
// the second launch outweigh what its narrower last round saves.
constexpr int kTailMinSlabs = 64;
bool tile_split(Params& prm) {
  if (prm.offsets == nullptr || prm.splits != 1 || prm.fuse_side != 0 || prm.ntiles < kCUs) return false;
  if (prm.Ktot < kTailMinSlabs * BK) return false;
  prm.tail = 1;
  return true;
}
Params tail_params(const Params& big) {
  Params t = big;
  t.tail = 2;
  t.nq = (int32_t)((t.Qtot + Narrow::BQ - 1) / Narrow::BQ);
  t.ntiles = kCUs;
  return t;
}

// The tile counts and order of a call on C tiles (prm from base_params, with
// any split plan already set).
template <class C>
Params cfg_params(const GemmCall& call, Params prm) {
  prm.nq = (int32_t)((prm.Qtot + C::BQ - 1) / C::BQ);
  if (call.offsets == nullptr && prm.splits == 1)
    prm.gm = tile_group(C::BP * code_bytes2(call.grad->fmt), C::BQ * code_bytes2(call.other->fmt),
                        (prm.Ptot + C::BP - 1) / C::BP);
  if (!call.dw) {
    const int64_t ptiles = call.offsets ? (call.M / C::BP + call.groups) : (call.M + C::BP - 1) / C::BP;
    prm.ntiles = (int32_t)(ptiles * prm.nq * prm.splits);
  } else {
    const int64_t np = (prm.Ptot + C::BP - 1) / C::BP;
    prm.ntiles = (int32_t)(np * prm.nq * call.groups * prm.splits);
  }
  return prm;
}

template <class C>
hipError_t launch_cfg(const GemmCall& call, Params prm, hipStream_t stream) {
  prm = cfg_params<C>(call, prm);
  if (!call.dw) {
    const bool mx = call.grad->fmt == LP_MXFP8;
    if constexpr (C::BQ == Big::BQ) {
      const bool split = tile_split(prm);
      const hipError_t e = mx ? dx_big_mxfp8(*call.other, prm, stream) : dx_big_bf16(*call.other, prm, stream);
      if (e != hipSuccess || !split) return e;
      const Params tail = tail_params(prm);
      return mx ? dx_narrow_mxfp8(*call.other, tail, stream) : dx_narrow_bf16(*call.other, tail, stream);
    } else {
      return mx ? dx_narrow_mxfp8(*call.other, prm, stream) : dx_narrow_bf16(*call.other, prm, stream);
    }
  }
  if constexpr (C::BQ == Big::BQ) return dw_big(*call.other, prm, stream);
  else return dw_narrow(*call.other, prm, stream);
}

constexpr int64_t kMinSplitSlabs = 16;     // contraction slabs per split, at least

// Output tiles of the 256 x 256 configuration.
int64_t big_tiles(const GemmCall& call) {
  const int64_t p = call.dw ? call.groups * ((call.N + 255) / 256) : (call.M + 255) / 256;
  return p * ((call.K + 255) / 256);
}

// Output tiles of the 256 x 128 configuration.
int64_t narrow_tiles(const GemmCall& call) {
  const int64_t p = call.dw ? call.groups * ((call.N + 255) / 256) : (call.M + 255) / 256;
  return p * ((call.K + 127) / 128);
}

// Split plan of a dense contraction whose output tiles would leave most CUs
// idle even at 256 x 128 (fewer than half as many tiles as CUs): as many
// splits of 256 x 256 tiles as keep one workgroup per CU, each split at
// least kMinSplitSlabs slabs long.  splits == 1: no split.  Measured on the
// 4096 x 2048 output of an 8192-long contraction (128 big tiles, two
// splits), the partials' write-back and re-read cost more than the narrower
// tiles lose, hence the threshold.
struct SplitPlan {
  int32_t splits, split_len;
  int64_t tiles;
  size_t bytes;
};

// dX of an MXFP8 gradient and an MXFP8 weight scaled along its rows: both
// scales run along the contraction, so the block-scaled MFMA applies them.
// Dense dW of an MXFP8 gradient and an MXFP8 input both scaled along their
// rows (the token axis, the contraction) likewise.
bool native_mx(const GemmCall& call) {
  if (call.grad->fmt != LP_MXFP8 || call.other->fmt != LP_MXFP8 || call.other->scale_axis != -2) return false;
  return !call.dw || (call.grad->scale_axis == -2 && call.offsets == nullptr);
}

bool is_fp8t(int f) { return f == LP_FP8T_E4M3 || f == LP_FP8T_E5M2; }

// Per-tensor scaled FP8 on both sides of the product.
bool native_pt(const GemmCall& call) { return is_fp8t(call.grad->fmt) && is_fp8t(call.other->fmt); }

// E4M3 with fp32 scales per 128 on both sides.
bool native_b128(const GemmCall& call) { return call.grad->fmt == LP_FP8_R128; }

SplitPlan split_plan(const GemmCall& call) {
  SplitPlan sp{1, 0, big_tiles(call), 0};
  if (call.offsets != nullptr || native_mx(call) || native_pt(call) || native_b128(call) || narrow_tiles(call) >= kCUs / 2 || sp.tiles == 0) return sp;
  const int64_t ktot = call.dw ? call.M : call.N;
  const int64_t nk = (ktot + BK - 1) / BK;
  int64_t s = kCUs / sp.tiles;
  if (s > nk / kMinSplitSlabs) s = nk / kMinSplitSlabs;
  if (s < 2) return sp;
  const int64_t per = (nk + s - 1) / s;                 // slabs per split
  s = (nk + per - 1) / per;                             // no empty split
  if (s < 2) return sp;
  sp.splits = (int32_t)s;
  sp.split_len = (int32_t)(per * BK);
  const size_t counters = ((size_t)sp.tiles * 4 + 255) / 256 * 256;
  sp.bytes = counters + (size_t)sp.tiles * s * Big::BP * Big::BQ * sizeof(float);
  return sp;
}

}  // namespace
}  // namespace gk

using namespace gk;

namespace {

struct B128Plan {
  int tile;            // tile size
  int splits;          // workgroups that share a tile's contraction
  int split_len;       // its elements for each
  size_t bytes;        // workspace, 0 without splits
};
B128Plan b128_plan(const GemmCall& call);

}  // namespace

size_t gemm_workspace_bytes(const GemmCall& call) {
  return native_b128(call) ? b128_plan(call).bytes : split_plan(call).bytes;
}

namespace {

Params base_params(const GemmCall& call) {
  Params prm{};
  prm.P = make_op(*call.grad);
  prm.Q = make_op(*call.other);
  prm.C = static_cast<uint16_t*>(call.out);
  prm.ldc = (int32_t)call.K;
  prm.Qtot = (int32_t)call.K;
  prm.offsets = call.offsets;
  prm.groups = call.groups;
  prm.splits = 1;
  prm.fuse_rows = call.fuse_rows;
  prm.fuse_side = call.fuse_side;
  if (!call.dw) {
    prm.Ptot = (int32_t)call.M;
    prm.Ktot = (int32_t)call.N;
    prm.c_batch = 0;
  } else {
    prm.Ptot = (int32_t)call.N;
    prm.Ktot = (int32_t)call.M;
    prm.c_batch = call.N * call.K;
  }
  return prm;
}

// Tile counts of a contraction on the FP8 MFMA kernel (256 x 256 tiles).
Params native_params(const GemmCall& call) {
  Params prm = base_params(call);
  prm.nq = (int32_t)((prm.Qtot + Big::BQ - 1) / Big::BQ);
  // Dense calls order their tiles in blocks of gm row tiles; grouped grad_X
  // does the same inside each group (a group of fewer row tiles is one
  // block).
  if (call.offsets == nullptr || !call.dw)
    prm.gm = tile_group(Big::BP * code_bytes2(call.grad->fmt), Big::BQ * code_bytes2(call.other->fmt),
                        call.offsets == nullptr ? (prm.Ptot + Big::BP - 1) / Big::BP : kCUsPerXcd);
  if (call.dw) {
    prm.ntiles = (int32_t)(((call.N + Big::BP - 1) / Big::BP) * prm.nq * call.groups);
  } else {
    const int64_t ptiles = call.offsets ? (call.M / Big::BP + call.groups) : (call.M + Big::BP - 1) / Big::BP;
    prm.ntiles = (int32_t)(ptiles * prm.nq);
  }
  return prm;
}

// Tile counts and order of a product with fp32 scales per 128 on b x b tiles.
// rows: output rows; groups split them (grad_X, forward) unless dw, where
// every group has all of them.
void b128_tiles(Params& prm, int b, bool dw) {
  const int64_t np = (prm.Ptot + b - 1) / b;
  prm.nq = (prm.Qtot + b - 1) / b;
  if (prm.offsets == nullptr || !dw) prm.gm = tile_group(b, b, prm.offsets == nullptr ? np : kCUsPerXcd);
  const int64_t pt = dw ? np * prm.groups : prm.offsets ? prm.Ptot / b + prm.groups : np;
  prm.ntiles = (int32_t)(pt * prm.nq);
}

// Dense products, grouped grad_X and forward split by dispatch round, as
// tile_split does: the whole rounds of 256 x 256 tiles, then a short last round
// in parts of tiles by a second launch (rounds_of and b128_tail_kernel have the
// rules).  For contractions of at least 16 stages over at most five rounds:
// 4112 x 4112 x 8208 forward 212 -> 168 us, grad_W 198 -> 173; 8192 x 2560 x 4096 98 -> 85;
// 16384 rows over 8 uneven experts, forward 2048 x 4096 159 -> 149, grad_X of
// 4096 x 2048 161 -> 150 (in halves); shorter ones and more rounds only pay for the
// second launch (grad_X of 1536 x 6144, 10000 rows: 103 -> 110; forward of 64
// experts, six rounds: 568 -> 573).
bool b128_split(Params& prm) {
  if (prm.ntiles < kCUs || prm.ntiles > 5 * kCUs || prm.Ktot < 16 * 128) return false;
  const int rest = prm.ntiles % kCUs;                            // dense: known here
  if (prm.offsets == nullptr && (prm.ntiles == rest || rest == 0 || 2 * rest > kCUs)) return false;
  prm.tail = 1;
  return true;
}

// The tile size of a product with fp32 scales per 128: the least estimated
// time of one contraction stage over all dispatch rounds, in units of 10 ns
// (measured per stage and round on a GPU that is not yet hot: 256 x 256 tiles
// 1.35 us, 128 x 128 0.50 us for up to 128 tiles and 0.62 us above, 64 x 64 0.20
// and 0.28 us; a second round of 64 x 64 tiles lost to 128 x 128 in every
// case).  Over 24 dense and grouped products the choice was within 6% of the best
// of the three, but for two (7% and 13%).  Grouped grad_X and
// grad_W keep 256 x 256 unless 128 x 128 fits one round: their narrow tiles
// read or write 128-byte pieces of long rows (64 experts of 2048 x 7168, 1024
// tokens: grad_X 293 us on 256 x 256 tiles, 377 us on 128 x 128).
enum class B128Op { kFwd, kDx, kDw };
int b128_tile(const Params& prm, B128Op op) {
  auto count = [&](int b) {
    Params t = prm;
    b128_tiles(t, b, op == B128Op::kDw);
    return (int64_t)t.ntiles;
  };
  const int64_t t256 = count(256), t128 = count(128), t64 = count(64);
  const bool one_round = prm.offsets != nullptr && op != B128Op::kFwd;
  const int64_t c256 = 135 * ((t256 + kCUs - 1) / kCUs);
  const int64_t c128 = t128 <= kCUs / 2 ? 50 : one_round && t128 > kCUs ? INT64_MAX : 62 * ((t128 + kCUs - 1) / kCUs);
  const int64_t c64 = t64 <= kCUs / 2 ? 20 : t64 <= kCUs ? 28 : INT64_MAX;
  return c64 <= c128 && c64 <= c256 ? 64 : c128 <= c256 ? 128 : 256;
}

// The first 4 KiB of a workspace hold what other products need zero between calls
// (their tiles' counters): left alone.
constexpr size_t kB128WsHead = 4096;

// A dense grad_X or grad_W of few tiles over a long contraction, given a
// workspace: several workgroups to a tile, an fp32 tile from each, and a
// second launch that adds them.  By the same estimate as b128_tile, plus 5 us
// for that launch and the way of the fp32 tiles to memory and back (8 bytes an
// element at 5 TB/s); at least 16 stages to a workgroup.  grad_W of 240 x 240 over 21648
// rows 81.9 us without, 19.8 with; 16 x 4096 over 32768 96.4, 35.0; 64 x 4096 over 8192
// 27.1, 17.2; 1024 x 1024 over 32768 99.5, 52.1, over 8192 (64 stages, 64 tiles of 128 x
// 128) left whole at 28.2.
B128Plan b128_plan(const GemmCall& call) {
  const B128Op op = call.dw ? B128Op::kDw : B128Op::kDx;
  const Params prm = base_params(call);
  B128Plan best{b128_tile(prm, op), 1, prm.Ktot, 0};
  const int64_t runs = (prm.Ktot + 127) / 128;
  if (call.offsets != nullptr || best.tile == 256 || runs < 32) return best;
  auto stage = [](int tile, int64_t n) { return tile == 64 ? (n <= kCUs / 2 ? 20 : 28) : (n <= kCUs / 2 ? 50 : 62); };
  int64_t cost = INT64_MAX;
  for (int tile : {64, 128}) {
    Params t = prm;
    b128_tiles(t, tile, call.dw);
    if (t.ntiles <= 0 || t.ntiles > kCUs) continue;
    for (int64_t s = 1; s * t.ntiles <= kCUs && runs / s >= 16; ++s) {
      const int64_t per = (runs + s - 1) / s;
      if (s > 1 && (runs + per - 1) / per != s) continue;        // no empty split
      const int64_t joint = s > 1 ? 500 + t.ntiles * s * tile * tile / 6250 : 0;
      const int64_t c = stage(tile, t.ntiles * s) * per + joint;
      if (c >= cost) continue;
      cost = c;
      best = B128Plan{tile, (int)s, (int)(per * 128), s > 1 ? kB128WsHead + (size_t)t.ntiles * s * tile * tile * 4 : 0};
    }
  }
  return best;
}

}  // namespace

hipError_t launch_gemm(const GemmCall& call, hipStream_t stream) {
  if (native_b128(call)) {
    Params prm = base_params(call);
    const B128Plan plan = b128_plan(call);
    if (plan.splits > 1 && call.ws != nullptr && call.ws_bytes >= plan.bytes) {
      b128_tiles(prm, plan.tile, call.dw);
      prm.splits = plan.splits;
      prm.split_len = plan.split_len;
      prm.ws = reinterpret_cast<float*>(static_cast<uint8_t*>(call.ws) + kB128WsHead);
      const hipError_t e = call.dw ? b128_dw(prm, plan.tile, stream) : b128_dx(prm, plan.tile, stream);
      return e != hipSuccess ? e : b128_join(prm, plan.tile, stream);
    }
    const int tile = b128_tile(prm, call.dw ? B128Op::kDw : B128Op::kDx);
    b128_tiles(prm, tile, call.dw);
    const bool split = tile == 256 && !(call.dw && call.offsets != nullptr) && b128_split(prm);
    const hipError_t e = call.dw ? b128_dw(prm, tile, stream) : b128_dx(prm, tile, stream);
    if (e != hipSuccess || !split) return e;
    return call.dw ? b128_dw_tail(prm, stream) : b128_dx_tail(prm, stream);
  }
  if (native_mx(call) || native_pt(call)) {
    const Params prm = native_params(call);
    const int fp = call.grad->fmt, fq = call.other->fmt;
    if (native_pt(call)) return call.dw ? dw_pt(prm, fp, fq, stream) : dx_pt(prm, fp, fq, stream);
    return call.dw ? dw_mx(prm, stream) : dx_mx(prm, stream);
  }
  Params prm = base_params(call);
  if (big_tiles(call) >= kCUs) return launch_cfg<Big>(call, prm, stream);
  // Fewer than one full wave of 256 x 256 tiles across the CUs: split the
  // contraction when a large enough workspace is given, else halve the tile
  // width so that every CU gets work.
  const SplitPlan sp = split_plan(call);
  if (sp.splits > 1 && call.ws != nullptr && call.ws_bytes >= sp.bytes) {
    const size_t counters = ((size_t)sp.tiles * 4 + 255) / 256 * 256;
    prm.splits = sp.splits;
    prm.split_len = sp.split_len;
    prm.cnt = static_cast<uint32_t*>(call.ws);
    prm.ws = reinterpret_cast<float*>(static_cast<uint8_t*>(call.ws) + counters);
    return launch_cfg<Big>(call, prm, stream);
  }
  return launch_cfg<Narrow>(call, prm, stream);
}

namespace {

// Shapes and operands of a forward.
Params fwd_params(const lp_qtensor& x, const lp_qtensor& w, const int32_t* offsets, int32_t groups, void* y) {
  Params prm{};
  prm.P = make_op(x);
  prm.Q = make_op(w);
  prm.C = static_cast<uint16_t*>(y);
  prm.Ptot = (int32_t)x.rows;
  prm.Qtot = (int32_t)w.rows;
  prm.Ktot = (int32_t)x.cols;
  prm.ldc = prm.Qtot;
  prm.offsets = offsets;
  prm.groups = groups;
  prm.splits = 1;
  return prm;
}

}  // namespace

hipError_t launch_fwd(const lp_qtensor& x, const lp_qtensor& w, const int32_t* offsets, int32_t groups, void* y,
                      hipStream_t stream) {
  Params prm = fwd_params(x, w, offsets, groups, y);
  if (x.fmt == LP_FP8_R128) {
    if (b128_skinny_fits(prm)) return b128_fwd_skinny(prm, stream);
    const int tile = b128_tile(prm, B128Op::kFwd);
    b128_tiles(prm, tile, false);
    const bool split = tile == 256 && b128_split(prm);
    const hipError_t e = b128_fwd(prm, tile, stream);
    return e != hipSuccess || !split ? e : b128_fwd_tail(prm, stream);
  }
  // MX operands run on the block-scaled MFMA (256 x 256 tiles); the others
  // through bf16 tiles, 256 x 256 unless both are bf16 (256 x 128: three
  // stages of both tiles fit in LDS only at that width).
  const bool mx = x.fmt == LP_MXFP4 || x.fmt == LP_MXFP8;
  const int BP = 256, BQ = w.fmt == LP_BF16 ? 128 : 256;
  prm.nq = (int32_t)((prm.Qtot + BQ - 1) / BQ);
  if (offsets == nullptr)
    prm.gm = tile_group(BP * code_bytes2(x.fmt), BQ * code_bytes2(w.fmt), (prm.Ptot + BP - 1) / BP);
  const int64_t ptiles = offsets ? (x.rows / BP + groups) : (x.rows + BP - 1) / BP;
  prm.ntiles = (int32_t)(ptiles * prm.nq);
  if (mx) return fwd_mx(prm, x.fmt == LP_MXFP4, stream);
  // (An MXFP4 weight comes here for contractions too short for a split: with longer
  // ones 128 x 256 rows and columns a workgroup, lp_gemm_w4.hip, always take less.)
  const bool split = BQ == Big::BQ && w.fmt != LP_MXFP4 && tile_split(prm);
  const hipError_t e = fwd_dec(prm, x.fmt, w.fmt, false, stream);
  if (e != hipSuccess || !split) return e;
  return fwd_dec(tail_params(prm), x.fmt, w.fmt, true, stream);
}

hipError_t launch_fwd_w4(const lp_qtensor& x, const lp_qtensor& w, const int32_t* offsets, int32_t groups, void* y,
                         hipStream_t stream) {
  const Params prm = fwd_params(x, w, offsets, groups, y);
  bool done = false;
  const hipError_t e = w4_fwd(prm, w.fmt, &done, stream);
  return done ? e : launch_fwd(x, w, offsets, groups, y, stream);
}

hipError_t launch_fwd_dyn(const void* x, const lp_qtensor& xq, const lp_qtensor& w, const int32_t* offsets,
                          int32_t groups, void* x_codes, void* x_scales, void* y, hipStream_t stream) {
  const Params prm = fwd_params(xq, w, offsets, groups, y);
  if (fwd_dyn_fuses(xq.rows, xq.cols, offsets != nullptr)) return b128_fwd_fused(prm, x, stream);
  if (xq.cols > 0) {
    const hipError_t e = launch_r128_cols(x, 1, xq.rows, xq.cols, x_codes, x_scales, stream);
    if (e != hipSuccess) return e;
  }
  return launch_fwd(xq, w, offsets, groups, y, stream);
}

hipError_t launch_grouped_dx_deferred(const lp_qtensor& grad, const void* w, int64_t K, const int32_t* offsets,
                                      int32_t groups, int64_t fuse_rows, void* w_codes, void* w_scales,
                                      void* grad_x, hipStream_t stream) {
  const int64_t M = grad.rows, N = grad.cols;
  // The fused kernel takes the gradient's scales in 16-byte chunks of its
  // scale rows (N % 512 == 0), and the quantizer that leaves out the fused
  // groups works on 32 x 32 tiles (K % 32 == 0); otherwise every weight is
  // quantized first.
  const bool can_fuse = N % 512 == 0 && K % 32 == 0;
  const int32_t fr = can_fuse ? (int32_t)(fuse_rows < M ? fuse_rows : M) : 0;
  // Groups of more than fr rows: weight quantized first, then the
  // block-scaled product on its codes.
  if (fr < M) {
    hipError_t e = fr > 0 ? launch_mx_quant_rows_groups(w, groups, N, K, offsets, M, fr, w_codes, w_scales, stream)
                          : launch_mx_quant(w, groups, N, K, -2, LP_MXFP8, w_codes, w_scales, stream);
    if (e != hipSuccess) return e;
    const lp_qtensor wq{LP_MXFP8, -2, groups, N, K, w_codes, w_scales, nullptr};
    GemmCall c{false, &grad, &wq, offsets, groups, M, N, K, grad_x, nullptr, 0};
    c.fuse_rows = fr;
    c.fuse_side = fr > 0 ? 1 : 0;
    if ((e = launch_gemm(c, stream)) != hipSuccess) return e;
  }
  // Groups of at most fr rows: the weight quantized inside the product.
  if (fr > 0) {
    const lp_qtensor wb{LP_BF16, -1, groups, N, K, w, nullptr, nullptr};
    GemmCall c{false, &grad, &wb, offsets, groups, M, N, K, grad_x, nullptr, 0};
    Params prm = base_params(c);
    prm.fuse_rows = fr;
    prm.fuse_side = 2;
    prm.nq = (int32_t)((K + 255) / 256);
    // Row tiles of the listed groups: at most M / 256 + G, and at most
    // G ceil(fr / 256).
    int64_t rt = M / 256 + groups;
    const int64_t rt2 = (int64_t)groups * ((fr + 255) / 256);
    rt = rt2 < rt ? rt2 : rt;
    prm.ntiles = (int32_t)(rt * prm.nq);
    return dx_wquant(prm, stream);
  }
  return hipSuccess;
}

hipError_t launch_gemm_pair(const GemmCall& dx, const GemmCall& dw, hipStream_t stream) {
  if (native_pt(dx) && native_pt(dw) && dx.other->fmt == dw.other->fmt)
    return pt_pair(native_params(dx), native_params(dw), dx.grad->fmt, dx.other->fmt, stream);
  // A grouped layer's grad_X and grad_W from a bf16 gradient and FP4 W and X
  // (scaled along their last axis), both on 256 x 256 tiles: one launch.
  const int fq = dx.other->fmt;
  if (dx.offsets != nullptr && dx.grad->fmt == LP_BF16 && (fq == LP_MXFP4 || fq == LP_NVFP4) &&
      dw.other->fmt == fq && dx.other->scale_axis == -1 && dw.other->scale_axis == -1 && dx.ws == nullptr &&
      dw.ws == nullptr && big_tiles(dx) >= kCUs && big_tiles(dw) >= kCUs)
    return dec_pair(cfg_params<Big>(dx, base_params(dx)), cfg_params<Big>(dw, base_params(dw)), fq, stream);
  const hipError_t e = launch_gemm(dx, stream);
  return e != hipSuccess ? e : launch_gemm(dw, stream);
}

}  // namespace lp

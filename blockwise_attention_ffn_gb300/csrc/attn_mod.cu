// attn_mod.cu -- the C entry points of the modified attention: argument checks
// and the debug checks around the launches in attn_mod_fwd.cu, attn_mod_bwd.cu.
#include <cuda_runtime.h>
#include <math.h>

#include "../../include/bpt.h"
#include "internal.h"

using namespace bpt;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check(const bpt_config* cfg, const bpt_score_mod* mod, PackedDims* D) {
  const int rc = packed_dims(cfg, D);
  if (rc) return rc;
  if (!mod) return BPT_EINVAL;
  if ((reinterpret_cast<uintptr_t>(mod->row_begin) & 3) || (reinterpret_cast<uintptr_t>(mod->row_end) & 3) ||
      (reinterpret_cast<uintptr_t>(mod->slopes) & 3))
    return BPT_EINVAL;
  // 0: no cap; outside these the powers in the cap's first polynomial would leave
  // fp32, and no score is that small or large
  if (!(mod->softcap == 0.f || (mod->softcap >= 0x1p-10f && mod->softcap <= 0x1p20f))) return BPT_EINVAL;
  // grid sizes, 32-bit columns and the extra rows' 32-bit row coordinate
  if (D->width > INT32_MAX || D->b * D->H * D->s_pad > INT32_MAX) return BPT_EUNSUPPORTED;
  return BPT_OK;
}

struct ModSpans {
  Span sp[3];
  ModSpans(const PackedDims& D, const bpt_score_mod* mod)
      : sp{{mod->row_begin, mod->row_begin ? D.rows * 4 : 0},
           {mod->row_end, mod->row_end ? D.rows * 4 : 0},
           {mod->slopes, mod->slopes ? D.H * 4 : 0}} {}
};

}  // namespace

extern "C" {

int bpt_attention_mod_fwd(const bpt_config* cfg, const bpt_score_mod* mod, const void* qkv, void* o, void* lse,
                          void* stream) {
  PackedDims D;
  int rc = check(cfg, mod, &D);
  if (rc) return rc;
  if (!qkv || !o || !aligned16(qkv) || !aligned16(o) || !aligned16(lse)) return BPT_EINVAL;
  const Span sp[] = {{qkv, D.rows * D.width * 2}, {o, D.rows * D.H * D.d * 2},
                     {lse, lse ? D.b * D.H * D.s_pad * 4 : 0}};
  const ModSpans ms(D, mod);
  if (overlaps(sp[1], sp, 1) || (lse && overlaps(sp[2], sp, 2))) return BPT_EINVAL;
  if (overlaps(sp[1], ms.sp, 3) || (lse && overlaps(sp[2], ms.sp, 3))) return BPT_EINVAL;
  if (D.debug && (debug_spans(sp, 3) || debug_spans(ms.sp, 3))) return BPT_EINVAL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if ((rc = attention_mod_fwd(D, cfg->causal, *mod, qkv, o, reinterpret_cast<float*>(lse), st))) return rc;
  return D.debug ? debug_finish(st) : BPT_OK;
}

size_t bpt_attention_mod_bwd_workspace_bytes(const bpt_config* cfg) {
  PackedDims D;
  return packed_dims(cfg, &D) ? 0 : attention_mod_bwd_ws_bytes(D);
}

int bpt_attention_mod_bwd(const bpt_config* cfg, const bpt_score_mod* mod, const void* qkv, const void* o,
                          const void* lse, const void* dout, void* dqkv, void* ws, size_t ws_bytes, void* stream) {
  PackedDims D;
  int rc = check(cfg, mod, &D);
  if (rc) return rc;
  if (!qkv || !o || !lse || !dout || !dqkv || !ws) return BPT_EINVAL;
  if (!aligned16(qkv) || !aligned16(o) || !aligned16(lse) || !aligned16(dout) || !aligned16(dqkv) || !aligned16(ws))
    return BPT_EINVAL;
  const size_t need = attention_mod_bwd_ws_bytes(D);
  if (ws_bytes < need) return BPT_ENOSPC;
  const int64_t packed = D.rows * D.width * 2, hd = D.rows * D.H * D.d * 2;
  const Span sp[] = {{qkv, packed}, {o, hd}, {lse, D.b * D.H * D.s_pad * 4}, {dout, hd}, {dqkv, packed},
                     {ws, (int64_t)need}};
  const ModSpans ms(D, mod);
  if (overlaps(sp[4], sp, 4) || overlaps(sp[5], sp, 5)) return BPT_EINVAL;
  if (overlaps(sp[4], ms.sp, 3) || overlaps(sp[5], ms.sp, 3)) return BPT_EINVAL;
  if (D.debug && (debug_spans(sp, 6) || debug_spans(ms.sp, 3))) return BPT_EINVAL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if ((rc = attention_mod_bwd(D, cfg->causal, *mod, qkv, o, reinterpret_cast<const float*>(lse), dout, dqkv, ws, st)))
    return rc;
  return D.debug ? debug_finish(st) : BPT_OK;
}

}  // extern "C"

"""MuonClip (Muon + per-head QK-Clip) optimizer step for GB300 (sm_103a).

The compute lives in libmuonclip.so (CUDA, built by muon_qk_clip_gb300.build);
this package is its binding plus seeded synthetic inputs for tests and the
benchmark.
"""
from .abi import MuonClipError  # noqa: F401
from .binding import (AdamHparams, ClipLayer, ClipSegment, Hparams, adamw_state, adamw_step,  # noqa: F401
                      alloc_workspace, default_hparams, gqa_segments, mha_segments, mla_segments,
                      muon_momentum, muon_newton_schulz, muonclip_step, qk_attention_backward,
                      qk_attention_forward, qk_attention_packed_backward, qk_attention_packed_forward,
                      qk_clip_apply, qk_max_logit, qk_norm_rope, qk_norm_rope_backward, workspace_size)

__all__ = ["AdamHparams", "ClipLayer", "ClipSegment", "Hparams", "MuonClipError", "adamw_state", "adamw_step",
           "alloc_workspace", "default_hparams", "gqa_segments", "mha_segments", "mla_segments",
           "muon_momentum", "muon_newton_schulz", "muonclip_step", "qk_attention_backward",
           "qk_attention_forward", "qk_attention_packed_backward", "qk_attention_packed_forward",
           "qk_clip_apply", "qk_max_logit", "qk_norm_rope", "qk_norm_rope_backward", "workspace_size"]

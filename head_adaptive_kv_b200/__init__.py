"""B200-native decode hot path of HARD-KV's Cascade Cache.

Five steps per (sequence, KV head): score the sparse tier against the current
query, Logits Calibration, a clamped per-head Top-p budget, order-preserving
compaction into a static layout (Rewrite Cache / Flatten Index), and cascade
decode attention over the dense, compacted-sparse and condensed tiers. All of it
runs in ``libhkv.so`` (hand-written CUDA for sm_100a, C ABI in ``include/hkv.h``);
the ``hkv`` module only marshals arguments. ``workloads`` makes seeded inputs.

``prompt`` is the side before the first step (``include/hkv_prompt.h``): page
plans, per-head norms with the position rotation, the attention of prompt
chunks over a paged cache, and the tiers filled from finished prompts.
"""
_EXPORTS = {
    "FLAT_SUM", "PAD_MAX", "Cut", "HkvError", "Problem", "StepOutputs", "Tier", "Workspace",
    "calibrate", "cascade_decode", "compact", "debug_withhold_publish", "launch_count", "score",
    "set_wait_limit_ns", "step", "status_string", "topp_select",
}
_PROMPT_EXPORTS = {
    "Chunk", "ChunkWorkspace", "PageState", "Pages", "Rope", "StatusWorkspace", "chunk_attention", "fill_tiers",
    "page_plan", "page_release", "qk_norm_rope",
}


def __getattr__(name):
    if name in _EXPORTS:
        from . import hkv  # loads libhkv.so; raises if it is missing

        return getattr(hkv, name)
    if name in _PROMPT_EXPORTS:
        from . import prompt

        return getattr(prompt, name)
    raise AttributeError(name)

"""gsort: GB300-native stable LSD radix sort, stream compaction and segmented
bitonic sort, and the selection and grouping operators of language models, in
hand-written CUDA for sm_103a behind a C ABI (libgsort.so).

The torch-facing wrappers live in `bitonic_networks_gb300.gsort` and
`bitonic_networks_gb300.model_ops`; they are
loaded on first attribute access so that importing the package (for example
to reach the input generators in `synth`) does not require the CUDA library.
"""
import importlib

__all__ = [
    "sort", "sort_keys", "sort_pairs", "compact_positive", "segmented_sort_", "segmented_sort",
    "partition", "split_sort",
    "digit_histograms", "GsortError", "library_path",
    "radix_workspace_bytes", "sort_workspace_bytes", "segmented_sort_workspace_bytes",
    "compact_workspace_bytes",
]
_MODEL_OPS = [
    "route_experts", "route_experts_backward", "group_by_expert", "group_capacity",
    "group_workspace_bytes", "dispatch_rows", "combine_rows", "combine_rows_backward",
    "token_logprobs", "token_logprobs_backward", "ExpertGroups", "TokenLogprobs",
    "embed_tokens", "embed_tokens_backward", "embed_workspace_bytes", "adjust_logits", "adjust_logits_backward",
    "gradient_norm", "clip_gradients", "ClippedGradients",
]
__all__ += _MODEL_OPS


def __getattr__(name):
    if name in __all__:
        mod = importlib.import_module(".model_ops" if name in _MODEL_OPS else ".gsort", __name__)
        value = globals()[name] = getattr(mod, name)   # the next access finds it at once
        return value
    raise AttributeError(name)

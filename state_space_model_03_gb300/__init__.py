"""GB300-native Mamba-1 selective-scan forward, decode step and causal conv1d.

``selective_scan_fn`` (with an optional start state), ``selective_state_update``,
``causal_conv1d_fn`` and ``causal_conv1d_update`` run the hand-written sm_103a
kernels of ``libssfwd.so`` through its C ABI (``include/ssfwd.h``). Packed
requests (``include/ssfwd_packed.h``) have ``request_tables``,
``packed_conv1d_fn``, ``packed_conv1d_update``, ``head_scan_fn`` and
``head_state_update``. A gated recurrent layer (``include/ssfwd_layer.h``) has
``gated_scan_fn``, ``packed_gated_scan_fn``, ``gated_state_update``,
``rms_norm_fn`` and ``rms_norm_quant_fn``. There is no CPU fallback: the calls raise if the CUDA
library is missing or no GPU is present.
"""

__all__ = ["selective_scan_fn", "selective_scan_fn_host", "selective_scan_bwd", "SelectiveScanFn",
           "selective_state_update", "causal_conv1d_fn", "causal_conv1d_update"]
_PACKED = ["request_tables", "RequestTables", "packed_conv1d_fn", "packed_conv1d_update", "head_scan_fn",
           "head_scan_block", "head_state_update"]
_LAYER = ["gated_scan_fn", "packed_gated_scan_fn", "gated_state_update", "rms_norm_fn", "rms_norm_quant_fn"]
__all__ += _PACKED + _LAYER


def __getattr__(name):
    # Lazy: importing the package (e.g. for the input generator) does not load
    # the CUDA library; the first use of the API does, and fails loudly.
    if name in _PACKED:
        from . import packed
        return getattr(packed, name)
    if name in _LAYER:
        from . import layer
        return getattr(layer, name)
    if name in __all__:
        from . import api
        return getattr(api, name)
    raise AttributeError(name)

"""libdwconv: depthwise 2-D convolution on GB300 (sm_103a), forward,
backward-data and backward-weight, behind a C ABI (include/dwconv.h).

The Python surface is the binding in ``binding`` (same names as the C entry
points). ``build.build()`` compiles the CUDA library in-tree. ``synth`` draws
seeded synthetic inputs and holds no convolution arithmetic.
"""
from .binding import (  # noqa: F401
    Act8, DTYPES, Desc, DwconvError, ESIZE, NormDesc, SYMBOLS, dwconv2d_bwd_data, dwconv2d_bwd_data_multi,
    dwconv2d_bwd_nhwc, dwconv2d_bwd_nhwc_plan_name, dwconv2d_bwd_nhwc_workspace_size, dwconv2d_group_norm_nhwc,
    dwconv2d_group_norm_nhwc_bwd, dwconv2d_group_norm_nhwc_plan_name, dwconv2d_group_norm_nhwc_workspace_size,
    dwconv2d_bwd_weight, dwconv2d_bwd_weight_noalloc, dwconv2d_bwd_weight_workspace_size, dwconv2d_fwd, dwconv2d_fwd_multi,
    dwconv2d_multi_plan_name, dwconv2d_output_shape, dwconv2d_plan_name, dwconv_act8_decode, dwconv_act8_encode, dwconv_device_timeouts, dwconv_fma_probe, dwconv_status_string, lib_path,
    load, make_act8, make_desc, make_norm_desc,
    Grad, RmsDesc, Weight8, dwconv2d_pointwise8, dwconv2d_pointwise8_plan_name, dwconv2d_pointwise8_workspace_size,
    dwconv_grad_norm_clip, dwconv_grad_norm_clip_workspace_size, dwconv_rms_norm, dwconv_rms_norm_bwd,
    dwconv_rms_norm_bwd_workspace_size, dwconv_rms_norm_plan_name, dwconv_weight8_encode, make_grads, make_rms_desc,
    make_weight8, weight8_pitch)

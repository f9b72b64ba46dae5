"""ctypes binding of the training-layer C ABI (include/scape_layers.h): argument
marshalling only, on the library that _scape.load() loads."""
from __future__ import annotations

import ctypes

_vp, _i64, _i32, _f32, _sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                              ctypes.c_size_t)

ACTIVATIONS = {None: 0, "relu": 1, "gelu": 2, "silu": 3}

PROTOS = {
    "scape_layer_last_error": (ctypes.c_char_p, []),
    "scape_layer_status": (_i32, [_vp, _vp]),
    "scape_layer_probe_wait": (_i32, [_i64, _vp]),
    "scape_layer_pack8": (_i32, [_vp, _i64, _i32, _i64, _i64, _vp, _i64, _vp, _vp]),
    "scape_layer_unpack8": (_i32, [_vp, _i64, _vp, _i64, _i64, _i32, _vp, _i64, _i32, _vp]),
    "scape_layer_act_grad": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i32, _vp, _i64, _i32,
                                    _vp]),
    "scape_layer_add_rmsnorm": (_i32, [_vp, _i64, _vp, _i64, _vp, _i32, _i64, _i64, _f32, _i32,
                                       _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp]),
    "scape_layer_add_rmsnorm_bwd_workspace": (_i32, [_i64, _i64, _vp]),
    "scape_layer_add_rmsnorm_bwd": (_i32, [_vp, _i64, _vp, _i64, _vp, _i32, _vp, _vp, _i64, _i64,
                                           _i64, _i32, _vp, _i64, _vp, _i32, _vp, _sz, _vp]),
    "scape_layer_linear_workspace": (_i32, [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp]),
    "scape_layer_linear": (_i32, [_vp, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _i32,
                                  _vp, _i64, _vp, _i64, _vp, _vp, _sz, _vp]),
    "scape_layer_linear_bwd_input_workspace": (_i32, [_vp, _i64, _vp, _i64, _i64, _i64, _i64,
                                                      _vp]),
    "scape_layer_linear_bwd_input": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i32, _i64,
                                            _i64, _i64, _vp, _i64, _vp, _sz, _vp]),
    "scape_layer_linear_bwd_weight_workspace": (_i32, [_vp, _i64, _vp, _i64, _i64, _i64, _i64,
                                                       _vp]),
    "scape_layer_linear_bwd_weight": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i32, _i64,
                                             _i64, _i64, _vp, _i64, _vp, _i32, _vp, _sz, _vp]),
    "scape_layer_linear_plan": (_i32, [_i32, _i64, _i64, _i64, _i32, _vp, _vp, _vp]),
}

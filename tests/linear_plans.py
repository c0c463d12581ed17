"""What kernel a product takes: the library's own plan (ssd::linear_plan, a host function without a C entry point), and
sizes that between them reach every tile, split and not, in every form that it is built for.

A case is (kind, type, rows, in, out) and the plan it has to take: (columns of the tile's rows and columns, split or
not, the second tile's where the last columns take another). tests/test_linear_plans.py holds the plans to it without
a GPU, so that a change to the plan cannot take a kernel out of the GPU tests unseen."""
from __future__ import annotations

import ctypes


class _Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("bm", "bn", "nm", "nn", "steps", "splits", "steps_per_split", "n_main",
                                            "rest_bm", "rest_bn", "rest_nm", "rest_nn")]


def _plan(ssd, rows, cols, kbytes, f32, along_k):
    f = ssd.load()._ZN3ssd11linear_planElllbb
    f.restype, f.argtypes = _Plan, [ctypes.c_int64] * 3 + [ctypes.c_bool] * 2
    return f(rows, cols, kbytes, f32, along_k)


def plan_of(ssd, kind, dtype, rows, k, n):
    """((bm, bn), split?, (rest_bm, rest_bn) or None) of a forward product ("fwd", "mx") or a gradient ("dx", "dw")."""
    es, f32 = (2, False) if dtype == "bf16" else (4, True)

    def whole(values):  # bytes of a row of this many values, in 16-byte chunks
        return (values * es + 15) // 16 * 16
    if kind == "fwd":
        p = _plan(ssd, rows, n, whole(k), f32, False)
    elif kind == "mx":
        p = _plan(ssd, rows, n, k, False, False)
    elif kind == "dx":
        p = _plan(ssd, rows, k, whole(n), f32, not f32)
    else:
        p = _plan(ssd, n, k, whole(rows), f32, not f32)
    return (p.bm, p.bn), p.splits > 1, (p.rest_bm, p.rest_bn) if p.n_main else None


T128, T192, T256, T64 = (128, 128), (256, 192), (256, 256), (64, 64)

# rows of whole 16-byte chunks and not, columns in groups of 4 and not
FORWARD = [
    ("bf16", 407, 208, 9624, T128, False, None), ("bf16", 407, 210, 9621, T128, False, None),
    ("bf16", 840, 8232, 4608, T128, True, None), ("bf16", 839, 8234, 4607, T128, True, None),
    ("bf16", 8737, 208, 908, T192, False, None), ("bf16", 8737, 210, 907, T192, False, None),
    ("bf16", 341, 4224, 11536, T192, True, None), ("bf16", 341, 4226, 11533, T192, True, None),
    ("bf16", 1157, 208, 10024, T256, False, None), ("bf16", 1157, 210, 10023, T256, False, None),
    ("bf16", 8305, 3776, 480, T256, True, None), ("bf16", 8305, 3778, 479, T256, True, None),
    ("bf16", 1157, 211, 10023, T256, False, None),   # an odd row length: copies of both operands
    ("bf16", 3899, 224, 5396, T256, False, T128), ("bf16", 3899, 226, 5395, T256, False, T128),
    ("bf16", 3847, 256, 6948, T256, False, T192), ("bf16", 3847, 258, 6945, T256, False, T192),
    ("bf16", 3859, 248, 4868, T256, False, T64), ("bf16", 3859, 250, 4867, T256, False, T64),
    ("f32", 6693, 208, 588, T128, False, None), ("f32", 6693, 209, 587, T128, False, None),
    ("f32", 75, 2188, 7588, T128, True, None), ("f32", 75, 2189, 7587, T128, True, None),
    ("f32", 8737, 212, 908, T192, False, None), ("f32", 8737, 213, 907, T192, False, None),
    ("f32", 5365, 6424, 140, T192, True, None), ("f32", 5365, 6425, 137, T192, True, None),
    ("f32", 3859, 252, 4868, T192, False, T128), ("f32", 3859, 253, 4867, T192, False, T128),
    ("f32", 7967, 236, 10692, T192, False, T192), ("f32", 7967, 237, 10691, T192, False, T192),
    ("f32", 1937, 208, 6332, T192, False, T64), ("f32", 1937, 209, 6331, T192, False, T64),
]

# 8 bits: a row's scales in whole words and not
EIGHT_BITS = [
    (449, 256, 8384, T128, False, None), (407, 224, 9620, T128, False, None),
    (7429, 256, 1095, T192, False, None), (8737, 224, 907, T192, False, None),
    (1077, 256, 9839, T256, False, None), (1157, 224, 10022, T256, False, None),
    (3899, 256, 5394, T256, False, T128), (3847, 288, 6944, T256, False, T192), (3883, 288, 5017, T256, False, T64),
]

# (type, rows, in, out, plan of dx, plan of dw; None: any)
BACKWARD = [
    ("bf16", 16384, 768, 3352, (T192, False, None), (T256, True, None)),   # the 125M layer's input projection
    ("bf16", 711, 5552, 136, (T128, False, None), None), ("bf16", 711, 5551, 131, (T128, False, None), None),
    ("bf16", 205, 5336, 10424, (T128, True, None), None), ("bf16", 205, 5331, 10417, (T128, True, None), None),
    ("bf16", 9463, 848, 136, (T192, False, None), None), ("bf16", 9463, 843, 133, (T192, False, None), None),
    ("bf16", 3857, 1064, 2736, (T192, True, None), None), ("bf16", 3857, 1063, 2731, (T192, True, None), None),
    ("bf16", 1819, 6320, 136, (T256, False, None), None), ("bf16", 1567, 6945, 137, (T256, False, None), None),
    ("bf16", 933, 4496, 3344, (T256, True, None), None), ("bf16", 933, 4489, 3341, (T256, True, None), None),
    ("bf16", 131, 424, 9544, None, (T128, False, None)), ("bf16", 131, 419, 9537, None, (T128, False, None)),
    ("bf16", 7593, 6456, 200, None, (T128, True, None)), ("bf16", 9685, 3065, 321, None, (T128, True, None)),
    ("bf16", 133, 2600, 3184, None, (T192, False, None)), ("bf16", 133, 2597, 3179, None, (T192, False, None)),
    ("bf16", 2859, 728, 5464, None, (T192, True, None)), ("bf16", 2859, 725, 5461, None, (T192, True, None)),
    ("bf16", 131, 1752, 6528, None, (T256, False, None)), ("bf16", 131, 1745, 6521, None, (T256, False, None)),
    ("bf16", 3453, 936, 4392, None, (T256, True, None)), ("bf16", 3453, 935, 4387, None, (T256, True, None)),
    ("f32", 711, 5552, 136, (T128, False, None), None), ("f32", 321, 2167, 3529, (T128, True, None), None),
    ("f32", 9463, 843, 133, (T192, False, None), None), ("f32", 2515, 1093, 3535, (T192, True, None), None),
    ("f32", 4037, 4311, 153, (T192, False, T128), None), ("f32", 1819, 6320, 136, (T192, False, T64), None),
    ("f32", 131, 419, 9537, None, (T128, False, None)), ("f32", 3569, 3275, 205, None, (T128, True, None)),
    ("f32", 133, 2600, 3184, None, (T192, False, None)), ("f32", 2659, 527, 6815, None, (T192, True, None)),
    ("f32", 145, 2099, 7989, None, (T192, False, T128)), ("f32", 131, 3144, 4056, None, (T192, False, T64)),
]

"""The scratch that attention's pieces are left in, on the CPU: every plan of either cache's calls fits what a context allocates."""

import ctypes
import itertools

import pytest

from cross_model_kv_amd import kvmap as K


class Plan(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("row_blocks", ctypes.c_int), ("grid", ctypes.c_int), ("splits", ctypes.c_bool),
                ("prompt", ctypes.c_bool)]


def _fn(name, res, n):
    f = getattr(K.lib(), name)
    f.restype, f.argtypes = res, [ctypes.c_int] * n
    return f


@pytest.mark.parametrize("cus", [1, 32, 80, 256, 304])
@pytest.mark.parametrize("call,scratch", [("q8_attend_plan", "q8_scratch_bytes"), ("paged_attend_plan", "paged_scratch_bytes")])
def test_every_plan_fits(call, scratch, cus):
    plan = _fn(f"_ZN5kvmap{len(call)}{call}ENS_4ElemEiiiiiii", Plan, 8)
    room = _fn(f"_ZN5kvmap{len(scratch)}{scratch}Ei", ctypes.c_size_t, 1)(cus)
    piece = _fn("_ZN5kvmap14q8_piece_bytesEiii", ctypes.c_size_t, 3)
    cut, largest = 0, 0
    for elem, d, H, G, n_q, B, max_len in itertools.product((0, 1), (64, 128), (1, 3, 8), (1, 2, 8, 16, 33), (1, 2, 4, 16),
                                                            (1, 2, 16, 70, 600), (0, 1, 200, 300, 1100, 2100, 40000, 1 << 20)):
        p = plan(elem, B, n_q, H * G, H, d, max_len, cus)
        assert p.rows in (16, 32) or p.prompt
        assert p.grid >= 1 and p.rows * p.row_blocks >= n_q * G
        if p.splits:
            cut += 1
            largest = max(largest, piece(p.grid, p.rows, d))
    assert cut and largest <= room, (largest, room)

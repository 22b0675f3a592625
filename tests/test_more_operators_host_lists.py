"""Lists of buffers and sizes as the binding takes them: refusals come from the
library, whatever kind of sequence was given.  The pointers are never
dereferenced."""

import ctypes

import pytest

import double_binary_tree_gb300 as vr
from tests.test_more_operators_host import adamw_args, values_args
from tests.test_operators_host import A, INV, STEP, code

KINDS = [list, tuple, lambda x: (ctypes.c_void_p * 2)(*x), lambda x: (ctypes.c_size_t * 2)(*x),
         lambda x: (ctypes.c_longlong * 2)(*x), vr.pointer_array]
IDS = ["list", "tuple", "void_p", "size_t", "longlong", "pointer_array"]


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_pointers(kind):
    src, dst = kind([A, A + STEP]), kind([A + 2 * STEP, A + 3 * STEP])
    got = vr._ptrs(src)
    assert got._type_ is ctypes.c_void_p and list(got) == [A, A + STEP]
    # steps = 0 is refused by the library
    assert code(vr.vr_orthogonalize, src, dst, 2, 8, 8, vr.VR_FLOAT32, 0, None, 1e-7, 1.0,
                A + 4 * STEP, 1 << 20) == INV


@pytest.mark.parametrize("kind", [list, tuple, lambda x: (ctypes.c_size_t * 2)(*x),
                                  lambda x: (ctypes.c_int * 2)(*x),
                                  lambda x: (ctypes.c_longlong * 2)(*x), vr.size_array])
def test_sizes(kind):
    assert list(vr.size_array(kind([1000, 300]))) == [1000, 300]
    args = adamw_args(sizes=kind([1000, 300]), step=0)
    assert code(vr.vr_adamw, *args) == INV


def test_prepared_lists_are_taken_as_they_are():
    for prepared in (vr.pointer_array([A, 0, None]), vr.size_array([1, 2])):
        again = vr._ptrs(prepared) if prepared._type_ is ctypes.c_void_p else vr.size_array(prepared)
        assert again is prepared
    assert vr.pointer_array(None) is None


def test_lists_shorter_than_the_count():
    """Refused instead of read on."""
    for name in ("params", "grads", "m", "v", "mScales", "vScales", "masters", "sizes"):
        short = adamw_args()
        at = ["params", "grads", "m", "v", "mScales", "vScales", "masters", "sizes"].index(name)
        for cut in (short[at][:1], [],
                    (vr.size_array if name == "sizes" else vr.pointer_array)(short[at][:1])):
            args = list(short)
            args[at] = cut
            assert code(vr.vr_adamw, *args) == INV, name
    for at in range(4):
        args = values_args()
        args[at] = args[at][:1]
        assert code(vr.vr_adamw_values, *args) == INV
    for at in (6, 7):
        args = values_args()
        args[at] = args[at][:1]
        assert code(vr.vr_adamw_values, *args) == INV
    # what is not read may be any list (the refusal is the sizes')
    args = values_args(mValues=None, m=[], mScales=[], sizes=[1 << 41, 1])
    assert code(vr.vr_adamw_values, *args) == INV

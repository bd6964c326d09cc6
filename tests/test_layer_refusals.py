"""CPU tests of the entry points around the scan: what they refuse before any
CUDA call, with the documented status.  Every call is invalid in one way and
uses placeholder pointers that are never dereferenced."""
import pytest

import selective_state_space_selscan_b200 as ss

C = ss.STATUS_CODE
FAKE = 0x7f0000000000
BF, F32, I32 = ss.SELSCAN_BF16, ss.SELSCAN_F32, ss.SELSCAN_I32


def t(shape, dtype=BF, strides=None, data=FAKE):
    if strides is None:
        strides, acc = [], 1
        for s in reversed(shape):
            strides.insert(0, acc)
            acc *= s
    n = len(shape)
    return ss._DESC.pack(data, dtype, n, *shape, *(0,) * (4 - n), *strides, *(0,) * (4 - n))


def conv(**over):
    a = dict(x=t((2, 24, 40)), w=t((24, 4), F32), bias=t((24,), F32), h0=t((2, 24, 3)),
             y=t((2, 24, 40)), last=t((2, 24, 3)))
    a.update(over)
    return ss.lib().selscan_conv(a["x"], a["w"], a["bias"], 1, a["h0"], a["y"], a["last"], None)


CONV = [
    (dict(x=None), "NULL"), (dict(y=None), "NULL"), (dict(w=None), "NULL"),
    (dict(x=t((2, 24, 40), data=0)), "NULL"),
    (dict(h0=t((2, 24, 3), data=0)), "NULL"),
    (dict(x=t((2, 24))), "SHAPE"), (dict(y=t((2, 24, 39))), "SHAPE"),
    (dict(w=t((23, 4), F32)), "SHAPE"), (dict(w=t((24,), F32)), "SHAPE"),
    (dict(bias=t((23,), F32)), "SHAPE"), (dict(h0=t((2, 24, 4))), "SHAPE"),
    (dict(last=t((2, 24, 2))), "SHAPE"), (dict(last=t((24, 3))), "SHAPE"),
    (dict(x=t((2, 24, 40), 7)), "DTYPE"), (dict(x=t((2, 24, 40), I32)), "DTYPE"),
    (dict(y=t((2, 24, 40), F32)), "DTYPE"), (dict(w=t((24, 4))), "DTYPE"),
    (dict(h0=t((2, 24, 3), F32)), "DTYPE"), (dict(last=t((2, 24, 3), F32)), "DTYPE"),
    (dict(x=t((2, 24, 40), strides=(960, -40, 1))), "STRIDE"),
    (dict(y=t((2, 24, 40), strides=(0, 40, 1))), "STRIDE"),
    (dict(y=t((2, 24, 40), strides=(960, 40, 0))), "STRIDE"),
    (dict(w=t((24, 4), F32, strides=(1, 24))), "STRIDE"),
    (dict(h0=t((2, 24, 3), strides=(72, 1, 24))), "STRIDE"),
    (dict(x=t((2, 24, 40), data=FAKE + 1)), "ALIGN"), (dict(y=t((2, 24, 40), data=FAKE + 1)), "ALIGN"),
    (dict(last=t((2, 24, 3), data=FAKE + 1)), "ALIGN"), (dict(w=t((24, 4), F32, data=FAKE + 2)), "ALIGN"),
    (dict(w=t((24, 5), F32), h0=None, last=None), "UNSUPPORTED"),
    (dict(w=t((24, 1), F32), h0=None, last=None), "UNSUPPORTED"),
    (dict(x=t((65536, 24, 40)), y=t((65536, 24, 40)), h0=None, last=None), "UNSUPPORTED"),
]


@pytest.mark.parametrize("over,expect", CONV)
def test_conv_rejects(over, expect):
    assert conv(**over) == C["SELSCAN_ERR_" + expect]


def conv_bwd(**over):
    a = dict(x=t((2, 24, 40)), w=t((24, 4), F32), bias=t((24,), F32), h0=t((2, 24, 3)),
             dy=t((2, 24, 40)), dlast=t((2, 24, 3)), dx=t((2, 24, 40)), dw=t((24, 4), F32),
             db=t((24,), F32), dh0=t((2, 24, 3)))
    a.update(over)
    return ss.lib().selscan_conv_bwd(a["x"], a["w"], a["bias"], 1, a["h0"], a["dy"], a["dlast"],
                                     a["dx"], a["dw"], a["db"], a["dh0"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(dy=None), "NULL"), (dict(dx=None), "NULL"), (dict(dw=None), "NULL"),
    (dict(dy=t((2, 24, 41))), "SHAPE"), (dict(dw=t((24, 3), F32)), "SHAPE"),
    (dict(db=t((24, 1), F32)), "SHAPE"), (dict(dlast=t((2, 24, 2))), "SHAPE"),
    (dict(dy=t((2, 24, 40), F32)), "DTYPE"), (dict(dw=t((24, 4))), "DTYPE"),
    (dict(dh0=t((2, 24, 3), F32)), "DTYPE"),
    (dict(dx=t((2, 24, 40), strides=(960, 0, 1))), "STRIDE"),
    (dict(dlast=t((2, 24, 3), strides=(72, 1, 24))), "STRIDE"),
    (dict(dx=t((2, 24, 40), data=FAKE + 1)), "ALIGN"),
    (dict(w=t((24, 6), F32), dw=t((24, 6), F32), h0=None, dlast=None, dh0=None), "UNSUPPORTED"),
])
def test_conv_bwd_rejects(over, expect):
    assert conv_bwd(**over) == C["SELSCAN_ERR_" + expect]


def conv_step(**over):
    a = dict(state=t((9, 24, 3)), slots=t((5,), I32), x=t((5, 24)), w=t((24, 4), F32),
             bias=t((24,), F32), y=t((5, 24)))
    a.update(over)
    return ss.lib().selscan_conv_step(a["state"], a["slots"], a["x"], a["w"], a["bias"], 1, a["y"],
                                      None)


@pytest.mark.parametrize("over,expect", [
    (dict(state=None), "NULL"), (dict(x=None), "NULL"), (dict(y=None), "NULL"),
    (dict(slots=t((5,), I32, data=0)), "NULL"),
    (dict(slots=None), "SHAPE"),  # the state then has one row per token
    (dict(slots=t((4,), I32)), "SHAPE"), (dict(slots=t((5, 1), I32)), "SHAPE"),
    (dict(state=t((9, 24, 2))), "SHAPE"), (dict(y=t((5, 23))), "SHAPE"),
    (dict(slots=t((5,), F32)), "DTYPE"), (dict(state=t((9, 24, 3), F32)), "DTYPE"),
    (dict(slots=t((5,), I32, strides=(2,))), "STRIDE"),
    (dict(state=t((9, 24, 3), strides=(72, 1, 24))), "STRIDE"),
    (dict(y=t((5, 24), strides=(0, 1))), "STRIDE"), (dict(x=t((5, 24), strides=(24, -1))), "STRIDE"),
    (dict(slots=t((5,), I32, data=FAKE + 2)), "ALIGN"),
    (dict(state=t((9, 24, 3), data=FAKE + 1)), "ALIGN"),
    (dict(w=t((24, 5), F32), state=t((9, 24, 4))), "UNSUPPORTED"),
])
def test_conv_step_rejects(over, expect):
    assert conv_step(**over) == C["SELSCAN_ERR_" + expect]


def conv_packed(**over):
    a = dict(state=t((9, 24, 3)), x=t((40, 24)), w=t((24, 4), F32), bias=None,
             start=t((6,), I32), slots=t((5,), I32), seen=t((5,), I32), y=t((40, 24)))
    a.update(over)
    return ss.lib().selscan_conv_packed(a["state"], a["x"], a["w"], a["bias"], 1, a["start"],
                                        a["slots"], a["seen"], a["y"], None)


PACKED = [
    (dict(state=None), "NULL"), (dict(start=None), "NULL"), (dict(slots=None), "NULL"),
    (dict(y=None), "NULL"), (dict(seen=t((5,), I32, data=0)), "NULL"),
    (dict(start=t((5,), I32)), "SHAPE"), (dict(seen=t((6,), I32)), "SHAPE"),
    (dict(slots=t((5, 1), I32)), "SHAPE"), (dict(y=t((40, 23))), "SHAPE"),
    (dict(start=t((6,), F32)), "DTYPE"), (dict(slots=t((5,), BF)), "DTYPE"),
    (dict(y=t((40, 24), F32)), "DTYPE"),
    (dict(start=t((6,), I32, strides=(2,))), "STRIDE"),
    (dict(y=t((40, 24), strides=(23, 1))), "STRIDE"),
    (dict(y=t((40, 24), strides=(48, 2))), "STRIDE"),
    (dict(seen=t((5,), I32, data=FAKE + 1)), "ALIGN"),
]


@pytest.mark.parametrize("over,expect", PACKED + [
    (dict(x=t((40, 24), strides=(48, 2))), "STRIDE"), (dict(x=t((40, 24), I32)), "DTYPE"),
    (dict(w=t((24, 5), F32), state=t((9, 24, 4))), "UNSUPPORTED"),
    (dict(slots=t((65536,), I32), start=t((65537,), I32), seen=None), "UNSUPPORTED"),
])
def test_conv_packed_rejects(over, expect):
    assert conv_packed(**over) == C["SELSCAN_ERR_" + expect]


def fwd_packed(**over):
    a = dict(state=t((9, 24, 16), F32), u=t((40, 24)), delta=t((40, 24)), bias=t((24,), F32),
             A=t((24, 16), F32), B=t((40, 16)), C=t((40, 16)), D=t((24,), F32), z=t((40, 24)),
             start=t((6,), I32), slots=t((5,), I32), seen=t((5,), I32), y=t((40, 24)))
    a.update(over)
    return ss.lib().selscan_fwd_packed(a["state"], a["u"], a["delta"], a["bias"], 1, a["A"], a["B"],
                                       a["C"], a["D"], a["z"], a["start"], a["slots"], a["seen"],
                                       a["y"], None)


@pytest.mark.parametrize("over,expect", PACKED + [
    (dict(u=None), "NULL"), (dict(delta=None), "NULL"), (dict(B=None), "NULL"),
    (dict(z=t((40, 24), data=0)), "NULL"),
    (dict(A=t((23, 16), F32)), "SHAPE"), (dict(B=t((40, 15))), "SHAPE"),
    (dict(C=t((39, 16))), "SHAPE"), (dict(state=t((9, 24, 8), F32)), "SHAPE"),
    (dict(z=t((40, 24), F32)), "DTYPE"), (dict(state=t((9, 24, 16))), "DTYPE"),
    (dict(delta=t((40, 24), F32)), "DTYPE"),
    (dict(u=t((40, 24), strides=(1, 40))), "STRIDE"), (dict(B=t((40, 16), strides=(1, 40))), "STRIDE"),
    (dict(state=t((9, 24, 16), F32, strides=(384, 1, 24))), "STRIDE"),
    (dict(A=t((24, 16), F32, data=FAKE + 4)), "ALIGN"),
    (dict(state=t((9, 24, 16), F32, data=FAKE + 8)), "ALIGN"),
    (dict(u=t((40, 24), data=FAKE + 1)), "ALIGN"),
    (dict(A=t((24, 32), F32), B=t((40, 32)), C=t((40, 32)), state=t((9, 24, 32), F32)), "UNSUPPORTED"),
])
def test_fwd_packed_rejects(over, expect):
    assert fwd_packed(**over) == C["SELSCAN_ERR_" + expect]


def step_slots(scalar=False, **over):
    if scalar:
        a = dict(state=t((9, 2, 64, 128), F32), u=t((5, 128)), delta=t((5, 2), F32), bias=None,
                 A=t((2,), F32), B=t((5, 128)), C=t((5, 128)), D=None, z=None, y=t((5, 128)))
    else:
        a = dict(state=t((9, 24, 16), F32), u=t((5, 24)), delta=t((5, 24)), bias=None,
                 A=t((24, 16), F32), B=t((5, 16)), C=t((5, 16)), D=None, z=None, y=t((5, 24)))
    a["slots"] = t((5,), I32)
    a.update(over)
    head = (a["state"], a["slots"], a["u"], a["delta"], a["bias"], 1, a["A"], a["B"], a["C"],
            a["D"], a["z"])
    if scalar:
        return ss.lib().selscan_step_scalarA_slots(*head, 64, a["y"], None)
    return ss.lib().selscan_step_slots(*head, a["y"], None)


@pytest.mark.parametrize("scalar", [False, True])
@pytest.mark.parametrize("over,expect", [
    (dict(slots=None), "NULL"), (dict(slots=t((5,), I32, data=0)), "NULL"),
    (dict(slots=t((6,), I32)), "SHAPE"), (dict(slots=t((5,), F32)), "DTYPE"),
    (dict(slots=t((5,), I32, strides=(3,))), "STRIDE"),
    (dict(slots=t((5,), I32, data=FAKE + 2)), "ALIGN"),
    (dict(state=None), "NULL"), (dict(y=None), "NULL"),
])
def test_step_slots_rejects(scalar, over, expect):
    assert step_slots(scalar, **over) == C["SELSCAN_ERR_" + expect]


def test_step_slots_rejects_state_shapes():
    assert step_slots(state=t((9, 23, 16), F32)) == C["SELSCAN_ERR_SHAPE"]
    assert step_slots(True, state=t((9, 2, 63, 128), F32)) == C["SELSCAN_ERR_SHAPE"]


def test_nothing_to_do_is_accepted_without_a_device():
    """Calls without rows, channels or sequences launch nothing."""
    assert conv(x=t((0, 24, 40)), y=t((0, 24, 40)), h0=None, last=None) == 0
    assert conv_step(x=t((0, 24)), y=t((0, 24)), slots=t((0,), I32)) == 0
    assert conv_packed(start=t((1,), I32), slots=t((0,), I32), seen=t((0,), I32)) == 0
    assert fwd_packed(start=t((1,), I32), slots=t((0,), I32), seen=None) == 0
    assert step_slots(u=t((0, 24)), delta=t((0, 24)), B=t((0, 16)), C=t((0, 16)), y=t((0, 24)),
                      slots=t((0,), I32)) == 0


@pytest.mark.parametrize("bound", [True, False])
def test_host_tensors_are_refused(bound, monkeypatch):
    """By the C++ binding and by the ctypes one."""
    import torch
    assert ss._binding(), "_bind.so is not built"
    monkeypatch.setattr(ss, "_bound", ss._binding() if bound else False)
    x = torch.zeros(2, 24, 40)
    w, s = torch.zeros(24, 4), torch.zeros(2, 24, 3)
    i = torch.zeros(3, dtype=torch.int32)
    A, st = -torch.ones(24, 16), torch.zeros(4, 24, 16)
    r = torch.zeros(8, 24)
    bc = torch.zeros(8, 16)
    for call in (lambda: ss.selscan_conv(x, w), lambda: ss.selscan_conv_bwd(x, w, x),
                 lambda: ss.selscan_conv_step(s, x[..., 0], w),
                 lambda: ss.selscan_conv_packed(s, r, w, i, i[:2]),
                 lambda: ss.selscan_fwd_packed(st, r, r, A, bc, bc, i, i[:2]),
                 lambda: ss.selscan_step(st, r, r, A, bc, bc, slots=i)):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()


def test_index_status_has_a_name():
    assert C["SELSCAN_ERR_INDEX"] == 9 and "slot" in ss._strerror(9)


def test_binding_checks_its_arguments():
    import torch
    call = ss._binding()
    with pytest.raises(TypeError, match="torch tensors"):
        call(ss._ENTRY["selscan_conv"], None, "x", None, None, 1, None, None, None)
    with pytest.raises(TypeError, match="too few"):
        call(ss._ENTRY["selscan_conv"], None, None, None)
    with pytest.raises(ValueError, match="entry point"):
        call(99, None)
    with pytest.raises(TypeError):
        call(ss._ENTRY["selscan_conv"], None, None, None, None, "silu", None, None, None)
    assert call(ss._ENTRY["selscan_conv"], None, None, None, None, 1, None, None, None) == \
        C["SELSCAN_ERR_NULL"]

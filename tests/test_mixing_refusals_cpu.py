"""Group norm and window attention refuse outputs that lie over what other blocks of the call still read
or write, and scales that float32 does not hold. Addresses only: every call here is refused before any GPU work."""
import ctypes

import pytest

import submanifold_sparse_convolution_amd as smc

ARG = 1
BASE = 1 << 30          # addresses that are never read
ROWS, C, GROUPS, SAMPLES = 100, 32, 4, 3
PLACES = {name: BASE + 65536 * i for i, name in enumerate(
    ("x", "y", "dy", "dx", "weight", "bias", "offsets", "stats", "dweight", "dbias", "workspace"))}


def group(**changed):
    a = smc.GroupNormArgs(ROWS, C, GROUPS, SAMPLES, 0, 0, 1e-5)
    for name, at in {**PLACES, **changed}.items():
        setattr(a, name, at)
    a.ldx = a.ldy = a.ld_dy = a.ld_dx = 48
    a.workspace_bytes = 1 << 20
    return a


def message(call, a):
    assert call(ctypes.byref(a), None) == ARG
    return smc.lib().smc_last_error().decode()


# (output moved onto, at a distance in bytes): rows are 64 bytes, 96 apart, vectors 64 (offsets 16, stats 96)
@pytest.mark.parametrize("out,on,by", [("y", "weight", 0), ("y", "bias", 62), ("y", "offsets", 12), ("y", "stats", -9500),
                                       ("stats", "x", 9560), ("stats", "weight", -92), ("stats", "bias", 60), ("stats", "offsets", 0)])
def test_group_norm(out, on, by):
    assert "shares memory" in message(smc.lib().smc_group_norm, group(**{out: PLACES[on] + by}))


@pytest.mark.parametrize("out", ["dweight", "dbias"])
@pytest.mark.parametrize("on,by", [("weight", 0), ("weight", 62), ("bias", -62), ("bias", 0), ("x", 96), ("x", 9500), ("x", -10),
                                   ("dy", 0), ("dx", 32), ("stats", 94), ("offsets", 4)])
def test_gradients_of_the_weights(out, on, by):
    assert "shares memory" in message(smc.lib().smc_group_norm_backward, group(**{out: PLACES[on] + by}))


def test_gradients_on_each_other():
    assert "shares memory" in message(smc.lib().smc_group_norm_backward, group(dweight=PLACES["dbias"]))
    assert "shares memory" in message(smc.lib().smc_group_norm_backward, group(dx=PLACES["dbias"] - 9504))
    for on in ("weight", "bias", "offsets", "stats"):
        assert "shares memory" in message(smc.lib().smc_group_norm_backward, group(dx=PLACES[on]))


@pytest.mark.parametrize("changed", [dict(dweight=PLACES["x"] + 64, ld=True), dict(dweight=PLACES["weight"] + 64),
                                     dict(dbias=PLACES["bias"] - 64), dict(dweight=PLACES["x"] + 99 * 96 + 64),
                                     dict(dx=PLACES["x"]), dict(dx=PLACES["dy"]), dict(bias=PLACES["weight"])])
def test_neighbours_are_taken(changed):
    """Between rows, right behind and right before: the next check (of the scratch memory) refuses the call."""
    changed = dict(changed)
    wide = changed.pop("ld", False)
    a = group(**changed)
    if wide:
        a.ldx = 64
    a.workspace_bytes = 0
    assert "workspace" in message(smc.lib().smc_group_norm_backward, a)


def attention(**changed):
    w = smc.WindowsArgs(8, 1)
    w.ex = w.ey = w.ez = 2
    w.plan, w.plan_bytes = BASE, smc.lib().smc_windows_bytes(8, 1)
    w.tiles32 = w.tiles64 = w.tiles128 = w.longest = 1
    w.pairs = 64
    a = smc.AttentionArgs(ctypes.pointer(w), 2, 1, 16, 0, 0.25, 1)
    names = ("q", "k", "v", "out", "dout", "dq", "dk", "dv", "bias", "lse", "dbias", "workspace")
    at = {name: BASE + 65536 * (i + 1) for i, name in enumerate(names)}
    for name, value in changed.items():
        at[name] = at[value[0]] + value[1]
    for name, value in at.items():
        setattr(a, name, value)
    for name in ("ldq", "ldk", "ldv", "ld_out", "ld_dout", "ld_dq", "ld_dk", "ld_dv"):
        setattr(a, name, 32)
    a.workspace_bytes = 1 << 20
    return a


@pytest.mark.parametrize("out,on,by", [("out", "bias", 0), ("out", "lse", 60), ("lse", "q", 508), ("lse", "k", 0), ("lse", "v", 32),
                                       ("lse", "bias", 32)])
def test_attention(out, on, by):
    assert "shares memory" in message(smc.lib().smc_window_attention, attention(**{out: (on, by)}))


@pytest.mark.parametrize("out,on,by", [(o, i, 0) for o in ("dq", "dk", "dv") for i in ("bias", "lse", "dbias")]
                         + [("dbias", i, 16) for i in ("q", "k", "v", "out", "dout", "lse", "dq", "dk", "dv")])
def test_attention_gradients(out, on, by):
    assert "shares memory" in message(smc.lib().smc_window_attention_backward, attention(**{out: (on, by)}))


def test_attention_neighbours_are_taken():
    for changed in (dict(), dict(dbias=("k", 512)), dict(dbias=("bias", 36)), dict(lse=("q", 512))):
        a = attention(**changed)
        a.workspace_bytes = 0
        assert "workspace" in message(smc.lib().smc_window_attention_backward, a)


@pytest.mark.parametrize("scale", [0.0, -1.0, float("nan"), float("inf"), 3e38])
def test_scales(scale):
    """Above 2^126 the scale's product with log2 e is no float32 number."""
    a = attention()
    a.scale = scale
    for call in (smc.lib().smc_window_attention, smc.lib().smc_window_attention_backward):
        assert "scale" in message(call, a)

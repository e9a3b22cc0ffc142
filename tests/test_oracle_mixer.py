"""CPU: the fp64 oracle of the short convolution and the selective scan against
closed forms, brute force and central differences."""
import numpy as np
import pytest

import oracle.mixer as om


def _conv_case(seed, W, silu, lens):
    r = np.random.default_rng(seed)
    T, D, N = sum(lens), 3, len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    return dict(x=r.normal(size=(T, D)), w=r.normal(size=(D, W)), bias=r.normal(size=D), cu=cu,
                s0=r.normal(size=(N, W - 1, D)), silu=silu), r.normal(size=(T, D)), r.normal(size=(N, W - 1, D))


def _ssm_case(seed, lens, S=3, G=2, **kw):
    r = np.random.default_rng(seed)
    T, D, N = sum(lens), 4, len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    c = dict(x=r.normal(size=(T, D)), dt=r.normal(size=(T, D)), A=-np.exp(r.normal(size=(D, S))),
             B=r.normal(size=(T, G, S)), C=r.normal(size=(T, G, S)), skip=r.normal(size=D), z=r.normal(size=(T, D)),
             dt_bias=r.normal(size=D), s0=r.normal(size=(N, D, S)))
    c.update(kw)
    return c, cu, r.normal(size=(T, D)), r.normal(size=(N, D, S))


def _differences(f, a, eps=1e-6):
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + eps
        hi = f()
        a[i] = keep - eps
        lo = f()
        a[i] = keep
        g[i] = (hi - lo) / (2 * eps)
    return g


def test_conv_is_a_padded_convolution():
    c, _, _ = _conv_case(0, 4, False, [9])
    y, _ = om.conv(c["x"], c["w"], None, c["cu"], None, False)
    for d in range(3):
        assert np.allclose(y[:, d], np.convolve(c["x"][:, d], c["w"][d][::-1])[:9])


@pytest.mark.parametrize("cut", [1, 2, 3, 5])
def test_conv_state_resumes(cut):
    c, _, _ = _conv_case(1, 4, True, [7])
    y, s = om.conv(**c)
    y1, s1 = om.conv(c["x"][:cut], c["w"], c["bias"], [0, cut], c["s0"])
    y2, s2 = om.conv(c["x"][cut:], c["w"], c["bias"], [0, 7 - cut], s1)
    assert np.allclose(np.concatenate([y1, y2]), y) and np.array_equal(s2, s)


@pytest.mark.parametrize("W,silu", [(2, True), (3, False), (4, True)])
def test_conv_gradients_match_differences(W, silu):
    c, gy, gsT = _conv_case(2 + W, W, silu, [5, 0, 1, 2])

    def loss():
        y, s = om.conv(**c)
        return (y * gy).sum() + (s * gsT).sum()
    got = om.conv(**c, gy=gy, gsT=gsT)
    for g, name in zip(got, ("x", "w", "bias", "s0")):
        assert np.allclose(g, _differences(loss, c[name]), atol=1e-7), name


def test_ssm_equals_the_materialised_sum():
    """y_t = sum_s C_t . (prod of decays) B_s u_s, with no recurrence."""
    c, cu, _, _ = _ssm_case(10, [6], z=None, dt_bias=None, s0=None)
    y, _ = om.ssm(**c, cu=cu)
    delta = om.softplus(c["dt"])
    for t in range(6):
        for d in range(4):
            tot = c["skip"][d] * c["x"][t, d]
            for s in range(t + 1):
                k = np.exp(c["A"][d] * delta[s + 1:t + 1, d].sum())
                tot += (c["C"][t, d // 2] * k * c["B"][s, d // 2]).sum() * delta[s, d] * c["x"][s, d]
            assert abs(tot - y[t, d]) < 1e-12


@pytest.mark.parametrize("kw", [{}, {"z": None}, {"skip": None, "dt_bias": None}, {"use_softplus": False}])
def test_ssm_gradients_match_differences(kw):
    c, cu, gy, gsT = _ssm_case(11, [4, 0, 1, 3], **kw)
    if not kw.get("use_softplus", True):
        c["dt"], c["dt_bias"] = np.abs(c["dt"]) + 0.1, np.abs(c["dt_bias"])

    def loss():
        y, s = om.ssm(**c, cu=cu)
        return (y * gy).sum() + (s * gsT).sum()
    got = om.ssm(**c, cu=cu, gy=gy, gsT=gsT)
    for g, name in zip(got, ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "s0")):
        if c[name] is not None:
            assert np.allclose(g, _differences(loss, c[name]), atol=1e-6, rtol=1e-5), name


def test_absolute_bounds_the_values():
    c, cu, gy, gsT = _ssm_case(12, [5, 2])
    for kw in ({}, {"gy": gy, "gsT": gsT}):
        for v, b in zip(om.ssm(**c, cu=cu, **kw), om.ssm(**c, cu=cu, **kw, absolute=True)):
            assert (np.abs(v) <= b + 1e-12).all()
    c, gy, gsT = _conv_case(13, 4, True, [5, 2])
    for kw in ({}, {"gy": gy, "gsT": gsT}):
        for v, b in zip(om.conv(**c, **kw), om.conv(**c, **kw, absolute=True)):
            assert (np.abs(v) <= b + 1e-12).all()

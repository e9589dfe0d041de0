"""Pins of oracle/step.py: the scan against a dense transition-matrix form, a closed form and
its own splits, the norm against torch's float64 operations, the pages against hand-checked
steps; planted mistakes are rejected."""
import numpy as np
import pytest
import torch

from oracle import step as os_


def _scan_case(rng, lens, D, S, G, slots=6):
    T = sum(lens)
    return dict(x=rng.normal(size=(T, D)), dt=rng.normal(size=(T, D)), A=-np.exp(rng.normal(size=(D, S))),
                B=rng.normal(size=(T, G, S)), C=rng.normal(size=(T, G, S)), cu=np.concatenate([[0], np.cumsum(lens)]),
                slot=rng.permutation(slots)[:len(lens)], pool=rng.normal(size=(slots, D, S)), D=rng.normal(size=D),
                z=rng.normal(size=(T, D)), dt_bias=rng.normal(size=D))


def _call(c, **over):
    c = {**c, **over}
    return os_.selective_scan(c["x"], c["dt"], c["A"], c["B"], c["C"], c["cu"], c["slot"], c["pool"], D=c["D"], z=c["z"],
                              dt_bias=c["dt_bias"], has_init=c.get("has_init"))


def _dense(c):
    """Every output of a sequence as one sum over earlier tokens: decays exp(A (S_t - S_s))."""
    out = np.zeros_like(c["x"])
    D, G = c["x"].shape[1], c["B"].shape[1]
    for n in range(len(c["slot"])):
        a, b = c["cu"][n], c["cu"][n + 1]
        for d in range(D):
            g = d // (D // G)
            delta = np.log1p(np.exp(c["dt"][a:b, d] + c["dt_bias"][d]))
            S = np.cumsum(delta)
            for t in range(b - a):
                h = np.exp(c["A"][d] * S[t]) * c["pool"][c["slot"][n], d]
                h = h + (np.exp(c["A"][d][None] * (S[t] - S[:t + 1])[:, None]) * (delta * c["x"][a:b, d])[:t + 1, None]
                         * c["B"][a:a + t + 1, g]).sum(0)
                z = c["z"][a + t, d]
                out[a + t, d] = (h @ c["C"][a + t, g] + c["D"][d] * c["x"][a + t, d]) * z * (0.5 + 0.5 * np.tanh(z / 2))
    return out


def test_scan_matches_the_dense_form():
    c = _scan_case(np.random.default_rng(0), [5, 1, 9], 6, 3, 2)
    out, _, _ = _call(c)
    np.testing.assert_allclose(out, _dense(c), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("mistake", ["A", "B", "D", "group", "z"])
def test_planted_mistakes_are_rejected(mistake):
    c = _scan_case(np.random.default_rng(0), [5, 1, 9], 6, 3, 2)
    want = _dense(c)
    over = {"A": dict(A=-c["A"]), "B": dict(B=c["C"], C=c["B"]), "D": dict(D=None), "group": dict(B=c["B"][:, ::-1]),
            "z": dict(z=None)}[mistake]
    assert not np.allclose(_call(c, **over)[0], want, rtol=1e-6)


def test_scan_closed_forms():
    """A = 0: a prefix sum; dt so small that delta is 0: the state stays."""
    rng = np.random.default_rng(1)
    c = _scan_case(rng, [7], 4, 2, 1)
    c.update(A=np.zeros((4, 2)), D=None, z=None, C=np.ones((7, 1, 2)), has_init=[0])
    out, pool, _ = _call(c)
    delta = np.log1p(np.exp(c["dt"] + c["dt_bias"]))
    np.testing.assert_allclose(out, np.cumsum(delta * c["x"] * c["B"].sum(2), 0), rtol=1e-12)
    c.update(dt=np.full((7, 4), -1e4), A=-np.ones((4, 2)), has_init=[1])
    out, pool, _ = _call(c)
    np.testing.assert_array_equal(pool, c["pool"])


def test_scan_splits_and_slots():
    rng = np.random.default_rng(2)
    c = _scan_case(rng, [11, 0, 4], 5, 4, 1)
    c["has_init"] = [1, 0, 0]
    whole, pool, _ = _call(c)
    assert (pool[c["slot"][1]] == 0).all()
    untouched = [s for s in range(6) if s not in c["slot"]]
    np.testing.assert_array_equal(pool[untouched], c["pool"][untouched])
    first = {k: (v[:6] if k in ("x", "dt", "B", "C", "z") else v) for k, v in c.items()}
    a, p, _ = _call(first, cu=[0, 6], slot=c["slot"][:1], has_init=[1])
    rest = {k: (v[6:11] if k in ("x", "dt", "B", "C", "z") else v) for k, v in c.items()}
    for t in range(5):                       # token by token
        one = {k: (v[t:t + 1] if k in ("x", "dt", "B", "C", "z") else v) for k, v in rest.items()}
        y, p, _ = os_.selective_update(one["x"], one["dt"], c["A"], one["B"], one["C"], c["slot"][:1], p, D=c["D"], z=one["z"],
                                       dt_bias=c["dt_bias"])
        np.testing.assert_allclose(y[0], whole[6 + t], rtol=1e-12)
    np.testing.assert_allclose(p[c["slot"][0]], pool[c["slot"][0]], rtol=1e-12)
    skipped = _call(c, slot=np.array([-1, -1, c["slot"][2]]))
    assert np.isnan(skipped[0][:11]).all() and np.isfinite(skipped[0][11:]).all()


def test_bound_covers_fp32_arithmetic_and_is_not_loose():
    """The recurrence in fp32 by another route (torch) stays in the bound, within three digits of it."""
    rng = np.random.default_rng(3)
    c = _scan_case(rng, [60], 8, 4, 1)
    out, pool, (err, perr) = _call(c)
    t = {k: torch.from_numpy(np.asarray(v, np.float32)) for k, v in c.items() if k not in ("cu", "slot")}
    c64 = {k: (v.double().numpy() if k in t else c[k]) for k, v in {**{k: None for k in c}, **t}.items()}
    out, pool, (err, perr) = _call({**c, **{k: v for k, v in c64.items() if k in t}})
    h = t["pool"][int(c["slot"][0])].clone()
    worst = 0.0
    for i in range(60):
        v = t["dt"][i] + t["dt_bias"]
        delta = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
        h = torch.exp(delta[:, None] * t["A"]) * h + (delta * t["x"][i])[:, None] * t["B"][i]
        y = (h * t["C"][i]).sum(1) + t["D"] * t["x"][i]
        y = y * t["z"][i] / (1 + torch.exp(-t["z"][i]))
        worst = max(worst, float((np.abs(y.double().numpy() - out[i]) / err[i]).max()))
    assert 1e-3 < worst < 1


def test_norm_matches_torch():
    rng = np.random.default_rng(4)
    x, r, g, w = (rng.normal(size=s) for s in ((3, 2, 10), (3, 2, 10), (3, 2, 10), (10,)))
    tx, tr, tg, tw = (torch.from_numpy(v) for v in (x, r, g, w))
    y, u = os_.rms_norm(x, w, eps=1e-5, offset=1.0, residual=r)
    want = torch.nn.functional.rms_norm(tx + tr, (10,), tw + 1, 1e-5)
    np.testing.assert_allclose(y, want.numpy(), rtol=1e-12)
    np.testing.assert_array_equal(u, x + r)
    y, _ = os_.rms_norm(x, w, gate=g)
    np.testing.assert_allclose(y, (torch.nn.functional.rms_norm(tx, (10,), tw, 1e-6) * torch.nn.functional.silu(tg)).numpy(), rtol=1e-12)
    y, _ = os_.rms_norm(x, None, gate=g, gate_first=True)
    np.testing.assert_allclose(y, torch.nn.functional.rms_norm(tx * torch.nn.functional.silu(tg), (10,), None, 1e-6).numpy(), rtol=1e-12)
    assert not np.allclose(os_.rms_norm(x, w)[0], os_.rms_norm(x, w, offset=1.0)[0])


def test_scales_and_codes():
    y = np.array([[448.0, -1.0, 3.0, np.nan, 0.5]])
    s = os_.group_scales(y, 3)
    np.testing.assert_array_equal(s, [[1.0, 0.5 / 448]])
    c = os_.e4m3_codes(y, s, 3)
    np.testing.assert_array_equal(os_.E4M3[c[0, :3]], [448.0, -1.0, 3.0])
    assert c[0, 3] & 0x7f == 0x7f and os_.E4M3[c[0, 4]] == 448.0
    assert os_.group_scales(np.zeros((1, 4)), 0)[0, 0] == 2.0 ** -64


def test_plan_by_hand():
    """Page 4.  Request 0 holds 3 rows and brings 2: one page; 1 is padding; 2 holds 4 and brings
    1: one page; 3 needs two but one is left: it and 4 get none; token room 9."""
    table = np.full((5, 3), -1)
    table[0, 0], table[2, 0], table[4, 0] = 7, 8, 9
    got = os_.plan_pages([1, 2, 3], 9, table, [3, -1, 4, 0, 1], [2, 5, 1, 5, 1], 4, 9)
    stack, t, cu, cl, kv, slots, pos, seq = got
    assert stack == [1] and t[0].tolist() == [7, 3, -1] and t[2].tolist() == [8, 2, -1] and t[4].tolist() == [9, -1, -1]
    assert cu == [0, 2, 2, 3, 8, 9] and cl == [3, -1, 4, -1, -1] and kv == [5, -1, 5, -1, -1]
    assert slots == [31, 12, 8, -1, -1, -1, -1, -1, -1] and pos == [3, 4, 4, -1, -1, -1, -1, -1, -1]
    assert seq == [0, 0, 2, -1, -1, -1, -1, -1, -1]
    # a request whose table is too narrow is passed over; tokens past the room end the service
    got = os_.plan_pages([1, 2, 3], 9, np.full((3, 1), -1), [0, 0, 0], [5, 2, 4], 4, 10)
    assert got[3] == [-1, 0, -1] and got[2] == [0, 5, 7, 10] and got[0] == [1, 2]
    # back: the pages behind the kept rows, in order, as far as the stack's capacity goes
    assert os_.release_pages([1], 9, t, [0, -1, 4, 5, 2], [5, 9, 5, 5, 1], 4) == [1, 7, 3, 2]
    assert os_.release_pages([1], 3, t, [0, -1, 4, 5, 2], [5, 9, 5, 5, 1], 4) == [1, 7, 3]


def test_release_passes_over_holes():
    table = np.array([[5, -1, 6], [-1, -2, 7]])
    assert os_.release_pages([1], 9, table, [0, 0], [12, 12], 4) == [1, 5, 6, 7]
    assert os_.release_pages([1], 3, table, [0, 0], [12, 12], 4) == [1, 5, 6]
    assert os_.release_pages([], 3, table, [1, 0], [8, 5], 4) == []

"""Pins of the paged-cache oracle (CPU), each independent of its code."""
import numpy as np
import torch

import oracle
from moda_inputs import Workload, make_inputs
from paged_util import Paged, make


def test_paged_forward_is_the_dense_forward():
    """Sequences cut into shuffled pages, all tokens new: the dense oracle's rows."""
    w = Workload("dense", 2, 21, 4, 2, 8, 3, "f32", 5)
    x = make_inputs(w)
    want, wl = oracle.forward(x["q"], x["k"], x["v"], x["kd"], x["vd"], w.scale)
    P, blocks = 4, 6
    order = np.random.default_rng(0).permutation(2 * blocks)
    table = torch.tensor(order.reshape(2, blocks), dtype=torch.int32)
    kp, vp = np.full((12, 2, P, 8), np.nan), np.full((12, 2, P, 8), np.nan)
    for b in range(2):
        for t in range(21):
            kp[table[b, t // P], :, t % P], vp[table[b, t // P], :, t % P] = x["k"][b, t], x["v"][b, t]
    flat = lambda t: t.reshape(42, *t.shape[2:])  # noqa: E731
    out, lse, _, _ = oracle.paged_forward(flat(x["q"]), kp, vp, table, [0, 21, 42], [21, 21], flat(x["kd"]),
                                          flat(x["vd"]), 3, w.scale)
    np.testing.assert_allclose(out, want.reshape(42, 4, 8), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(lse, wl.transpose(0, 2, 1).reshape(42, 4), rtol=1e-12)


def test_rotation_is_a_complex_product_and_keeps_relative_logits():
    c = Paged("rot", ((9, 9),), Hq=2, Hkv=1, d=16, P=4, rot=16, dtype="f32")
    x = make(c)
    qo, kp, _, _, _ = oracle.paged_append(x["q"], x["k"], x["v"], x["k_pages"], x["v_pages"], x["table"], x["cu_q"],
                                          x["ctx"], x["rope"])
    f = 10000.0 ** (-np.arange(8) / 8)
    q, k = x["q"].double().numpy(), x["k"].double().numpy()
    for i in (0, 3, 8):
        z = (q[i, 1, :8] + 1j * q[i, 1, 8:]) * np.exp(1j * i * f)
        np.testing.assert_allclose(qo[i, 1], np.concatenate([z.real, z.imag]), atol=2e-6)
    # <rot_p q, rot_r k> depends on p - r only
    row = x["rope"].double().numpy()
    a = oracle.rotate(q[0], row[5], False)[0] @ oracle.rotate(k[0], row[2], False)[0]
    b = oracle.rotate(q[0], row[7], False)[0] @ oracle.rotate(k[0], row[4], False)[0]
    assert abs(a - b) < 1e-5


def test_append_leaves_everything_else_alone():
    c = Paged("left", ((7, 2), (5, 0), (3, 3)), P=4, d=8, Hq=2, Hkv=1, dtype="f32", cap=2, spare_rows=2)
    x = make(c)
    mark = torch.full_like(x["q"], 3.0)
    qo, kp, _, kd, _ = oracle.paged_append(x["q"], x["k"], x["v"], x["k_pages"], x["v_pages"], x["table"], x["cu_q"],
                                           x["ctx"], kd=x["kd"], vd=x["vd"], slot=1, q_out=mark)
    assert np.all(qo[5:] == 3.0)
    np.testing.assert_array_equal(kd[:, 0], x["kd"][:, 0].double().numpy())
    np.testing.assert_array_equal(kd[5:], x["kd"][5:].double().numpy())
    t = x["table"]
    np.testing.assert_array_equal(kp[t[0, 1], 0, 2], x["k"][1, 0].double().numpy())  # position 6
    np.testing.assert_array_equal(kp[t[0, 0]], x["k_pages"][t[0, 0]].double().numpy())


def test_scale_is_the_smallest_power_of_two():
    for a, want in ((127.0, 1.0), (127.5, 2.0), (63.5, 0.5), (63.51, 1.0), (1e-45, 2.0 ** -126), (0.0, 0.0)):
        assert oracle.scale_for(a) == want


def test_q8_growth_stays_within_one_step():
    """Tokens appended one by one, each larger than all before: a code has been
    moved at every step, yet stands within one step of its value."""
    rng = np.random.default_rng(3)
    P, d = 16, 8
    codes = [np.zeros((1, 1, P, d)) for _ in range(2)]
    scale = [np.full((1, 1), np.nan) for _ in range(2)]
    rows = [rng.standard_normal((1, 1, d)) * 1.7 ** t for t in range(P)]
    for t, r in enumerate(rows):
        codes[0], codes[1], scale[0], scale[1] = oracle.paged_append_q8(
            r, r, codes[0], codes[1], scale[0], scale[1], torch.zeros(1, 1, dtype=torch.int32), [0, 1], [t + 1])
    got = codes[0][0, 0] * scale[0][0, 0]
    # rotations run in fp32, so do the inputs here
    want = np.array([r[0, 0].astype(np.float32) for r in rows])
    assert np.abs(got - want).max() <= scale[0][0, 0]
    assert np.abs(codes[0]).max() <= 127


def test_empty_rows_and_missing_pages():
    c = Paged("gap", ((9, 1), (0, 1)), P=4, d=8, Hq=2, Hkv=1, dtype="f32")
    x = make(c)
    x["table"][0, 1] = 99
    out, lse, _, _ = oracle.paged_forward(x["q"], x["k_pages"], x["v_pages"], x["table"], x["cu_q"], x["ctx"], None,
                                          None, 0, 0.3)
    assert np.all(np.isneginf(lse[1])) and np.all(out[1] == 0)
    full = [0, 1, 2, 3, 8]  # block 1 (positions 4..7) has no page
    t = x["table"]
    k = np.array([x["k_pages"][t[0, j // 4], 0, j % 4].double().numpy() for j in full])
    z = k @ x["q"][0, 0].double().numpy() * 0.3
    assert abs(lse[0, 0] - np.log(np.exp(z).sum())) < 1e-12

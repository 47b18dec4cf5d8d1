"""Pins of the oracle's MXFP4 and expert-routing parts: values the format
fixes, an independent rounding rule, planted mistakes, and invariants."""
import inspect
import textwrap

import numpy as np
import pytest

import oracle
import oracle.lora_oracle as lo


def test_decode_specification_values():
    codes = np.arange(256, dtype=np.uint8).reshape(16, 16)
    v = oracle.decode_mxfp4(codes, np.full((16, 1), 127, np.uint8))
    mags = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    for b in range(256):
        row, col = divmod(b, 16)
        for half in range(2):
            code = b >> (4 * half) & 15
            want = mags[code & 7] * (-1 if code & 8 else 1)
            assert v[row, 2 * col + half] == want
    one = np.full((1, 16), 0x22, np.uint8)
    for b, want in ((127, 1.0), (0, 2.0 ** -127), (254, 2.0 ** 127), (130, 8.0)):
        assert np.all(oracle.decode_mxfp4(one, np.array([[b]], np.uint8)) == want)
    assert np.isnan(oracle.decode_mxfp4(one, np.array([[255]], np.uint8))).all()


def _block(values):
    x = np.zeros((1, 32))
    x[0, :len(values)] = values
    q, s = oracle.quantize_mxfp4(x)
    return oracle.decode_mxfp4(q, s)[0], int(s[0, 0])


def test_quantize_known_blocks():
    # amax 6: floor(log2 6) - 2 = 0, so the grid is the format's own
    v, b = _block([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -5, 0.26, 4.99, 5.01])
    assert b == 127
    assert v[:13].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -4, 0.5, 4, 6]
    assert np.signbit(v[8])
    # amax 7.5 rounds to 8, past the largest value: saturates at 6
    assert _block([7.5, -7.9])[0][:2].tolist() == [6, -6]
    # a power of two and just below it
    assert _block([8.0])[1] == 128 and _block([np.nextafter(8.0, 0)])[1] == 127
    # nothing, and less than the least scale holds
    assert _block([])[1] == 0 and _block([2.0 ** -140])[0][0] == 0
    for bad in (np.inf, -np.inf, np.nan):
        v, b = _block([1.0, bad])
        assert b == 255 and np.isnan(v).all()


def test_quantize_by_another_rule():
    """Nearest value by comparison with the midpoints between neighbours, and
    quantizing the decoded values changes nothing."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((6, 96)) * np.exp2(rng.integers(-20, 20, size=(6, 96)))
    x[0, :32] = np.round(x[0, :32] * 4) / 4
    q, s = oracle.quantize_mxfp4(x)
    v = oracle.decode_mxfp4(q, s)
    scale = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5])
    m = np.abs(x) / scale
    up = (m[..., None] > mids).sum(-1)
    tie = (m[..., None] == mids).any(-1)
    up = np.where(tie & (up % 2 == 1), up + 1, up)
    assert np.array_equal(np.abs(v), np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])[up] * scale)
    q2, s2 = oracle.quantize_mxfp4(v)
    assert np.array_equal(oracle.decode_mxfp4(q2, s2), v)


MUTATIONS = {
    "high_half_first": ("np.stack([c & 15, c >> 4], axis=-1)", "np.stack([c >> 4, c & 15], axis=-1)"),
    "bias_128": ("np.ldexp(1.0, b - 127)", "np.ldexp(1.0, b - 128)"),
    "sign_dropped": ("np.where(c & 8, -1.0, 1.0)", "1.0"),
    "no_nan": ("np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))", "np.ldexp(1.0, b - 127)"),
}


@pytest.mark.parametrize("name", sorted(MUTATIONS))
def test_decode_mutants_fail(name):
    old, new = MUTATIONS[name]
    src = textwrap.dedent(inspect.getsource(lo.decode_mxfp4))
    assert old in src
    ns = dict(lo.__dict__)
    exec(src.replace(old, new), ns)
    real, ns_f = oracle.decode_mxfp4, ns["decode_mxfp4"]
    oracle.decode_mxfp4 = ns_f
    try:
        with pytest.raises(AssertionError):
            test_decode_specification_values()
    finally:
        oracle.decode_mxfp4 = real


def test_layer_with_one_scale_equals_the_plain_oracle():
    """A weight both formats hold exactly gives the plain oracle's output."""
    import workloads as wl
    w = wl.make_random(91, 9, 64, 24, 3, 8, dtype="bf16")
    codes, scales = wl.make_mxfp4(91, 24, 64, lo=125, hi=129)
    W = wl._encode(oracle.decode_mxfp4(codes, scales).astype(np.float32), "bf16")
    a = oracle.lora_forward_mxfp4w(w.X, codes, scales, w.A, w.B, w.row_slot, w.slot_rank,
                                   w.slot_alpha, w.r_max, "bf16")
    b = oracle.lora_forward(w.X, W, w.A, w.B, w.row_slot, w.slot_rank, w.slot_alpha, w.r_max, "bf16")
    for x, y in zip(a, b):
        assert np.allclose(x, y, rtol=1e-12, atol=1e-12)


def test_routing_worked_example_and_invariants():
    r = oracle.expert_routing([[2, 0], [0, 2], [-1, 1], [7, 2]], 3)
    assert r["expert_offsets"].tolist() == [0, 2, 3, 6]
    assert r["sorted_choice"].tolist() == [1, 2, 5, 0, 3, 7]
    assert r["choice_position"].tolist() == [[3, 0], [1, 4], [-1, 2], [-1, 5]]
    assert r["status"] == 1
    ids = np.random.default_rng(3).integers(-1, 5, size=(50, 3))
    r = oracle.expert_routing(ids, 5)
    flat = ids.reshape(-1)
    kept = np.flatnonzero(flat >= 0)
    assert np.array_equal(r["sorted_choice"], kept[np.argsort(flat[kept], kind="stable")])
    assert np.array_equal(r["choice_position"].reshape(-1)[r["sorted_choice"]], np.arange(len(kept)))
